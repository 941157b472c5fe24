"""The limits that the header states for the expert operators are the ones
that are enforced, and the status that reports them names no other entry
point's (no GPU is needed for these checks)."""
import os
import re

import pytest

import block_scaled_mxfp4_bf16_amd as mx
from tests.test_experts_abi import GEMV
from tests.test_grouped_abi import GROUPED
from tests.test_route_combine_abi import COMBINE, FAKE, ROUTE

UNSUPPORTED = 2
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mxfp4.h")


def call(name, base, **change):
    args = dict(base)
    assert set(change) <= set(args)
    args.update(change)
    return getattr(mx.lib(), name)(*args.values(), None)


def stated(name):
    """The text of the comment before an entry point's declaration."""
    with open(HEADER) as f:
        text = f.read()
    before = text[:re.search(r"MXFP4_API mxfp4_status_t %s\(" % name, text).start()]
    return re.sub(r"[\s*/]+", " ", before[before.rindex("UNSUPPORTED ("):])


CASES = [
    ("mxfp4_moe_combine", COMBINE, dict(T=(1 << 26) + 1), "T > 2^26"),
    ("mxfp4_moe_combine", COMBINE, dict(rows=(1 << 30) + 1), "rows > 2^30"),
    ("mxfp4_moe_combine", COMBINE, dict(ld_y=(1 << 30) + 1), "a row stride > 2^30"),
    ("mxfp4_moe_combine", COMBINE, dict(ld_out=(1 << 30) + 1), "a row stride > 2^30"),
    ("mxfp4_moe_combine", COMBINE, dict(residual=FAKE, ld_res=(1 << 30) + 1), "a row stride > 2^30"),
    ("mxfp4_moe_route", ROUTE, dict(ld=(1 << 40) + 1), "ld > 2^40"),
    ("mxfp4_gemv", GEMV, dict(ids=FAKE, experts=1 << 31), "experts or repeat >= 2^31"),
    ("mxfp4_gemv", GEMV, dict(ids=FAKE, repeat=1 << 31), "experts or repeat >= 2^31"),
    ("mxfp4_gemm_grouped", GROUPED, dict(repeat=1 << 31), "repeat >= 2^31"),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_limits_are_stated(i):
    name, base, change, text = CASES[i]
    assert call(name, base, **change) == UNSUPPORTED
    assert text in stated(name), stated(name)


def test_status_names_no_other_limits():
    text = mx.lib().mxfp4_status_string(UNSUPPORTED).decode()
    assert text.startswith("MXFP4_ERR_UNSUPPORTED") and "%" not in text and "mxfp4.h" in text
    with pytest.raises(RuntimeError, match="mxfp4_moe_route.*MXFP4_ERR_UNSUPPORTED") as e:
        mx.mxfp4_moe_route(FAKE, 0, 2000, None, 4, 2000, 8, 0, True, FAKE, FAKE, FAKE, FAKE, FAKE, stream=0)
    assert "K %" not in str(e.value)
