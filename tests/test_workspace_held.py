"""A call that hands data from one launch to the next through the library's
workspace keeps it until its last launch is enqueued: host threads that call
on one stream cannot mix their launches, threads on different streams do not
wait for each other, and the per-thread stream is a stream of each thread.  Host-only: the entry points are built here with
g++ against stand-ins for HIP and the launchers, once plainly and once with
ThreadSanitizer."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_scaled_mxfp4_bf16_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


def _build(path, extra):
    # device qualifiers mean nothing to g++; the one device array becomes a host one
    flags = ["-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-D__align__(x)=__attribute__((aligned(x)))",
             "-DHIP_SYMBOL(x)=x", "-isystem", os.path.join(ROCM, "include"), *extra]
    exe = str(path / "check")
    subprocess.check_call(["g++", *flags, "-o", exe, os.path.join(ROOT, "tests", "workspace_held_check.cpp"), "-x", "c++",
                           os.path.join(CSRC, "experts_api.hip"), os.path.join(CSRC, "mxfp4_api.hip"), "-lpthread"])
    return exe


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    return _build(tmp_path_factory.mktemp("held"), [])


def run(exe, what):
    r = subprocess.run([exe, what], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    assert what + " ok" in r.stdout
    return r.stderr


@pytest.mark.parametrize("what", ["one_stream", "two_streams", "stream_per_thread"])
def test_launches_of_two_calls_do_not_mix(check, what):
    run(check, what)


def test_no_exception_leaves_a_c_entry(check):
    run(check, "no_host_memory")


def test_no_data_race(tmp_path):
    probe = subprocess.run(["g++", "-fsanitize=thread", "-x", "c++", "-", "-o", str(tmp_path / "t")],
                           input="int main(){return 0;}", capture_output=True, text=True)
    if probe.returncode != 0 or subprocess.run([str(tmp_path / "t")], capture_output=True).returncode != 0:
        pytest.skip("ThreadSanitizer is not usable with this g++")
    err = run(_build(tmp_path, ["-fsanitize=thread", "-g"]), "one_stream")
    assert "WARNING: ThreadSanitizer" not in err, err[-2000:]
