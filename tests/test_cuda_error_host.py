"""A CUDA error that the library returns is not left behind for the caller's next
CUDA call (torch's, say): a stand-in for the runtime fails one call and keeps the
last error as the runtime does."""

import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKE = """
static int last;
int cudaGetDevice(int* dev) { *dev = 0; return last = 46; }  /* devices unavailable */
int cudaPeekAtLastError(void) { return last; }
int cudaGetLastError(void) { const int e = last; last = 0; return e; }
"""
CALL = """
import ctypes, sys
sys.path[:0] = [{root!r}, {tests!r}]
import test_prompt_host as H
p, keep_alive = H.prompt()
for call in (H.attention, H.weights, H.evict):
    status = call(p)
    assert status == H.B.KVQ_ECUDA, status
    assert H.kvq.load_library().kvq_last_error().startswith(b"cudaGetDevice"), H.kvq.load_library().kvq_last_error()
    assert ctypes.CDLL(None).cudaPeekAtLastError() == 0
"""


def test_a_returned_error_is_cleared(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    (tmp_path / "fake.c").write_text(FAKE)
    subprocess.run([cc, "-shared", "-fPIC", str(tmp_path / "fake.c"), "-o", str(tmp_path / "fake.so")], check=True)
    run = subprocess.run([sys.executable, "-c", CALL.format(root=ROOT, tests=os.path.join(ROOT, "tests"))],
                         env={**os.environ, "LD_PRELOAD": str(tmp_path / "fake.so")}, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr
