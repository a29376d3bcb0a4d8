"""Calls of several host threads and caches at once: what one of them asks of a
kernel must not reach another's launch."""

import ctypes
import shutil
import subprocess
import threading

import pytest

pytestmark = pytest.mark.gpu

# the calls of one thread, back to back in C: Python's own lock would let the threads take turns
CALLS = """
#include "kvq.h"
int weights_calls(kvq_status (*fn)(const kvq_prompt*, const void*, const void*, const float*, int64_t, float*, void*),
                  const kvq_prompt* p, const void* q, const void* k, const float* lse, float* w, void* stream, int n) {
  int failed = 0;
  for (int i = 0; i < n; ++i) failed += fn(p, q, k, lse, 32, w, stream) != KVQ_OK;
  return failed;
}
int restore_calls(kvq_status (*fn)(const kvq_cache*, int32_t, int32_t, void*, void*, int64_t, kvq_dtype, void*),
                  const kvq_cache* c, void* k, void* v, int64_t t_stride, void* stream, int n) {
  int failed = 0;
  for (int i = 0; i < n; ++i) failed += fn(c, 0, 1, k, v, t_stride, KVQ_BF16, stream) != KVQ_OK;
  return failed;
}
"""


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


@pytest.fixture(scope="module")
def kvq(torch):
    import quantized_kv_cache_02_gb300 as kvq
    kvq.load_library()
    return kvq


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    import os
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    at = tmp_path_factory.mktemp("calls")
    (at / "calls.c").write_text(CALLS)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([cc, "-O2", "-shared", "-fPIC", "-I", os.path.join(root, "include"), str(at / "calls.c"), "-o",
                    str(at / "calls.so")], check=True)
    return ctypes.CDLL(str(at / "calls.so"))


def test_weights_of_several_head_dims(torch, kvq, calls):
    """The CUDA-core weights kernel serves every head_dim, each with its own shared memory."""
    lens, threads, outs, failed = [70, 31], [], [], []
    gate = threading.Barrier(4)

    def run(p, q, k, lse, out, stream):
        gate.wait()
        failed.append(calls.weights_calls(kvq.load_library().kvq_prompt_weights, ctypes.byref(p.c), *(ctypes.c_void_p(x.data_ptr())
                                          for x in (q, k, lse, out)), ctypes.c_void_p(stream.cuda_stream), 20000))

    for d in (256, 16, 256, 64):
        q = torch.randn(sum(lens), 4, d, device="cuda")
        k = torch.randn(sum(lens), 2, d, device="cuda")
        lse = kvq.prompt_attention(q, k, k, lens)[1]
        p = kvq.binding._Prompt(k, lens)
        p.queries(q)
        out = torch.empty(2, sum(lens), device="cuda")
        outs.append((out, kvq.prompt_weights(q, k, lse, lens, 32)))
        threads.append(threading.Thread(target=run, args=(p, q, k, lse, out, torch.cuda.Stream())))
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0, 0, 0, 0]
    assert all(torch.equal(a, b) for a, b in outs)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_second_cache_leaves_the_first_ones_appends_alone(torch, kvq, dtype):
    """An append's shared memory goes by its cache's group and head_dim: a later cache needs less here."""
    big = kvq.KVQCache(1, 2, 4, 128, 64, 128, 7, 512, dtype=dtype)
    alone = kvq.KVQCache(1, 2, 4, 128, 64, 128, 7, 512, dtype=dtype)
    k, v = (torch.randn(1, 2, 400, 128, device="cuda").to(big.dtype) for _ in range(2))
    alone.append(k, v)
    kvq.KVQCache(1, 2, 4, 32, 16, 8, 7, 64, dtype=dtype)
    big.append(k, v)
    torch.cuda.synchronize()
    a, b = big.export_unit(0, 1), alone.export_unit(0, 1)
    assert big.seq_state(0) == alone.seq_state(0) and all((a[x] == b[x]).all() for x in a)


def test_restores_of_two_caches(torch, kvq, calls):
    """A restore's shared memory goes by its cache's group."""
    threads, results, failed = [], [], []
    gate = threading.Barrier(4)

    def run(cache, k, v, stream):
        gate.wait()
        failed.append(calls.restore_calls(kvq.load_library().kvq_restore, ctypes.c_void_p(cache.handle),
                                          ctypes.c_void_p(k.data_ptr()), ctypes.c_void_p(v.data_ptr()),
                                          ctypes.c_int64(k.shape[2]), ctypes.c_void_p(stream.cuda_stream), 20000))

    for group in (128, 64, 128, 64):
        cache = kvq.KVQCache(1, 2, 4, 128, 64, group, 7, 512)
        cache.append(*(torch.randn(1, 2, 400, 128, device="cuda").bfloat16() for _ in range(2)))
        want = cache.restore()
        got = [torch.empty_like(t) for t in want]
        results.append((cache, want, got))
        threads.append(threading.Thread(target=run, args=(cache, *got, torch.cuda.Stream())))
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0, 0, 0, 0]
    for _, want, got in results:
        assert all(torch.equal(a, b) for a, b in zip(want, got))
