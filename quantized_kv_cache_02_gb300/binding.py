"""ctypes binding of libkvq.so (include/kvq.h): the same entry points under the
same names, plus ``KVQCache``, a small owner object that allocates the arena
with torch and passes torch's current CUDA stream.  Argument marshalling only:
all work runs in the library's CUDA kernels.  Importing fails loudly when the
library has not been built; there is no other implementation to fall back on.
"""

from __future__ import annotations

import ctypes
import numbers
import os
from operator import index

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvq.so")

KVQ_OK, KVQ_EINVAL, KVQ_ECAPACITY, KVQ_ENOMEM, KVQ_ECUDA, KVQ_EUNSUPPORTED, KVQ_EDEVICE = range(7)
KVQ_BF16, KVQ_FP32 = 0, 1
STATUS_NAMES = {0: "KVQ_OK", 1: "KVQ_EINVAL", 2: "KVQ_ECAPACITY", 3: "KVQ_ENOMEM", 4: "KVQ_ECUDA",
                5: "KVQ_EUNSUPPORTED", 6: "KVQ_EDEVICE"}

MAX_FLUSHED_GROUPS = 4096  # of one sequence in one append to a paged cache

# Every function include/kvq.h declares.
EXPORTED = ("kvq_required_bytes", "kvq_create", "kvq_append", "kvq_decode_attention",
            "kvq_decode_attention_ex", "kvq_bytes", "kvq_ledger", "kvq_seq_state", "kvq_export_unit",
            "kvq_export_pages", "kvq_device_status", "kvq_page_bytes", "kvq_kernel_launches", "kvq_destroy",
            "kvq_last_error", "kvq_decode_attention_noalloc", "kvq_restore", "kvq_dense_decode_attention",
            "kvq_compare", "kvq_required_bytes_paged", "kvq_create_paged", "kvq_release", "kvq_pool_state",
            "kvq_required_bytes_segmented", "kvq_create_segmented", "kvq_decode_step",
            "kvq_prompt_attention", "kvq_prompt_weights", "kvq_evict")


class kvq_config(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("residual_len", ctypes.c_int32), ("group", ctypes.c_int32),
                ("qmax", ctypes.c_int32), ("dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class kvq_bytes_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("code_bytes", "n_scales", "scale_bytes", "window_elems",
                                              "window_bytes", "total", "allocated")]


class kvq_seq_info(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("total", "quantized", "window", "last_flushed", "n_groups",
                                              "capacity")]


class kvq_unit_view(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("window_k", ctypes.c_void_p), ("window_v", ctypes.c_void_p)]


class kvq_decode_opts(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int32), ("chunk_pages", ctypes.c_int32), ("split_start", ctypes.c_void_p),
                ("split_stop", ctypes.c_void_p)]


class kvq_compare_t(ctypes.Structure):
    _fields_ = [("key_mse", ctypes.c_double), ("value_mse", ctypes.c_double)] + [
        (n, ctypes.c_int64) for n in ("n_key_scales", "n_value_scales", "raw_bytes", "container_quantized_bytes",
                                      "packed_quantized_bytes")]


class kvq_prompt(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_seqs", "n_q_heads", "n_kv_heads", "head_dim", "dtype")] + [
        ("seq_lens", ctypes.POINTER(ctypes.c_int64))] + [
        (n, ctypes.c_int64) for n in ("n_tokens", "q_token_stride", "q_head_stride", "k_token_stride",
                                      "k_head_stride", "v_token_stride", "v_head_stride", "out_token_stride",
                                      "out_head_stride")] + [("status", ctypes.c_void_p)]


class KVQError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libkvq.so and declare its signatures (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} not found: build it with __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P, V, I32, I64, SZ = ctypes.POINTER, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    sigs = {
        "kvq_required_bytes": ([P(kvq_config), P(I64), P(SZ)], ctypes.c_int),
        "kvq_create": ([P(kvq_config), P(I64), V, SZ, P(V)], ctypes.c_int),
        "kvq_append": ([V, V, V, I64, I32, I32, V], ctypes.c_int),
        "kvq_decode_attention": ([V, V, V, V], ctypes.c_int),
        "kvq_decode_attention_ex": ([V, V, V, V, P(kvq_decode_opts)], ctypes.c_int),
        "kvq_bytes": ([V, P(kvq_bytes_t)], ctypes.c_int),
        "kvq_ledger": ([P(kvq_config), P(I64), P(kvq_bytes_t)], ctypes.c_int),
        "kvq_seq_state": ([V, I32, P(kvq_seq_info)], ctypes.c_int),
        "kvq_export_unit": ([V, I32, I32, P(kvq_unit_view), V], ctypes.c_int),
        "kvq_export_pages": ([V, I32, I32, V, SZ, V], ctypes.c_int),
        "kvq_device_status": ([V, P(I32), V], ctypes.c_int),
        "kvq_page_bytes": ([P(kvq_config)], SZ),
        "kvq_kernel_launches": ([], ctypes.c_uint64),
        "kvq_decode_attention_noalloc": ([V, V, V, V], ctypes.c_int),
        "kvq_decode_step": ([V, V, V, V, V, V, P(kvq_decode_opts)], ctypes.c_int),
        "kvq_restore": ([V, I32, I32, V, V, I64, ctypes.c_int, V], ctypes.c_int),
        "kvq_dense_decode_attention": ([V, V, V, I64, V, V, V], ctypes.c_int),
        "kvq_compare": ([V, V, I64, I32, I64, I32, ctypes.c_int, I32, ctypes.c_float, I32, V, P(kvq_compare_t), V],
                        ctypes.c_int),
        "kvq_required_bytes_paged": ([P(kvq_config), P(I64), I64, P(SZ)], ctypes.c_int),
        "kvq_create_paged": ([P(kvq_config), P(I64), I64, V, SZ, P(V)], ctypes.c_int),
        "kvq_required_bytes_segmented": ([P(kvq_config), P(I64), P(SZ)], ctypes.c_int),
        "kvq_create_segmented": ([P(kvq_config), P(I64), V, SZ, P(V)], ctypes.c_int),
        "kvq_release": ([V, I32, I32], ctypes.c_int),
        "kvq_pool_state": ([V, P(I64), P(I64)], ctypes.c_int),
        "kvq_prompt_attention": ([P(kvq_prompt), V, V, V, V, V, V], ctypes.c_int),
        "kvq_prompt_weights": ([P(kvq_prompt), V, V, V, I64, V, V], ctypes.c_int),
        "kvq_evict": ([P(kvq_prompt), V, V, V, P(I64), I64, I64, V, V, V, V], ctypes.c_int),
        "kvq_destroy": ([V], None),
        "kvq_last_error": ([], ctypes.c_char_p),
    }
    for name, (args, res) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != KVQ_OK:
        raise KVQError(status, load_library().kvq_last_error().decode())


def make_config(batch, n_kv_heads, n_q_heads, head_dim, residual_len, group, qmax, dtype=KVQ_BF16, eps=1e-8):
    return kvq_config(batch, n_kv_heads, n_q_heads, head_dim, residual_len, group, qmax, dtype, eps)


def _i64_array(values):
    values = [int(v) for v in values]
    return (ctypes.c_int64 * len(values))(*values)


# ---- thin wrappers with the C names --------------------------------------------

def kvq_required_bytes(cfg: kvq_config, capacity) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().kvq_required_bytes(ctypes.byref(cfg), _i64_array(capacity), ctypes.byref(out)))
    return out.value


def kvq_ledger(cfg: kvq_config, tokens) -> dict:
    out = kvq_bytes_t()
    _check(load_library().kvq_ledger(ctypes.byref(cfg), _i64_array(tokens), ctypes.byref(out)))
    return {n: getattr(out, n) for n, _ in kvq_bytes_t._fields_}


def kvq_page_bytes(cfg: kvq_config) -> int:
    return load_library().kvq_page_bytes(ctypes.byref(cfg))


def kvq_required_bytes_paged(cfg: kvq_config, capacity, pool_blocks: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().kvq_required_bytes_paged(ctypes.byref(cfg), _i64_array(capacity), pool_blocks,
                                                   ctypes.byref(out)))
    return out.value


def kvq_create_paged(cfg: kvq_config, capacity, pool_blocks: int, device_ptr: int, device_bytes: int) -> int:
    handle = ctypes.c_void_p()
    _check(load_library().kvq_create_paged(ctypes.byref(cfg), _i64_array(capacity), pool_blocks,
                                           ctypes.c_void_p(device_ptr), device_bytes, ctypes.byref(handle)))
    return handle.value


def kvq_required_bytes_segmented(cfg: kvq_config, capacity) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().kvq_required_bytes_segmented(ctypes.byref(cfg), _i64_array(capacity), ctypes.byref(out)))
    return out.value


def kvq_create_segmented(cfg: kvq_config, capacity, device_ptr: int, device_bytes: int) -> int:
    handle = ctypes.c_void_p()
    _check(load_library().kvq_create_segmented(ctypes.byref(cfg), _i64_array(capacity), ctypes.c_void_p(device_ptr),
                                               device_bytes, ctypes.byref(handle)))
    return handle.value


def kvq_release(handle, seq_begin: int, n_seqs: int) -> None:
    _check(load_library().kvq_release(handle, seq_begin, n_seqs))


def kvq_pool_state(handle) -> tuple:
    free, total = ctypes.c_int64(0), ctypes.c_int64(0)
    _check(load_library().kvq_pool_state(handle, ctypes.byref(free), ctypes.byref(total)))
    return free.value, total.value


def kvq_create(cfg: kvq_config, capacity, device_ptr: int, device_bytes: int) -> int:
    handle = ctypes.c_void_p()
    _check(load_library().kvq_create(ctypes.byref(cfg), _i64_array(capacity), ctypes.c_void_p(device_ptr),
                                     device_bytes, ctypes.byref(handle)))
    return handle.value


def kvq_append(handle, new_k_ptr, new_v_ptr, n_tokens, seq_begin, n_seqs, stream) -> None:
    _check(load_library().kvq_append(handle, new_k_ptr, new_v_ptr, n_tokens, seq_begin, n_seqs, stream))


def kvq_decode_attention(handle, q_ptr, out_ptr, stream) -> None:
    _check(load_library().kvq_decode_attention(handle, q_ptr, out_ptr, stream))


def kvq_decode_attention_ex(handle, q_ptr, out_ptr, stream, kernel=0, chunk_pages=0, split_start=None,
                            split_stop=None) -> None:
    opts = kvq_decode_opts(kernel, chunk_pages, split_start, split_stop)
    _check(load_library().kvq_decode_attention_ex(handle, q_ptr, out_ptr, stream, ctypes.byref(opts)))


def kvq_decode_step(handle, k_ptr, v_ptr, q_ptr, out_ptr, stream, kernel=0, split_start=None, split_stop=None):
    opts = kvq_decode_opts(kernel, 0, split_start, split_stop)
    _check(load_library().kvq_decode_step(handle, k_ptr, v_ptr, q_ptr, out_ptr, stream, ctypes.byref(opts)))


def kvq_decode_attention_noalloc(handle, q_ptr, out_ptr, stream) -> None:
    """Decode attention with the split scratch in the library's fixed device
    array (for callers that cannot allocate device memory at call time)."""
    _check(load_library().kvq_decode_attention_noalloc(handle, q_ptr, out_ptr, stream))


def kvq_bytes(handle) -> dict:
    out = kvq_bytes_t()
    _check(load_library().kvq_bytes(handle, ctypes.byref(out)))
    return {n: getattr(out, n) for n, _ in kvq_bytes_t._fields_}


def kvq_seq_state(handle, seq: int) -> dict:
    out = kvq_seq_info()
    _check(load_library().kvq_seq_state(handle, seq, ctypes.byref(out)))
    return {n: getattr(out, n) for n, _ in kvq_seq_info._fields_}


def kvq_export_unit(handle, seq, kv_head, view: kvq_unit_view, stream) -> None:
    _check(load_library().kvq_export_unit(handle, seq, kv_head, ctypes.byref(view), stream))


def kvq_export_pages(handle, seq, kv_head, dst_ptr, dst_bytes, stream) -> None:
    _check(load_library().kvq_export_pages(handle, seq, kv_head, dst_ptr, dst_bytes, stream))


def kvq_device_status(handle, stream) -> int:
    word = ctypes.c_int32(0)
    status = load_library().kvq_device_status(handle, ctypes.byref(word), stream)
    if status not in (KVQ_OK, KVQ_EDEVICE):
        _check(status)
    return word.value


def kvq_restore(handle, seq_begin, n_seqs, k_ptr, v_ptr, t_stride, out_dtype, stream) -> None:
    _check(load_library().kvq_restore(handle, seq_begin, n_seqs, k_ptr, v_ptr, t_stride, out_dtype, stream))


def kvq_dense_decode_attention(handle, k_ptr, v_ptr, t_stride, q_ptr, out_ptr, stream) -> None:
    _check(load_library().kvq_dense_decode_attention(handle, k_ptr, v_ptr, t_stride, q_ptr, out_ptr, stream))


def kvq_compare(key_ptr, value_ptr, batch, heads, tokens, head_dim, dtype, qmax, eps, group, workspace_ptr,
                stream) -> dict:
    out = kvq_compare_t()
    _check(load_library().kvq_compare(key_ptr, value_ptr, batch, heads, tokens, head_dim, dtype, qmax, eps, group,
                                      workspace_ptr, ctypes.byref(out), stream))
    return {n: getattr(out, n) for n, _ in kvq_compare_t._fields_}


def compare(key, value, qmax=7, eps=1e-8, group=0) -> dict:
    """The page's compare on device tensors key, value [batch, heads, tokens,
    head_dim] (bf16 or fp32, contiguous, same shape and dtype)."""
    import torch
    assert key.is_cuda and key.shape == value.shape and key.dtype == value.dtype
    assert key.is_contiguous() and value.is_contiguous() and key.dim() == 4
    dt = {torch.bfloat16: KVQ_BF16, torch.float32: KVQ_FP32}[key.dtype]
    ws = torch.empty(2, dtype=torch.float64, device=key.device)
    b, h, t, d = key.shape
    return kvq_compare(key.data_ptr(), value.data_ptr(), b, h, t, d, dt, qmax, eps, group, ws.data_ptr(),
                       torch.cuda.current_stream(key.device).cuda_stream)


def kvq_prompt_attention(prompt: kvq_prompt, q_ptr, k_ptr, v_ptr, out_ptr, lse_ptr, stream) -> None:
    _check(load_library().kvq_prompt_attention(ctypes.byref(prompt), q_ptr, k_ptr, v_ptr, out_ptr, lse_ptr, stream))


def kvq_prompt_weights(prompt: kvq_prompt, q_ptr, k_ptr, lse_ptr, last, weights_ptr, stream) -> None:
    _check(load_library().kvq_prompt_weights(ctypes.byref(prompt), q_ptr, k_ptr, lse_ptr, last, weights_ptr, stream))


def kvq_evict(prompt: kvq_prompt, k_ptr, v_ptr, weights_ptr, keep, first, recent, k_out_ptr, v_out_ptr, index_ptr,
              stream) -> None:
    _check(load_library().kvq_evict(ctypes.byref(prompt), k_ptr, v_ptr, weights_ptr, _counts(keep), first, recent,
                                    k_out_ptr, v_out_ptr, index_ptr, stream))


# ---- prompt operators on torch tensors ---------------------------------------
#
# A short prompt's call is bound by the host (the kernels take 5 to 15 us), so
# these read each attribute of a tensor once.

_prompt_status = {}  # device index -> int32 status word that the prompt kernels report to


def _status_word(device_index):
    import torch
    word = _prompt_status.get(device_index)
    if word is None and not torch.cuda.is_current_stream_capturing():
        word = _prompt_status[device_index] = torch.zeros(1, dtype=torch.int32, device=f"cuda:{device_index}")
        torch.cuda.synchronize(device_index)  # cleared before any stream can report to it
    return word  # None in a capture that no eager call came before: those kernels report nowhere


def prompt_status(device=None) -> int:
    """The prompt kernels' status word on a device (synchronizes): 0 unless a
    bounded wait gave up there since the process started, which leaves that
    call's results undefined.  No call looks at it by itself.  Kernels captured
    before any eager call on the device report nowhere."""
    import torch
    with torch.cuda.device(device):
        return int(_status_word(torch.cuda.current_device()).item())


def _counts(values):
    try:
        return (ctypes.c_int64 * len(values))(*values)
    except TypeError:  # integers of other kinds (numpy, tensors); a fraction is no count
        return (ctypes.c_int64 * len(values))(*[index(v) for v in values])


class _Prompt:
    """The checked arguments of one prompt operator: the C struct, and how to
    call on k's device and torch's current stream there."""

    __slots__ = ("torch", "c", "k", "device", "tokens", "heads", "dim")

    def __init__(self, k, seq_lens):
        import torch
        self.torch, self.k = torch, k
        assert k.is_cuda and k.dim() == 3, "k must be a CUDA tensor [tokens, heads, head_dim]"
        dtype = k.dtype
        assert dtype == torch.bfloat16 or dtype == torch.float32, f"expected bfloat16 or float32, got {dtype}"
        self.device = k.get_device()
        self.tokens, self.heads, self.dim = k.shape
        lens = _counts(seq_lens)
        self.c = c = kvq_prompt(len(lens), self.heads, self.heads, self.dim,
                                KVQ_BF16 if dtype == torch.bfloat16 else KVQ_FP32, lens, self.tokens)
        c.k_token_stride, c.k_head_stride = self.strides("k", k, None)
        word = _prompt_status.get(self.device)
        if word is None:
            word = _status_word(self.device)
        if word is not None:
            c.status = word.data_ptr()

    def strides(self, name, t, heads):
        shape, stride, k = t.shape, t.stride(), self.k
        assert len(shape) == 3 and shape[0] == self.tokens and shape[2] == self.dim and heads in (None, shape[1]), \
            f"{name} of shape {tuple(shape)} does not go with k of shape {tuple(k.shape)}"
        assert t.get_device() == self.device and t.dtype == k.dtype, f"{name} must match the device and dtype of k"
        assert stride[2] == 1, f"{name}'s last dimension must be contiguous"
        return stride[:2]

    def queries(self, q):
        self.c.n_q_heads = q.shape[1]
        self.c.q_token_stride, self.c.q_head_stride = self.strides("q", q, None)

    def values(self, v):
        self.c.v_token_stride, self.c.v_head_stride = self.strides("v", v, self.heads)

    def rows(self, name, t, heads):
        """A float32 [heads, tokens] tensor; made where t is None."""
        torch = self.torch
        if t is None:
            return torch.empty((heads, self.tokens), dtype=torch.float32, device=self.k.device)
        assert t.dtype == torch.float32 and t.is_contiguous() and t.get_device() == self.device, \
            f"{name} must be a contiguous float32 tensor on k's device"
        assert t.shape == (heads, self.tokens), f"expected {name} of shape {(heads, self.tokens)}, got {tuple(t.shape)}"
        return t

    def call(self, fn, *args):
        cuda = self.torch.cuda
        if cuda.current_device() != self.device:
            with cuda.device(self.device):
                return self.call(fn, *args)
        status = fn(ctypes.byref(self.c), *args, self.torch._C._cuda_getCurrentRawStream(self.device))
        if status:
            _check(status)


def prompt_attention(q, k, v, seq_lens, out=None, lse=None):
    """Causal attention over packed prompts: q [tokens, n_q_heads, head_dim],
    k, v [tokens, n_kv_heads, head_dim] (bf16 or fp32; any strides of whole
    16-byte steps), seq_lens the sequences' lengths in order.  Returns (out,
    lse): out like q, lse float32 [n_q_heads, tokens].  No gradient."""
    p = _Prompt(k, seq_lens)
    p.queries(q)
    p.values(v)
    if out is None:
        out = p.torch.empty(q.shape, dtype=q.dtype, device=q.device)
    p.c.out_token_stride, p.c.out_head_stride = p.strides("out", out, q.shape[1])
    lse = p.rows("lse", lse, q.shape[1])
    p.call(load_library().kvq_prompt_attention, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
           lse.data_ptr())
    return out, lse


def prompt_weights(q, k, lse, seq_lens, last, out=None):
    """The attention weight every prompt token gathers from the last ``last``
    queries of its sequence, summed over the query heads of its KV head
    (float32 [n_kv_heads, tokens]); lse as prompt_attention returned it."""
    assert lse is not None, "lse is needed"
    p = _Prompt(k, seq_lens)
    p.queries(q)
    p.rows("lse", lse, q.shape[1])
    out = p.rows("out", out, p.heads)
    p.call(load_library().kvq_prompt_weights, q.data_ptr(), k.data_ptr(), lse.data_ptr(), index(last), out.data_ptr())
    return out


class Kept:
    """What evict kept.  k, v [rows, head_dim] and index [rows] hold one block
    [n_kv_heads, counts[i]] per sequence, back to back."""

    def __init__(self, k, v, index, counts, n_kv_heads):
        self.k, self.v, self.index, self.counts, self.n_kv_heads = k, v, index, counts, n_kv_heads

    def sequence(self, i):
        """(k, v, index) of sequence i: k, v [1, n_kv_heads, counts[i],
        head_dim] as KVQCache.append takes them, index [n_kv_heads, counts[i]]
        (positions in the sequence, rising)."""
        at, n = sum(self.counts[:i]) * self.n_kv_heads, self.counts[i]
        rows = slice(at, at + n * self.n_kv_heads)
        shape = (1, self.n_kv_heads, n, self.k.shape[1])
        return self.k[rows].view(shape), self.v[rows].view(shape), self.index[rows].view(self.n_kv_heads, n)


def evict(k, v, weights, seq_lens, keep, first=0, recent=0):
    """Keep ``keep`` tokens of every sequence and KV head (an int, cut to each
    sequence's length, or a count per sequence): the first ``first``, the last
    ``recent`` and the heaviest between, equal weights by lowest token.  k, v
    [tokens, n_kv_heads, head_dim]; weights float32 [n_kv_heads, tokens].
    Returns a Kept."""
    assert weights is not None, "weights are needed"
    p = _Prompt(k, seq_lens)
    p.values(v)
    p.rows("weights", weights, p.heads)
    if isinstance(keep, numbers.Integral):
        counts = [min(index(keep), index(n)) for n in seq_lens]
    else:
        counts = [index(n) for n in keep]
    assert len(counts) == len(seq_lens), f"expected {len(seq_lens)} counts in keep, got {len(counts)}"
    torch, device = p.torch, k.device
    # (counts past a sequence's length are refused by the call, not tried on the allocator)
    rows = sum(max(0, min(n, index(most))) for n, most in zip(counts, seq_lens)) * p.heads
    k_out = torch.empty((rows, p.dim), dtype=k.dtype, device=device)
    v_out = torch.empty_like(k_out)
    at = torch.empty(rows, dtype=torch.int32, device=device)
    p.call(load_library().kvq_evict, k.data_ptr(), v.data_ptr(), weights.data_ptr(),
           _counts(counts), index(first), index(recent), k_out.data_ptr(), v_out.data_ptr(),
           at.data_ptr())
    return Kept(k_out, v_out, at, counts, p.heads)


def kvq_kernel_launches() -> int:
    return load_library().kvq_kernel_launches()


def kvq_destroy(handle) -> None:
    if handle:
        load_library().kvq_destroy(handle)


# ---- owner object ------------------------------------------------------------

class KVQCache:
    """One layer's quantized cache on the current CUDA device.  The arena is a
    torch uint8 tensor kept alive by this object; every call runs on torch's
    current stream."""

    def __init__(self, batch, n_kv_heads, n_q_heads, head_dim, residual_len, group, qmax, capacity,
                 dtype="bf16", eps=1e-8, device=None, pool_blocks=0, segmented=False):
        """pool_blocks > 0 makes a paged cache: ``capacity`` then bounds each
        sequence's length and the pool of blocks is shared.  segmented=True
        makes a cache that flushes each append's whole overflow as one segment
        (``group`` is then unused)."""
        import torch
        self.torch = torch
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.dtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.cfg = make_config(batch, n_kv_heads, n_q_heads, head_dim, residual_len, group, qmax,
                               KVQ_BF16 if dtype == "bf16" else KVQ_FP32, eps)
        if isinstance(capacity, int):
            capacity = [capacity] * batch
        self.capacity = list(capacity)
        self.pool_blocks = pool_blocks
        self.segmented = segmented
        if segmented:
            self.nbytes = kvq_required_bytes_segmented(self.cfg, self.capacity)
        elif pool_blocks:
            self.nbytes = kvq_required_bytes_paged(self.cfg, self.capacity, pool_blocks)
        else:
            self.nbytes = kvq_required_bytes(self.cfg, self.capacity)
        self.arena = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=self.device)
        base = self.arena.data_ptr()
        self._base = (base + 255) // 256 * 256
        with torch.cuda.device(self.device):
            if segmented:
                self.handle = kvq_create_segmented(self.cfg, self.capacity, self._base, self.nbytes)
            elif pool_blocks:
                self.handle = kvq_create_paged(self.cfg, self.capacity, pool_blocks, self._base, self.nbytes)
            else:
                self.handle = kvq_create(self.cfg, self.capacity, self._base, self.nbytes)

    def _stream(self):
        return self.torch.cuda.current_stream(self.device).cuda_stream

    def _check_input(self, t, shape):
        assert t.is_cuda and t.device == self.device, "input must live on the cache's device"
        assert t.dtype == self.dtype and t.is_contiguous(), f"input must be contiguous {self.dtype}"
        assert tuple(t.shape) == tuple(shape), f"expected shape {tuple(shape)}, got {tuple(t.shape)}"

    def append(self, new_k, new_v, seq_begin=0):
        """new_k, new_v: [n_seqs, n_kv_heads, n_tokens, head_dim] on the device."""
        n_seqs, _, n, _ = new_k.shape
        shape = (n_seqs, self.cfg.n_kv_heads, n, self.cfg.head_dim)
        self._check_input(new_k, shape)
        self._check_input(new_v, shape)
        kvq_append(self.handle, new_k.data_ptr(), new_v.data_ptr(), n, seq_begin, n_seqs, self._stream())

    def append_kept(self, kept, seq_begin=0):
        """Append what evict kept: its sequence i to sequence seq_begin + i.
        Lengths, and a paged cache's blocks, are checked for all of them before
        the first is appended: all or none."""
        assert 0 <= seq_begin and seq_begin + len(kept.counts) <= self.cfg.batch, \
            f"{len(kept.counts)} sequences from {seq_begin} on do not fit a batch of {self.cfg.batch}"
        blocks = 0  # that the appends will take from the pool
        for i, n in enumerate(kept.counts):
            seq, state = seq_begin + i, self.seq_state(seq_begin + i)
            if state["total"] + n > self.capacity[seq]:
                raise KVQError(KVQ_ECAPACITY, f"sequence {seq}: {state['total']} + {n} tokens exceed its capacity")
            if n and self.pool_blocks:
                flushed = max(0, state["window"] + n - self.cfg.residual_len) // self.cfg.group
                if flushed > MAX_FLUSHED_GROUPS:
                    raise KVQError(KVQ_EUNSUPPORTED, f"sequence {seq} would flush {flushed} groups in one append; a "
                                                     f"paged cache takes at most {MAX_FLUSHED_GROUPS}")
                blocks += flushed
        if blocks and blocks > self.pool_state()[0]:
            raise KVQError(KVQ_ECAPACITY, f"the appends need {blocks} new blocks; the pool has {self.pool_state()[0]} free")
        for i, n in enumerate(kept.counts):
            if n:
                k, v, _ = kept.sequence(i)
                self.append(k, v, seq_begin + i)

    def decode_attention(self, q, out=None, kernel=0, chunk_pages=0, split_start=None, split_stop=None):
        """q: [batch, n_q_heads, head_dim]; returns float32 [batch, n_q_heads, head_dim]."""
        shape = (self.cfg.batch, self.cfg.n_q_heads, self.cfg.head_dim)
        self._check_input(q, shape)
        if out is None:
            out = self.torch.empty(shape, dtype=self.torch.float32, device=self.device)
        if kernel == 0 and chunk_pages == 0 and split_start is None and split_stop is None:
            kvq_decode_attention(self.handle, q.data_ptr(), out.data_ptr(), self._stream())
        else:
            kvq_decode_attention_ex(self.handle, q.data_ptr(), out.data_ptr(), self._stream(), kernel, chunk_pages,
                                    split_start, split_stop)
        return out

    def restore(self, seq_begin=0, n_seqs=None, t_stride=None, out_dtype="bf16", k_out=None, v_out=None):
        """Dense restored Keys and Values [n_seqs, n_kv_heads, t_stride, head_dim]
        (rows past each sequence's length are left as allocated)."""
        n_seqs = self.cfg.batch - seq_begin if n_seqs is None else n_seqs
        if t_stride is None:
            t_stride = max(1, max(self.seq_state(b)["total"] for b in range(seq_begin, seq_begin + n_seqs)))
        dt = self.torch.bfloat16 if out_dtype == "bf16" else self.torch.float32
        shape = (n_seqs, self.cfg.n_kv_heads, t_stride, self.cfg.head_dim)
        if k_out is None:
            k_out = self.torch.zeros(shape, dtype=dt, device=self.device)
        if v_out is None:
            v_out = self.torch.zeros(shape, dtype=dt, device=self.device)
        assert tuple(k_out.shape) == shape and tuple(v_out.shape) == shape
        assert k_out.dtype == dt and v_out.dtype == dt and k_out.is_contiguous() and v_out.is_contiguous()
        kvq_restore(self.handle, seq_begin, n_seqs, k_out.data_ptr(), v_out.data_ptr(), t_stride,
                    KVQ_BF16 if out_dtype == "bf16" else KVQ_FP32, self._stream())
        return k_out, v_out

    def dense_decode_attention(self, k, v, q, out=None):
        """Standard decode attention over dense restored k, v [batch, n_kv_heads,
        t_stride, head_dim] (bf16), lengths from this cache."""
        shape = (self.cfg.batch, self.cfg.n_q_heads, self.cfg.head_dim)
        self._check_input(q, shape)
        assert k.shape == v.shape and k.dim() == 4 and k.shape[:2] == (self.cfg.batch, self.cfg.n_kv_heads)
        assert k.dtype == self.dtype and v.dtype == self.dtype and k.is_contiguous() and v.is_contiguous()
        if out is None:
            out = self.torch.empty(shape, dtype=self.torch.float32, device=self.device)
        kvq_dense_decode_attention(self.handle, k.data_ptr(), v.data_ptr(), k.shape[2], q.data_ptr(), out.data_ptr(),
                                   self._stream())
        return out

    def decode_step(self, new_k, new_v, q, out=None, kernel=0, split_start=None, split_stop=None):
        """Append one token per sequence (new_k, new_v: [batch, n_kv_heads, 1,
        head_dim]) and attend with q [batch, n_q_heads, head_dim]."""
        shape = (self.cfg.batch, self.cfg.n_kv_heads, 1, self.cfg.head_dim)
        self._check_input(new_k, shape)
        self._check_input(new_v, shape)
        qshape = (self.cfg.batch, self.cfg.n_q_heads, self.cfg.head_dim)
        self._check_input(q, qshape)
        if out is None:
            out = self.torch.empty(qshape, dtype=self.torch.float32, device=self.device)
        kvq_decode_step(self.handle, new_k.data_ptr(), new_v.data_ptr(), q.data_ptr(), out.data_ptr(), self._stream(),
                        kernel, split_start, split_stop)
        return out

    def bytes(self):
        return kvq_bytes(self.handle)

    def release(self, seq_begin=0, n_seqs=1):
        kvq_release(self.handle, seq_begin, n_seqs)

    def pool_state(self):
        """(free blocks, pool blocks) of a paged cache."""
        return kvq_pool_state(self.handle)

    def seq_state(self, seq):
        return kvq_seq_state(self.handle, seq)

    def export_unit(self, seq, kv_head):
        """Host numpy copies of one unit: dict of k_codes, v_codes, k_scales,
        v_scales, window_k, window_v (token order)."""
        import numpy as np
        st = self.seq_state(seq)
        Q, W, D = st["quantized"], st["window"], self.cfg.head_dim
        arrs = {"k_codes": np.zeros((Q, D), np.int8), "v_codes": np.zeros((Q, D), np.int8),
                "k_scales": np.zeros((st["n_groups"], D), np.float32), "v_scales": np.zeros((Q,), np.float32),
                "window_k": np.zeros((W, D), np.float32), "window_v": np.zeros((W, D), np.float32)}
        view = kvq_unit_view(*[a.ctypes.data for a in arrs.values()])
        kvq_export_unit(self.handle, seq, kv_head, view, self._stream())
        return arrs

    def export_pages(self, seq, kv_head):
        import numpy as np
        st = self.seq_state(seq)
        n = (st["quantized"] // self.cfg.group) * kvq_page_bytes(self.cfg)
        buf = np.zeros(max(n, 1), np.uint8)
        kvq_export_pages(self.handle, seq, kv_head, buf.ctypes.data, buf.nbytes, self._stream())
        return buf[:n].tobytes()

    def device_status(self):
        return kvq_device_status(self.handle, self._stream())

    def close(self):
        if getattr(self, "handle", None):
            kvq_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
