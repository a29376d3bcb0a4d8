"""Refusals of the prompt operators, before any launch and without a GPU: every
bad shape, stride, length and pointer is an error code, and a prompt without
tokens is no work.  The pointers are never dereferenced."""

import ctypes

import pytest

kvq = pytest.importorskip("quantized_kv_cache_02_gb300")
B = kvq.binding

PTR = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)


def prompt(lens=(5, 0, 3), **kw):
    a = dict(n_q_heads=8, n_kv_heads=2, head_dim=64, dtype=B.KVQ_BF16, n_tokens=8, n_seqs=len(lens))
    a.update(kw)
    arr = (ctypes.c_int64 * max(1, len(lens)))(*lens)
    p = B.kvq_prompt(a["n_seqs"], a["n_q_heads"], a["n_kv_heads"], a["head_dim"], a["dtype"], arr, a["n_tokens"])
    for t, h in (("q", 8), ("k", 2), ("v", 2), ("out", 8)):
        setattr(p, f"{t}_token_stride", a.get(f"{t}_token_stride", h * 64))
        setattr(p, f"{t}_head_stride", a.get(f"{t}_head_stride", 64))
    return p, arr


def attention(p, q=PTR, k=PTR, v=PTR, out=PTR, lse=None):
    return kvq.load_library().kvq_prompt_attention(p and ctypes.byref(p), q, k, v, out, lse, None)


def weights(p, q=PTR, k=PTR, lse=PTR, last=4, w=PTR):
    return kvq.load_library().kvq_prompt_weights(p and ctypes.byref(p), q, k, lse, last, w, None)


def evict(p, keep=(2, 0, 3), first=0, recent=0, k=PTR, v=PTR, w=PTR, ko=PTR, vo=PTR, index=PTR):
    keep = keep and (ctypes.c_int64 * len(keep))(*keep)
    return kvq.load_library().kvq_evict(p and ctypes.byref(p), k, v, w, keep, first, recent, ko, vo, index, None)


SHAPES = [(dict(n_seqs=0), B.KVQ_EINVAL), (dict(n_kv_heads=0), B.KVQ_EINVAL), (dict(n_q_heads=0), B.KVQ_EINVAL),
          (dict(n_q_heads=7), B.KVQ_EINVAL), (dict(n_q_heads=18), B.KVQ_EUNSUPPORTED),
          (dict(head_dim=8), B.KVQ_EUNSUPPORTED), (dict(head_dim=72), B.KVQ_EUNSUPPORTED),
          (dict(head_dim=272), B.KVQ_EUNSUPPORTED), (dict(dtype=2), B.KVQ_EINVAL), (dict(n_tokens=7), B.KVQ_EINVAL),
          (dict(n_tokens=-1), B.KVQ_EINVAL), (dict(n_tokens=(1 << 30) + 1), B.KVQ_EINVAL),
          (dict(lens=(5, -1, 3)), B.KVQ_EINVAL), (dict(lens=(1 << 62, 1 << 62, 1 << 62)), B.KVQ_EINVAL),
          (dict(n_kv_heads=70000, n_q_heads=70000), B.KVQ_EUNSUPPORTED)]


@pytest.mark.parametrize("bad,status", SHAPES)
def test_shapes_and_lengths(bad, status):
    p, keep_alive = prompt(**bad)
    assert attention(p) == status
    assert weights(p) == status
    assert evict(p) == status
    assert kvq.load_library().kvq_last_error()


@pytest.mark.parametrize("bad,status", [
    (dict(k_token_stride=60), B.KVQ_EINVAL), (dict(k_token_stride=132), B.KVQ_EINVAL),
    (dict(k_token_stride=0), B.KVQ_EINVAL), (dict(k_head_stride=0), B.KVQ_EINVAL),
    (dict(k_head_stride=-64), B.KVQ_EINVAL), (dict(k_head_stride=68), B.KVQ_EINVAL),
    (dict(k_token_stride=1 << 40), B.KVQ_EUNSUPPORTED)])
def test_strides(bad, status):
    p, keep_alive = prompt(**bad)
    assert attention(p) == weights(p) == evict(p) == status


def test_rows_of_out_do_not_overlap():
    p, keep_alive = prompt(out_token_stride=64, out_head_stride=64)
    assert attention(p) == B.KVQ_EINVAL
    p, keep_alive = prompt(out_token_stride=448, out_head_stride=64)
    assert attention(p) == B.KVQ_EINVAL
    assert b"overlap" in kvq.load_library().kvq_last_error()
    # strides of a dimension of one entry are not looked at
    p, keep_alive = prompt(lens=(1,), n_tokens=1, k_token_stride=0, k_head_stride=60)
    assert attention(p) == B.KVQ_EINVAL and b"k strides" in kvq.load_library().kvq_last_error()


def test_pointers():
    p, keep_alive = prompt()
    null = ctypes.c_void_p()
    for bad in (null, ODD):
        for name in ("q", "k", "v", "out"):
            assert attention(p, **{name: bad}) == B.KVQ_EINVAL, name
        for name in ("q", "k"):
            assert weights(p, **{name: bad}) == B.KVQ_EINVAL, name
        for name in ("k", "v", "ko", "vo"):
            assert evict(p, **{name: bad}) == B.KVQ_EINVAL, name
    assert attention(None) == weights(None) == evict(None) == B.KVQ_EINVAL
    p.seq_lens = None
    assert attention(p) == weights(p) == evict(p) == B.KVQ_EINVAL


def test_counts():
    p, keep_alive = prompt()
    assert weights(p, last=0) == B.KVQ_EINVAL
    assert evict(p, keep=None) == B.KVQ_EINVAL
    for bad in [dict(keep=(6, 0, 3)), dict(keep=(-1, 0, 3)), dict(keep=(2, 1, 3)), dict(first=-1), dict(recent=-1),
                dict(first=3), dict(recent=3), dict(first=1, recent=2), dict(first=1 << 62, recent=1 << 62),
                dict(keep=(0, 0, 3), recent=1)]:
        assert evict(p, **bad) == B.KVQ_EINVAL, bad


def test_a_prompt_without_tokens_is_no_work():
    p, keep_alive = prompt(lens=(0, 0))
    null = ctypes.c_void_p()
    before = kvq.kvq_kernel_launches()
    assert attention(p, null, null, null, null) == B.KVQ_OK
    assert weights(p, null, null, null, 1, null) == B.KVQ_OK
    assert evict(p, (0, 0), 0, 0, null, null, null, null, null, null) == B.KVQ_OK
    p, keep_alive = prompt()
    assert evict(p, (0, 0, 0), 0, 0, null, null, null, null, null, null) == B.KVQ_OK
    assert kvq.kvq_kernel_launches() == before


def test_prompt_struct_matches_header(tmp_path):
    import test_abi_layout as L
    structs, L.STRUCTS = L.STRUCTS, [B.kvq_prompt]
    try:
        L.test_binding_structs_match_header(tmp_path)
    finally:
        L.STRUCTS = structs
