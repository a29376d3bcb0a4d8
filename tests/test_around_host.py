"""Refusals of the cross attention, the rotary positions and the fork, before any
launch and without a GPU.  The pointers are never dereferenced."""

import ctypes
import math

import pytest

kvq = pytest.importorskip("quantized_kv_cache_02_gb300")
B = kvq.binding

PTR = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)
NULL = ctypes.c_void_p()


def i64(values):
    return (ctypes.c_int64 * max(1, len(values)))(*values)


def refusal():
    return kvq.load_library().kvq_last_error()


def cross(q_lens=(5, 0, 3), kv_lens=(4, 2, 6), kv_starts=None, **kw):
    a = dict(n_q_heads=8, n_kv_heads=2, head_dim=64, dtype=B.KVQ_BF16, n_q_tokens=8, n_kv_tokens=12, n_seqs=len(q_lens))
    a.update(kw)
    keep = [i64(q_lens), i64(kv_lens)]
    c = B.kvq_cross(a["n_seqs"], a["n_q_heads"], a["n_kv_heads"], a["head_dim"], a["dtype"],
                    *[ctypes.addressof(x) for x in keep])
    if kv_starts is not None:
        keep.append(i64(kv_starts))
        c.kv_starts = ctypes.addressof(keep[-1])
    c.n_q_tokens, c.n_kv_tokens = a["n_q_tokens"], a["n_kv_tokens"]
    for t, h in (("q", 8), ("k", 2), ("v", 2), ("out", 8)):
        setattr(c, f"{t}_token_stride", a.get(f"{t}_token_stride", h * 64))
        setattr(c, f"{t}_head_stride", a.get(f"{t}_head_stride", 64))
    return c, keep


def attend(c, q=PTR, k=PTR, v=PTR, out=PTR, lse=None):
    return kvq.load_library().kvq_cross_attention(c and ctypes.byref(c), q, k, v, out, lse, None)


@pytest.mark.parametrize("bad,status", [
    (dict(n_seqs=0), 1), (dict(n_kv_heads=0), 1), (dict(n_q_heads=0), 1), (dict(n_q_heads=7), 1),
    (dict(n_q_heads=18), 5), (dict(head_dim=8), 5), (dict(head_dim=72), 5), (dict(head_dim=272), 5), (dict(dtype=2), 1),
    (dict(n_q_tokens=7), 1), (dict(n_q_tokens=-1), 1), (dict(n_q_tokens=(1 << 30) + 1), 1), (dict(n_kv_tokens=11), 1),
    (dict(n_kv_tokens=-1), 1), (dict(n_kv_tokens=(1 << 30) + 1), 1), (dict(q_lens=(5, -1, 3)), 1),
    (dict(kv_lens=(4, -1, 3)), 1), (dict(q_lens=(1 << 62,) * 3), 1), (dict(kv_lens=(1 << 62,) * 3), 1),
    (dict(kv_starts=(0, 0, 7)), 1), (dict(kv_starts=(-1, 0, 0)), 1), (dict(kv_starts=(0, 1 << 62, 0)), 1),
    (dict(kv_starts=(0, 13, 0), kv_lens=(1, 0, 1)), 1), (dict(n_kv_heads=70000, n_q_heads=70000), 5),
    (dict(q_token_stride=60), 1), (dict(k_token_stride=132), 1), (dict(v_token_stride=0), 1), (dict(k_head_stride=-64), 1),
    (dict(v_head_stride=68), 1), (dict(k_token_stride=1 << 40), 5), (dict(out_token_stride=64), 1)])
def test_cross(bad, status):
    c, keep_alive = cross(**bad)
    assert attend(c) == status and refusal()


def test_cross_pointers():
    c, keep_alive = cross()
    for bad in (NULL, ODD):
        for name in ("q", "k", "v", "out"):
            assert attend(c, **{name: bad}) == B.KVQ_EINVAL and refusal().startswith(name.encode()), name
    assert attend(None) == B.KVQ_EINVAL
    for name in ("q_lens", "kv_lens"):
        c, keep_alive = cross()
        setattr(c, name, None)
        assert attend(c) == B.KVQ_EINVAL
    # no states at all: k and v are not looked at
    c, keep_alive = cross(kv_lens=(0, 2, 0), k_token_stride=1)
    assert attend(c, k=NULL, v=NULL, out=NULL) == B.KVQ_EINVAL and refusal().startswith(b"out")


def test_cross_without_queries_is_no_work():
    c, keep_alive = cross(q_lens=(0, 0))
    before = kvq.kvq_kernel_launches()
    assert attend(c, NULL, NULL, NULL, NULL) == B.KVQ_OK and kvq.kvq_kernel_launches() == before


def turn(positions=PTR, position_bytes=8, ps=2, pa=1, tokens=8, dtype=B.KVQ_BF16, n=2, plan=None, frequency=(1.0, 0.5),
         axis=(0, 1), tensor=None, **kw):
    a = dict(head_dim=64, n_axes=2, n_pairs=len(frequency), interleaved=0)
    a.update(kw)
    p = B.kvq_rotary_plan(a["head_dim"], a["n_axes"], a["n_pairs"], a["interleaved"],
                          (ctypes.c_double * 2)(*frequency), (ctypes.c_int32 * 2)(*axis))
    t = (B.kvq_rotary_tensor * 2)(*[B.kvq_rotary_tensor(PTR, ctypes.c_void_p(1 << 30), 512, 64, 512, 64, 8) for _ in range(2)])
    for field, value in (tensor or {}).items():
        setattr(t[1], field, value)
    return kvq.load_library().kvq_rotary(ctypes.byref(p) if plan is None else plan, positions, position_bytes, ps, pa,
                                         tokens, dtype, t, n, 0, None)


@pytest.mark.parametrize("bad,status", [
    (dict(head_dim=72), 5), (dict(head_dim=0), 5), (dict(head_dim=272), 5), (dict(n_axes=0), 1), (dict(n_axes=5), 1),
    (dict(n_pairs=0), 1), (dict(n_pairs=33), 1), (dict(frequency=(math.nan, 1.0)), 1), (dict(frequency=(math.inf, 1.0)), 1),
    (dict(frequency=(1.0, -2.0 ** 21)), 1), (dict(axis=(0, 2)), 1), (dict(axis=(-1, 0)), 1), (dict(dtype=2), 1),
    (dict(position_bytes=2), 1), (dict(tokens=-1), 1), (dict(tokens=(1 << 30) + 1), 1), (dict(n=0), 1), (dict(n=3), 1),
    (dict(ps=-1), 1), (dict(pa=-1), 1), (dict(ps=(1 << 30) + 1), 1), (dict(positions=NULL), 1),
    (dict(positions=ctypes.c_void_p((1 << 20) + 4)), 1), (dict(tensor=dict(n_heads=0)), 1),
    (dict(tensor=dict(n_heads=65536)), 1), (dict(tensor=dict(input=0)), 1), (dict(tensor=dict(out=8)), 1),
    (dict(tensor=dict(in_token_stride=60)), 1), (dict(tensor=dict(out_head_stride=0)), 1),
    (dict(tensor=dict(in_token_stride=1 << 40)), 5), (dict(tensor=dict(out_token_stride=64)), 1),
    (dict(tensor=dict(out=1 << 20, out_token_stride=1024)), 1), (dict(tensor=dict(out=1 << 20, out_head_stride=72)), 1)])
def test_rotary(bad, status):
    assert turn(**bad) == status and refusal()


def test_rotary_null_and_no_tokens():
    assert turn(plan=ctypes.POINTER(B.kvq_rotary_plan)()) == B.KVQ_EINVAL
    before = kvq.kvq_kernel_launches()
    assert turn(tokens=0, positions=NULL) == B.KVQ_OK and kvq.kvq_kernel_launches() == before
    # one token, one axis: their strides are not looked at
    assert turn(tokens=1, ps=-5, pa=-5, n_axes=1, axis=(0, 0), tensor=dict(in_token_stride=3)) != B.KVQ_OK
    assert b"strides" not in refusal()


def test_rotary_sections():
    plan = kvq.Rotary.sections(64, [3, 2], theta=100.0)
    assert plan.axes == [0, 0, 0, 1, 1] and plan.n_axes == 2
    assert plan.frequencies == pytest.approx([100.0 ** (-i / 5) for i in range(5)])
    plan = kvq.Rotary.sections(64, [3, 2], theta=100.0, restart=True, interleaved=True)
    assert plan.frequencies == pytest.approx([1, 100.0 ** (-1 / 3), 100.0 ** (-2 / 3), 1, 0.1]) and plan.interleaved
    for bad in [dict(frequencies=[]), dict(frequencies=[1.0], axes=[0, 1]), dict(frequencies=[1.0], axes=[-1])]:
        with pytest.raises(AssertionError):
            kvq.Rotary(64, **bad)
    with pytest.raises(TypeError):
        kvq.Rotary(64, [1.0], [0.5])


def test_fork_without_a_cache():
    pair = (ctypes.c_int32 * 1)(0)
    assert kvq.load_library().kvq_fork(None, pair, pair, 1, None) == B.KVQ_EINVAL


def test_structs_match_header(tmp_path):
    import test_abi_layout as L
    structs, L.STRUCTS = L.STRUCTS, [B.kvq_cross, B.kvq_rotary_plan, B.kvq_rotary_tensor]
    try:
        L.test_binding_structs_match_header(tmp_path)
    finally:
        L.STRUCTS = structs
