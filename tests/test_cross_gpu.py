"""Cross attention against its formula in 64 bits.

Tolerances as of the causal attention (tests/test_prompt_gpu.py): with u = 2^-24 a
score is off by at most ds = (d + 8) u max_j sum_c |q_c k_c| / sqrt(d), which moves
every weight by the factor 1 +- ds; 2^x is good to 2^-21; sums over n states add n u;
with A = sum_j p_j |v_j|, |d out| <= (2 ds + 2 n u + 2^-20) A.  For bf16 the weights
are rounded once where the tensor cores take them (2^-8 of each) and so is the output:
2^-8 (A + |out|) more.
"""

import math

import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


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


def inputs(torch, nq, nkv, hq, hkv, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = getattr(torch, dtype)
    q = torch.randn(nq, hq, d, generator=g, device="cuda").to(dt)
    k = torch.randn(nkv, hkv, d, generator=g, device="cuda")
    k = (k * torch.exp(0.5 * torch.randn(hkv, d, generator=g, device="cuda"))).to(dt)
    v = (torch.randn(nkv, hkv, d, generator=g, device="cuda") + 0.25).to(dt)
    return q, k, v


def check(torch, out, lse, q, k, v, q_lens, kv_lens, kv_starts=None):
    hq, d = q.shape[1:]
    g = hq // k.shape[1]
    i = j = 0
    for b, (n, m) in enumerate(zip(q_lens, kv_lens)):
        at = j if kv_starts is None else kv_starts[b]
        for h in range(hq if n else 0):
            got = out[i:i + n, h].double()
            if m == 0:
                assert (got == 0).all() and (lse is None or (lse[h, i:i + n] == -math.inf).all())
                continue
            kk, vv = k[at:at + m, h // g].double(), v[at:at + m, h // g].double()
            z = q[i:i + n, h].double() @ kk.T / math.sqrt(d)
            ds = (d + 8) * U * (q[i:i + n, h].double().abs() @ kk.abs().T / math.sqrt(d)).amax(1)
            e = torch.logsumexp(z, 1)
            p = torch.exp(z - e[:, None])
            ref, size = p @ vv, p @ vv.abs()
            tol = (2 * ds[:, None] + 2 * m * U + 2.0 ** -20) * size + 1e-37
            if out.dtype == torch.bfloat16:
                tol += 2.0 ** -8 * (size + ref.abs())
            bad = (got - ref).abs() - tol
            assert torch.isfinite(got).all() and bad.max() <= 0, (b, h, n, m, int(bad.argmax()), float(bad.max()))
            if lse is not None:
                off = (lse[h, i:i + n].double() - e).abs()
                assert (off <= 2 * ds + m * U + 2.0 ** -20 + 4 * U * e.abs()).all(), (b, h, n, m, float(off.max()))
        i, j = i + n, j + m


SHAPES = [(8, 2, 64, "bfloat16"), (4, 4, 128, "bfloat16"), (7, 1, 128, "bfloat16"), (8, 1, 64, "bfloat16"),
          (6, 2, 80, "bfloat16"), (2, 1, 256, "bfloat16"), (2, 2, 16, "bfloat16"), (5, 1, 128, "float32"),
          (4, 2, 16, "float32"), (8, 1, 256, "float32"), (3, 3, 64, "float32")]


@pytest.mark.parametrize("hq,hkv,d,dtype", SHAPES)
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([1], [1]), ([1], [1000]), ([3], [0]), ([130], [127]), ([64, 0, 1, 257], [129, 5, 640, 1]), ([5, 1, 2], [0, 300, 64]),
    ([1] * 9, [7, 0, 64, 65, 128, 1, 2, 1500, 333]), ([31, 200], [500, 128])])
def test_shapes(torch, kvq, hq, hkv, d, dtype, q_lens, kv_lens):
    q, k, v = inputs(torch, sum(q_lens) + 2, sum(kv_lens) + 3, hq, hkv, d, dtype)
    out, lse = torch.full_like(q, 7.0), torch.full((hq, len(q)), 7.0, device="cuda")
    # what lies behind the sequences stays, and is not looked at
    q[sum(q_lens):] = math.nan
    k[sum(kv_lens):] = math.nan
    v[sum(kv_lens):] = math.inf
    kvq.cross_attention(q, k, v, q_lens, kv_lens, out=out, lse=lse)
    check(torch, out, lse, q, k, v, q_lens, kv_lens)
    assert (out[sum(q_lens):] == 7.0).all() and (lse[:, sum(q_lens):] == 7.0).all()
    again, lse2 = kvq.cross_attention(q, k, v, q_lens, kv_lens)
    assert torch.equal(again[:sum(q_lens)], out[:sum(q_lens)]) and torch.equal(lse2[:, :sum(q_lens)], lse[:, :sum(q_lens)])
    assert kvq.prompt_status() == 0


@pytest.mark.parametrize("hq,hkv,d,dtype", [(8, 2, 128, "bfloat16"), (4, 4, 64, "bfloat16"), (6, 2, 80, "bfloat16"),
                                            (4, 2, 128, "float32")])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_neighbours_and_later_states_stay_out(torch, kvq, hq, hkv, d, dtype, n):
    """Padded batches and shared states: whatever lies between the states is not seen."""
    lens, starts, rows = [100, 1, 333, 100, 0], [600, 7, 200, 600, 0], 800
    q, k, v = inputs(torch, 5 * n, rows, hq, hkv, d, dtype)
    seen = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for a, m in zip(starts, lens):
        seen[a:a + m] = True
    k[~seen], v[~seen] = math.nan, math.inf
    k[~seen][::2] = -math.inf
    out, lse = kvq.cross_attention(q, k, v, [n] * 5, lens, starts)
    check(torch, out, lse, q, k, v, [n] * 5, lens, starts)
    # the same states, the same queries: the same bits
    q[3 * n:4 * n] = q[:n]
    out, lse = kvq.cross_attention(q, k, v, [n] * 5, lens, starts)
    assert torch.equal(out[3 * n:4 * n], out[:n]) and torch.equal(lse[:, 3 * n:4 * n], lse[:, :n])


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n", [1, 9, 200])
def test_strides(torch, kvq, dtype, n):
    """A fused key-value projection, head-major queries and a padded output."""
    hq, hkv, d, m = 8, 2, 64, 150
    q, k, v = inputs(torch, n, m, hq, hkv, d, dtype)
    fused = torch.stack((k, v), 1)
    out = torch.zeros(n, hq, 2 * d, device="cuda", dtype=q.dtype)
    kvq.cross_attention(q.transpose(0, 1).contiguous().transpose(0, 1), fused[:, 0], fused[:, 1], [n], [m], out=out[..., :d])
    want, _ = kvq.cross_attention(q, k, v, [n], [m])
    assert torch.equal(out[..., :d], want) and (out[..., d:] == 0).all()
    major = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (k, v)]
    assert torch.equal(kvq.cross_attention(q, *major, [n], [m])[0], want)


@pytest.mark.parametrize("dtype,d", [("bfloat16", 128), ("bfloat16", 64), ("float32", 128), ("bfloat16", 48)])
@pytest.mark.parametrize("n", [1, 20, 260])
def test_infinities(torch, kvq, dtype, d, n):
    """A state whose scores are minus infinity weighs nothing; a row of only such is
    NaN; an infinite Value is infinite for everyone who sees it, and only in its channel."""
    hq, m = 2, 140
    q, k, v = inputs(torch, n, m, hq, hq, d, dtype)
    q = q.abs() + 0.5
    k[:130] = -math.inf
    v[3, :, 1] = 5.0
    out, lse = kvq.cross_attention(q, k, v, [n], [m])
    check(torch, out, lse, q, k[130:], v[130:], [n], [10])
    out, lse = kvq.cross_attention(q, k, v, [n], [130])
    assert out.isnan().all() and (lse == -math.inf).all()
    q, k, v = inputs(torch, n, m, hq, hq, d, dtype, 1)
    v[5, 0, 2] = math.inf
    v[139, 1, 3] = math.nan
    out, _ = kvq.cross_attention(q, k, v, [n], [m])
    assert (out[:, 0, 2] == math.inf).all() and out[:, 1, 3].isnan().all()
    out[:, 0, 2] = out[:, 1, 3] = 0
    assert torch.isfinite(out).all()


def test_many_sequences(torch, kvq):
    """More sequences than a launch holds, with and without queries or states."""
    g = torch.Generator().manual_seed(3)
    for dtype, d in (("bfloat16", 64), ("float32", 32)):
        q_lens = torch.randint(0, 4, (600,), generator=g).tolist()
        kv_lens = torch.randint(0, 30, (600,), generator=g).tolist()
        q_lens[17], kv_lens[500] = 400, 1000
        q, k, v = inputs(torch, sum(q_lens), sum(kv_lens), 2, 1, d, dtype)
        out, lse = kvq.cross_attention(q, k, v, q_lens, kv_lens)
        check(torch, out, lse, q, k, v, q_lens, kv_lens)


@pytest.mark.parametrize("n", [1, 100])
def test_streams_and_graphs(torch, kvq, n):
    """Two calls at once on streams of their own, and a captured call replayed on other inputs."""
    args = [inputs(torch, n, 700, 8, 2, 128, "bfloat16", s) for s in range(2)]
    want = [kvq.cross_attention(*a, [n], [700])[0] for a in args]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in args], [None] * 2
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = kvq.cross_attention(*args[i], [n], [700])[0]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    q, k, v = (t.clone() for t in args[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = kvq.cross_attention(q, k, v, [n], [700])
    for i in (1, 0):
        for t, s in zip((q, k, v), args[i]):
            t.copy_(s)
        graph.replay()
        assert torch.equal(out, want[i])


def test_no_work_and_refusals(torch, kvq):
    q, k, v = inputs(torch, 8, 12, 4, 2, 64, "bfloat16")
    before = kvq.kvq_kernel_launches()
    out, lse = kvq.cross_attention(q[:0], k, v, [0, 0], [5, 7])
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0) and kvq.kvq_kernel_launches() == before
    out, lse = kvq.cross_attention(q, k[:0], v[:0], [8], [0])
    assert (out == 0).all() and (lse == -math.inf).all()
    for args in [(q.half(), k, v, [8], [12]), (q, k.float(), v, [8], [12]), (q, k, v[:11], [8], [12]),
                 (q, k, v, [8], [6, 6]), (q, k, v, [8], [12], [0, 0]), (q[..., :32], k, v, [8], [12])]:
        with pytest.raises(AssertionError):
            kvq.cross_attention(*args)
    for args in [([9], [12]), ([8], [13]), ([8], [-1]), ([8], [12], [1]), ([8], [1], [-1]), ([4, 5], [1, 1])]:
        with pytest.raises(kvq.KVQError):
            kvq.cross_attention(q, k, v, *args)
    with pytest.raises(TypeError):
        kvq.cross_attention(q, k, v, [8], [1.5])


@pytest.mark.parametrize("hq,hkv,d,dtype", [(8, 2, 64, "bfloat16"), (7, 1, 128, "bfloat16"), (2, 2, 128, "bfloat16"),
                                            (5, 1, 64, "bfloat16"), (4, 2, 128, "float32"), (3, 1, 80, "bfloat16")])
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([1], [5000]), ([2, 1, 1], [1027, 0, 2500]), ([100], [5000]), ([33, 1, 70], [1500, 2000, 130]),
    ([40, 50, 60], [0, 3000, 129]), ([64], [1025]), ([300, 2], [700, 4100]), ([129], [2049])])
def test_split_states(torch, kvq, hq, hkv, d, dtype, q_lens, kv_lens):
    """Few tiles over many states: clusters of CTAs, some without states, join their results."""
    q, k, v = inputs(torch, sum(q_lens) + 1, sum(kv_lens) + 5, hq, hkv, d, dtype, 9)
    out, lse = torch.full_like(q, 7.0), torch.full((hq, len(q)), 7.0, device="cuda")
    k[sum(kv_lens):], v[sum(kv_lens):] = math.nan, math.inf
    kvq.cross_attention(q, k, v, q_lens, kv_lens, out=out, lse=lse)
    check(torch, out, lse, q, k, v, q_lens, kv_lens)
    assert (out[sum(q_lens):] == 7.0).all() and (lse[:, sum(q_lens):] == 7.0).all()
    again, lse2 = kvq.cross_attention(q, k, v, q_lens, kv_lens)
    assert torch.equal(again[:-1], out[:-1]) and torch.equal(lse2[:, :-1], lse[:, :-1]) and kvq.prompt_status() == 0


def test_split_states_minus_infinity(torch, kvq):
    """Ranks that see only scores of minus infinity weigh nothing."""
    for n in (1, 90):
        q, k, v = inputs(torch, n, 3000, 2, 2, 128, "bfloat16", 4)
        q = q.abs() + 0.5
        k[:2900] = -math.inf
        out, lse = kvq.cross_attention(q, k, v, [n], [3000])
        check(torch, out, lse, q, k[2900:], v[2900:], [n], [100])
        out, lse = kvq.cross_attention(q, k, v, [n], [2900])
        assert out.isnan().all() and (lse == -math.inf).all()


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 64), (16, 4, 128), (7, 1, 128), (6, 6, 128)])
@pytest.mark.parametrize("q_lens,kv_lens", [([9000], [100]), ([20000], [128]), ([5000, 3000, 1, 6000], [300, 0, 40, 129]),
                                            ([2500] * 8, [64, 700, 128, 1, 256, 513, 16, 1000])])
def test_more_tiles_than_ctas(torch, kvq, hq, hkv, d, q_lens, kv_lens):
    """CTAs that take tile after tile, of one block of states and of several."""
    q, k, v = inputs(torch, sum(q_lens), sum(kv_lens), hq, hkv, d, "bfloat16", 5)
    for _ in range(3):
        out, lse = kvq.cross_attention(q, k, v, q_lens, kv_lens)
    check(torch, out, lse, q, k, v, q_lens, kv_lens)
    assert kvq.prompt_status() == 0


@pytest.mark.parametrize("n", [1, 200])
@pytest.mark.parametrize("dtype,d", [("bfloat16", 64), ("float32", 64)])
def test_offsets_past_32_bits(torch, kvq, dtype, d, n):
    """States whose rows lie a megabyte apart: the last ones past 2^32 elements."""
    m, step = 4200, 1 << 20
    dt = getattr(torch, dtype)
    buffer = torch.empty(m * step, dtype=dt, device="cuda")
    k, v = (buffer.as_strided((m, 2, d), (step, d, 1), at) for at in (0, step // 2))
    q, kk, vv = inputs(torch, n, m, 4, 2, d, dtype)
    k.copy_(kk), v.copy_(vv)
    out, lse = kvq.cross_attention(q, k, v, [n], [m])
    want, want_lse = kvq.cross_attention(q, kk, vv, [n], [m])
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    check(torch, out, lse, q, kk, vv, [n], [m])


@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (8, 2, 128)])
def test_mixed_sequences(torch, kvq, hq, hkv, d):
    """One call of two launches: a token, few queries over many states, many queries over
    fewer."""
    q_lens, kv_lens = [1500, 40, 1, 60, 2, 700], [200, 4000, 1000, 6000, 0, 129]
    q, k, v = inputs(torch, sum(q_lens), sum(kv_lens), hq, hkv, d, "bfloat16", 8)
    before = kvq.kvq_kernel_launches()
    out, lse = kvq.cross_attention(q, k, v, q_lens, kv_lens)
    assert kvq.kvq_kernel_launches() == before + 2
    check(torch, out, lse, q, k, v, q_lens, kv_lens)
    again, _ = kvq.cross_attention(q, k, v, q_lens, kv_lens)
    assert torch.equal(out, again) and kvq.prompt_status() == 0
