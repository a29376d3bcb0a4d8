"""The prompt operators against their formulas in 64 bits.

Tolerances, per element, from the arithmetic.  With u = 2^-24 (half an fp32
step), a score's products and sum are off by at most
    ds = (d + 8) u max_j sum_c |q_c k_c| / sqrt(d)
(one rounding a product and addition, a few for the scale and the exponent's
argument), which moves every softmax weight by the factor 1 +- ds, and 2^x is
good to 2^-21.  Sums over n keys add at most n u.  For bf16 each weight is
rounded once (2^-8 of it) and so is the output (2^-8 of it).  With
A = sum_j p_j |v_j| that gives |d out| <= (2 ds + 2 n u + 2^-20) A, plus
2^-8 (A + |out|) for bf16.  Maxima that differ between steps only rescale by
powers that are rounded like the weights.
"""

import math

import numpy as np
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


def inputs(torch, tokens, hq, hkv, d, dtype, seed=0, q_gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = getattr(torch, dtype)
    q = (torch.randn(tokens, hq, d, generator=g, device="cuda") * q_gain).to(dt)
    k = torch.randn(tokens, hkv, d, generator=g, device="cuda")
    k = (k * torch.exp(torch.randn(hkv, d, generator=g, device="cuda"))).to(dt)
    v = (torch.randn(tokens, hkv, d, generator=g, device="cuda") + 0.25).to(dt)
    return q, k, v


def scores(torch, q, k, first=0):
    """z, p, lse, ds of one head of one sequence; queries from row ``first`` on."""
    d, n = q.shape[1], k.shape[0]
    z = q[first:].double() @ k.double().T / math.sqrt(d)
    size = (q[first:].double().abs() @ k.double().abs().T / math.sqrt(d)).amax(1)
    hidden = torch.arange(n, device="cuda")[None, :] > torch.arange(first, n, device="cuda")[:, None]
    z = z.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(z, 1)
    return z, torch.exp(z - lse[:, None]), lse, (d + 8) * U * size


def check_attention(torch, out, lse, q, k, v, lens):
    g = q.shape[1] // k.shape[1]
    at = 0
    for n in lens:
        for h in range(q.shape[1] if n else 0):
            kk, vv = k[at:at + n, h // g], v[at:at + n, h // g].double()
            z, p, e, ds = scores(torch, q[at:at + n, h], kk)
            ref, size = p @ vv, p @ vv.abs()
            tol = (2 * ds[:, None] + 2 * n * U + 2.0 ** -20) * size + 1e-37
            if out.dtype == torch.bfloat16:
                tol += 2.0 ** -8 * (size + ref.abs())
            got = out[at:at + n, h].double()
            bad = (got - ref).abs() - tol
            assert torch.isfinite(got).all() and bad.max() <= 0, (n, h, int(bad.argmax()), float(bad.max()))
            if lse is not None:
                off = (lse[h, at:at + n].double() - e).abs()
                assert (off <= 2 * ds + n * U + 2.0 ** -20 + 4 * U * e.abs()).all(), (n, h, float(off.max()))
        at += n


def check_weights(torch, w, q, k, lse, lens, last):
    g = q.shape[1] // k.shape[1]
    at = 0
    for n in lens:
        first = max(0, n - last)
        for hk in range(k.shape[1] if n else 0):
            ref = torch.zeros(n, dtype=torch.float64, device="cuda")
            tol = torch.zeros_like(ref)
            for h in range(hk * g, hk * g + g):
                z, _, _, ds = scores(torch, q[at:at + n, h], k[at:at + n, hk], first)
                e = lse[h, at + first:at + n].double()
                p = torch.exp(z - e[:, None])
                # the argument's rounding: a few half steps of |lse| and |score|
                arg = 8 * U * (e.abs()[:, None] + z.nan_to_num(neginf=0.0).abs())
                ref += p.sum(0)
                tol += (p * (2 * ds[:, None] + arg + 2.0 ** -20 + (n - first) * g * U)).sum(0)
            off = (w[hk, at:at + n].double() - ref).abs()
            assert (off <= tol + 1e-37).all(), (n, hk, float((off - tol).max()))
        at += n


SHAPES = [
    ([1], 1, 1, 16), ([2], 2, 1, 64), ([1, 1, 1], 4, 4, 128), ([63, 64, 65], 8, 2, 128), ([127, 128, 129], 8, 8, 64),
    ([1, 0, 300, 0, 17], 8, 2, 128), ([511, 31, 257], 6, 2, 64), ([1000], 4, 1, 128), ([385, 5], 5, 1, 128),
    ([200, 90], 14, 2, 64), ([33, 160], 8, 1, 128), ([260], 12, 2, 128), ([130, 70], 4, 2, 48), ([97], 3, 1, 80),
    ([150], 2, 2, 256), ([700, 123], 2, 2, 128), ([1025], 2, 2, 64), ([641], 32, 8, 128),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("lens,hq,hkv,d", SHAPES)
def test_attention(torch, kvq, lens, hq, hkv, d, dtype):
    q, k, v = inputs(torch, sum(lens), hq, hkv, d, dtype)
    out, lse = kvq.prompt_attention(q, k, v, lens)
    check_attention(torch, out, lse, q, k, v, lens)
    again, _ = kvq.prompt_attention(q, k, v, lens)
    assert torch.equal(out, again)
    assert kvq.prompt_status() == 0


@pytest.mark.parametrize("dtype,d", [("bfloat16", 128), ("bfloat16", 64), ("float32", 128), ("bfloat16", 32)])
def test_attention_of_scores_that_rise(torch, kvq, dtype, d):
    """Running maxima that move at every step and by far, one heavy key, and equal keys."""
    n = 700
    q, k, v = inputs(torch, n, 4, 2, d, dtype, 3, q_gain=4.0)
    k = (k * torch.linspace(0.1, 3.0, n, device="cuda")[:, None, None]).to(k.dtype)
    check_attention(torch, *kvq.prompt_attention(q, k, v, [n]), q, k, v, [n])
    up = (q[:1, :2].expand(n, 2, d) * torch.linspace(-2.0, 2.0, n, device="cuda")[:, None, None]).to(k.dtype)
    check_attention(torch, *kvq.prompt_attention(q, up, v, [n]), q, up, v, [n])
    down = up.flip(0).contiguous()
    check_attention(torch, *kvq.prompt_attention(q, down, v, [n]), q, down, v, [n])
    same = k[:1].expand(n, 2, d).contiguous()
    check_attention(torch, *kvq.prompt_attention(q, same, v, [n]), q, same, v, [n])


@pytest.mark.parametrize("d,dtype", [(128, "bfloat16"), (64, "bfloat16"), (128, "float32")])
def test_other_sequences_and_rows_behind_the_last_stay_out(torch, kvq, d, dtype):
    lens, tail = [70, 45, 200, 3], 90
    q, k, v = inputs(torch, sum(lens) + tail, 8, 2, d, dtype, 4)
    for t in (q, k, v):
        t[:70] = math.nan
        t[115:315:2] = math.inf
        t[116:315:2] = -math.inf
        t[sum(lens):] = math.nan
    out = torch.full_like(q, 7.0)
    lse = torch.full((8, q.shape[0]), 5.0, device="cuda")
    kvq.prompt_attention(q, k, v, lens, out=out, lse=lse)
    assert (out[sum(lens):] == 7.0).all() and (lse[:, sum(lens):] == 5.0).all()
    w = torch.full((2, q.shape[0]), 3.0, device="cuda")
    kvq.prompt_weights(q, k, lse, lens, 64, out=w)
    assert (w[:, sum(lens):] == 3.0).all()
    for a, n in ((70, 45), (315, 3)):
        s = slice(a, a + n)
        check_attention(torch, out[s], lse[:, s], q[s], k[s], v[s], [n])
        check_weights(torch, w[:, s], q[s], k[s], lse[:, s], [n], 64)


@pytest.mark.parametrize("hq,hkv", [(8, 2), (2, 2), (5, 1)])
@pytest.mark.parametrize("d,dtype", [(128, "bfloat16"), (64, "bfloat16"), (96, "bfloat16"), (256, "bfloat16"),
                                     (128, "float32")])
def test_infinities_and_nan_of_later_tokens_stay_out(torch, kvq, d, dtype, hq, hkv):
    """A Value reaches the tokens from its own on: infinities and NaN make those
    elements infinite or NaN and leave every other bit as zeros in their place do."""
    lens = [700, 70, 1]
    q, k, v = inputs(torch, sum(lens), hq, hkv, d, dtype, 11)
    bad = torch.zeros(v.shape, device="cuda")
    for token, channel, x in ((3, 5, math.inf), (130, 2, math.nan), (131, 3, -math.inf), (150, 3, math.inf),
                              (300, slice(16, 32), math.inf), (301, 17, -math.inf), (555, 0, math.nan),
                              (556, slice(40, 48), -math.inf), (690, d - 1, math.inf), (699, slice(0, d), math.nan),
                              (700, 7, math.inf), (740, 8, math.nan), (769, 9, -math.inf)):
        bad[token, hkv - 1, channel] = x
    v = torch.where(bad != 0, torch.zeros_like(v), v)
    want, lse = kvq.prompt_attention(q, k, v, lens)
    check_attention(torch, want, lse, q, k, v, lens)
    got, l2 = kvq.prompt_attention(q, k, torch.where(bad != 0, bad.to(v.dtype), v), lens)
    at = 0
    for n in lens:
        seen = bad[at:at + n].cumsum(0).repeat_interleave(hq // hkv, 1)  # infinite or NaN from the first one on
        expect = torch.where(seen == 0, want[at:at + n].float(), seen)
        assert torch.equal(got[at:at + n].float().nan_to_num(nan=1e30), expect.nan_to_num(nan=1e30))
        at += n
    assert torch.equal(lse, l2) and kvq.prompt_status() == 0


@pytest.mark.parametrize("d,dtype", [(128, "bfloat16"), (64, "bfloat16"), (96, "bfloat16"), (128, "float32")])
def test_infinities_and_nan_of_keys_and_queries(torch, kvq, d, dtype):
    """A key counts from its token on, a query at its own row; a score of minus infinity weighs nothing."""
    n, hq, hkv = 500, 4, 2
    q, k, v = inputs(torch, n, hq, hkv, d, dtype, 12)
    want, lse = kvq.prompt_attention(q, k, v, [n])
    k2, q2 = k.clone(), q.clone()
    k2[333, 1], q2[77, 0] = math.nan, math.nan
    got, l2 = kvq.prompt_attention(q2, k2, v, [n])
    rows = torch.zeros(n, hq, dtype=torch.bool, device="cuda")
    rows[333:, 2:] = True
    rows[77, 0] = True
    assert got[rows].isnan().all() and torch.equal(got[~rows], want[~rows])
    assert l2.T[rows].isnan().all() and torch.equal(l2.T[~rows], lse.T[~rows])
    # the weights that the last queries give: a NaN query reaches the keys up to its own, a NaN key itself
    w = kvq.prompt_weights(q, k, lse, [n], 450)
    w2 = kvq.prompt_weights(q2, k2, lse, [n], 450)
    nan = torch.zeros(hkv, n, dtype=torch.bool, device="cuda")
    nan[0, :78] = True
    nan[1, 333] = True
    assert w2[nan].isnan().all() and torch.equal(w2[~nan], w[~nan])
    # the first 260 keys at minus infinity for queries of positive first channel
    q, k = q.clone(), k.clone()
    q[..., 0], k[..., 0] = 1.0, 0.0
    k[:260, :, 0] = -math.inf
    got, lse = kvq.prompt_attention(q, k, v, [n])
    check_attention(torch, got[260:], lse[:, 260:], q[260:], k[260:], v[260:], [n - 260])
    assert got[:260].isnan().all() and kvq.prompt_status() == 0


@pytest.mark.parametrize("d,dtype", [(128, "bfloat16"), (64, "bfloat16"), (96, "float32")])
def test_infinite_weights_stay_infinite(torch, kvq, d, dtype):
    """A query whose weights overflow makes those of the keys it sees infinite, never NaN, whatever is added later."""
    n, at = 900, 300
    q, k, v = inputs(torch, n, 4, 2, d, dtype, 13)
    lse = kvq.prompt_attention(q, k, v, [n])[1]
    w = kvq.prompt_weights(q, k, lse, [n], n)
    lse[0, at] = -1000.0
    got = kvq.prompt_weights(q, k, lse, [n], n)
    assert got[0, :at + 1].isposinf().all()
    assert torch.equal(got[0, at + 1:], w[0, at + 1:]) and torch.equal(got[1], w[1])


@pytest.mark.parametrize("d,dtype", [(128, "bfloat16"), (64, "bfloat16"), (96, "float32")])
def test_strides(torch, kvq, d, dtype):
    """Slices of one fused projection, head-major tensors, a strided output, one head out of many."""
    lens, hq, hkv = [100, 61], 8, 2
    n = sum(lens)
    q, k, v = inputs(torch, n, hq, hkv, d, dtype, 5)
    want, lse = kvq.prompt_attention(q, k, v, lens)
    check_attention(torch, want, lse, q, k, v, lens)
    fused = torch.cat([q, k, v], 1)
    fq, fk, fv = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    hm = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]
    wide = torch.full((n, hq, 3 * d), 2.0, dtype=q.dtype, device="cuda")
    for a in ((fq, fk, fv), hm, (fq, hm[1], v)):
        out = wide[:, :, d:2 * d]
        out, l2 = kvq.prompt_attention(*a, lens, out=out)
        assert torch.equal(out, want) and torch.equal(l2, lse)
        assert (wide[:, :, :d] == 2.0).all() and (wide[:, :, 2 * d:] == 2.0).all()
        w = kvq.prompt_weights(a[0], a[1], lse, lens, 50)
        assert torch.equal(w, kvq.prompt_weights(q, k, lse, lens, 50))
        kept = kvq.evict(a[1], a[2], w, lens, 40, 2, 5)
        plain = kvq.evict(k, v, w, lens, 40, 2, 5)
        assert torch.equal(kept.k, plain.k) and torch.equal(kept.v, plain.v) and torch.equal(kept.index, plain.index)
    one, l1 = kvq.prompt_attention(fq[:, 3:4], fk[:, :1], fv[:, :1], lens)
    check_attention(torch, one, l1, q[:, 3:4], k[:, :1], v[:, :1], lens)


@pytest.mark.parametrize("d", [64, 32])
def test_offsets_past_31_bits(torch, kvq, d):
    n, wide = 2200, 1 << 20
    big = torch.zeros(n, wide, dtype=torch.bfloat16, device="cuda")
    q, k, v = inputs(torch, n, 4, 1, d, "bfloat16", 6)
    last = wide - 4 * d
    big[:, :4 * d] = q.reshape(n, -1)
    big[:, 4 * d:5 * d] = k[:, 0]
    big[:, 5 * d:6 * d] = v[:, 0]
    bq, bk, bv = (big[:, a:b].view(n, -1, d) for a, b in ((0, 4 * d), (4 * d, 5 * d), (5 * d, 6 * d)))
    out, lse = kvq.prompt_attention(bq, bk, bv, [n], out=big[:, last:].view(n, 4, d))
    check_attention(torch, out, lse, q, k, v, [n])
    w = kvq.prompt_weights(bq, bk, lse, [n], 33)
    check_weights(torch, w, q, k, lse, [n], 33)
    kept = kvq.evict(bk, bv, w, [n], 700, 1, 9)
    index = kept.index.long()
    assert torch.equal(kept.k, k[index, 0]) and torch.equal(kept.v, v[index, 0])


@pytest.mark.parametrize("dtype,d", [("bfloat16", 128), ("float32", 16)])
def test_more_sequences_than_one_launch_takes(torch, kvq, dtype, d):
    lens = [(7 * i) % 41 for i in range(600)]
    q, k, v = inputs(torch, sum(lens), 4, 2, d, dtype, 7)
    out, lse = kvq.prompt_attention(q, k, v, lens)
    check_attention(torch, out, lse, q, k, v, lens)
    w = kvq.prompt_weights(q, k, lse, lens, 10)
    check_weights(torch, w, q, k, lse, lens, 10)
    check_evict(torch, kvq, k, v, w, lens, 8, 1, 3)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("last", [1, 16, 50, 1 << 40])
@pytest.mark.parametrize("lens,hq,hkv,d", [([1], 1, 1, 16), ([129, 1, 0, 40], 8, 2, 128), ([700], 4, 1, 64),
                                           ([300, 64], 3, 1, 128), ([250], 14, 2, 64), ([130], 8, 1, 80),
                                           ([515], 2, 2, 128)])
def test_weights(torch, kvq, lens, hq, hkv, d, dtype, last):
    q, k, v = inputs(torch, sum(lens), hq, hkv, d, dtype, 8)
    _, lse = kvq.prompt_attention(q, k, v, lens)
    full = lse.clone()
    at = 0
    for n in lens:  # what does not count is not read
        lse[:, at:at + max(0, n - last)] = math.nan
        at += n
    w = kvq.prompt_weights(q, k, lse, lens, last)
    check_weights(torch, w, q, k, full, lens, last)
    # every counted query hands out weight 1 a head
    at = 0
    for n in lens:
        counted = min(n, last) * (hq // hkv)
        assert torch.allclose(w[:, at:at + n].double().sum(1), torch.tensor(float(counted), dtype=torch.float64,
                                                                           device="cuda"), rtol=2e-4)
        at += n
    assert torch.equal(w, kvq.prompt_weights(q, k, lse, lens, last))


def check_evict(torch, kvq, k, v, w, lens, keep, first, recent):
    kept = kvq.evict(k, v, w, lens, keep, first, recent)
    begin = np.concatenate([[0], np.cumsum(lens)])
    counts = [min(keep, n) for n in lens] if isinstance(keep, int) else keep
    assert kept.counts == list(counts)
    ws = w.cpu().numpy()
    for i, n in enumerate(lens):
        ks, vs, index = kept.sequence(i)
        for h in range(k.shape[1]):
            x = ws[h, begin[i]:begin[i + 1]]
            if counts[i] >= n:
                want = np.arange(n)
            else:
                x = np.where(np.isnan(x), -np.inf, x).astype(np.float64)
                nan = np.isnan(ws[h, begin[i]:begin[i + 1]])
                free = np.arange(first, n - recent)
                best = free[np.lexsort((free, nan[free], -x[free]))[:counts[i] - first - recent]]
                want = np.sort(np.concatenate([np.arange(first), best, np.arange(n - recent, n)]))
            got = index[h].cpu().numpy()
            assert np.array_equal(got, want), (i, h)
            rows = torch.from_numpy(want).cuda() + int(begin[i])
            assert torch.equal(ks[0, h], k[rows, h]) and torch.equal(vs[0, h], v[rows, h])
    return kept


@pytest.mark.parametrize("dtype,d", [("bfloat16", 128), ("float32", 80), ("bfloat16", 16)])
@pytest.mark.parametrize("lens,keep,first,recent", [
    ([1], 1, 0, 0), ([1], 0, 0, 0), ([2], 1, 0, 0), ([2], 1, 1, 0), ([2], 1, 0, 1), ([300], 128, 4, 32),
    ([1024, 0, 1025, 1023], 100, 0, 0), ([5000, 17, 700], 16, 4, 12), ([5000, 17, 700], 699, 1, 1),
    ([2049, 33], [2048, 0], 0, 0), ([70001], 3001, 2, 64), ([4096, 4096], [1, 4095], 0, 1)])
def test_evict(torch, kvq, lens, keep, first, recent, dtype, d):
    _, k, v = inputs(torch, sum(lens), 2, 2, d, dtype, 9)
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.exp(3 * torch.randn(2, sum(lens), generator=g, device="cuda"))
    if first + recent > (keep if isinstance(keep, int) else max(keep)):
        pytest.skip("refused")
    counts = [min(keep, n) for n in lens] if isinstance(keep, int) else keep
    if any(c < n and first + recent > c for c, n in zip(counts, lens)):
        with pytest.raises(kvq.KVQError):
            kvq.evict(k, v, w, lens, keep, first, recent)
        return
    check_evict(torch, kvq, k, v, w, lens, keep, first, recent)


@pytest.mark.parametrize("lens,hkv,keep", [([1000003], 1, 5001), ([57001] * 80, 2, 300), ([20000, 9000, 33], 3, 7000)])
def test_evict_long_runs_and_many_units(torch, kvq, lens, hkv, keep):
    """Runs longer than shared memory holds (in a cluster and alone), and clusters of several sizes."""
    _, k, v = inputs(torch, sum(lens), hkv, hkv, 16, "bfloat16", 15)
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.exp(2 * torch.randn(hkv, sum(lens), generator=g, device="cuda")).bfloat16().float()
    check_evict(torch, kvq, k, v, w, lens, keep, 1, 5)


def test_evict_equal_and_special_weights(torch, kvq):
    n = 3000
    _, k, v = inputs(torch, n, 4, 4, 64, "bfloat16", 10)
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randint(0, 5, (4, n), generator=g, device="cuda").float()
    w[1] = 0.0
    w[1, ::3] = -0.0
    w[2, 5::7] = math.inf
    w[2, 6::7] = math.nan
    w[2, 8::9] = -math.inf
    w[3] = -1e-42
    w[3, ::2] = 1e-42
    for keep in (1, 17, 400, 1500, 2600, 2999):
        check_evict(torch, kvq, k, v, w, [n], keep, 0, 1)
    # rows pass unchanged, whatever bits they hold
    bits = torch.randint(-32768, 32767, (n, 4, 64), generator=g, device="cuda", dtype=torch.int32).to(torch.int16)
    kept = kvq.evict(bits.view(torch.bfloat16), v, w, [n], 50)
    rows = kept.index.view(4, 50).long()
    want = torch.stack([bits[rows[h], h] for h in range(4)]).view(-1, 64)
    assert torch.equal(kept.k.view(torch.int16), want)


def test_streams_and_graphs(torch, kvq):
    """Two calls at once on two streams, and a captured run of all three, replayed on new inputs."""
    lens = [900, 30]
    sets = [inputs(torch, sum(lens), 8, 2, 128, "bfloat16", s) for s in (11, 12)]

    def chain(q, k, v):
        out, lse = kvq.prompt_attention(q, k, v, lens)
        w = kvq.prompt_weights(q, k, lse, lens, 32)
        kept = kvq.evict(k, v, w, lens, 64, 2, 16)
        return out, lse, w, kept.k, kept.v, kept.index

    want = [chain(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for st, s in zip(streams, sets):
        with torch.cuda.stream(st):
            got.append([chain(*s) for _ in range(5)][-1])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    static = [t.clone() for t in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = chain(*static)
    for i in (1, 0, 1):
        for t, s in zip(static, sets[i]):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(res, want[i]))
    assert kvq.prompt_status() == 0


@pytest.mark.parametrize("d", [128, 48])
def test_c_entry_without_lse_and_status(torch, kvq, d):
    q, k, v = inputs(torch, 150, 4, 2, d, "bfloat16", 16)
    want, _ = kvq.prompt_attention(q, k, v, [150])
    out = torch.zeros_like(q)
    p = kvq.binding._Prompt(k, [150])
    p.queries(q)
    p.values(v)
    p.c.out_token_stride, p.c.out_head_stride = out.stride()[:2]
    p.c.status = None
    before = kvq.kvq_kernel_launches()
    kvq.kvq_prompt_attention(p.c, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), None,
                             torch.cuda.current_stream().cuda_stream)
    assert torch.equal(out, want) and kvq.kvq_kernel_launches() == before + 1


def test_integers_of_other_kinds(torch, kvq):
    q, k, v = inputs(torch, 60, 2, 2, 64, "bfloat16", 17)
    lens = np.array([40, 20])
    out, lse = kvq.prompt_attention(q, k, v, lens)
    assert torch.equal(out, kvq.prompt_attention(q, k, v, [40, 20])[0])
    w = kvq.prompt_weights(q, k, lse, torch.tensor([40, 20]), np.int64(8))
    kept = kvq.evict(k, v, w, lens, np.int32(16), np.int64(1), np.int64(2))
    plain = kvq.evict(k, v, w, [40, 20], [16, 16], 1, 2)
    assert kept.counts == plain.counts and torch.equal(kept.index, plain.index)


def test_append_kept_checks_before_it_appends(torch, kvq):
    _, k, v = inputs(torch, 200, 2, 2, 64, "bfloat16", 18)
    kept = kvq.evict(k, v, torch.rand(2, 200, device="cuda"), [100, 100], [30, 80])
    cache = kvq.KVQCache(2, 2, 2, 64, 16, 8, 7, 64)
    with pytest.raises(kvq.KVQError):
        cache.append_kept(kept)
    assert cache.seq_state(0)["total"] == 0
    with pytest.raises(AssertionError):
        cache.append_kept(kept, 1)


def test_tensor_refusals(torch, kvq):
    q, k, v = inputs(torch, 40, 8, 2, 64, "bfloat16", 13)
    lse = torch.zeros(8, 40, device="cuda")
    w = torch.zeros(2, 40, device="cuda")
    with pytest.raises(kvq.KVQError):
        kvq.prompt_attention(q, k, v, [41])
    with pytest.raises(kvq.KVQError):
        kvq.prompt_attention(q[:, :, 4:20], k[:, :, 4:20], v[:, :, 4:20], [40])  # 8-byte offset
    with pytest.raises(kvq.KVQError):
        kvq.prompt_attention(q[:, :7], k, v, [40])
    with pytest.raises(kvq.KVQError):
        kvq.evict(k, v, w, [40], 10, 6, 6)
    with pytest.raises(kvq.KVQError):
        kvq.prompt_weights(q, k, lse, [40], 0)
    for bad in [lambda: kvq.prompt_attention(q.float(), k, v, [40]), lambda: kvq.prompt_attention(q, k, v[:39], [39]),
                lambda: kvq.prompt_attention(q.half(), k.half(), v.half(), [40]),
                lambda: kvq.prompt_attention(q, k.cpu(), v, [40]),
                lambda: kvq.prompt_weights(q, k, lse[:, :39], [40], 4),
                lambda: kvq.prompt_weights(q, k, lse.double(), [40], 4), lambda: kvq.evict(k, v, lse, [40], 10),
                lambda: kvq.evict(k, v, w, [20, 20], [5])]:
        with pytest.raises(AssertionError):
            bad()


def test_prompt_to_cache(torch, kvq):
    """The operators as a serving loop runs them: attend the prompts, cut them
    to a budget, quantize what stays and decode, against the oracle's cache of
    the kept rows."""
    from oracle import kvq_oracle as O
    lens, hq, hkv, d, keep = [600, 90, 333], 8, 2, 128, 256
    q, k, v = inputs(torch, sum(lens), hq, hkv, d, "bfloat16", 14)
    out, lse = kvq.prompt_attention(q, k, v, lens)
    check_attention(torch, out, lse, q, k, v, lens)
    w = kvq.prompt_weights(q, k, lse, lens, 32)
    kept = check_evict(torch, kvq, k, v, w, lens, keep, 4, 32)
    cache = kvq.KVQCache(len(lens), hkv, hq, d, 64, 32, 7, keep + 8)
    cache.append_kept(kept)
    qd = q[:len(lens)].contiguous()
    got = cache.decode_attention(qd).cpu().numpy()
    for i in range(len(lens)):
        seq = O.GroupedSequence(hkv, d, 64, 32, 7)
        ks, vs, _ = kept.sequence(i)
        seq.append(ks[0].float().cpu().numpy(), vs[0].float().cpu().numpy())
        ref = seq.attend(qd[i].float().cpu().numpy())
        assert cache.seq_state(i)["total"] == min(keep, lens[i])
        assert (np.abs(got[i] - ref) <= 1e-3 + 1e-2 * np.abs(ref)).all()
