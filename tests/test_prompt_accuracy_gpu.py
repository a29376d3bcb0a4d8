"""What the tensor-core gathered weights do beyond fp32 sums of tensor-core scores,
held by tolerances that are tighter than those of any order of summation.

A long sum.  With queries of 0 and one lse for all rows every weight is the same
number p times the rows that see its key.  For a p of 18 significant bits every
sum inside a tile is exact (at most 64 p in one number), so all that is left are
the running sums over the tiles: two of them, each within 2 u of its exact sum
however long (Kahan; u = 2^-24), and the addition of the two, u: 3 u, and 2^-40
for the products of these.  Added plainly, a sum past 64 tiles rounds every
further one the same way.

Scores.  The tensor cores round toward zero.  A score that is two sums of D / 32
steps, the second of which ends with lse taken off, loses on average half a step
of each partial sum, together 1.0 (D = 64) or 2.0 (D = 128) times the score: a
share ``loss`` of it.  That moves a weight p by p * loss * score, the sum of all
weights by the sum of these; the kernel puts it back.  Where partial sums grow
evenly at most half of it may be left over.  With the heavy channels all first
the loss is up to twice as much, with all of them last it may be none: all of it
may be left over, with either sign, and no more.
"""

import math

import pytest

from test_prompt_gpu import kvq, torch  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("n,hq,hkv", [(8192, 32, 8), (5003, 16, 16), (6001, 60, 20)])
def test_sums_over_many_tiles(torch, kvq, n, hq, hkv, d):  # noqa: F811
    zero = torch.zeros(n, hq, d, dtype=torch.bfloat16, device="cuda")
    # single tokens give single weights: take an lse whose weight has 18 significant bits
    many = torch.linspace(0.1, 0.6, 4096, device="cuda")
    one = torch.zeros(4096, 1, d, dtype=torch.bfloat16, device="cuda")
    p = kvq.prompt_weights(one, one, many[None].contiguous(), [1] * 4096, 1)[0]
    short = ((p.view(torch.int32) & 127) == 64).nonzero()[:, 0]
    assert len(short)
    for i in short[:3].tolist():
        w = kvq.prompt_weights(zero, zero[:, :hkv], torch.full((hq, n), float(many[i]), device="cuda"), [n], n)
        seen = (n - torch.arange(n, dtype=torch.float64, device="cuda")) * (hq // hkv)
        off = (w.double() / (seen * p[i].double()) - 1).abs()
        assert off.max() <= 3 * U + 2.0 ** -40, float(off.max()) / U


@pytest.mark.parametrize("seed", [1, 2, 3])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("heavy,left", [("even", 0.5), ("first", 1.0), ("last", 1.0)])
def test_scores_lose_nothing_on_average(torch, kvq, d, heavy, left, seed):  # noqa: F811
    n, g, hkv = 1024, 4, 4
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    # Keys with a scale per channel and a ten times heavier channel in every 16, or 8 heavy ones at one end
    sigma = torch.exp(torch.rand(hkv, d, generator=gen, device="cuda") * math.log(100.0)) * 0.05
    if heavy == "even":
        sigma[:, 5::16] *= 10.0
    else:
        sigma = torch.ones(hkv, d, device="cuda")
        sigma[:, slice(0, 8) if heavy == "first" else slice(d - 8, d)] = 10.0
    q, k = normal(n, g * hkv, d).bfloat16(), (normal(n, hkv, d) * sigma).bfloat16()
    z = torch.einsum("ihgd,jhd->hgij", q.double().view(n, hkv, g, d), k.double()) / math.sqrt(d)
    hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
    lse = torch.logsumexp(z.masked_fill(hidden, -math.inf), 3).float()
    p = torch.exp(z - lse.double()[..., None]).masked_fill(hidden, 0.0)
    w = kvq.prompt_weights(q, k, lse.view(g * hkv, n).contiguous(), [n], n).double()
    loss = (d / 64) * 0.5 * 2.0 ** -23 / (2 * math.log(2))
    assert abs(float(w.sum() - p.sum())) <= left * loss * float((p * z).sum())
