"""The tensor-core gathered weights where a CTA streams a run of key pairs past
query tiles that stay, and where eight CTAs share a pair's query tiles."""

import pytest

from test_prompt_gpu import check_weights, inputs, kvq, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("lens,hq,hkv,last", [
    # runs of four pairs, ends inside one, a pair whose second tile is empty; one query tile and two
    ([8192, 5003, 257, 1024], 32, 8, 32), ([8192, 5003, 257, 1024], 32, 8, 64), ([8192, 5003, 257, 1024], 32, 8, 17),
    # runs of thirteen pairs: both places for a pair are used again and again
    ([60000], 32, 8, 50), ([3, 41003, 1, 19001], 24, 8, 84),
    # clusters of eight, whose ranks take up to nine query tiles of a pair, and for the last keys some none
    ([1100], 8, 1, 1 << 40), ([2200, 130], 8, 2, 1050), ([4096], 1, 1, 1 << 40)])
def test_runs_of_pairs_and_clusters(torch, kvq, lens, hq, hkv, last, d):  # noqa: F811
    q, k, v = inputs(torch, sum(lens), hq, hkv, d, "bfloat16", 19)
    _, lse = kvq.prompt_attention(q, k, v, lens)
    w = kvq.prompt_weights(q, k, lse, lens, last)
    check_weights(torch, w, q, k, lse, lens, last)
    for _ in range(3):
        assert torch.equal(w, kvq.prompt_weights(q, k, lse, lens, last))
    assert kvq.prompt_status() == 0


@pytest.mark.parametrize("last", [1 << 40, 40])
@pytest.mark.parametrize("d,dtype", [(128, "bfloat16"), (64, "bfloat16"), (96, "bfloat16"), (128, "float32")])
def test_infinite_lse(torch, kvq, d, dtype, last):  # noqa: F811
    """exp(score - lse) of a row whose lse is infinite or far beyond the scores: nothing for plus infinity,
    infinity for minus infinity, and NaN only where the score is that infinity itself or NaN."""
    n, hq, hkv = 300, 4, 2
    q, k, v = inputs(torch, n, hq, hkv, d, dtype, 21)
    lse = kvq.prompt_attention(q, k, v, [n])[1]
    lse[0, 270], lse[1, 280], lse[0, 275], lse[1, 290], lse[0, 291] = torch.inf, torch.inf, 3e38, 1e38, 1e10
    w = kvq.prompt_weights(q, k, lse, [n], last)
    plain = lse.clone()
    plain[0, 270] = plain[1, 280] = plain[0, 275] = plain[1, 290] = plain[0, 291] = 1e4
    assert torch.equal(w, kvq.prompt_weights(q, k, plain, [n], last)) and w.isfinite().all()
    # minus infinity reaches the keys up to its own row, the other KV head keeps its bits
    lse[0, 277] = -torch.inf
    low = kvq.prompt_weights(q, k, lse, [n], last)
    assert low[0, :278].isposinf().all() and torch.equal(low[0, 278:], w[0, 278:]) and torch.equal(low[1], w[1])
    # a score that is the row's infinity has no weight
    q[295, 2, 0], k[..., 0] = torch.inf, 1.0
    k[7, 1, 0] = -1.0
    lse[2, 295] = torch.inf
    both = kvq.prompt_weights(q, k, lse, [n], last)
    nan = torch.zeros(n, dtype=torch.bool, device="cuda")
    nan[:296], nan[7] = True, False
    assert both[1][nan].isnan().all() and both[1][~nan].isfinite().all()
