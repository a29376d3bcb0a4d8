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
