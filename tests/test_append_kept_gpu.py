"""KVQCache.append_kept on a paged cache: all of a Kept or nothing."""

import pytest

from test_prompt_gpu import inputs, kvq, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def test_paged_append_is_all_or_none(torch, kvq):  # noqa: F811
    lens, counts, batch = [200, 100, 150], [96, 60, 130], 3
    _, k, v = inputs(torch, sum(lens), 2, 2, 64, "bfloat16", 20)
    kept = kvq.evict(k, v, torch.rand(2, sum(lens), device="cuda"), lens, counts)
    # groups of 8 past a window of 16: 10, 5 and 14
    small = kvq.KVQCache(batch, 2, 2, 64, 16, 8, 7, 256, pool_blocks=28)
    with pytest.raises(kvq.KVQError):
        small.append_kept(kept)
    assert small.pool_state() == (28, 28) and [small.seq_state(i)["total"] for i in range(batch)] == [0, 0, 0]
    enough = kvq.KVQCache(batch, 2, 2, 64, 16, 8, 7, 256, pool_blocks=29)
    enough.append_kept(kept)
    assert enough.pool_state() == (0, 29)
    plain = kvq.KVQCache(batch, 2, 2, 64, 16, 8, 7, 256)
    plain.append_kept(kept)
    for i in range(batch):
        assert enough.seq_state(i) == plain.seq_state(i)
        for h in range(2):
            a, b = enough.export_unit(i, h), plain.export_unit(i, h)
            assert all((a[x] == b[x]).all() for x in a)
