"""KVQCache.append_kept appends all of a Kept or nothing: what an append would
refuse is found before the first one, on stand-ins for the cache and its pool."""

from types import SimpleNamespace

import pytest

kvq = pytest.importorskip("quantized_kv_cache_02_gb300")
B = kvq.binding


class Cache:
    """The host state of a paged (or, with pool None, contiguous) cache and the
    C library's rules for an append."""

    append_kept = kvq.KVQCache.append_kept

    def __init__(self, pool, capacity, batch=3, residual=8, group=4):
        self.cfg = SimpleNamespace(batch=batch, residual_len=residual, group=group)
        self.pool_blocks, self.free, self.capacity = pool or 0, pool, [capacity] * batch
        self.total, self.quantized, self.appended = [0] * batch, [0] * batch, []

    def seq_state(self, i):
        return {"total": self.total[i], "quantized": self.quantized[i], "window": self.total[i] - self.quantized[i]}

    def pool_state(self):
        return self.free, self.pool_blocks

    def append(self, k, v, i):
        over = self.total[i] - self.quantized[i] + k - self.cfg.residual_len
        groups = over // self.cfg.group if over > 0 else 0
        if self.free is not None:
            assert groups <= 4096 and groups <= self.free, "the library refuses this append"
            self.free -= groups
        self.total[i] += k
        self.quantized[i] += groups * self.cfg.group
        self.appended.append((i, k))


def kept(*counts):
    return SimpleNamespace(counts=list(counts), sequence=lambda i: (counts[i], counts[i], None))


def test_a_pool_that_is_too_small_for_all_takes_none():
    # 20 tokens flush 3 groups of 4 past a window of 8
    c = Cache(pool=8, capacity=100)
    with pytest.raises(kvq.KVQError) as e:
        c.append_kept(kept(20, 20, 20))
    assert e.value.status == B.KVQ_ECAPACITY and "pool" in str(e.value) and c.appended == [] and c.free == 8
    c.append_kept(kept(20, 19))
    assert c.appended == [(0, 20), (1, 19)] and c.free == 3
    # windows count: 3 more tokens on a window of 8 flush nothing, on one of 11 a group
    c.append_kept(kept(3, 0, 20))
    assert c.free == 0 and c.total == [23, 19, 20]
    with pytest.raises(kvq.KVQError):
        c.append_kept(kept(0, 3, 1))
    assert c.total == [23, 19, 20]
    c.append_kept(kept(0, 0, 3))
    c.append_kept(kept(0, 0, 0))
    assert c.free == 0 and c.total == [23, 19, 23]


def test_more_groups_than_one_append_takes():
    c = Cache(pool=10000, capacity=10 ** 6)
    with pytest.raises(kvq.KVQError) as e:
        c.append_kept(kept(20, 8 + 4 * 4097))
    assert e.value.status == B.KVQ_EUNSUPPORTED and c.appended == []
    c.append_kept(kept(20, 8 + 4 * 4096 + 3))
    assert c.appended == [(0, 20), (1, 8 + 4 * 4096 + 3)]


def test_a_contiguous_cache_has_no_pool():
    c = Cache(pool=None, capacity=50)
    c.append_kept(kept(50, 40, 1))
    with pytest.raises(kvq.KVQError) as e:
        c.append_kept(kept(0, 10, 50))
    assert e.value.status == B.KVQ_ECAPACITY and c.total == [50, 40, 1]
