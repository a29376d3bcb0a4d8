"""Forks: a copied sequence is its source, bit for bit, and from then on its own."""

import pytest

pytestmark = pytest.mark.gpu


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


KINDS = ["contiguous", "paged", "segmented"]
CONFIGS = [dict(d=128, R=64, G=32, qmax=7, dtype="bf16", hkv=2, hq=8), dict(d=16, R=5, G=8, qmax=127, dtype="fp32", hkv=3, hq=3),
           dict(d=64, R=128, G=64, qmax=1, dtype="bf16", hkv=1, hq=2), dict(d=80, R=17, G=24, qmax=7, dtype="bf16", hkv=2, hq=2)]


def make(kvq, kind, c, capacity, pool=400):
    return kvq.KVQCache(len(capacity), c["hkv"], c["hq"], c["d"], c["R"], c["G"], c["qmax"], capacity, dtype=c["dtype"],
                        pool_blocks=pool if kind == "paged" else 0, segmented=kind == "segmented")


def rows(torch, c, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    return [torch.randn(1, c["hkv"], n, c["d"], generator=g, device="cuda").to(dt) * (1 + i) for i in range(2)]


def fill(torch, cache, c, lens, chunk=0):
    for b, n in enumerate(lens):
        if n:
            k, v = rows(torch, c, n, 100 + b)
            step = chunk or n
            for a in range(0, n, step):
                cache.append(k[:, :, a:a + step].contiguous(), v[:, :, a:a + step].contiguous(), b)


def unit(cache, b, h):
    got = cache.export_unit(b, h)
    return {name: x.tobytes() for name, x in got.items()}


def everything(cache, c, batch):
    return [(cache.seq_state(b), [unit(cache, b, h) for h in range(c["hkv"])]) for b in range(batch)]


def same(one, other):
    state = [{k: v for k, v in s[0].items() if k != "capacity"} for s in (one, other)]
    return state[0] == state[1] and one[1] == other[1]


MAPS = [([0], [3]), ([0, 0, 0], [1, 2, 3]), ([1, 0], [0, 1]), ([1, 2, 3, 0], [0, 1, 2, 3]), ([0, 1, 2], [1, 2, 3]),
        ([1, 0, 0, 1], [0, 1, 2, 3]), ([1, 2, 0, 1], [0, 1, 2, 3]), ([4, 0], [0, 2]), ([2, 2], [2, 4]), ([5, 5, 1], [1, 0, 5]),
        ([1, 2, 0, 4, 3, 4], [0, 1, 2, 3, 4, 5])]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("c", CONFIGS, ids=lambda c: f"d{c['d']}q{c['qmax']}")
def test_every_map(torch, kvq, kind, c):
    """All copies at once, whatever the order: chains, cycles, trees on cycles, an empty source."""
    lens = [300, 1, c["R"] + c["G"], 77, 0, 1000]
    for src, dst in MAPS:
        cache = make(kvq, kind, c, [1100] * 6)
        fill(torch, cache, c, lens)
        before = everything(cache, c, 6)
        cache.fork(src, dst)
        after = everything(cache, c, 6)
        for b in range(6):
            at = src[dst.index(b)] if b in dst else b
            assert same(after[b], before[at]), (src, dst, b)
        cache.close()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("c", CONFIGS[:3], ids=lambda c: f"d{c['d']}q{c['qmax']}")
def test_copies_go_their_own_way(torch, kvq, kind, c):
    """Appends, decodes and releases after a fork: as in a cache that was filled by itself."""
    n, batch = 210, 3
    cache, other = (make(kvq, kind, c, [n + 200] * batch) for _ in range(2))
    fill(torch, cache, c, [n, 5, 0], 90)
    for b in range(batch):
        k, v = rows(torch, c, n, 100)
        for a in range(0, n, 90):
            other.append(k[:, :, a:a + 90].contiguous(), v[:, :, a:a + 90].contiguous(), b)
    cache.fork(0, [1, 2])
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    for step in range(c["G"] + 3):
        k, v = (torch.cat([rows(torch, c, 1, 1000 + 10 * step + b)[i] for b in range(batch)]) for i in range(2))
        q = torch.randn(batch, c["hq"], c["d"], generator=torch.Generator(device="cuda").manual_seed(step),
                        device="cuda").to(dt)
        if step % 2:
            out, want = cache.decode_step(k, v, q), other.decode_step(k, v, q)
        else:
            cache.append(k, v)
            other.append(k, v)
            out, want = cache.decode_attention(q), other.decode_attention(q)
        assert torch.equal(out, want), step
    assert everything(cache, c, batch) == everything(other, c, batch)
    assert cache.bytes() == other.bytes()
    cache.release(0)
    cache.append(*rows(torch, c, n, 5), 0)  # blocks that the copies still hold are not handed out
    assert [everything(cache, c, batch)[b] == everything(other, c, batch)[b] for b in range(batch)] == [False, True, True]


def test_blocks_are_shared_and_come_back(torch, kvq):
    c = CONFIGS[0]
    cache = make(kvq, "paged", c, [1100] * 4, pool=40)
    fill(torch, cache, c, [64 + 30 * 32, 64 + 5 * 32, 0, 0])
    assert cache.pool_state() == (5, 40)
    cache.fork([0, 0], [2, 3])
    assert cache.pool_state() == (5, 40)
    cache.release(0)
    cache.release(2)
    assert cache.pool_state() == (5, 40)
    cache.fork(1, 3)  # the last that held them
    assert cache.pool_state() == (35, 40)
    cache.release(1)
    assert cache.pool_state() == (35, 40)
    cache.release(3)
    assert cache.pool_state() == (40, 40)
    # every block once in the pool: a full pool's worth of appends does not collide
    fill(torch, cache, c, [64 + 20 * 32, 64 + 20 * 32])
    one = make(kvq, "contiguous", c, [1100] * 4)
    fill(torch, one, c, [64 + 20 * 32, 64 + 20 * 32])
    assert everything(cache, c, 2) == everything(one, c, 2)


def test_many_sequences(torch, kvq):
    """More sequences than one launch's steps hold, chains among them."""
    c = dict(d=16, R=8, G=8, qmax=7, dtype="bf16", hkv=1, hq=1)
    for kind in KINDS:
        batch = 1500
        cache = make(kvq, kind, c, [40] * batch, pool=6 * batch)
        k, v = (torch.randn(batch, 1, 33, 16, device="cuda").bfloat16() for _ in range(2))
        cache.append(k, v)
        before = [t.clone() for t in cache.restore()]
        g = torch.Generator().manual_seed(1)
        src = [(b // 300) * 300 + int(torch.randint(300, (1,), generator=g)) for b in range(batch)]
        cache.fork(src, list(range(batch)))
        for x, y in zip(cache.restore(), before):
            assert torch.equal(x, y[src])
        with pytest.raises(kvq.KVQError) as e:
            cache.fork(0, list(range(1, 514)))
        assert e.value.status == kvq.binding.KVQ_EUNSUPPORTED
        cache.fork(list(range(512, 0, -1)), list(range(511, -1, -1)))
        for x, y in zip(cache.restore(), before):
            assert torch.equal(x[:512], y[src][1:513])


def test_refusals_change_nothing(torch, kvq):
    c = CONFIGS[0]
    for kind in KINDS:
        cache = make(kvq, kind, c, [400, 400, 100, 400])
        fill(torch, cache, c, [300, 50, 90, 0])
        before = everything(cache, c, 4)
        for src, dst, status in [([0], [4], 1), ([-1], [0], 1), ([0, 1], [3, 3], 1), ([1, 0], [3, 2], 2), ([4], [0], 1)]:
            with pytest.raises(kvq.KVQError) as e:
                cache.fork(src, dst)
            assert e.value.status == status
        with pytest.raises(AssertionError):
            cache.fork([0, 1], [3])
        with pytest.raises(TypeError):
            cache.fork([0.5], [3])
        launches = kvq.kvq_kernel_launches()
        cache.fork([], [])
        cache.fork([0, 3], [0, 3])
        assert everything(cache, c, 4) == before and kvq.kvq_kernel_launches() == launches


def test_on_a_side_stream(torch, kvq):
    c = CONFIGS[0]
    cache = make(kvq, "contiguous", c, [1100] * 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        k, v = rows(torch, c, 1000, 1)
        torch.cuda._sleep(1000000)
        cache.append(k, v, 0)
        cache.fork(0, [1, 2])
        ks, vs = cache.restore()
    side.synchronize()
    assert torch.equal(ks[1], ks[0]) and torch.equal(vs[2], vs[0]) and cache.device_status() == 0


def test_offsets_past_32_bits(torch, kvq):
    """Sequences whose pages lie past 2^32 bytes of the arena."""
    c = dict(d=128, R=128, G=64, qmax=127, dtype="bf16", hkv=8, hq=8)
    n = 1000
    cache = make(kvq, "contiguous", c, [1200000, 1200, 1200, 1200000, 1200])
    k, v = rows(torch, c, n, 3)
    cache.append(k, v, 1)
    cache.fork([1, 1], [3, 4])
    ks, vs = cache.restore()
    for b in (3, 4):
        assert torch.equal(ks[b, :, :n], ks[1, :, :n]) and torch.equal(vs[b, :, :n], vs[1, :, :n])
    cache.fork([4, 3], [0, 4])
    assert everything(cache, c, 1)[0][1] == everything(cache, c, 2)[1][1]
