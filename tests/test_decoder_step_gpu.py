"""One decoder layer's attention through the operators as they are used together: a
prompt's queries and Keys turned to their positions, its causal attention, its Keys and
Values into a cache, the cache forked into samples, and then steps of one token a
sample: turned, appended and attended, beside a cross attention to an encoder's states."""

import math

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


def turned(torch, x, at, plan):
    n = len(plan.frequencies)
    angle = (at[:, plan.axes].double() * torch.tensor(plan.frequencies, dtype=torch.float64, device="cuda"))[:, None]
    a, b = x[..., :n].double(), x[..., n:2 * n].double()
    return torch.cat((a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos(), x[..., 2 * n:].double()), -1)


def attend(torch, q, k, v, causal=False):
    """q [n, hq, d], k, v [m, hkv, d] in 64 bits."""
    g = q.shape[1] // k.shape[1]
    z = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(g, 1)) / math.sqrt(q.shape[2])
    if causal:
        z = z.masked_fill(torch.ones(z.shape[1:], dtype=torch.bool, device="cuda").triu(1), -math.inf)
    return torch.einsum("hij,jhd->ihd", z.softmax(2), v.repeat_interleave(g, 1))


@pytest.mark.parametrize("paged", [False, True])
def test_prompt_fork_and_steps(torch, kvq, paged):
    frames, height, width, hq, hkv, d, samples, steps = 3, 8, 10, 8, 2, 128, 4, 6
    n = frames * height * width
    g = torch.Generator(device="cuda").manual_seed(11)

    def rows(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    t = torch.arange(n, device="cuda")
    at = torch.stack((t // (height * width), t // width % height, t % width), 1)
    plan = kvq.Rotary.sections(d, [16, 20, 20])  # the last sixteen channels stay
    q, k, v = rows(n, hq, d), rows(n, hkv, d), rows(n, hkv, d)
    states = rows(77, hkv, d), rows(77, hkv, d)
    qr, kr = kvq.rotary(q, k, at, plan)
    # each rounded once: half a bf16 step, and as much again for all that is fp32
    for got, x in ((qr, q), (kr, k)):
        want = turned(torch, x, at, plan)
        assert ((got.double() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-5).all()
    out, _ = kvq.prompt_attention(qr, kr, v, [n])
    want = attend(torch, qr.double(), kr.double(), v.double(), True)
    # weights and output rounded to bf16, half a step each of at most max |v|, and as much again
    slack = 2.0 ** -6 * v.double().abs().max()
    assert ((out.double() - want).abs() <= slack).all()
    crossed, _ = kvq.cross_attention(out, *states, [n], [77])
    want = attend(torch, out.double(), states[0].double(), states[1].double())
    assert ((crossed.double() - want).abs() <= 2.0 ** -6 * states[1].double().abs().max()).all()

    cache = kvq.KVQCache(samples, hkv, hq, d, 64, 32, 127, n + steps, pool_blocks=samples * 8 if paged else 0)
    cache.append(kr.transpose(0, 1)[None].contiguous(), v.transpose(0, 1)[None].contiguous())
    cache.fork(0, list(range(1, samples)))
    assert all(cache.seq_state(b)["total"] == n for b in range(samples))
    held_k, held_v = cache.restore(out_dtype="fp32")
    assert all(torch.equal(held_k[b], held_k[0]) and torch.equal(held_v[b], held_v[0]) for b in range(samples))
    new = [[], []]
    for step in range(steps):
        q, k, v = rows(samples, hq, d), rows(samples, hkv, d), rows(samples, hkv, d)
        at = torch.tensor([[frames, step // width, step % width]], device="cuda").expand(samples, 3)
        qr, kr = kvq.rotary(q, k, at, plan)
        out = cache.decode_step(kr[:, :, None], v[:, :, None], qr)
        new[0].append(kr), new[1].append(v)
        for b in range(samples):
            # what the cache holds: the prompt's restored rows, then this sample's own tokens
            ks, vs = (torch.cat((h[b].transpose(0, 1).double(), torch.stack([x[b] for x in y]).double()))
                      for h, y in zip((held_k, held_v), new))
            want = attend(torch, qr[b][None].double(), ks, vs)[0]
            assert ((out[b].double() - want).abs() <= 1e-3 + 1e-2 * want.abs()).all(), (step, b)
        # the samples share the encoder's states
        crossed, _ = kvq.cross_attention(out.bfloat16(), *states, [1] * samples, [77] * samples, [0] * samples)
        want = attend(torch, out.bfloat16().double(), states[0].double(), states[1].double())
        assert ((crossed.double() - want).abs() <= 2.0 ** -6 * states[1].double().abs().max()).all()
    assert kvq.prompt_status() == 0 and cache.device_status() == 0
