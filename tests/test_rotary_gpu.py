"""Rotary positions against their formula in 64 bits.

Tolerances, per element, from the arithmetic, with u = 2^-24.  The angle in turns
is rounded to 2^-33, its part of a quadrant (at most an eighth of a turn, given to
sincospif as at most 1/4) to u of itself: 2 pi 2^-33 + pi u / 4 radians.  sincospif is
good to a step of values up to 1, u, taken twice.  The reference's own product of
position and frequency is off by u64 = 2^-53 of the angle, as is the fixed-point
fraction.  So cosine and sine are off by at most
    da = 2 pi 2^-33 + pi u / 4 + 2 u + 2 u64 |angle|,
an output by (|x1| + |x2|) da, u |x2| for the rounded product, u |y| for the sum, and
half a bf16 step, 2^-8 |y|, where it is rounded to bf16.
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


def normal(torch, shape, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(getattr(torch, dtype))


def reference(torch, x, positions, plan, inverse=False):
    """Output in 64 bits and its tolerance for x's dtype."""
    n = len(plan.frequencies)
    pos = positions if positions.dim() == 2 else positions[:, None]
    angle = pos[:, plan.axes].double() * torch.tensor(plan.frequencies, dtype=torch.float64, device="cuda")
    angle = (-angle if inverse else angle)[:, None]
    one, two = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if plan.interleaved else (slice(0, n), slice(n, 2 * n))
    y, tol = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    a, b = x[..., one].double(), x[..., two].double()
    y[..., one], y[..., two] = a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()
    da = 2 * math.pi * 2.0 ** -33 + math.pi * U / 4 + 2 * U + 2.0 ** -52 * angle.abs()
    tol[..., one] = (a.abs() + b.abs()) * da + U * (b.abs() + y[..., one].abs())
    tol[..., two] = (a.abs() + b.abs()) * da + U * (b.abs() + y[..., two].abs())
    if x.dtype == torch.bfloat16:
        tol[..., :2 * n] += 2.0 ** -8 * y[..., :2 * n].abs()
    return y, tol


def check(torch, got, x, positions, plan, inverse=False):
    want, tol = reference(torch, x, positions, plan, inverse)
    bad = (got.double() - want).abs() - tol
    assert bad.max() <= 0, (int(bad.argmax()), float(bad.max()))
    rest = 2 * len(plan.frequencies)
    assert torch.equal(got[..., rest:], x[..., rest:])


def positions_of(torch, tokens, axes, seed=0, reach=5000, dtype="int64"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-reach, reach, (tokens, axes), generator=g, device="cuda").to(getattr(torch, dtype))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("dim,sections", [(16, [8]), (128, [16, 24, 24]), (64, [32]), (64, [5, 9, 2, 3]), (128, [17]),
                                          (256, [128]), (256, [40, 88]), (80, [1]), (80, [12, 12, 16]), (48, [4, 4])])
def test_shapes(torch, kvq, dim, sections, dtype, interleaved):
    plan = kvq.Rotary.sections(dim, sections, interleaved=interleaved, restart=len(sections) == 3)
    for tokens, hq, hk in ((1, 8, 2), (33, 5, 1), (300, 3, 7)):
        q, k = normal(torch, (tokens, hq, dim), dtype, 1), normal(torch, (tokens, hk, dim), dtype, 2)
        at = positions_of(torch, tokens, len(sections), tokens)
        for inverse in (False, True):
            a, b = kvq.rotary(q, k, at, plan, inverse=inverse)
            check(torch, a, q, at, plan, inverse)
            check(torch, b, k, at, plan, inverse)


@pytest.mark.parametrize("tokens", [1, 2, 255, 4099])
def test_many_tokens_and_one_tensor(torch, kvq, tokens):
    plan = kvq.Rotary.sections(64, [32], theta=500000.0)
    q = normal(torch, (tokens, 40, 64), "bfloat16")
    at = torch.arange(tokens, device="cuda", dtype=torch.int32)
    a, b = kvq.rotary(q, None, at, plan)
    assert b is None
    check(torch, a, q, at, plan)


@pytest.mark.parametrize("at", [0, 1, 432000, 2 ** 31 - 1, -2 ** 31, 2 ** 40 + 12345])
def test_far_positions(torch, kvq, at):
    plan = kvq.Rotary(32, [1.0, 0.3, 1e-4, math.pi, 2 * math.pi, 0.0, -0.7, 1000.5])
    q = normal(torch, (5, 2, 32), "float32")
    for dtype in (torch.int64, torch.int32):
        if abs(at) < 2 ** 31 or dtype == torch.int64:
            p = torch.full((5, 1), at, device="cuda", dtype=dtype)
            check(torch, kvq.rotary(q, None, p, plan)[0], q, p, plan)


def test_strides_and_in_place(torch, kvq):
    """Slices of one fused projection, turned where they lie; head-major and padded
    outputs; positions by columns; rows past the tensors stay."""
    tokens, hq, hk, d = 77, 8, 2, 64
    plan = kvq.Rotary.sections(d, [8, 12, 12])
    at = positions_of(torch, tokens, 3).T.contiguous().T
    fused = normal(torch, (tokens + 1, (hq + 2 * hk) * d), "bfloat16")
    before = fused.clone()
    heads = fused[:tokens].view(tokens, hq + 2 * hk, d)
    q, k = heads[:, :hq], heads[:, hq:hq + hk]
    a, b = kvq.rotary(q, k, at, plan)
    assert torch.equal(fused, before)
    kvq.rotary(q, k, at, plan, q_out=q, k_out=k)
    assert torch.equal(q, a) and torch.equal(k, b)
    assert torch.equal(heads[:, hq + hk:], before[:tokens].view_as(heads)[:, hq + hk:]) and torch.equal(fused[-1], before[-1])
    for out in (torch.zeros(hq, tokens, d, device="cuda", dtype=torch.bfloat16).transpose(0, 1),
                torch.zeros(tokens, hq, 2 * d, device="cuda", dtype=torch.bfloat16)[..., :d]):
        kvq.rotary(before[:tokens].view_as(heads)[:, :hq], None, at, plan, q_out=out)
        assert torch.equal(out, a)


def test_turning_back_is_the_gradient(torch, kvq):
    plan = kvq.Rotary.sections(48, [7, 6], interleaved=True)
    x, w = normal(torch, (9, 3, 48), "float32", 1), normal(torch, (9, 3, 48), "float32", 2)
    at = positions_of(torch, 9, 2)
    grad = kvq.rotary(w, None, at, plan, inverse=True)[0]
    leaf = x.double().requires_grad_()
    (reference(torch, leaf, at, plan)[0] * w.double()).sum().backward()
    _, tol = reference(torch, w, at, plan, True)
    assert ((grad.double() - leaf.grad).abs() <= tol + 1e-15).all()
    # against differences: the loss is linear in x, so a difference of any step is the derivative but for
    # the two losses' rounding, that of their own outputs
    step = torch.zeros_like(x)
    step[4, 1, 5] = 0.5
    losses, slack = [], 0.0
    for y in (x + step, x - step):
        losses.append((kvq.rotary(y, None, at, plan)[0].double() * w.double()).sum())
        slack += float((reference(torch, y, at, plan)[1] * w.double().abs()).sum())
    assert abs(float(losses[0] - losses[1]) - float(grad[4, 1, 5])) <= slack + float(tol[4, 1, 5])


def test_infinite_channels_that_stay(torch, kvq):
    plan = kvq.Rotary(64, [1.0, 0.5, 0.25], interleaved=True)
    q = normal(torch, (4, 2, 64), "bfloat16")
    q[..., 6:] = math.inf
    q[1, 1, 7] = math.nan
    at = torch.arange(4, device="cuda")
    got = kvq.rotary(q, None, at, plan)[0]
    assert torch.equal(got[..., 6:].nan_to_num(7.0, 3.0), q[..., 6:].nan_to_num(7.0, 3.0))
    assert torch.isfinite(got[..., :6]).all()


def test_streams_and_graphs(torch, kvq):
    """On a stream of its own, and captured: a replay turns to the positions of its time."""
    plan = kvq.Rotary.sections(128, [64])
    q, k = normal(torch, (32, 32, 128), "bfloat16", 1), normal(torch, (32, 8, 128), "bfloat16", 2)
    at = torch.arange(32, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1000000)
        at += 1000
        a, b = kvq.rotary(q, k, at, plan)
    side.synchronize()
    check(torch, a, q, at, plan)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = kvq.rotary(q, k, at, plan)
    for step in (1, 500):
        at += step
        graph.replay()
        check(torch, a, q, at, plan)
        check(torch, b, k, at, plan)


def test_no_tokens(torch, kvq):
    plan = kvq.Rotary(64, [1.0])
    before = kvq.kvq_kernel_launches()
    a, b = kvq.rotary(torch.empty(0, 4, 64, device="cuda"), torch.empty(0, 1, 64, device="cuda"),
                      torch.empty(0, 1, device="cuda", dtype=torch.int64), plan)
    assert a.shape == (0, 4, 64) and b.shape == (0, 1, 64) and kvq.kvq_kernel_launches() == before


def test_refusals(torch, kvq):
    plan = kvq.Rotary.sections(64, [16, 16])
    q, at = normal(torch, (8, 4, 64), "bfloat16"), torch.zeros(8, 2, device="cuda", dtype=torch.int64)
    for args in [(q.half(), None, at), (q, None, at.double()), (q, None, at[:, :1]), (q, None, at[:7]),
                 (q, None, at.cpu()), (q[..., :32], None, at), (q, q[:7], at), (q, q.float(), at),
                 (q.transpose(1, 2), None, at), (q.cpu(), None, at), (q[0], None, at)]:
        with pytest.raises(AssertionError):
            kvq.rotary(*args, plan)
    with pytest.raises(AssertionError):
        kvq.rotary(q, None, at, plan, q_out=torch.empty(8, 4, 64, device="cuda"))
    wide = torch.empty(8, 4, 128, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(kvq.KVQError):  # in place with other strides
        kvq.rotary(wide[:4, :, :64], None, at[:4], plan, q_out=wide.view(16, 2, 128)[:4].view(4, 4, 64))
    with pytest.raises(kvq.KVQError):  # rows one over the other
        kvq.rotary(q, None, at, plan, q_out=wide.view(-1)[:64].expand(8, 4, 64))


@pytest.mark.parametrize("interleaved,pairs", [(False, 16), (True, 13), (False, 13)])
def test_offsets_past_32_bits(torch, kvq, interleaved, pairs):
    """Rows that lie a megabyte apart: the last ones past 2^32 elements."""
    tokens, step = 4200, 1 << 20
    buffer = torch.empty(tokens * step, dtype=torch.bfloat16, device="cuda")
    q, out = (buffer.as_strided((tokens, 2, 64), (step, 64, 1), at) for at in (0, step // 2))
    x = normal(torch, (tokens, 2, 64), "bfloat16")
    q.copy_(x)
    plan = kvq.Rotary.sections(64, [pairs], interleaved=interleaved)
    at = torch.arange(tokens, device="cuda")
    kvq.rotary(q, None, at, plan, q_out=out)
    assert torch.equal(out, kvq.rotary(x, None, at, plan)[0]) and torch.equal(q, x)
    check(torch, out, x, at, plan)
