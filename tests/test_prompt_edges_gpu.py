"""Calls of the prompt operators that the documentation allows at its edges, and refusals on the device."""

import pytest

from test_prompt_gpu import inputs, kvq, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def test_counts_past_the_lengths_are_refused(torch, kvq):  # noqa: F811
    """Whatever their size: nothing is allocated for them."""
    _, k, v = inputs(torch, 60, 2, 2, 64, "bfloat16", 22)
    w = torch.rand(2, 60, device="cuda")
    before = torch.cuda.max_memory_allocated()
    for keep in ([41, 20], [10 ** 11, 20], [10 ** 13, 20], [40, 10 ** 18], [-10 ** 13, 20], [-1, 10 ** 13]):
        with pytest.raises(kvq.KVQError) as e:
            kvq.evict(k, v, w, [40, 20], keep)
        assert e.value.status == kvq.binding.KVQ_EINVAL
    assert torch.cuda.max_memory_allocated() - before < 1 << 20


@pytest.mark.parametrize("d,dtype", [(128, "bfloat16"), (64, "bfloat16"), (48, "bfloat16"), (64, "float32")])
def test_strides_of_dimensions_of_one_entry_are_not_used(torch, kvq, d, dtype):  # noqa: F811
    q, k, v = inputs(torch, 1, 1, 1, d, dtype, 23)
    want, lse = kvq.prompt_attention(q, k, v, [1])
    odd = [t.as_strided((1, 1, d), s) for t, s in zip((q, k, v), ((3, 7, 1), (0, 0, 1), (1 << 40, 5, 1)))]
    out = torch.empty_like(q).as_strided((1, 1, d), (0, 1, 1))
    _, l2 = kvq.prompt_attention(*odd, [1], out=out)
    assert torch.equal(out.reshape(-1), v.reshape(-1)) and torch.equal(want.reshape(-1), v.reshape(-1))
    assert torch.equal(lse, l2)
    w = kvq.prompt_weights(odd[0], odd[1], lse, [1], 1)
    assert torch.equal(w, kvq.prompt_weights(q, k, lse, [1], 1))
    kept = kvq.evict(odd[1], odd[2], w, [1], 1)
    assert torch.equal(kept.k, k[:, 0]) and torch.equal(kept.v, v[:, 0])
    # one KV head of several tokens, one token of several heads
    q, k, v = inputs(torch, 70, 4, 1, d, dtype, 24)
    want, lse = kvq.prompt_attention(q, k, v, [70])
    one = [t.as_strided((70, 1, d), (d, s, 1)) for t, s in ((k, 3), (v, 0))]
    assert torch.equal(kvq.prompt_attention(q, *one, [70])[0], want)
    assert torch.equal(kvq.prompt_weights(q, one[0], lse, [70], 9), kvq.prompt_weights(q, k, lse, [70], 9))
    q, k, v = inputs(torch, 1, 4, 2, d, dtype, 25)
    one = [t.as_strided((1, t.shape[1], d), (s, d, 1)) for t, s in ((q, 9), (k, 0), (v, 1))]
    assert torch.equal(kvq.prompt_attention(*one, [1])[0], kvq.prompt_attention(q, k, v, [1])[0])


def test_fractions_are_no_counts(torch, kvq):  # noqa: F811
    q, k, v = inputs(torch, 40, 2, 2, 64, "bfloat16", 26)
    lse = torch.zeros(2, 40, device="cuda")
    w = torch.rand(2, 40, device="cuda")
    for bad in (lambda: kvq.prompt_attention(q, k, v, [39.5]), lambda: kvq.prompt_weights(q, k, lse, [40], 3.5),
                lambda: kvq.evict(k, v, w, [20, 20], [0.5, 0.5]), lambda: kvq.evict(k, v, w, [40], 0.5),
                lambda: kvq.evict(k, v, w, [40], 10, first=0.5), lambda: kvq.evict(k, v, w, [40], 10, recent=1.5)):
        with pytest.raises(TypeError):
            bad()


@pytest.mark.parametrize("d,dtype", [(128, "bfloat16"), (64, "bfloat16"), (96, "bfloat16"), (128, "float32")])
def test_infinite_scores(torch, kvq, d, dtype):  # noqa: F811
    """Plus infinity makes out and lse of its rows NaN and reaches no other; rows of minus infinity alone
    have an lse of minus infinity."""
    n, hq, hkv = 400, 4, 2
    q, k, v = inputs(torch, n, hq, hkv, d, dtype, 27)
    q[..., 0], k[..., 0] = 1.0, 0.0
    want, lse = kvq.prompt_attention(q, k, v, [n])
    high = k.clone()
    high[333, 1, 0] = torch.inf
    got, l2 = kvq.prompt_attention(q, high, v, [n])
    assert got[333:, 2:].isnan().all() and l2[2:, 333:].isnan().all()
    got[333:, 2:], l2[2:, 333:] = want[333:, 2:], lse[2:, 333:]
    assert torch.equal(got, want) and torch.equal(l2, lse)
    low = k.clone()
    low[:140, 0, 0] = -torch.inf
    got, l2 = kvq.prompt_attention(q, low, v, [n])
    assert got[:140, :2].isnan().all() and l2[:2, :140].isneginf().all()
    assert got[140:].isfinite().all() and l2[:2, 140:].isfinite().all()
    assert torch.equal(got[:, 2:], want[:, 2:]) and torch.equal(l2[2:], lse[2:])
