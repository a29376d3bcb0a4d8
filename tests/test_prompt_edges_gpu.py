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
