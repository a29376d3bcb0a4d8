"""Counts and lengths of the prompt operators are integers of any kind; a fraction
is refused, never cut to the integer below it."""

import numpy as np
import pytest

kvq = pytest.importorskip("quantized_kv_cache_02_gb300")


def test_integers_of_any_kind():
    import torch
    for values in ([3, 0, 7], (3, 0, 7), np.array([3, 0, 7], np.int32), torch.tensor([3, 0, 7]),
                   [np.int64(3), torch.tensor(0), 7]):
        assert list(kvq.binding._counts(values)) == [3, 0, 7]


def test_fractions_are_refused():
    import torch
    for values in ([3, 0.5], [3.0], np.array([3.0]), torch.tensor([3.0]), ["3"], [None]):
        with pytest.raises(TypeError):
            kvq.binding._counts(values)
