"""Strides of a dimension of one entry are not looked at: the call's next check is
what refuses it."""

import ctypes

import pytest

pytest.importorskip("quantized_kv_cache_02_gb300")
import test_prompt_host as H  # noqa: E402

NULL = ctypes.c_void_p()
BAD = [0, -64, 3, 60, 1 << 45]


def refusal():
    return H.kvq.load_library().kvq_last_error()


@pytest.mark.parametrize("bad", BAD)
def test_of_one_token(bad):
    for t in ("q", "k", "v"):
        p, keep_alive = H.prompt(lens=(1,), n_tokens=1, **{f"{t}_token_stride": bad})
        assert H.attention(p, out=NULL) == H.B.KVQ_EINVAL and refusal().startswith(b"out must"), t
        # the same stride counts with a second token
        p, keep_alive = H.prompt(lens=(1,), n_tokens=2, **{f"{t}_token_stride": bad})
        assert H.attention(p, out=NULL) != H.B.KVQ_OK and refusal().startswith(t.encode() + b" strides"), t
    p, keep_alive = H.prompt(lens=(1,), n_tokens=1, k_token_stride=bad)
    assert H.weights(p, k=NULL) == H.B.KVQ_EINVAL and refusal().startswith(b"k must")
    p, keep_alive = H.prompt(lens=(1,), n_tokens=1, k_token_stride=bad, v_token_stride=bad)
    assert H.evict(p, keep=(1,), ko=NULL) == H.B.KVQ_EINVAL and refusal().startswith(b"k_out")
    p, keep_alive = H.prompt(lens=(1,), n_tokens=1, out_token_stride=bad)
    assert H.attention(p) != H.B.KVQ_OK and b"strides" not in refusal()  # no device, or not its memory


@pytest.mark.parametrize("bad", BAD)
def test_of_one_head(bad):
    for t in ("k", "v"):
        p, keep_alive = H.prompt(n_kv_heads=1, **{f"{t}_head_stride": bad})
        assert H.attention(p, out=NULL) == H.B.KVQ_EINVAL and refusal().startswith(b"out must"), t
    one = dict(n_kv_heads=1, n_q_heads=1, q_token_stride=64, k_token_stride=64, v_token_stride=64, out_token_stride=64)
    p, keep_alive = H.prompt(**one, q_head_stride=bad, k_head_stride=bad, v_head_stride=bad, out_head_stride=bad)
    assert H.attention(p) != H.B.KVQ_OK and b"strides" not in refusal()
    assert H.evict(p, ko=NULL) == H.B.KVQ_EINVAL and refusal().startswith(b"k_out")
