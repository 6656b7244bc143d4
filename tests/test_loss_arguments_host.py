"""Arguments of the vocabulary-row losses that no call has in earnest, refused
before any CUDA call: extents past 64 bits, temperatures past fp32."""
import numpy as np
import pytest

import fsdp_sharded_mixed_gb300 as zs

BUF = np.zeros(1 << 12, np.uint8)
P = BUF.ctypes.data + (-BUF.ctypes.data) % 16   # an aligned host address


def _logprobs(dtype=zs.ZS_FP32, rows=1, vocab=8, stride=8, T=1.0):
    zs.zs_token_logprobs(P, dtype, rows, vocab, stride, None, T, lse=P + 256, stream=0)


def _logprobs_grad(dtype=zs.ZS_FP32, rows=1, vocab=8, stride=8, gstride=8, T=1.0):
    zs.zs_token_logprobs_grad(P, dtype, rows, vocab, stride, P + 64, T, P + 128, None, P + 192,
                              None, P + 256, gstride, stream=0)


# Extents whose bytes 64 bits would hold as 0, a few or negative, and the least one refused.
WRAPPING = [((1 << 24) + 1, 1 << 40), ((1 << 22) + 1, 1 << 40), ((1 << 31) - 1, 1 << 40),
            ((1 << 31) - 1, 1 << 33), ((1 << 30) + 1, 1 << 34), (17, 1 << 40)]


@pytest.mark.parametrize("dtype", [zs.ZS_BF16, zs.ZS_FP32])
@pytest.mark.parametrize("rows,stride", WRAPPING)
def test_extents_past_what_a_device_holds_are_refused(rows, stride, dtype):
    with pytest.raises(zs.ZsError, match="row_stride") as e:
        _logprobs(dtype, rows, stride=stride)
    assert e.value.status == zs.ZS_ERR_RANGE
    with pytest.raises(zs.ZsError, match="row_stride") as e:
        _logprobs_grad(dtype, rows, stride=stride)
    assert e.value.status == zs.ZS_ERR_RANGE
    with pytest.raises(zs.ZsError, match="grad_stride") as e:
        _logprobs_grad(dtype, rows, gstride=stride)
    assert e.value.status == zs.ZS_ERR_RANGE


def test_the_largest_extents_are_not():
    """They come to the next check (these addresses are the host's)."""
    for rows, stride in ((1, 1 << 40), (16, 1 << 40), ((1 << 31) - 1, 8192)):
        with pytest.raises(zs.ZsError) as e:
            _logprobs(zs.ZS_FP32, rows, stride=stride)
        assert e.value.status == zs.ZS_ERR_INVAL, str(e.value)


@pytest.mark.parametrize("T", [1e-39, 3e-39, 4.2e-39, 9e-39, 2e37, 1e38, 1e40, 7e44])
def test_temperatures_past_fp32_are_refused(T):
    """Of these 1/T or log2(e)/T is infinite in fp32 or below its normal range, or
    ln(vocab) T is infinite."""
    for call in (_logprobs, _logprobs_grad):
        with pytest.raises(zs.ZsError, match="temperature") as e:
            call(T=T)
        assert e.value.status == zs.ZS_ERR_INVAL


@pytest.mark.parametrize("T", [1e-38, 1e-9, 1.0, 1e9, 1e37])
def test_temperatures_within_fp32_are_not(T):
    for call in (_logprobs, _logprobs_grad):
        with pytest.raises(zs.ZsError) as e:
            call(T=T)
        assert "temperature" not in str(e.value)
