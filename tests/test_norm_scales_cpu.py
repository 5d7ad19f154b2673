"""The norms' scales: a number that could leave fp64's range on the way is refused, on the CPU."""
import ctypes

import pytest

import w4a8_quantized_gemm_token_amd as w4

EINVAL = 1


def call(res_scale, y_scale):
    f = lambda n: ctypes.c_void_p(4096 + n)  # noqa: E731
    return w4.load().w4a8_residual_norm_quantize(f(0), 0, 64, f(0), 0, 64, 4, 64, 1, None, None, None, 0, 0, res_scale, y_scale, f(65536),
                                                 64, 1, None, None, 1e-6, None, 0, 0, None, None, None)


@pytest.mark.parametrize("scale", [3.5e38, -1e39, 1e300, -1.7e308, float("inf"), float("nan")])
def test_scales_past_fp32(scale):
    assert call(scale, 1.0) == EINVAL and call(1.0, scale) == EINVAL
    assert b"scales" in w4.load().w4a8_last_error()
