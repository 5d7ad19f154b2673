"""GPU tests of the norms between blocks beside 80-bit forms, and at the ends of what the scales may be."""
from __future__ import annotations

import numpy as np
import pytest

from tests.gpu_common import cuda, to_dev, to_host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def test_largest_scales():
    """Rows of zeros, weights and gates of zero, and the largest scales: 1 / sqrt(eps) = 1e20 meets 3.4e38 and stays a number."""
    import w4a8_quantized_gemm_token_amd as w4
    M, H, top = 4, 520, float(np.finfo(np.float32).max)
    y = np.zeros((M, H), np.float32)
    y[1, ::2], y[2], y[3] = 1e-30, 3e38, 1.0
    w, g = np.ones(H, np.float32), np.ones(H, np.float32)
    w[::3], g[::5] = 0.0, 0.0
    for scale in (top, -top):
        out = torch.full((M, H), 7.0, device=cuda())
        w4.prepare_residual_norm_quantize(to_dev(np.zeros((M, H), np.float32)), to_dev(y), (out, None, None, None), post="rms",
                                          post_w=to_dev(w), gate=to_dev(g), y_scale=scale, res_scale=top, pre="none", eps=1e-40)()
        got = to_host(out).astype(np.float64)
        zero = (y == 0) | (w == 0) | (g == 0)
        assert not got[zero].any() and not np.isnan(got).any()
        # RMS of a row of 1e-30 in every other element, beside eps: 1e-30 / sqrt(5e-61 + 1e-40) = 1e-10; of one value: 1
        with np.errstate(over="ignore"):
            one = y[1, 0].astype(np.float64) / np.sqrt((y[1].astype(np.float64) ** 2).mean() + 1e-40) * scale
        live = ~zero
        assert np.allclose(got[1][live[1]], one, rtol=2.0 ** -22, atol=0)
        assert np.allclose(got[2:][live[2:]], scale, rtol=2.0 ** -22, atol=0)
