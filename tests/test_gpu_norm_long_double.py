"""GPU tests of the norms between blocks against an 80-bit form, with the bound that the kernel's own sums give."""
from __future__ import annotations

import numpy as np
import pytest

from tests.gpu_common import cuda, to_dev, to_host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

X = np.longdouble

# In half steps of fp64, 2^-53.  A thread adds 32 values at most (four chunks of 8; rows of more than 16384 have four chunks a
# thread), then four steps inside 16 lanes, two over a wave and four over the waves: 42 additions.  With 1/H and its product
# the mean is off by 44 of the mean |u|, and the mean square, whose terms add the rounding of u - mean twice, by 46; eps and the
# root make half of that and four for the two Newton steps, 28, of the result.  u - mean, the root's, the weight's, the bias's, the
# gate's, the scale's and the join's products and sums: 8.  Together 44 + 28 + 8 = 80 of the size below: under 2^-46.
BOUND = X(2.0) ** -46


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert np.finfo(X).nmant >= 63
    yield
    torch.cuda.synchronize()


def norm(u, kind, w, b, eps):
    if kind == "none":
        return u, np.abs(u)
    mean = u.mean(1, keepdims=True) if kind == "layer" else X(0)
    spread = np.abs(u).mean(1, keepdims=True) if kind == "layer" else X(0)
    inv = 1 / np.sqrt(((u - mean) ** 2).mean(1, keepdims=True) + X(eps))
    return (u - mean) * inv * w + b, (np.abs(u) + spread) * inv * np.abs(w) + np.abs(b)


def check(got, value, size):
    """fp32 outputs: value rounded, for a value within the bound."""
    slack = BOUND * size
    lo, hi = (value - slack).astype(np.float32), (value + slack).astype(np.float32)
    bad = (got < lo) | (got > hi)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside, {got[bad][0]!r} for {value[bad][0]!r}"
    assert (lo == hi).mean() > 0.99  # (the bound leaves next to every output one value)


@pytest.mark.parametrize("kind", ["none", "rms", "layer"])
@pytest.mark.parametrize("M,H", [(1, 7168), (3, 64), (5, 1031), (4, 8192), (3, 8200), (2, 16384), (2, 20001), (3, 32768), (600, 5003)])
def test_against_80_bits(M, H, kind):
    import w4a8_quantized_gemm_token_amd as w4
    rng = np.random.default_rng(M + H)
    eps, rs, ys = 1e-6, 0.9, 1.25
    f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    res, y, g = f(M, H), f(M, H) + np.float32(0.5), f(H)
    w, b = rng.uniform(0.5, 1.5, H).astype(np.float32), f(H)
    named = {} if kind == "none" else dict(post_w=to_dev(w), post_b=to_dev(b), pre_w=to_dev(w), pre_b=to_dev(b))
    stream, z = torch.zeros(M, H, device=cuda()), torch.zeros(M, H, device=cuda())
    w4.prepare_residual_norm_quantize(to_dev(res), to_dev(y), (stream, z, None, None), post=kind, pre=kind, gate=to_dev(g), res_scale=rs,
                                      y_scale=ys, eps=eps, **named)()
    got, gz = to_host(stream), to_host(z)
    W, B = w.astype(X), b.astype(X)
    p, size = norm(y.astype(X), kind, W, B, eps)
    scale = X(ys) * g.astype(X)
    check(got, p * scale + X(rs) * res.astype(X), size * np.abs(scale) + np.abs(X(rs) * res.astype(X)))
    value, size = norm(got.astype(X), kind, W, B, eps)
    check(gz, value, size)
