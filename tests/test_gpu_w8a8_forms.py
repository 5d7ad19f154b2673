"""GPU tests of the 8-bit product's forms that its sizes alone do not reach: launches cut in two."""
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
    torch.cuda.empty_cache()


def w4mod():
    import w4a8_quantized_gemm_token_amd as w4
    return w4


def repeated(block, n):
    """n entries along dim 0: `block` over and over."""
    out = torch.empty((n, *block.shape[1:]), dtype=block.dtype, device=block.device)
    for i in range(0, n, block.shape[0]):
        out[i:i + block.shape[0]] = block[:min(block.shape[0], n - i)]
    return out


def expected(qa, sa, qw, sw, bias, dtype):
    """The stated fp32 steps on the exact sums (|sum| < 2^53, so fp64 holds it): the output's bytes."""
    v = (qa.double() @ qw.double().t().contiguous()).float() * sa[:, None] * sw[None, :]
    return (v if bias is None else v + bias).to(dtype)


@pytest.mark.parametrize("long_rows", [True, False])
def test_more_tiles_than_a_launch_has_threads_for(long_rows):
    """2^30 rows by one column and 17 rows by 2^30 columns: at 256 threads a tile of 64 this is 2^32 threads and
    more, and one launch may have fewer.  The long side repeats a block, and so do the outputs."""
    gen = torch.Generator(device=cuda()).manual_seed(7)
    K, P, L = 16, (1 << 20) + 7, (1 << 30) + 65

    def codes(n):
        return torch.randint(-127, 128, (n, K), dtype=torch.int8, device=cuda(), generator=gen)

    block, other = codes(P), codes(1 if long_rows else 17)
    sb, so = torch.rand(P, device=cuda(), generator=gen), torch.rand(other.shape[0], device=cuda(), generator=gen)
    long, sl = repeated(block, L), repeated(sb, L)
    if long_rows:
        bias = torch.rand(1, device=cuda(), generator=gen)
        got = w4mod().gemm_w8a8(long, sl, other, so, bias=bias, out_dtype=torch.float16).t()
        ref = expected(block, sb, other, so, bias, torch.float16).t()
    else:
        bb = torch.rand(P, device=cuda(), generator=gen)
        got = w4mod().gemm_w8a8(other, so, long, sl, bias=repeated(bb, L), out_dtype=torch.bfloat16)
        ref = expected(other, so, block, sb, bb, torch.bfloat16)
    whole = L // P * P
    for r in range(ref.shape[0]):
        assert bool((got[r, :whole].view(-1, P) == ref[r]).all()) and bool((got[r, whole:] == ref[r, :L - whole]).all()), r
