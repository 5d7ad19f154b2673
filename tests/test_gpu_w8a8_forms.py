"""GPU tests of the 8-bit product by form: every split of k of the few-row loop, launches cut in two."""
from __future__ import annotations

import numpy as np
import pytest

from tests.gpu_common import cuda
from tests.test_gpu_w8a8 import dense, grouped

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


# k by which the few-row loop gives each wave 1, 2, 3 or 4 windows of 128 in one pass, or takes several passes;
# with and without a part window, waves and windows without a share, and the full 16 waves
FEW_ROW_K = [144, 2048, 2064, 3600, 4096, 2576, 4112, 4224, 5376, 6016, 6144, 3968, 7152, 7168, 8192, 8208, 24592]


@pytest.mark.parametrize("K", FEW_ROW_K)
@pytest.mark.parametrize("M", [1, 7, 16])
def test_few_rows_every_split_of_k(M, K):
    dense(np.random.default_rng(K + M), M, K, 16390, M == 7, "bf16" if M == 16 else "f32")


@pytest.mark.parametrize("K", FEW_ROW_K)
def test_few_slots_every_split_of_k(K):
    grouped(np.random.default_rng(K), [1, 16, 0, 3, 9, 2, 16, 1], K, 1552)


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
