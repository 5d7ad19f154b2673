"""GPU tests of the 8-bit product by form: every split of k of the few-row loop, special values through every form's
epilogue, offsets that are not ascending, launches cut in two."""
from __future__ import annotations

import numpy as np
import pytest

from tests.gpu_common import cuda
from tests.test_gpu_w8a8 import LOOPS, TYPES, dense, grouped

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


def expected(qa, sa, qw, sw, bias, dtype):
    """The stated fp32 steps on the exact sums (|sum| < 2^53, so fp64 holds it): the output's bytes."""
    v = (qa.double() @ qw.double().t().contiguous()).float() * sa[:, None] * sw[None, :]
    return (v if bias is None else v + bias).to(dtype)


def same(got, ref):
    """Equal, NaN where the other is."""
    return bool(((got == ref) | (got.isnan() & ref.isnan())).all())


def special(gen, rows, *cols):
    """Scales of rows and columns, zero, infinite, NaN, huge and subnormal ones among them, first and last."""
    sa = torch.rand(rows, device=cuda(), generator=gen)
    sw = torch.rand(*cols, device=cuda(), generator=gen)
    if rows > 4:
        sa[0], sa[1], sa[2], sa[-1] = 0.0, float("nan"), 1e-42, float("inf")
    sw[..., 0], sw[..., 5], sw[..., 6], sw[..., 7] = 0.0, float("inf"), 1e30, float("nan")
    sw[..., -2], sw[..., -1] = 1e-42, float("inf")
    return sa, sw


def ints(gen, *shape):
    return torch.randint(-127, 128, shape, dtype=torch.int8, device=cuda(), generator=gen)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("M,N", LOOPS + [(20, 70)])
def test_special_values_in_every_form(M, N, dtype):
    """Scales and biases that are not ordinary numbers reach exactly their row or column, and fp16 outputs past the
    range become infinite, in every loop and tile."""
    gen = torch.Generator(device=cuda()).manual_seed(M + N)
    K = 272
    qa, qw = ints(gen, M, K), ints(gen, N, K)
    sa, sw = special(gen, M, N)
    bias = torch.randn(N, device=cuda(), generator=gen)
    bias[3], bias[9], bias[N - 3] = float("-inf"), float("inf"), float("nan")
    for b in (None, bias):
        got = w4mod().gemm_w8a8(qa, sa, qw, sw, bias=b, out_dtype=TYPES[dtype])
        assert same(got, expected(qa, sa, qw, sw, b, TYPES[dtype])), b is None


def test_special_values_per_expert():
    """The same through both loops of the expert product."""
    gen = torch.Generator(device=cuda()).manual_seed(3)
    K, N, counts = 272, 530, [3, 40, 0, 16, 150, 1]
    S, E = sum(counts), len(counts)
    qa, qw = ints(gen, S, K), ints(gen, E, N, K)
    sa, sw = special(gen, S, E, N)
    off = [sum(counts[:e]) for e in range(E + 1)]
    got = w4mod().moe_grouped_gemm_w8a8(qa, sa, None, torch.tensor(off, dtype=torch.int32, device=cuda()), qw, sw, S)
    for e in range(E):
        s = slice(off[e], off[e + 1])
        assert same(got[s], expected(qa[s], sa[s], qw[e], sw[e], None, torch.float32)), e


@pytest.mark.parametrize("S", [12, 300])
def test_offsets_that_are_not_ascending_are_written(S):
    """Eight experts claim all slots and eight claim none: at least the first one's blocks fit under the limit on the
    work, so every row is written, each value by an expert that claims it, and none behind max_slots."""
    gen = torch.Generator(device=cuda()).manual_seed(11)
    K, N, E = 64, 48, 16
    qa, qw = ints(gen, S, K), ints(gen, E, N, K)
    sa, sw = torch.rand(S, device=cuda(), generator=gen), torch.rand(E, N, device=cuda(), generator=gen)
    off = torch.tensor([0, 2 ** 31 - 1] * 8 + [-5], dtype=torch.int32, device=cuda())
    buf = torch.full((S + 20, N), float("nan"), device=cuda())
    w4mod().moe_grouped_gemm_w8a8(qa, sa, None, off, qw, sw, S, out=buf[:S])
    assert bool(buf[S:].isnan().all())
    claims = torch.stack([expected(qa, sa, qw[e], sw[e], None, torch.float32) for e in range(0, E, 2)])
    assert bool((buf[:S] == claims).any(0).all())


def repeated(block, n):
    """n entries along dim 0: `block` over and over."""
    out = torch.empty((n, *block.shape[1:]), dtype=block.dtype, device=block.device)
    for i in range(0, n, block.shape[0]):
        out[i:i + block.shape[0]] = block[:min(block.shape[0], n - i)]
    return out


@pytest.mark.parametrize("long_rows", [True, False])
def test_more_tiles_than_a_launch_has_threads_for(long_rows):
    """2^30 rows by one column and 17 rows by 2^30 columns: at 256 threads a tile of 64 this is 2^32 threads and
    more, and one launch may have fewer.  The long side repeats a block, and so do the outputs."""
    gen = torch.Generator(device=cuda()).manual_seed(7)
    K, P, L = 16, (1 << 20) + 7, (1 << 30) + 65

    block, other = ints(gen, P, K), ints(gen, 1 if long_rows else 17, K)
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
