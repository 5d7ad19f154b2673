"""GPU tests of how many bits of fp32 rows and of the low-rank values the adapters' products hold: inputs whose sums are exact
in fp32 in any order, so that what is left out of an operand shows in the outputs of every type."""
from __future__ import annotations

import numpy as np
import pytest

from tests.blocks_oracle import STEP, TINY
from tests.gpu_common import cuda, to_host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def add(x, A, B, ab, out, scale=None):
    """Float64 outputs of one adapter for all rows, base 0."""
    import w4a8_quantized_gemm_token_amd as w4
    dev = lambda v, t: torch.as_tensor(np.ascontiguousarray(v)).to(cuda(), t)  # noqa: E731
    got = torch.zeros(x.shape[0], B.shape[0], dtype=TYPES[out], device=cuda())
    w4.lora_add(got, dev(x, torch.float32), torch.zeros(x.shape[0], dtype=torch.int32, device=cuda()), dev(A[None], TYPES[ab]),
                dev(B[None], TYPES[ab]), scale=None if scale is None else dev([scale], torch.float32))
    return to_host(got.double())


def full_rows(rng, M, K):
    """Values of [1, 2) with all 24 bits: sums of two of them, with signs that differ, are exact, and so are those of parts."""
    return (1.0 + rng.integers(0, 1 << 23, (M, K)) * 2.0 ** -23).astype(np.float32)


def check(got, value, error, out):
    """value is exact before the outputs' rounding but for `error`."""
    tol = STEP[out] * (np.abs(value) + error) + error + TINY[out]
    if out == "f32" and error == 0:
        tol = np.zeros_like(value)  # the differences have 24 bits at most
    bad = np.abs(got - value) > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside, {got[bad][0]!r} for {value[bad][0]!r}"


# v beside fp16 weights is two fp16 parts: half a step of 11 bits, and of what that leaves: 2^-23 of a value, here below 2
HELD = {"bf16": 0.0, "f16": 2.0 ** -22}


@pytest.mark.parametrize("M", [1, 20, 64, 150])
@pytest.mark.parametrize("out", sorted(TYPES))
@pytest.mark.parametrize("ab", ["f16", "bf16"])
def test_fp32_rows_that_cancel(ab, out, M):
    """v_j = x[k] - x[k'], each column one v_j: rows whose common part cancels leave the low bits of x."""
    rng = np.random.default_rng(M)
    K, R, N = 1032, 16, 80
    x, A, B = full_rows(rng, M, K), np.zeros((R, K)), np.zeros((N, R))
    for j in range(R):
        k = rng.choice(K, 2, replace=False)
        A[j, k] = 1.0, -1.0
    B[np.arange(N), np.arange(N) % R] = 1.0
    value = (x.astype(np.float64) @ A.T) @ B.T
    check(add(x, A, B, ab, out), value, HELD[ab], out)


@pytest.mark.parametrize("M", [1, 20, 64, 150])
@pytest.mark.parametrize("R", [16, 64, 128, 256])
@pytest.mark.parametrize("out", sorted(TYPES))
@pytest.mark.parametrize("ab", ["f16", "bf16"])
def test_low_rank_values_that_cancel(ab, out, R, M):
    """v_j = x[k_j] with all its bits, each column the difference of two."""
    rng = np.random.default_rng(M + R)
    K, N = 520, 150
    x, A, B = full_rows(rng, M, K), np.zeros((R, K)), np.zeros((N, R))
    A[np.arange(R), rng.choice(K, R, replace=False)] = 1.0
    for n in range(N):
        B[n, rng.choice(R, 2, replace=False)] = 1.0, -1.0
    value = (x.astype(np.float64) @ A.T) @ B.T
    check(add(x, A, B, ab, out), value, 2 * HELD[ab], out)


@pytest.mark.parametrize("out", sorted(TYPES))
def test_values_at_fp32s_end(out):
    """Values next to fp32's largest, which 8 bits would round to an infinity, stay what they are."""
    x = np.zeros((3, 64), np.float32)
    x[0, 3], x[1, 5], x[2, 7] = np.finfo(np.float32).max, -3.4e38, 3.3895e38
    A, B = np.zeros((8, 64)), np.zeros((20, 8))
    A[0, [3, 5, 7]] = 2.0 ** -20
    B[:, 0] = 2.0 ** -100  # (bf16: fp16 has no such weight)
    value = (x.astype(np.float64) @ A.T) @ B.T
    check(add(x, A, B, "bf16", out), value, 0.0, out)
