"""GPU tests of the adapters at the ends of fp32's range: rows of the low-rank values that are scaled by a power of two."""
from __future__ import annotations

import numpy as np
import pytest

from tests import blocks_oracle as o
from tests.gpu_common import cuda, to_host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def call(x, A, B, scale, ab, x_type=torch.bfloat16):
    import w4a8_quantized_gemm_token_amd as w4
    dev = lambda v, t: torch.as_tensor(np.ascontiguousarray(v)).to(cuda(), t)  # noqa: E731
    out = torch.zeros(x.shape[0], B.shape[1], device=cuda())
    w4.lora_add(out, dev(x, x_type), torch.zeros(x.shape[0], dtype=torch.int32, device=cuda()), dev(A, TYPES[ab]), dev(B, TYPES[ab]),
                scale=dev(scale, torch.float32))
    return to_host(out).astype(np.float64)


def case(M, K, R, N, low, high, scale, seed):
    """v = R of a row's bf16 entries, rows from 2^low to 2^high; fp16 weights."""
    rng = np.random.default_rng(seed)
    x = np.ldexp(rng.uniform(1, 2, (M, K)), np.rint(np.linspace(low, high, M)).astype(int)[:, None])
    x = torch.as_tensor(x).to(torch.bfloat16).double().numpy()
    A = np.zeros((1, R, K))
    A[0, np.arange(R), rng.choice(K, R, replace=False)] = 1.0
    B = torch.as_tensor(rng.standard_normal((1, N, R))).half().double().numpy()
    return x, A, B, np.array([scale], np.float32)


@pytest.mark.parametrize("ab", sorted(TYPES))
@pytest.mark.parametrize("M,N,R", [(1, 40, 8), (17, 130, 16), (70, 33, 64), (200, 96, 136)])
def test_tiny_rows(M, N, R, ab):
    """Terms of 2^-131 to 2^-90, of ordinary weights and a scale below one: as near as any, to fp32's last subnormal."""
    x, A, B, scale = case(M, 264, R, N, -125, -100, 0.7 * 2.0 ** -6, M)
    if ab == "bf16":
        B = torch.as_tensor(B).bfloat16().double().numpy()
    value, bound = o.lora(x, [0] * M, A, B, None, scale, np.zeros((M, N)), "f32", True)
    # the sum before the scale and the outputs are rounded to fp32's steps of 2^-149 at the least
    o.close(call(x, A, B, scale, ab), value, bound + 2.0 ** -148, "f32")


@pytest.mark.parametrize("M,N,R", [(1, 40, 8), (17, 130, 16), (70, 33, 64), (200, 96, 136)])
def test_huge_rows(M, N, R):
    """Rows up to 2^126 against weights of 2^-20 and 0, and a scale of 2^18: every term is finite, and those of 0 are 0."""
    x, A, B, scale = case(M, 264, R, N, 90, 126, 2.0 ** 18, M)
    B = torch.as_tensor(B * 2.0 ** -22 / R).half().double().numpy()
    B[:, ::3] = 0.0
    value, bound = o.lora(x, [0] * M, A, B, None, scale, np.zeros((M, N)), "f32", True)
    got = call(x, A, B, scale, "f16")
    assert np.isfinite(got).all() and not got[:, ::3].any()
    o.close(got, value, bound, "f32")
