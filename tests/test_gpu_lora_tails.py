"""GPU tests of the adapters' last, partial window of 64 k: every length of it, in calls where a wave has whole windows in front of
it, where it is a wave's first, and where it is the only one."""
from __future__ import annotations

import numpy as np
import pytest

from tests import blocks_oracle as o
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


def check(M, K, N, R, x, ab, out):
    import w4a8_quantized_gemm_token_amd as w4
    rng = np.random.default_rng(K + M)
    L = 9  # more than eight adapters in a tile, and a rank of each its own
    ids = rng.integers(-1, L, M)
    ranks = [max(1, R >> (a % 3)) for a in range(L)]
    dev = lambda v, t: torch.as_tensor(np.ascontiguousarray(v)).to(cuda(), t)  # noqa: E731
    xs = dev(rng.standard_normal((M, K + 3)), TYPES[x])[:, :K]
    A, B = dev(rng.standard_normal((L, R, K)) / np.sqrt(K), TYPES[ab]), dev(rng.standard_normal((L, N, R)) / np.sqrt(R), TYPES[ab])
    base, scale = dev(rng.standard_normal((M, N)), TYPES[out]), rng.uniform(0.5, 2, L).astype(np.float32)
    got = torch.zeros_like(base)
    w4.lora_add(got, xs, dev(ids, torch.int32), A, B, scale=dev(scale, torch.float32), ranks=dev(ranks, torch.int32), base=base)
    h = lambda t: to_host(t.double())  # noqa: E731
    # the bound of fp32 outputs: the bits of x and of v do not turn on the output's type
    value, bound = o.lora(h(xs), ids, h(A), h(B), ranks, scale, h(base), "f32", x != "f32")
    o.close(h(got), value, bound, out, f"K={K}")


@pytest.mark.parametrize("tail", [8, 16, 24, 32, 40, 48, 56])
@pytest.mark.parametrize("windows", [0, 1, 7, 8, 9, 64])
def test_every_tail(windows, tail):
    K = 64 * windows + tail
    for i, (x, ab, out) in enumerate((("f16", "f16", "f16"), ("bf16", "bf16", "f32"), ("f32", "bf16", "bf16"), ("f32", "f16", "f32"),
                                      ("f16", "bf16", "f32"), ("bf16", "f16", "f16"))):
        check((1, 20, 77)[i % 3], K, 45, (16, 24, 64)[i % 3], x, ab, out)
        check((77, 1, 20)[i % 3], K, 45, (24, 72, 8)[i % 3], x, ab, out)
