"""GPU tests of the adapters above 64 tiles of 64 rows with k shared out over several ranges: the table of groups that a launch of
its own makes, its ranges, their parts of the low-rank values, and a last slab with other ranges than the first."""
from __future__ import annotations

import pytest

from tests.blocks_oracle import STEP, TINY
from tests.gpu_common import cuda

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SLAB = 32768


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def ranges(ids, L, K, R):
    """Ranges of k of a slab of these rows."""
    rows, windows = len(ids), -(-K // 64)
    tiles = -(-rows // 64)
    groups = sum(len({a for a in ids[t * 64:t * 64 + 64] if 0 <= a < L}) for t in range(tiles))
    units = groups * (1 if R <= 64 else -(-R // 64))
    most = max(1, min(max(4, 512 // tiles), windows // 8))
    worth = 16384 * groups // (rows * R)
    wanted = max(1, min(max(-(-128 // units), min(max(4, 512 // units), worth)), most))
    per = -(-windows // wanted)
    return -(-windows // per)


def check(M, K, N, R, L, how, x, ab, out, ranks=None, in_place=True):
    import w4a8_quantized_gemm_token_amd as w4
    gen = torch.Generator(device=cuda()).manual_seed(M + K + R)
    rand = lambda *s: torch.randn(*s, generator=gen, device=cuda())  # noqa: E731
    xs = rand(M, K).mul_(torch.exp(0.5 * rand(M, 1))).to(TYPES[x])
    A, B = (rand(L, R, K) / K ** 0.5).to(TYPES[ab]), (rand(L, N, R) / R ** 0.5).to(TYPES[ab])
    base = rand(M, N).to(TYPES[out])
    ids = torch.randint(-1 if how == "holes" else 0, L, (M,), generator=gen, device=cuda(), dtype=torch.int32)
    if how == "sorted":
        ids = ids.sort().values.contiguous()
    scale = 0.5 + torch.rand(L, generator=gen, device=cuda())
    rk = None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device=cuda())
    host = ids.tolist()
    slabs = [ranges(host[m:m + SLAB], L, K, R) for m in range(0, M, SLAB)]
    assert all(n > 1 for n in slabs) and -(-min(M, SLAB) // 64) > 64, slabs
    got = base.clone() if in_place else torch.zeros_like(base)
    w4.lora_add(got, xs, ids, A, B, scale=scale, ranks=rk, base=None if in_place else base)
    del rand
    # the bound of blocks_oracle.lora, with all of x and of v held: a step 2^-23 for each of the 32 products of a matrix
    # instruction and the K / 32 (rank / 32) of them in a row and 8 waves and the ranges added up, 2^-21 for what is left of v
    u, held = 2.0 ** -23, 2.0 ** -21
    for a in range(-1, L):
        at = torch.nonzero(ids == a).flatten()
        for rows in at.split(4096):
            have = base[rows].double()
            j = R if rk is None or a < 0 else ranks[a]
            if a < 0 or j == 0:
                assert torch.equal(got[rows], base[rows])
                continue
            x64, A64, B64, s = xs[rows].double(), A[a, :j].double(), B[a, :, :j].double(), float(scale[a])
            v, size = x64 @ A64.t().contiguous(), x64.abs() @ A64.abs().t().contiguous()
            verr = size * ((32 + K / 32 + 24) * u + held)
            t = s * (v @ B64.t().contiguous())
            tsize = (v.abs() + verr) @ B64.abs().t().contiguous()
            err = s * (verr @ B64.abs().t().contiguous() + tsize * ((32 + j / 32 + 2) * u + held)) + u * (have.abs() + t.abs())
            value = have + t
            tol = err * (1 + STEP[out]) + STEP[out] * (value.abs() + err) + TINY[out]
            bad = (got[rows].double() - value).abs() > tol
            assert not bool(bad.any()), f"adapter {a}: {int(bad.sum())} of {bad.numel()} outside"
    return slabs


@pytest.mark.parametrize("out", sorted(TYPES))
@pytest.mark.parametrize("ab", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,R,how", [(4161, 2056, 24, "sorted"), (4161, 4096, 136, "mixed"), (5000, 4096, 24, "mixed"),
                                       (5000, 2056, 136, "holes")])
def test_several_ranges_of_many_tiles(M, K, R, how, ab, out):
    check(M, K, 130, R, 5, how, "f32", ab, out, in_place=how != "holes")


@pytest.mark.parametrize("x", sorted(TYPES))
def test_row_types(x):
    check(4500, 3000, 70, 64, 3, "mixed", x, "bf16", "f32")
    check(9000, 1024, 33, 8, 2, "holes", x, "f16", "bf16", in_place=False)


def test_mixed_ranks_of_many_tiles():
    check(4700, 2048, 90, 72, 5, "mixed", "bf16", "bf16", "f32", ranks=[0, 1, 17, 64, 72])


@pytest.mark.parametrize("K,ab", [(2048, "bf16"), (8192, "f16")])
def test_last_slab_has_ranges_of_its_own(K, ab):
    """32768 rows and 70 more: with k 8192 the short slab shares k out further than the first."""
    slabs = check(SLAB + 70, K, 40, 16, 4, "mixed", "bf16", ab, "f32")
    assert len(slabs) == 2 and (K == 2048 or slabs[1] > slabs[0]), slabs
