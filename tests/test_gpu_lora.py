"""GPU tests of the low-rank adapters against their 64-bit form (blocks_oracle.lora)."""
from __future__ import annotations

import numpy as np
import pytest

from tests import blocks_oracle as o
from tests.gpu_common import cuda, to_host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SENTINEL = -7.0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def w4mod():
    import w4a8_quantized_gemm_token_amd as w4
    return w4


def rows(values, kind, ld=None, shift=0):
    """Device rows of `values` in a wider matrix of sentinels, `shift` elements past its start."""
    M, W = values.shape
    ld = ld or W
    flat = torch.full((shift + M * ld + 8,), SENTINEL, dtype=TYPES[kind], device=cuda())
    view = flat[shift:shift + M * ld].view(M, ld)[:, :W]
    view.copy_(torch.as_tensor(values))
    return view, flat


def host64(t):
    return to_host(t.double())


def ids_of(rng, M, L, how):
    if how == "mixed":
        return rng.integers(0, L, M)
    if how == "sorted":
        return np.sort(rng.integers(0, L, M))
    if how == "one":
        return np.full(M, L - 1)
    if how == "none":
        return np.full(M, -1)
    if how == "distinct":
        return np.arange(M) % L
    ids = rng.integers(0, L, M)  # "holes": rows without an adapter, by every kind of id outside
    ids[rng.random(M) < 0.4] = -1
    ids[rng.random(M) < 0.2] = L
    ids[rng.random(M) < 0.1] = 2 ** 31 - 1
    ids[rng.random(M) < 0.1] = -2 ** 31
    return ids


class Case:
    def __init__(self, seed, M, K, N, R, L=5, ids="mixed", x="f32", ab="bf16", out="f32", ranks=None, scale=True, ldx=None,
                 ldo=None, shift=0):
        rng = np.random.default_rng(seed)
        self.out_type = out
        self.x, _ = rows(rng.standard_normal((M, K)) * np.exp(rng.uniform(-2, 2, (M, 1))), x, ldx, shift)
        self.A = torch.as_tensor(rng.standard_normal((L, R, K)) / np.sqrt(K)).to(cuda(), TYPES[ab])
        self.B = torch.as_tensor(rng.standard_normal((L, N, R)) / np.sqrt(R)).to(cuda(), TYPES[ab])
        self.ids = ids_of(rng, M, L, ids) if isinstance(ids, str) else np.asarray(ids)
        self.ranks = None if ranks is None else np.asarray(ranks, np.int32)
        self.scale = rng.uniform(-2, 2, L).astype(np.float32) if scale else None
        self.base, self.base_flat = rows(rng.standard_normal((M, N)), out, ldo, shift)
        self.M, self.N, self.ldo, self.shift, self.exact_x = M, N, ldo or N, shift, x != "f32"

    def dev(self, v, dtype):
        return None if v is None else torch.as_tensor(np.ascontiguousarray(v)).to(cuda(), dtype)

    def reference(self):
        return o.lora(host64(self.x), self.ids, host64(self.A), host64(self.B), self.ranks, self.scale, host64(self.base),
                      self.out_type, self.exact_x)

    def call(self, in_place=False, workspace=None):
        w4 = w4mod()
        args = dict(scale=self.dev(self.scale, torch.float32), ranks=self.dev(self.ranks, torch.int32), workspace=workspace)
        ids = self.dev(self.ids.astype(np.int32), torch.int32)
        if in_place:
            flat = self.base_flat.clone()
            out = flat[self.shift:self.shift + self.M * self.ldo].view(self.M, self.ldo)[:, :self.N]
            w4.lora_add(out, self.x, ids, self.A, self.B, **args)
        else:
            out, flat = rows(np.full((self.M, self.N), 3.0), self.out_type, self.ldo, self.shift)
            w4.lora_add(out, self.x, ids, self.A, self.B, base=self.base, **args)
        keep = torch.ones_like(flat, dtype=torch.bool)
        keep[self.shift:self.shift + self.M * self.ldo].view(self.M, self.ldo)[:, :self.N] = False
        assert bool((flat[keep] == SENTINEL).all()), "elements between or behind the rows were written"
        return out

    def check(self, what="", in_place=None):
        value, bound = self.reference()
        for place in ((False, True) if in_place is None else (in_place,)):
            out = self.call(place)
            o.close(host64(out), value, bound, self.out_type, f"{what} in_place={place}")
            none = (self.ids < 0) | (self.ids >= self.A.shape[0])
            if none.any():
                bare = np.flatnonzero(none)
                assert torch.equal(out[bare], self.base[bare]), "rows without an adapter changed"


# rows around the 16-row and 64-row tiles, columns and k off every width
@pytest.mark.parametrize("M", [1, 2, 3, 15, 16, 17, 31, 33, 48, 63, 64, 65, 127, 130, 200])
@pytest.mark.parametrize("K,N,R", [(8, 1, 8), (64, 17, 16), (72, 64, 24), (200, 255, 32), (1032, 130, 64)])
def test_sizes(M, K, N, R):
    Case(M * 100 + N, M, K, N, R).check()


@pytest.mark.parametrize("out", sorted(TYPES))
@pytest.mark.parametrize("ab", ["f16", "bf16"])
@pytest.mark.parametrize("x", sorted(TYPES))
@pytest.mark.parametrize("M,K,N,R", [(1, 520, 100, 16), (37, 328, 77, 40), (150, 256, 96, 128)])
def test_types(x, ab, out, M, K, N, R):
    Case(M + K, M, K, N, R, x=x, ab=ab, out=out, ids="holes").check()


@pytest.mark.parametrize("how", ["mixed", "sorted", "one", "none", "distinct", "holes"])
@pytest.mark.parametrize("M,L", [(1, 1), (7, 3), (64, 64), (64, 2), (100, 40), (300, 7), (300, 300)])
def test_orders(how, M, L):
    Case(M + L, M, 136, 70, 16, L=L, ids=how, x="bf16", out="bf16").check()


@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 48, 56, 64, 72, 96, 120, 128, 136, 192, 200, 256])
@pytest.mark.parametrize("M", [3, 70])
def test_ranks_of_the_stack(R, M):
    Case(R + M, M, 264, 90, R, L=3, out="f16", ab="f16", x="f16").check()


@pytest.mark.parametrize("M", [9, 64, 150])
def test_mixed_ranks(M):
    """Entries past an adapter's rank are not used, whatever they hold; ranks outside [0, R] are cut to it."""
    R, L = 40, 8
    ranks = [0, 1, 7, 8, 17, 40, 41, -3]
    c = Case(M, M, 200, 50, R, L=L, ranks=ranks, ids="distinct")
    for a, r in enumerate(ranks):
        r = min(max(r, 0), R)
        c.A[a, r:] = float("nan")
        c.B[a, :, r:] = float("inf")
    c.check()


def test_scale():
    Case(1, 20, 128, 40, 16, scale=False).check()
    c = Case(2, 20, 128, 40, 16)
    c.scale[:] = 0.0
    c.check()


@pytest.mark.parametrize("shift", [0, 1, 2, 3, 5])
@pytest.mark.parametrize("x,out", [("f32", "f32"), ("f16", "bf16"), ("bf16", "f16")])
def test_strides_and_alignment(shift, x, out):
    for M in (2, 70):
        Case(shift, M, 128, 33, 16, x=x, out=out, ldx=128 + 2 * shift + 1, ldo=33 + shift, shift=shift).check()
        Case(shift, M, 128, 96, 16, x=x, out=out, ldx=128 + 8 * shift, ldo=96 + 8 * shift, shift=shift).check()


def same_but(got, ref, where):
    """got equals ref bit for bit outside `where`, and is not finite inside it."""
    assert torch.equal(got[~where], ref[~where])
    assert not bool(torch.isfinite(got[where]).any())


@pytest.mark.parametrize("M", [5, 64, 100])
@pytest.mark.parametrize("x,ab,out", [("f32", "bf16", "f32"), ("f32", "f16", "bf16"), ("f16", "f16", "f16"), ("bf16", "f16", "f32"),
                                      ("f16", "bf16", "f32")])
def test_not_finite(M, x, ab, out):
    """NaN and infinities stay in their row (x), their adapter's rows (A) and their adapter's column (B)."""
    c = Case(M, M, 136, 50, 16, L=4, ids="distinct", x=x, ab=ab, out=out)
    ref = c.call().clone()
    ids = torch.as_tensor(c.ids).to(cuda())
    for bad in (float("nan"), float("inf")):
        x0, A0, B0 = c.x.clone(), c.A.clone(), c.B.clone()
        c.x[M // 2, 7] = bad
        where = torch.zeros_like(ref, dtype=torch.bool)
        where[M // 2] = True
        same_but(c.call(), ref, where)
        c.x.copy_(x0)
        c.A[2, 3, 9] = bad
        where = (ids == 2)[:, None].expand_as(ref)
        same_but(c.call(), ref, where)
        c.A.copy_(A0)
        c.B[1, 33, 5] = bad
        where = torch.zeros_like(ref, dtype=torch.bool)
        where[:, 33] = ids == 1
        same_but(c.call(), ref, where)
        c.B.copy_(B0)


def test_infinite_rows_have_their_sign():
    """An infinite x meets A's signs as in the formula: one-rank adapters, so v and the outputs are infinite."""
    for x in ("f32", "f16"):
        c = Case(3, 2, 64, 20, 8, L=1, ids="one", x=x, ranks=[1], scale=False)
        c.x[0, 5] = float("inf")
        got = to_host(c.call())
        want = np.sign(host64(c.A)[0, 0, 5]) * np.sign(host64(c.B)[0, :, 0]) * np.inf
        assert np.array_equal(got[0], want.astype(np.float32)) and np.isfinite(got[1]).all()


@pytest.mark.parametrize("x,ab,out", [("f32", "bf16", "f32"), ("f32", "f16", "f32"), ("f16", "f16", "f16"), ("bf16", "bf16", "bf16")])
def test_wide_ranges(x, ab, out):
    """Rows from tiny to huge and entries of v far apart in one row."""
    c = Case(5, 66, 520, 40, 24, x=x, ab=ab, out=out, ids="sorted")
    span = 6.0 if x == "f16" else 40.0
    c.x.mul_(torch.exp(torch.linspace(-span, span, c.M, device=cuda()))[:, None].to(c.x.dtype))
    c.A.mul_(torch.exp2(torch.linspace(-8, 0, 24, device=cuda()))[None, :, None].to(c.A.dtype))
    c.base.mul_(0)
    if out != "f32":  # inside the output's range
        c.scale *= 1e-6
    if out == "bf16" or out == "f32":
        c.check()
    else:
        c.check(in_place=False)


def test_largest_sizes_of_one_row():
    Case(1, 1, 1 << 20, 24, 8, L=1, ids="one").check(in_place=True)
    Case(2, 3, 64, 300_001, 8, L=2, x="bf16", out="bf16").check(in_place=True)


@pytest.mark.parametrize("M,K,N,R", [(1, 7168, 4096, 16), (64, 4096, 1040, 16), (700, 1024, 512, 32), (2100, 520, 264, 64),
                                     (4500, 256, 128, 16), (5000, 136, 70, 128)])
@pytest.mark.parametrize("how", ["sorted", "mixed"])
def test_larger(M, K, N, R, how):
    Case(M, M, K, N, R, L=6, ids=how, x="bf16", out="f32").check(in_place=True)


@pytest.mark.parametrize("M", [511, 513, 4096, 4097, 4161])
@pytest.mark.parametrize("how", ["sorted", "distinct", "holes"])
def test_many_tiles(M, how):
    """Around the numbers of tiles at which the groups are found another way; few and many groups a tile, copied rows."""
    Case(M, M, 72, 40, 8, L=70, ids=how, x="bf16", out="f32", ranks=np.arange(70) % 9).check()


def test_more_groups_than_workgroups():
    """10000 rows of 64 adapters in turn: ten thousand groups."""
    Case(1, 10000, 24, 130, 8, L=64, ids="distinct", x="f16", ab="f16", out="bf16").check()


def plain(x, ids, A, B, scale, base):
    """The definition in float64 on the device, adapter by adapter."""
    out = base.double()
    for a in range(A.shape[0]):
        at = torch.nonzero(ids == a).flatten()
        v = x[at].double() @ A[a].double().t().contiguous()
        out[at] += float(scale[a]) * (v @ B[a].double().t().contiguous())
    return out


def test_more_rows_than_one_launch():
    """Rows past one pair of launches, and past 2^31 elements of out; rows behind the last are left alone."""
    M, K, N, R, L, ldo = 33000, 64, 48, 8, 3, 70000
    gen = torch.Generator(device=cuda()).manual_seed(1)
    x = torch.randn(M, K, generator=gen, device=cuda(), dtype=torch.bfloat16)
    A = torch.randn(L, R, K, generator=gen, device=cuda()).div_(8).to(torch.bfloat16)
    B = torch.randn(L, N, R, generator=gen, device=cuda()).to(torch.bfloat16)
    ids = torch.randint(-1, L, (M,), generator=gen, device=cuda(), dtype=torch.int32)
    scale = torch.ones(L, device=cuda())
    out = torch.zeros(M + 1, ldo, dtype=torch.bfloat16, device=cuda())
    w4mod().lora_add(out[:M, :N], x, ids, A, B, scale=scale)
    want = plain(x, ids, A, B, scale, torch.zeros(M, N, device=cuda()))
    # v: fp32 sums of 64 products; out: one bf16 rounding (2^-8) and the 16 bits of v (2^-15)
    size = plain(x.abs(), ids, A.abs(), B.abs(), scale, torch.zeros(M, N, device=cuda()))
    assert bool(((out[:M, :N].double() - want).abs() <= want.abs() * 2.0 ** -8 + size * 2.0 ** -14).all())
    assert not bool(out[M].any()) and not bool(out[:, N:N + 64].any())


def test_stacks_past_32_bits():
    """Adapters whose offsets in A and in B pass 2^31 elements."""
    L, R, K, N, M = 260, 128, 65536, 80000, 5
    A = torch.empty(L, R, K, dtype=torch.bfloat16, device=cuda())
    B = torch.empty(L, N, R, dtype=torch.bfloat16, device=cuda())
    assert A.numel() > 1 << 31 and B.numel() > 1 << 31
    gen = torch.Generator(device=cuda()).manual_seed(2)
    for a in (0, L - 1):
        A[a] = torch.randn(R, K, generator=gen, device=cuda()).div_(256).to(torch.bfloat16)
        B[a] = torch.randn(N, R, generator=gen, device=cuda()).div_(11).to(torch.bfloat16)
    x = torch.randn(M, K, generator=gen, device=cuda())
    ids = torch.tensor([L - 1, 0, -1, L - 1, 0], dtype=torch.int32, device=cuda())
    out = torch.zeros(M, N, device=cuda())
    w4mod().lora_add(out, x, ids, A, B)
    pick = [0, L - 1]
    near = torch.tensor([1, 0, -1, 1, 0], device=cuda())
    want = plain(x, near, A[pick], B[pick], torch.ones(2), torch.zeros(M, N, device=cuda()))
    # 2-norm: roundings of 2^-24 in sums of 65536 and 128 terms, far inside 2^-18
    assert float((out.double() - want).norm() / want.norm()) < 2.0 ** -18


def test_accuracy_of_fp32():
    """fp32 outputs are as near to 64 bits as fp32 products are: 2-norm of the error at most 2^-20 of the term's."""
    for ab in ("bf16", "f16"):
        for M in (1, 40, 600):
            c = Case(M, M, 4096, 300, 32, ab=ab, ids="sorted")
            c.base.zero_()
            value, _ = c.reference()
            err = host64(c.call()) - value
            assert np.linalg.norm(err) <= 2.0 ** -20 * np.linalg.norm(value), (ab, M)


def test_same_bytes_again():
    c = Case(4, 200, 1032, 130, 24, x="f32", out="f32", ids="holes")
    first = c.call().clone()
    for _ in range(3):
        assert torch.equal(c.call(), first)


def test_streams_and_graphs():
    """Two calls side by side on streams of their own, then the same captured and replayed on changed inputs."""
    w4 = w4mod()
    cases = [Case(s, M, 1032, 260, 16, ids=how, out=out) for s, M, how, out in ((1, 64, "mixed", "f32"), (2, 500, "sorted", "bf16"))]
    dev = torch.int32
    parts = []
    for c in cases:
        out = torch.zeros(c.M, c.N, dtype=TYPES[c.out_type], device=cuda())
        ws = torch.empty(w4.lora_workspace(c.M, c.x.shape[1], c.A.shape[0], c.A.shape[1]), dtype=torch.uint8, device=cuda())
        parts.append((out, c.x, c.dev(c.ids.astype(np.int32), dev), c.A, c.B, ws, c.dev(c.scale, torch.float32), None, c.base))
    want = [c.call().clone() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for s, p in zip(streams, parts):
            with torch.cuda.stream(s):
                w4.lora_add(*p)
    torch.cuda.synchronize()
    for p, v in zip(parts, want):
        assert torch.equal(p[0], v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for p in parts:
            w4.lora_add(*p)
    for turn in range(4):
        for c in cases:
            c.x.mul_(0.5)
        want = [c.call().clone() for c in cases]
        for p in parts:
            p[0].zero_()
            p[5].fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for p, v in zip(parts, want):
            assert torch.equal(p[0], v), turn


def test_empty():
    w4 = w4mod()
    A, B = torch.zeros(2, 8, 16, dtype=torch.float16, device=cuda()), torch.zeros(2, 5, 8, dtype=torch.float16, device=cuda())
    out = torch.zeros(0, 5, device=cuda())
    assert w4.lora_add(out, torch.zeros(0, 16, device=cuda()), torch.zeros(0, dtype=torch.int32, device=cuda()), A, B) is out
