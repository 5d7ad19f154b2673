"""GPU tests of the 8-bit product, dense and per expert, against its 64-bit form.  The int32 sums are exact, so the
tolerance is the epilogue's roundings alone (w8_oracle.product)."""
from __future__ import annotations

import numpy as np
import pytest

from tests import w8_oracle as o
from tests.gpu_common import cuda, to_dev, to_host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def w4mod():
    import w4a8_quantized_gemm_token_amd as w4
    return w4


def codes(rng, *shape):
    return rng.integers(-127, 128, shape, dtype=np.int8)


def scales(rng, n):
    return np.exp(rng.uniform(-9, -2, n)).astype(np.float32)


def check(got, ref, bound, what):
    t = got.dtype
    eps = 0.0 if t == torch.float32 else torch.finfo(t).eps
    tiny = 0.0 if t == torch.float32 else torch.finfo(t).smallest_normal * torch.finfo(t).eps
    o.close(to_host(got.float()), ref, bound, eps, tiny, what)


def dense(rng, M, K, N, bias=False, dtype="f32", ldo=None):
    w4 = w4mod()
    qa, qw, sa, sw = codes(rng, M, K), codes(rng, N, K), scales(rng, M), scales(rng, N)
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    ref, bound = o.product(qa, sa, qw, sw, b)
    full = torch.full((M, ldo or N), -7.0, dtype=TYPES[dtype], device=cuda())
    got = w4.gemm_w8a8(to_dev(qa), to_dev(sa), to_dev(qw), to_dev(sw), bias=to_dev(b) if bias else None,
                       out=full[:, :N])
    check(got, ref, bound, f"M={M} K={K} N={N} {dtype}")
    assert bool((full[:, N:] == -7.0).all())
    return got


# rows around the tile heights, columns off every width, k in whole and part windows
MS = (1, 2, 15, 16, 17, 31, 33, 64, 65, 100, 128, 129, 200, 255, 256, 257, 300)


@pytest.mark.parametrize("M", MS)
@pytest.mark.parametrize("K,N", [(16, 1), (48, 17), (128, 64), (144, 255), (400, 130), (1024, 257)])
def test_dense_sizes(M, K, N):
    dense(np.random.default_rng(M * 1000 + N), M, K, N)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M,K,N,ldo", [(1, 512, 96, None), (7, 272, 40, 43), (40, 656, 100, 128), (150, 2064, 520, 520),
                                       (300, 384, 272, 301), (520, 256, 512, None)])
def test_dense_types_bias_strides(dtype, bias, M, K, N, ldo):
    dense(np.random.default_rng(M + K), M, K, N, bias, dtype, ldo)


# column counts at which each loop is taken: k shared out within a workgroup (up to 16 rows), and the tiles of 64 x 64,
# 128 x 128, 128 x 256 and 256 x 256 (the sizes above take 32 x 64)
LOOPS = [(1, 16400), (13, 16400), (16, 28677), (100, 8330), (130, 14341), (130, 28677), (257, 28677), (300, 57001)]


@pytest.mark.parametrize("M,N", LOOPS)
@pytest.mark.parametrize("K", [16, 128, 144, 400, 1040])
def test_dense_loops(M, N, K):
    dense(np.random.default_rng(M + N + K), M, K, N, bias=K % 3 == 0, dtype="f16" if K == 400 else "f32")


@pytest.mark.parametrize("M,N", LOOPS)
def test_dense_loops_strided_and_bf16(M, N):
    """Row strides that keep the stores 16-byte aligned, and that do not."""
    for ldo in (N + 8 - N % 8, N + 3):
        dense(np.random.default_rng(M + ldo), M, 272, N, True, "bf16", ldo)


@pytest.mark.parametrize("M", [1, 7, 16])
@pytest.mark.parametrize("K", [2048, 7168, 8192, 8208, 8320, 16384, 24592])
def test_dense_shared_k(M, K):
    """Few rows, k in one and in several passes over it, with and without a part window."""
    dense(np.random.default_rng(K + M), M, K, 16390 if K <= 8192 else 50, M == 7, "f32")


@pytest.mark.parametrize("M,K,N", [(1, 8192, 4100), (16, 8192, 2048), (77, 4112, 5003), (512, 4096, 1040),
                                   (1, 131056, 48), (33, 131056, 80), (1000, 1040, 3001)])
def test_dense_larger(M, K, N):
    dense(np.random.default_rng(M + N), M, K, N, True, "bf16")


@pytest.mark.parametrize("M", [1, 40, 300])
def test_dense_extreme_codes(M):
    """Codes at the ends of int8 at the largest K: |sum| = 2^14 (2^17 - 16), just inside int32."""
    w4 = w4mod()
    K, N = 131056, 20
    for a, w in ((-128, -128), (-128, 127), (127, 127)):
        qa = torch.full((M, K), a, dtype=torch.int8, device=cuda())
        qw = torch.full((N, K), w, dtype=torch.int8, device=cuda())
        got = to_host(w4.gemm_w8a8(qa, torch.ones(M, device=cuda()), qw, torch.ones(N, device=cuda())))
        assert (got == np.float32(a * w * K)).all()


@pytest.mark.parametrize("M", [3, 20, 70, 300])
def test_special_scales(M):
    """Zero, infinite and NaN scales and biases reach exactly their row or column; fp16 outputs past the range are
    infinite."""
    w4 = w4mod()
    rng = np.random.default_rng(M)
    K, N = 256, 70
    qa, qw, sa, sw = codes(rng, M, K), codes(rng, N, K), scales(rng, M), scales(rng, N)
    qa[:, 0], qw[:, 0] = 127, 127  # no sum is 0 by chance below
    sa[0], sa[1], sw[5], sw[6] = 0.0, np.nan, np.inf, 1e30
    b = rng.standard_normal(N).astype(np.float32)
    b[9] = np.inf
    ref, _ = o.product(qa, sa, qw, sw, b)
    got = to_host(w4.gemm_w8a8(to_dev(qa), to_dev(sa), to_dev(qw), to_dev(sw), to_dev(b)))
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(np.isposinf(got), np.isposinf(ref)) and np.array_equal(np.isneginf(got), np.isneginf(ref))
    keep = [n for n in range(N) if n not in (5, 6)]
    assert np.array_equal(got[0, keep], b[keep])
    half = to_host(w4.gemm_w8a8(to_dev(qa), to_dev(sa), to_dev(qw), to_dev(sw), out_dtype=torch.float16))
    big = np.abs(ref[2:, 6]) > 1e6
    assert np.isinf(half[2:, 6][big]).all()


def test_rows_do_not_depend_on_the_batch():
    """A row gives the same bytes alone and in every batch size (every loop)."""
    w4 = w4mod()
    rng = np.random.default_rng(3)
    for M, K, N in ((300, 1168, 520), (300, 144, 28700), (120, 528, 8330)):
        qa, qw, sa, sw = (to_dev(v) for v in (codes(rng, M, K), codes(rng, N, K), scales(rng, M), scales(rng, N)))
        whole = w4.gemm_w8a8(qa, sa, qw, sw)
        for m in (1, 16, 17, 40, 64, 100, 129, 256):
            part = w4.gemm_w8a8(qa[:m], sa[:m], qw, sw)
            assert torch.equal(part.view(torch.int32), whole[:m].view(torch.int32)), (N, m)


def test_weights_from_the_row_quantizer():
    """quantize_weights_w8 of W and quantize_act of x: the layer's error against fp64 is that of the codes."""
    w4 = w4mod()
    rng = np.random.default_rng(8)
    x = rng.standard_normal((33, 512)).astype(np.float32)
    W = (0.02 * rng.standard_normal((80, 512))).astype(np.float32)
    qa, sa = w4.quantize_act(to_dev(x))
    qw, sw = w4.quantize_weights_w8(to_dev(W))
    got = w4.gemm_w8a8(qa, sa, qw, sw)
    ref, bound = o.product(to_host(qa), to_host(sa), to_host(qw), to_host(sw))
    check(got, ref, bound, "codes")
    # each code is off by half a scale at most: |x w| errors add up to K (|x| sw/2 + |w| sa/2 + sa sw/4)
    xs, ws = np.abs(x.astype(np.float64)), np.abs(W.astype(np.float64))
    off = (xs.sum(1)[:, None] * to_host(sw)[None] + ws.sum(1)[None] * to_host(sa)[:, None]) / 2 + \
        512 / 4 * to_host(sa)[:, None].astype(np.float64) * to_host(sw)[None]
    assert (np.abs(to_host(got) - x.astype(np.float64) @ W.astype(np.float64).T) <= 1.001 * off + bound).all()


# ------------------------------------------------------------------ per expert
def grouped(rng, counts, K, N, R=None, rows="random", pad=0, repeat=False):
    """Slots by counts; `rows`: random rows, None (slot s is row s), or with indices outside [0, R) too."""
    w4 = w4mod()
    E, S = len(counts), int(sum(counts))
    R = R or max(S, 1)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    qa, sa, qw, sw = codes(rng, R, K), scales(rng, R), codes(rng, E, N, K), np.stack([scales(rng, N) for _ in range(E)])
    idx = np.arange(S + pad) if rows is None else rng.integers(0, R, S + pad)
    if rows == "outside":
        idx[::5] = rng.choice([-1, R, -2 ** 31, 2 ** 31 - 1], idx[::5].shape)
    out = torch.full((S + pad, N), -7.0, device=cuda())
    w4.moe_grouped_gemm_w8a8(to_dev(qa), to_dev(sa), None if rows is None else to_dev(idx.astype(np.int32)),
                             to_dev(off), to_dev(qw), to_dev(sw), S + pad, out=out)
    got = to_host(out)
    inside = (idx >= 0) & (idx < R)
    assert (got[S:] == -7.0).all() and (got[:S][~inside[:S]] == -7.0).all(), "rows of no expert are left as they were"
    for e in range(E):
        s = np.arange(off[e], off[e + 1])
        s = s[inside[s]]
        if s.size:
            ref, bound = o.product(qa[idx[s]], sa[idx[s]], qw[e], sw[e])
            o.close(got[s], ref, bound, 0.0, 0.0, f"expert {e} of {counts}")


@pytest.mark.parametrize("counts", [[1], [0, 3, 0], [16, 17, 0, 1], [64, 65, 63], [5, 0, 130, 40], [129, 300, 2, 33],
                                    [0, 0, 0, 0, 0, 0, 0, 9]])
@pytest.mark.parametrize("K,N", [(16, 5), (400, 132), (1040, 257)])
def test_grouped_sizes(counts, K, N):
    grouped(np.random.default_rng(sum(counts) + N), counts, K, N)


@pytest.mark.parametrize("K", [128, 2048, 3600, 7168, 8208, 16512])
def test_grouped_few_slots(K):
    """Up to 16 slots each: k in one and in several passes; more tiles than workgroups, so that runs cross experts."""
    grouped(np.random.default_rng(K), [1, 16, 0, 3, 9, 2, 16, 1], K, 1552)


@pytest.mark.parametrize("counts,K,N", [([17, 300, 0, 129, 64], 2064, 520), ([40] * 30, 144, 2570), ([1000, 3, 20], 656, 300)])
def test_grouped_more_slots(counts, K, N):
    """Row blocks of 128, several of an expert, more units than workgroups."""
    grouped(np.random.default_rng(K), counts, K, N)


@pytest.mark.parametrize("rows", [None, "random", "outside"])
@pytest.mark.parametrize("pad", [0, 37])
def test_grouped_rows_and_padding(rows, pad):
    rng = np.random.default_rng(5)
    counts = [3, 70, 0, 18, 140, 1]
    R = 240 + pad if rows is None else 90
    grouped(rng, counts, 272, 96, R=R, rows=rows, pad=pad)


@pytest.mark.parametrize("E", [1, 65, 384, 1024])
def test_grouped_many_experts(E):
    rng = np.random.default_rng(E)
    counts = rng.choice([0, 0, 1, 2, 9, 20], E)
    counts[rng.integers(0, E)] = 150
    grouped(rng, counts.tolist(), 64, 48)


def test_grouped_no_slots_and_clamped_offsets():
    """Every expert empty: nothing is written.  Offsets past max_slots are clamped to it."""
    w4 = w4mod()
    rng = np.random.default_rng(1)
    grouped(rng, [0, 0, 0], 64, 32, pad=9)
    qa, sa, qw, sw = codes(rng, 40, 64), scales(rng, 40), codes(rng, 2, 32, 64), np.stack([scales(rng, 32)] * 2)
    buf = torch.full((40, 32), -7.0, device=cuda())
    off = to_dev(np.array([0, 10, 1 << 30], np.int32))
    w4.moe_grouped_gemm_w8a8(to_dev(qa), to_dev(sa), None, off, to_dev(qw), to_dev(sw), 30, out=buf[:30])
    got = to_host(buf)
    assert (got[30:] == -7.0).all()
    for e, s in ((0, slice(0, 10)), (1, slice(10, 30))):
        ref, bound = o.product(qa[s], sa[s], qw[e], sw[e])
        o.close(got[s], ref, bound, 0.0, 0.0)


def test_grouped_offsets_that_are_not_ascending():
    """Offsets that go back and forth: the call ends, writes rows below max_slots only, and each written row is the
    product with one of the experts that claim it."""
    w4 = w4mod()
    rng = np.random.default_rng(11)
    S, K, N, E = 300, 64, 48, 16
    qa, sa, qw, sw = codes(rng, S, K), scales(rng, S), codes(rng, E, N, K), np.stack([scales(rng, N) for _ in range(E)])
    off = np.array([0, 2 ** 31 - 1] * 8 + [-5], np.int32)
    buf = torch.full((S + 20, N), -7.0, device=cuda())
    w4.moe_grouped_gemm_w8a8(to_dev(qa), to_dev(sa), None, to_dev(off), to_dev(qw), to_dev(sw), S, out=buf[:S])
    got = to_host(buf)
    assert (got[S:] == -7.0).all()
    near = np.zeros((S, N), bool)
    for e in range(E):
        ref, bound = o.product(qa, sa, qw[e], sw[e])
        near |= np.abs(got[:S] - ref) <= bound
    assert (near | (got[:S] == -7.0)).all()


def test_grouped_large_arrays():
    """Expert weights past 2^32 bytes and activation rows past 2^32 bytes: rows and experts on both sides."""
    w4 = w4mod()
    E, N, K = 40, 1024, 131056            # 5.4 GB of weights
    R = 33000                             # 4.3 GB of rows
    gen = torch.Generator(device=cuda()).manual_seed(4)
    qw = torch.randint(-127, 128, (E, N, K), dtype=torch.int8, device=cuda(), generator=gen)
    qa = torch.randint(-127, 128, (R, K), dtype=torch.int8, device=cuda(), generator=gen)
    sa, sw = torch.full((R,), 0.01, device=cuda()), torch.full((E, N), 0.02, device=cuda())
    counts = [0] * E
    counts[1], counts[20], counts[38], counts[39] = 5, 70, 20, 300
    off = to_dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    rows = torch.randint(0, R, (395,), dtype=torch.int32, device=cuda(), generator=gen)
    rows[::3] = R - 1 - rows[::3] % 100
    rows[1::7] = rows[1::7] % 100
    got = w4.moe_grouped_gemm_w8a8(qa, sa, rows, off, qw, sw, 395)
    for e in (1, 20, 38, 39):
        a, b = int(off[e]), int(off[e + 1])
        isum = qa[rows[a:b].long()].double() @ qw[e].double().t().contiguous()
        ref = isum * float(np.float32(0.01)) * float(np.float32(0.02))
        assert bool(((got[a:b].double() - ref).abs() <= 3.001 * o.U * ref.abs()).all()), e


# ------------------------------------------------------------------ streams and graphs
def test_graph_replays_with_new_inputs():
    """Both products captured into one graph; each replay on new inputs gives the eager bytes."""
    w4 = w4mod()
    gen = torch.Generator(device=cuda()).manual_seed(2)

    def ints(*shape):
        return torch.randint(-127, 128, shape, dtype=torch.int8, device=cuda(), generator=gen)

    M, K, N, E = 48, 528, 200, 6
    qa, qw, we = ints(M, K), ints(N, K), ints(E, N, K)
    sa = torch.rand(M, device=cuda(), generator=gen)
    sw, se = torch.rand(N, device=cuda(), generator=gen), torch.rand(E, N, device=cuda(), generator=gen)
    off = to_dev(np.array([0, 1, 1, 20, 40, 40, 48], np.int32))
    out, oute = torch.zeros(M, N, device=cuda()), torch.zeros(M, N, device=cuda())

    def both():
        w4.gemm_w8a8(qa, sa, qw, sw, out=out)
        w4.moe_grouped_gemm_w8a8(qa, sa, None, off, we, se, M, out=oute)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for cut in (48, 5, 30):
        qa.copy_(ints(M, K))
        off.copy_(to_dev(np.minimum([0, 1, 1, 20, 40, 40, 48], cut).astype(np.int32)))
        oute.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        got, gote = out.clone(), oute.clone()
        oute.fill_(-7.0)
        both()
        torch.cuda.synchronize()
        assert torch.equal(got, out) and torch.equal(gote, oute)
        assert bool((gote[cut:] == -7.0).all())


def test_two_streams_at_once():
    """Calls on two streams share nothing: the results are those of one after the other."""
    w4 = w4mod()
    gen = torch.Generator(device=cuda()).manual_seed(6)
    qa = torch.randint(-127, 128, (64, 2048), dtype=torch.int8, device=cuda(), generator=gen)
    ws = [torch.randint(-127, 128, (1000, 2048), dtype=torch.int8, device=cuda(), generator=gen) for _ in range(2)]
    sa, sw = torch.ones(64, device=cuda()), torch.ones(1000, device=cuda())
    ref = [w4.gemm_w8a8(qa, sa, w, sw) for w in ws]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [torch.zeros_like(ref[0]) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, w, g in zip(streams, ws, got):
            with torch.cuda.stream(s):
                w4.gemm_w8a8(qa, sa, w, sw, out=g)
    torch.cuda.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("T", [1, 37, 300])
def test_moe_layer_of_8_bit_experts(T):
    """Scored router -> quantizer -> gate/up product -> SiLU requant -> down product -> combine, each stage against
    its 64-bit form on the stage's own inputs, the shared expert as index E."""
    w4 = w4mod()
    rng = np.random.default_rng(T)
    E, k, H, I = 12, 4, 256, 144
    x = rng.standard_normal((T, H)).astype(np.float32)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    gw, gs = codes(rng, E + 1, 2 * I, H), np.stack([scales(rng, 2 * I) for _ in range(E + 1)])
    dw, ds = codes(rng, E + 1, H, I), np.stack([scales(rng, H) for _ in range(E + 1)])
    cfg = dict(bias=bias, score="sigmoid", n_groups=4, topk_groups=2, group_lead=2, renorm=True, scale=2.5)
    ids, w, off, perm, rows, sop = w4.moe_route_scored(to_dev(logits), k, **{**cfg, "bias": to_dev(bias)},
                                                       with_shared=True)
    S = T * k + T
    qa, sa = w4.quantize_act(to_dev(x))
    gu = w4.moe_grouped_gemm_w8a8(qa, sa, rows, off, to_dev(gw), to_dev(gs), S)
    qh, hs = w4.silu_mul_quantize(gu)
    y = w4.moe_grouped_gemm_w8a8(qh, hs, None, off, to_dev(dw), to_dev(ds), S)
    out = w4.moe_combine(y, sop, w, y_shared=y[T * k:])

    ids_r, w_r = o.route(logits, k, **cfg)
    assert np.array_equal(to_host(ids), ids_r)
    off_r, _, rows_r, sop_r = o.tables(ids_r, E, True)
    assert np.array_equal(to_host(off), off_r) and np.array_equal(to_host(rows), rows_r)
    for e in range(E + 1):
        s = slice(off_r[e], off_r[e + 1])
        ref, bound = o.product(to_host(qa)[rows_r[s]], to_host(sa)[rows_r[s]], gw[e], gs[e])
        o.close(to_host(gu)[s], ref, bound, 0.0, 0.0)
        ref, bound = o.product(to_host(qh)[s], to_host(hs)[s], dw[e], ds[e])
        o.close(to_host(y)[s], ref, bound, 0.0, 0.0)
    yh = to_host(y).astype(np.float64)
    terms = to_host(w).astype(np.float64)[:, :, None] * yh[sop_r.reshape(T, k)]
    ref = terms.sum(1) + yh[T * k:]
    # k fused multiply-adds and one addition: each rounds a partial sum of at most the magnitudes' sum
    bound = (k + 1) * 1.001 * o.U * (np.abs(terms).sum(1) + np.abs(yh[T * k:]))
    o.close(to_host(out), ref, bound, 0.0, 0.0)
