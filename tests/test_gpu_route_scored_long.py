"""GPU tests of the scored router over very long batches and hot experts: the tables against sorting on the device,
the weights against fp64, the time per pair, and the layer of 4-bit experts behind the router."""
from __future__ import annotations

import numpy as np
import pytest

from tests import w8_oracle as o
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


def check_tables(ids, E, off, perm, rows, sop):
    """The tables of ids [T][k] on the device: stable order of the pairs by expert."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(perm.long(), order)
    counts = torch.stack([(flat == e).sum() for e in range(E)])
    assert off[:E + 1].tolist() == [0] + counts.cumsum(0).tolist()
    assert torch.equal(rows[:T * k].long(), order // k)
    back = torch.empty_like(order)
    back[order] = torch.arange(T * k, device=ids.device)
    assert torch.equal(sop.long(), back)


def hot_logits(T, E, hot, share, gen):
    """Tokens of which `share` want the experts 0 .. hot - 1 first, the others any."""
    x = torch.randn(T, E, device=cuda(), generator=gen)
    x[:, :hot] += 50.0 * (torch.rand(T, 1, device=cuda(), generator=gen) < share)
    return x


@pytest.mark.parametrize("T,E,k,share", [(700, 40, 3, 1.0), (3001, 40, 3, 0.7), (70001, 40, 3, 1.0), (100003, 40, 3, 0.5),
                                         (262144, 8, 2, 0.999), (250000, 160, 6, 0.05)])
def test_hot_buckets(T, E, k, share):
    """Buckets that take many rounds of a workgroup's list, dense and sparse in the ids."""
    gen = torch.Generator(device=cuda()).manual_seed(T)
    x = hot_logits(T, E, k, share, gen)
    ids, w, off, perm, rows, sop = w4mod().moe_route_scored(x, k, score="sigmoid", renorm=False, with_shared=True)
    assert torch.equal(ids.long(), torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k])
    check_tables(ids, E, off, perm, rows, sop)
    assert int(off[E + 1]) == T * k + T and torch.equal(rows[T * k:].long(), torch.arange(T, device=cuda()))


def test_time_is_linear_in_the_pairs():
    """Every token picks the same experts: 8 times the tokens take about 8 times as long (1.0 and 8.0 ms), where
    reading all ids again for every 8192 pairs of a bucket took 60 times as long (2.6 and 156 ms)."""
    w4 = w4mod()
    E, k = 40, 3
    took = []
    for T in (1 << 18, 1 << 21):
        x = torch.arange(E, dtype=torch.float32, device=cuda()).repeat(T, 1)
        outs = w4.moe_route_scored(x, k)
        call = w4.prepare_moe_route_scored(x, k, outs)
        best = []
        for _ in range(3):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            call()
            b.record()
            torch.cuda.synchronize()
            best.append(a.elapsed_time(b))
        took.append(min(best))
        for j in range(k):
            assert int(outs[2][E - k + j]) == j * T
            assert torch.equal(outs[3][j * T:(j + 1) * T], torch.arange(T, device=cuda(), dtype=torch.int32) * k + k - 1 - j)
    assert took[1] < 24 * took[0], took


def test_more_tokens_than_a_launch_has_threads_for():
    """2^26 tokens and some: a wave for each is 2^32 threads, more than one launch may have."""
    T, E = (1 << 26) + 5, 8
    gen = torch.Generator(device=cuda()).manual_seed(1)
    x = torch.empty(T, E, dtype=torch.float16, device=cuda()).normal_(generator=gen)
    ids, w, off, perm, rows, sop = w4mod().moe_route_scored(x, 1, score="sigmoid", renorm=False)
    best = x.amax(1)
    want = torch.full((T,), E, dtype=torch.int32, device=cuda())
    for e in reversed(range(E)):
        want[x[:, e] == best] = e
    assert torch.equal(ids[:, 0], want)
    ref = torch.sigmoid(best.double())
    # fp64 scores, then one rounding to fp32
    assert bool(((w[:, 0].double() - ref).abs() <= 1.0001 * o.U * ref).all())
    check_tables(ids, E, off, perm, rows, sop)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("score,biased,lead,renorm", [("softmax", False, 1, False), ("softmax", True, 2, True),
                                                      ("sigmoid", True, 2, True), ("sigmoid", False, 1, False)])
def test_long_grouped_batches(dtype, score, biased, lead, renorm):
    """20011 tokens, 3 of 8 groups of 20 experts: ids, weights and tables against fp64 on the device."""
    T, E, k, n, keep, scale = 20011, 160, 6, 8, 3, 16.0
    gen = torch.Generator(device=cuda()).manual_seed(41)
    x = (1.5 * torch.randn(T, E, device=cuda(), generator=gen)).to(dtype)
    bias = 0.05 * torch.randn(E, device=cuda(), generator=gen) if biased else None
    ids, w, off, perm, rows, sop = w4mod().moe_route_scored(x, k, bias=bias, score=score, n_groups=n, topk_groups=keep,
                                                            group_lead=lead, renorm=renorm, scale=scale)
    xd = x.double()
    s = torch.sigmoid(xd) if score == "sigmoid" else torch.softmax(xd, 1)
    v = s + bias.double() if biased else s
    value = torch.sort(v.view(T, n, E // n), dim=2, descending=True).values[:, :, :lead].sum(2)
    kept = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :keep]
    open_ = torch.zeros(T, n, dtype=torch.bool, device=cuda()).scatter_(1, kept, True).repeat_interleave(E // n, 1)
    key = torch.where(open_, v if biased else xd, -float("inf"))
    want = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.long(), want)
    ref = s.gather(1, want)
    ref = scale * (ref / ref.sum(1, keepdim=True) if renorm else ref)
    # fp64 scores and sums (a few 1e-16), then one rounding to fp32
    assert bool(((w.double() - ref).abs() <= 1.0001 * o.U * ref).all())
    check_tables(ids, E, off, perm, rows, sop)


@pytest.mark.parametrize("T", [1, 37, 300])
def test_layer_of_4_bit_experts(orc, T):
    """Scored router -> quantizer -> gate/up product -> SiLU requant -> down product -> combine with the 4-bit expert
    product, the shared expert as index E; each stage against the oracle on the stage's own inputs."""
    w4 = w4mod()
    rng = np.random.default_rng(T)
    E, k, H, I = 6, 3, 256, 256
    x = rng.standard_normal((T, H)).astype(np.float32)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)

    def experts(N, K):
        per = [orc.quantize_weights((0.05 * rng.standard_normal((N, K))).astype(np.float32)) for _ in range(E + 1)]
        packed = np.stack([orc.pack_nibbles(q) for q, _, _ in per])
        return per, [to_dev(packed)] + [to_dev(np.stack([p[i] for p in per]).view(np.int16)) for i in (1, 2)]

    gate_up, gd = experts(2 * I, H)
    down, dd = experts(H, I)
    cfg = dict(score="sigmoid", n_groups=3, topk_groups=2, group_lead=2, renorm=True, scale=2.5)
    ids, w, off, _, rows, sop = w4.moe_route_scored(to_dev(logits), k, bias=to_dev(bias), with_shared=True, **cfg)
    S = T * k + T
    qa, sa = w4.quantize_act(to_dev(x))
    gu = w4.moe_grouped_gemm(qa, sa, rows, off, *gd, max_slots=S)
    qh, hs = w4.silu_mul_quantize(gu)
    y = w4.moe_grouped_gemm(qh, hs, None, off, *dd, max_slots=S)
    out = w4.moe_combine(y, sop, w, y_shared=y[T * k:])

    ids_r, w_r = o.route(logits, k, bias=bias, **cfg)
    off_r, _, rows_r, sop_r = o.tables(ids_r, E, True)
    assert np.array_equal(to_host(ids), ids_r) and np.array_equal(to_host(off), off_r)
    assert np.array_equal(to_host(rows), rows_r) and np.array_equal(to_host(sop), sop_r)
    for e in range(E + 1):
        s = slice(off_r[e], off_r[e + 1])
        if s.start == s.stop:
            continue
        for got, a, a_scale, per in ((gu, to_host(qa)[rows_r[s]], to_host(sa)[rows_r[s]], gate_up),
                                     (y, to_host(qh)[s], to_host(hs)[s], down)):
            ref, mag = orc.gemm(a, a_scale, *per[e])
            assert (np.abs(to_host(got)[s].astype(np.float64) - ref) <= 1e-5 * mag + 1e-6).all(), e
    yh = to_host(y).astype(np.float64)
    terms = to_host(w).astype(np.float64)[:, :, None] * yh[sop_r.reshape(T, k)]
    ref = terms.sum(1) + yh[T * k:]
    # k fused multiply-adds and one addition: each rounds a partial sum of at most the magnitudes' sum
    bound = (k + 1) * 1.001 * o.U * (np.abs(terms).sum(1) + np.abs(yh[T * k:]))
    o.close(to_host(out), ref, bound, 0.0, 0.0)
