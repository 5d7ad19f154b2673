"""GPU tests of the scored router against its 64-bit form: ids and tables equal, weights within one fp32 rounding."""
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


def run(logits, k, dtype="f32", with_shared=False, pad=0, **cfg):
    """The router on logits (numpy float32) held in `dtype`, with `pad` more elements between rows, against the
    oracle."""
    w4 = w4mod()
    T, E = logits.shape
    full = torch.full((T, E + pad), 99.0, dtype=TYPES[dtype], device=cuda())
    full[:, :E] = to_dev(np.ascontiguousarray(logits))
    x = full[:, :E]
    dev = {**cfg, "bias": to_dev(cfg["bias"])} if cfg.get("bias") is not None else cfg
    got = [to_host(v) for v in w4.moe_route_scored(x, k, with_shared=with_shared, **dev)]
    ids, w = o.route(to_host(x.float()), k, **cfg)
    assert np.array_equal(got[0], ids), np.argwhere(got[0] != ids)[:4].tolist()
    # fp64 throughout (a few 1e-16), then one rounding to fp32
    assert (np.abs(got[1].astype(np.float64) - w) <= 1.0001 * o.U * np.abs(w) + 2.0 ** -150).all()
    for name, g, r in zip(("offsets", "perm", "row_index", "slot_of_pair"), got[2:], o.tables(ids, E, with_shared)):
        assert np.array_equal(g, r), name
    return got


def logits_of(seed, T, E, spread=1.5):
    return (spread * np.random.default_rng(seed).standard_normal((T, E))).astype(np.float32)


def bias_of(seed, E):
    return (0.05 * np.random.default_rng(seed + 77).standard_normal(E)).astype(np.float32)


CONFIGS = [  # n_groups, topk_groups, group_lead
    (1, 1, 1), (2, 1, 1), (4, 2, 2), (8, 4, 2), (8, 8, 1)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("groups", CONFIGS)
def test_forms(score, bias, renorm, groups):
    n, keep, lead = groups
    run(logits_of(n, 50, 64), 6, score=score, bias=bias_of(n, 64) if bias else None, renorm=renorm, n_groups=n,
        topk_groups=keep, group_lead=lead, scale=2.5, with_shared=bias)


@pytest.mark.parametrize("T", [1, 2, 4, 5, 16, 17, 63, 300, 3001])
def test_token_counts(T):
    run(logits_of(T, T, 96), 8, score="sigmoid", bias=bias_of(1, 96), with_shared=True)


@pytest.mark.parametrize("E,k,n,keep,lead", [(1, 1, 1, 1, 1), (2, 2, 1, 1, 1), (7, 7, 1, 1, 1), (60, 8, 5, 2, 2),
                                             (63, 32, 7, 5, 1), (64, 32, 64, 40, 1), (65, 3, 13, 2, 2), (160, 6, 8, 3, 1),
                                             (256, 8, 8, 4, 2), (384, 8, 1, 1, 1), (384, 10, 3, 1, 2), (513, 32, 1, 1, 1),
                                             (1000, 20, 50, 10, 2), (1024, 32, 2, 1, 1), (1024, 8, 64, 8, 2)])
@pytest.mark.parametrize("bias", [False, True])
def test_expert_counts(E, k, n, keep, lead, bias):
    run(logits_of(E, 33, E), k, score="sigmoid" if E % 2 else "softmax", bias=bias_of(E, E) if bias else None,
        n_groups=n, topk_groups=keep, group_lead=lead, with_shared=not bias)


@pytest.mark.parametrize("T", [1, 3, 16])
@pytest.mark.parametrize("E,k,n,keep,lead", [(1, 1, 1, 1, 1), (60, 8, 5, 2, 2), (384, 8, 1, 1, 1), (513, 32, 27, 20, 2),
                                             (1000, 32, 50, 10, 2), (1024, 32, 64, 33, 1)])
def test_few_tokens(T, E, k, n, keep, lead):
    """The one-launch form over the expert counts, its pairs up to 16 tokens of 32."""
    run(logits_of(E + T, T, E), k, score="softmax", bias=bias_of(E, E), n_groups=n, topk_groups=keep, group_lead=lead,
        with_shared=True)
    run(logits_of(E + T, T, E), k, score="sigmoid", n_groups=n, topk_groups=keep, group_lead=lead, renorm=False)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("pad", [0, 1, 24])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_types_and_strides(dtype, pad, score):
    """16-bit logits tie often: equal keys go to the lower id."""
    run(logits_of(3, 70, 128, 0.3), 8, dtype=dtype, pad=pad, score=score, n_groups=4, topk_groups=3, group_lead=2)
    run(logits_of(4, 70, 128, 0.3), 8, dtype=dtype, pad=pad, score=score, bias=np.zeros(128, np.float32))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_close_keys(score, bias):
    """Logits a few fp32 steps apart: the picks are those of the exact scores, not of rounded ones."""
    rng = np.random.default_rng(12)
    x = np.empty((64, 96), np.float32)
    for t in range(64):
        base = np.float32(rng.uniform(-4, 4))
        x[t] = base + np.spacing(base) * rng.integers(-40, 41, 96).astype(np.float32)
    b = (1e-7 * rng.integers(-3, 4, 96)).astype(np.float32) if bias else None
    run(x, 8, score=score, bias=b)
    run(x, 8, score=score, bias=b, n_groups=8, topk_groups=3, group_lead=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups", [(1, 1, 1), (4, 2, 2)])
@pytest.mark.parametrize("renorm", [False, True])
def test_masked_and_special_logits(score, bias, groups, renorm):
    """Rows of -inf, NaN, +inf, one live expert, fewer live experts than k, lowest finite values, equal rows, far
    tails of the sigmoid; biases of -inf and NaN."""
    n, keep, lead = groups
    E, k = 32, 6
    x = logits_of(9, 16, E)
    lowest = np.finfo(np.float32).min
    x[0] = -np.inf
    x[1] = np.nan
    x[2] = np.inf
    x[3] = -np.inf
    x[3, 17] = 0.25
    x[4, ::2] = -np.inf
    x[5, 1::3] = np.nan
    x[6, 5], x[6, 30] = np.inf, np.inf
    x[7] = lowest
    x[8] = lowest
    x[8, 3] = 1.0
    x[9] = 1.5
    x[10] = -200 - np.arange(E, dtype=np.float32)
    x[11] = 50 + np.arange(E, dtype=np.float32) % 5
    x[12, 8:] = -np.inf
    x[13] = 3e38
    x[14] = np.where(np.arange(E) % 2 == 0, 0.0, -0.0)
    b = bias_of(2, E) if bias else None
    if bias:
        b[4], b[20], b[21] = -np.inf, np.nan, -np.inf
    got = run(x, k, score=score, bias=b, renorm=renorm, n_groups=n, topk_groups=keep, group_lead=lead)
    assert np.isfinite(got[1]).all()
    assert all(len(set(r)) == k for r in got[0].tolist()) and got[0].min() >= 0 and got[0].max() < E


def test_matches_the_plain_router():
    """Softmax, renormalised, no bias, no groups: the picks and tables of moe_route, the weights within its fp32
    steps (an exponential and a quotient of a sum of k)."""
    w4 = w4mod()
    x = to_dev(logits_of(21, 200, 384))
    a = [to_host(v) for v in w4.moe_route(x, 8, with_shared=True)]
    b = [to_host(v) for v in w4.moe_route_scored(x, 8, with_shared=True)]
    assert all(np.array_equal(a[i], b[i]) for i in (0, 2, 3, 4, 5))
    assert np.allclose(a[1], b[1], rtol=16 * o.U * 8, atol=0)


def test_no_tokens():
    w4 = w4mod()
    for shared in (False, True):
        got = w4.moe_route_scored(torch.zeros((0, 12), device=cuda()), 3, with_shared=shared)
        assert to_host(got[2]).tolist() == [0] * (13 + shared)


@pytest.mark.parametrize("T", [17, 700, 9001, 20011])
def test_every_token_picks_the_same_experts(T):
    """All pairs in k buckets (longer than a workgroup's list), the others empty."""
    x = np.tile(logits_of(8, 1, 40), (T, 1))
    run(x, 3, score="sigmoid", with_shared=True)


@pytest.mark.parametrize("T,E,k", [(20011, 160, 6), (9000, 384, 8)])
def test_long_batches(T, E, k):
    """Many chunks of pairs: the tables against stable sorting, the picks against the fp64 keys' order."""
    w4 = w4mod()
    x = to_dev(logits_of(31, T, E))
    b = to_dev(bias_of(31, E))
    ids, w, off, perm, rows, sop = w4.moe_route_scored(x, k, bias=b, score="sigmoid", with_shared=True)
    key = 1.0 / (1.0 + torch.exp(-x.double())) + b.double()
    assert torch.equal(ids.long(), torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k])
    for g, r in zip((off, perm, rows, sop), o.tables(to_host(ids), E, True)):
        assert np.array_equal(to_host(g), r)


@pytest.mark.parametrize("T", [1, 40])
def test_graph_replays_with_new_logits(T):
    w4 = w4mod()
    E, k = 64, 6
    x, b = torch.zeros(T, E, device=cuda()), to_dev(bias_of(5, E))
    cfg = dict(bias=b, score="sigmoid", n_groups=8, topk_groups=4, group_lead=2, with_shared=True)
    outs = w4.moe_route_scored(x, k, **cfg)
    call = None
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call = w4.prepare_moe_route_scored(x, k, outs, **cfg)
        call()
    for seed in range(4):
        x.copy_(to_dev(logits_of(seed, T, E)))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in outs]
        ref = w4.moe_route_scored(x, k, **cfg)
        assert all(torch.equal(g, r) for g, r in zip(got, ref)), seed
