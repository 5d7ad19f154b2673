"""Timed cases of the scored expert routing and of the 8-bit products (dense and per expert).

`run` computes an operator in elementary torch operations where `own` is false, and calls the library where it is
true; `exact` gives the same outputs from the definitions in 64 bits.

  route    logits [T][E] (and a balance bias per expert) -> picked experts, their weights, and the bucket tables the
           expert products read (offsets, pairs by expert, activation row of each slot, slot of each pair)
  gemm     int8 rows [M][K] times int8 weights [N][K], scaled per token and per output channel
  grouped  the same product where each slot's weights are those of its expert
"""
import math
import statistics

import torch

own = False

DEVICE = "cuda:0"
TYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


def listed():
    return [
        # one token of a decoding request, every expert scored: latency is all that counts
        dict(name="route one token", op="route", T=1, E=384, k=8, score="sigmoid", bias=True, groups=1, keep=1, lead=1,
             renorm=True, scale=2.5, shared=True, type="float32"),
        # a decode batch with group-limited picks: 8 groups, the 4 with the best two-expert sums stay
        dict(name="route decode batch", op="route", T=64, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4,
             lead=2, renorm=True, scale=2.5, shared=True, type="float32"),
        # a prefill chunk
        dict(name="route prefill", op="route", T=4096, E=384, k=8, score="sigmoid", bias=True, groups=1, keep=1, lead=1,
             renorm=True, scale=1.0, shared=True, type="float32"),
        # a long ragged prefill from a bf16 router: softmax scores, groups by their best expert, weights as they are
        dict(name="route long", op="route", T=20011, E=160, k=6, score="softmax", bias=False, groups=8, keep=3, lead=1,
             renorm=False, scale=16.0, shared=False, type="bfloat16"),
        # one token through a large projection: the weight stream
        dict(name="gemm one token", op="gemm", M=1, K=8192, N=28672, bias=False, type="float32"),
        # a decode batch through the same projection, bf16 out with a channel bias
        dict(name="gemm decode batch", op="gemm", M=16, K=8192, N=28672, bias=True, type="bfloat16"),
        # a small mixed batch through a layer of odd sizes
        dict(name="gemm ragged", op="gemm", M=77, K=4112, N=5003, bias=True, type="float16"),
        # a prefill chunk through a square projection
        dict(name="gemm prefill", op="gemm", M=4096, K=8192, N=8192, bias=False, type="bfloat16"),
        # one token through its 8 experts of 384 (gate and up stacked)
        dict(name="experts one token", op="grouped", T=1, E=384, k=8, K=7168, N=4096),
        # a decode batch: most experts that are hit see a few tokens
        dict(name="experts decode batch", op="grouped", T=64, E=384, k=8, K=7168, N=4096),
        # few large experts, about a hundred tokens each, ragged columns
        dict(name="experts ragged", op="grouped", T=500, E=8, k=2, K=4096, N=14340),
        # a prefill chunk over all experts, from cold ones to hot ones
        dict(name="experts prefill", op="grouped", T=4096, E=384, k=8, K=7168, N=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "gemm", "grouped"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 5, 8])
        size = rng.randint(6, 384 // groups)
        keep = rng.randint((groups + 1) // 2, groups)
        score = rng.choice(["sigmoid", "softmax"])
        return dict(op=op, T=_log(rng, 1, 20011), E=groups * size, k=rng.randint(1, min(8, keep * size)), score=score,
                    bias=rng.random() < 0.6, groups=groups, keep=keep, lead=rng.choice([1, 2]), renorm=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5, 16.0]), shared=rng.random() < 0.5, type=rng.choice(sorted(TYPES)))
    if op == "gemm":
        M, K = _log(rng, 1, 4096), 16 * _log(rng, 16, 512)
        most = min(235_000_000 // K, 4096 * 8192 * 8192 // (M * K), 28672)
        return dict(op=op, M=M, K=K, N=_log(rng, 64, most), bias=rng.random() < 0.5, type=rng.choice(sorted(TYPES)))
    E, K = _log(rng, 4, 384), 16 * _log(rng, 16, 448)
    T, k = _log(rng, 1, 4096), rng.randint(1, min(8, E))
    N = _log(rng, 64, min(14336, 384 * 7168 * 4096 // (E * K), 8 * 4096 * 7168 * 4096 // (T * k * K)))
    return dict(op=op, T=T, E=E, k=k, K=K, N=N)


# ---------------------------------------------------------------- inputs

def _popularity(E):
    """Log-weights of the experts: normal quantiles, so a few are hot and many are cold."""
    q = [statistics.NormalDist().inv_cdf((e + 0.5) / E) for e in range(E)]
    return [q[(e * 97 + 13) % E] for e in range(E)] if E % 97 else q


def _codes(x):
    """Symmetric 8-bit codes of each row and the row's scale."""
    s = x.abs().amax(-1) / 127.0
    q = torch.round(x / s[..., None]).clamp(-127, 127).to(torch.int8)
    return q, s


def _activations(rows, K, gen):
    """Normal rows of differing size, with a few channels far above the others."""
    x = torch.randn(rows, K, generator=gen, device=DEVICE)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device=DEVICE))
    x[:, torch.randint(0, K, (4,), generator=gen, device=DEVICE)] *= 8.0
    return _codes(x)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    state = dict(case)
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        x = 1.5 * torch.randn(T, E, generator=gen, device=DEVICE)
        x += 0.5 * torch.tensor(_popularity(E), device=DEVICE)
        state["logits"] = x.to(TYPES[case["type"]])
        state["b"] = 0.05 * torch.randn(E, generator=gen, device=DEVICE) if case["bias"] else None
        pairs, extra = T * k, T if case["shared"] else 0
        whole = dict(dtype=torch.int32, device=DEVICE)
        state["out"] = (torch.zeros(T, k, **whole), torch.zeros(T, k, device=DEVICE),
                        torch.zeros(E + 1 + bool(extra), **whole), torch.zeros(pairs, **whole),
                        torch.zeros(pairs + extra, **whole), torch.zeros(pairs, **whole))
    elif case["op"] == "gemm":
        M, K, N = case["M"], case["K"], case["N"]
        state["qa"], state["sa"] = _activations(M, K, gen)
        state["qw"], state["sw"] = _codes(0.02 * torch.randn(N, K, generator=gen, device=DEVICE))
        state["b"] = 0.1 * torch.randn(N, generator=gen, device=DEVICE) if case["bias"] else None
        state["out"] = torch.zeros(M, N, dtype=TYPES[case["type"]], device=DEVICE)
    else:
        T, E, k, K, N = (case[n] for n in ("T", "E", "k", "K", "N"))
        state["qa"], state["sa"] = _activations(T, K, gen)
        state["qw"] = torch.empty(E, N, K, dtype=torch.int8, device=DEVICE)
        state["sw"] = torch.empty(E, N, device=DEVICE)
        for e in range(E):
            state["qw"][e], state["sw"][e] = _codes(0.02 * torch.randn(N, K, generator=gen, device=DEVICE))
        noise = -torch.log(-torch.log(torch.rand(T, E, generator=gen, device=DEVICE).clamp(1e-9, 1 - 1e-7)))
        ids = torch.topk(noise + torch.tensor(_popularity(E), device=DEVICE), k).indices.reshape(-1)
        order = torch.sort(ids, stable=True).indices
        counts = torch.bincount(ids, minlength=E)
        state["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        state["rows"] = (order // k).to(torch.int32)
        state["out"] = torch.zeros(T * k, N, device=DEVICE)
    state["call"] = _handle(state) if own else None
    return state


def _handle(s):
    """The prepared library call that a serving loop keeps for its buffers."""
    import w4a8_quantized_gemm_token_amd as w4
    if s["op"] == "route":
        return w4.prepare_moe_route_scored(s["logits"], s["k"], s["out"], bias=s["b"], score=s["score"],
                                           n_groups=s["groups"], topk_groups=s["keep"], group_lead=s["lead"],
                                           renorm=s["renorm"], scale=s["scale"], with_shared=s["shared"])
    if s["op"] == "gemm":
        return w4.prepare_gemm_w8a8(s["qa"], s["sa"], s["qw"], s["sw"], s["out"], bias=s["b"])
    return w4.prepare_moe_grouped_gemm_w8a8(s["qa"], s["sa"], s["rows"], s["offsets"], s["qw"], s["sw"],
                                            s["out"].shape[0], s["out"])


# ---------------------------------------------------------------- the operators

def run(state):
    if own:
        state["call"]()
        return state["out"]
    return {"route": _route, "gemm": _gemm, "grouped": _grouped}[state["op"]](state)


def _route(s):
    # scores and keys in 64 bits: two experts' keys are often closer than 32 bits can tell
    T, E, k, groups = s["T"], s["E"], s["k"], s["groups"]
    x = s["logits"].double()
    if s["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        score = torch.exp(x - x.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    # without a bias the scores have the logits' order
    key = x if s["b"] is None else score + s["b"].double()
    if groups > 1:
        value = score if s["b"] is None else key
        best = torch.sort(value.view(T, groups, -1), dim=2, descending=True).values[:, :, :s["lead"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["keep"]]
        open_ = torch.zeros(T, groups, dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        key = torch.where(open_.repeat_interleave(E // groups, 1), key, -math.inf)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = (w * s["scale"]).float()
    flat = ids.reshape(-1)
    perm = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    rows = perm // k
    if s["shared"]:
        offsets = torch.cat([offsets, offsets[-1:] + T])
        rows = torch.cat([rows, torch.arange(T, device=x.device)])
    slot = torch.empty_like(perm)
    slot[perm] = torch.arange(T * k, device=x.device)
    return (ids.to(torch.int32), w, offsets.to(torch.int32), perm.to(torch.int32), rows.to(torch.int32),
            slot.to(torch.int32))


def _gemm(s):
    acc = s["qa"].float() @ s["qw"].float().t()
    out = acc * s["sa"][:, None] * s["sw"]
    if s["b"] is not None:
        out = out + s["b"]
    return out.to(TYPES[s["type"]])


def _grouped(s):
    out = torch.empty(s["rows"].shape[0], s["N"], device=DEVICE)
    ends = s["offsets"].tolist()
    for e in range(s["E"]):
        a, b = ends[e], ends[e + 1]
        if a < b:
            rows = s["rows"][a:b].long()
            acc = s["qa"][rows].float() @ s["qw"][e].float().t()
            out[a:b] = acc * s["sa"][rows][:, None] * s["sw"][e]
    return out


# ---------------------------------------------------------------- work and exact values

def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        extra = 1 if case["shared"] else 0
        size = 4 if case["type"] == "float32" else 2
        return {"bytes": T * E * size + 4 * E * case["bias"] + 4 * (5 * T * k + extra * T + E + 1 + extra),
                "flops": 10 * T * E}
    if case["op"] == "gemm":
        M, K, N = case["M"], case["K"], case["N"]
        size = 4 if case["type"] == "float32" else 2
        return {"bytes": M * K + N * K + 4 * (M + N + N * case["bias"]) + M * N * size, "flops": 2 * M * N * K}
    T, E, k, K, N = (case[n] for n in ("T", "E", "k", "K", "N"))
    # experts that at least one token picks, from the popularity that prepare() draws them by
    p = [math.exp(v) for v in _popularity(E)]
    hit = sum(1.0 - (1.0 - min(1.0, k * v / sum(p))) ** T for v in p)
    hit = min(max(hit, k), E)
    return {"bytes": int(T * (K + 4) + hit * N * (K + 4) + 4 * T * k + 4 * (E + 1) + 4 * T * k * N),
            "flops": 2 * T * k * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "gemm":
        scale = s["sa"].double()[:, None] * s["sw"].double()[None]
        value = torch.mm(s["qa"].double(), s["qw"].double().t().contiguous()) * scale
        return value if s["b"] is None else value + s["b"].double()[None]
    out = torch.empty(s["rows"].shape[0], s["N"], dtype=torch.float64, device=DEVICE)
    first = s["offsets"].long().cpu()
    for e in torch.nonzero(first[1:] > first[:-1]).flatten().tolist():
        at = slice(int(first[e]), int(first[e + 1]))
        r = s["rows"].long()[at]
        scale = s["sa"].double()[r].unsqueeze(1) * s["sw"][e].double().unsqueeze(0)
        out[at] = torch.mm(s["qa"].double()[r], s["qw"][e].double().t().contiguous()) * scale
    return out


def _before(v):
    """How many entries of a row come before each of its entries: larger ones, and equal ones to the left."""
    n = v.shape[1]
    left = torch.ones(n, n, dtype=torch.bool, device=v.device).tril(-1)
    mine, other = v[:, :, None], v[:, None, :]
    return ((other > mine) | ((other == mine) & left)).sum(2)


def _exact_route(s):
    T, E, k, groups = s["T"], s["E"], s["k"], s["groups"]
    all_ids, all_w = [], []
    for x in s["logits"].double().split(512):
        t = x.shape[0]
        score = torch.sigmoid(x) if s["score"] == "sigmoid" else torch.softmax(x, 1)
        value = score if s["b"] is None else score + s["b"].double()
        key = x if s["b"] is None else value
        g = value.reshape(t * groups, E // groups)
        lead = _before(g) < s["lead"]
        total = torch.where(lead, g, 0.0).sum(1).view(t, groups)
        closed = (_before(total) >= s["keep"]).repeat_interleave(E // groups, 1)
        place = _before(torch.where(closed, -math.inf, key))
        ids = torch.argsort(place, 1)[:, :k]
        w = torch.take_along_dim(score, ids, 1)
        all_ids.append(ids)
        all_w.append(w * s["scale"] / (w.sum(1, keepdim=True) if s["renorm"] else 1.0))
    ids = torch.cat(all_ids)
    pair = torch.arange(T * k, device=DEVICE)
    perm = torch.argsort(ids.reshape(-1) * (T * k) + pair)
    bounds = torch.searchsorted(ids.reshape(-1)[perm].contiguous(), torch.arange(E + 1, device=DEVICE))
    rows = torch.div(perm, k, rounding_mode="floor")
    if s["shared"]:
        bounds = torch.cat([bounds, torch.tensor([T * k + T], device=DEVICE)])
        rows = torch.cat([rows, torch.arange(T, device=DEVICE)])
    slot = torch.argsort(perm)
    return tuple(v.to(torch.int32) if v.dtype == torch.int64 else v
                 for v in (ids, torch.cat(all_w), bounds, perm, rows, slot))
