"""Plain 64-bit forms of the 8-bit product and of the scored router, for the tests."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half an fp32 step, relative


def product(qa, sa, qw, sw, bias=None):
    """(value, bound) of a_scale[m] w_scale[n] sum_k qa qw + bias in float64: |sum| < 2^31, so the float64
    product of the codes is exact.  The bound counts the kernel's fp32 roundings: the sum's conversion and
    the two scalings (three relative half steps of the product), the bias addition (one of the result)."""
    isum = qa.astype(np.float64) @ qw.astype(np.float64).T
    p = isum * sa.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :]
    v = p if bias is None else p + bias.astype(np.float64)[None, :]
    # (1 + U)^3 - 1 < 3.001 U for the product, then U of |p| (1 + 3.001 U) + |bias|
    bound = 3.001 * U * np.abs(p)
    if bias is not None:
        bound = bound + 1.001 * U * (np.abs(p) + np.abs(bias.astype(np.float64))[None, :])
    return v, bound


def close(got, value, bound, eps, tiny, what=""):
    """|got - value| within the fp32 bound plus half a step of the output's type (eps / 2 relative, or half its
    smallest subnormal `tiny`)."""
    tol = bound * (1 + eps) + eps / 2 * (np.abs(value) + bound) + tiny / 2
    err = np.abs(got.astype(np.float64) - value)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside, first at "
                           f"{np.argwhere(bad)[0].tolist()}: {got[bad][0]!r} for {value[bad][0]!r}")


def tame(x):
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    return np.minimum(x, float(np.finfo(np.float32).max))


def route(logits, k, bias=None, score="softmax", n_groups=1, topk_groups=1, group_lead=1, renorm=True, scale=1.0):
    """(ids [T][k], w [T][k] float64), token by token from the definition."""
    x = tame(logits)
    T, E = x.shape
    b = np.zeros(E) if bias is None else tame(bias)
    ids, w = np.zeros((T, k), np.int64), np.zeros((T, k))
    for t in range(T):
        xt = x[t]
        live = np.isfinite(xt)
        s = np.zeros(E)
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                s[live] = 1.0 / (1.0 + np.exp(-xt[live]))
        elif live.any():
            e = np.exp(xt[live] - xt[live].max())
            s[live] = e / e.sum()
        v = np.where(live & (b > -np.inf), s + np.where(b > -np.inf, b, 0.0), -np.inf)
        key = xt if bias is None else v
        gs = E // n_groups
        value = [sum(sorted(v[g * gs:(g + 1) * gs], reverse=True)[:group_lead]) for g in range(n_groups)]
        kept = sorted(range(n_groups), key=lambda g: (-value[g], g))[:topk_groups]
        open_ = [e for g in kept for e in range(g * gs, (g + 1) * gs)]
        pick = sorted(open_, key=lambda e: (-key[e], e))[:k]
        wt = np.array([s[e] if key[e] > -np.inf else 0.0 for e in pick])
        if renorm:
            wt = wt / wt.sum() if wt.sum() > 0 else np.zeros(k)
        ids[t], w[t] = pick, wt * scale
    return ids, w


def tables(ids, E, with_shared):
    """offsets, perm, row_index, slot_of_pair of the picks."""
    T, k = ids.shape
    flat = ids.reshape(-1)
    perm = np.argsort(flat, kind="stable")
    off = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))])
    rows = perm // k
    if with_shared:
        off = np.concatenate([off, [off[-1] + T]])
        rows = np.concatenate([rows, np.arange(T)])
    sop = np.empty_like(perm)
    sop[perm] = np.arange(perm.size)
    return off, perm, rows, sop
