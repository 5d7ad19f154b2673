"""Plain 64-bit forms of the low-rank adapters and of the norms, gate and residual between blocks, for the tests."""
from __future__ import annotations

import numpy as np

STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}       # half a step of a type, relative
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}    # half its smallest subnormal


def lora(x, ids, A, B, ranks, scale, base, out, exact_x):
    """(value, bound) of the adapters' rows.  x, A, B, base hold the values of their types in float64.

    The bound counts, with u = 2^-23 (a step, so that accumulation may cut off): the 32 products of a matrix instruction
    and the K / 32 instructions in a row, of sum |x||A|; the representation of x (2^-22 of fp32 outputs, 2^-16 of 16-bit
    ones, twice for the products of parts that are left out); the same for v over B's rank; scale, sum and rounding."""
    u = 2.0 ** -23
    held = 2.0 ** (-21 if out == "f32" else -15)
    value, bound = base.copy(), np.zeros_like(base)
    L, R, K = A.shape
    for m, a in enumerate(ids):
        if not 0 <= a < L:
            continue
        rank = R if ranks is None else int(min(max(ranks[a], 0), R))
        if rank == 0:
            continue
        s = 1.0 if scale is None else float(scale[a])
        Ar, Br = A[a, :rank], B[a, :, :rank]
        v, size = Ar @ x[m], np.abs(Ar) @ np.abs(x[m])
        verr = size * ((32 + K / 32) * u + (0.0 if exact_x else held))
        t, tsize = Br @ v, np.abs(Br) @ (np.abs(v) + verr)
        terr = np.abs(Br) @ verr + tsize * ((32 + rank / 32) * u + held)
        value[m] = base[m] + s * t
        bound[m] = abs(s) * (terr + 2 * u * tsize) + u * (np.abs(base[m]) + np.abs(s * t))
    return value, bound


def close(got, value, bound, out, what=""):
    """|got - value| within the bound and half a step of the output's type."""
    got = np.asarray(got, np.float64)
    tol = bound * (1 + STEP[out]) + STEP[out] * (np.abs(value) + bound) + TINY[out]
    same = (got == value) | (np.isnan(got) & np.isnan(value))
    bad = ~(same | (np.abs(got - value) <= tol))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside, first at {np.argwhere(bad)[0].tolist()}: "
                           f"{got[bad][0]!r} for {value[bad][0]!r}, tolerance {tol[bad][0]!r}")


def norm(u, kind, w, b, eps):
    """(value, size) of a norm of the rows of u: `size` is the magnitude that 64-bit roundings are relative to."""
    if kind == "none":
        return u.copy(), np.abs(u)
    mean = u.mean(1, keepdims=True) if kind == "layer" else np.zeros((u.shape[0], 1))
    spread = np.abs(u).mean(1, keepdims=True) if kind == "layer" else mean
    d = u - mean
    inv = 1.0 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    w = np.ones(u.shape[1]) if w is None else w.astype(np.float64)
    v, size = d * inv * w, (np.abs(u) + spread) * inv * np.abs(w)
    if b is not None:
        v, size = v + b.astype(np.float64), size + np.abs(b.astype(np.float64))
    return v, size


def joined(res, y, post, post_w, post_b, gate, res_scale, y_scale, eps):
    """(value, size) of the stream before its rounding."""
    v, size = 0.0, 0.0
    if y is not None:
        v, size = norm(y, post, post_w, post_b, eps)
        g = np.ones(1) if gate is None else gate
        v, size = v * g * y_scale, size * np.abs(g * y_scale)
    if res is not None:
        v, size = v + res_scale * res, size + np.abs(res_scale * res)
    return v, size


# 64-bit sums with up to 500 additions in a row (rows of 32768 are summed by 64 threads at least, then as a tree), products,
# roots and quotients: 512 half steps 2^-53 of the size
SLACK = 2.0 ** -44


def quantized(z):
    """Codes and scales of fp32 rows: s = max |z| times the fp32 number next to 1/127, q = rint(z / s)."""
    z = z.astype(np.float32)
    with np.errstate(invalid="ignore", divide="ignore"):
        s = np.abs(z).max(1) * (np.float32(1.0) / np.float32(127.0))
        q = np.clip(np.rint(z / s[:, None]), -127, 127)
    return np.where(s[:, None] == 0, 0, q).astype(np.int8), s.astype(np.float32)
