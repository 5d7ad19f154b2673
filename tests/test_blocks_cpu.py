"""Refusals of the low-rank adapters and of the norms between blocks, on the CPU: a rejected call launches nothing."""
import ctypes

import numpy as np
import pytest

import w4a8_quantized_gemm_token_amd as w4
from tests import blocks_oracle as o

EINVAL, EUNSUPPORTED, EWORKSPACE = 1, 2, 4
F = ctypes.c_void_p(4096)
BIG = 1 << 40


def off(n):
    return ctypes.c_void_p(4096 + n)


LORA = dict(x=F, x_type=0, ldx=256, M=4, K=256, ids=F, A=F, B=F, ab=2, L=8, R=16, ranks=None, scale=None, base=F, ldb=40,
            N=40, out=F, out_type=0, ldo=40, ws=F, ws_bytes=BIG, stream=None)


@pytest.mark.parametrize("change,status", [
    ({"x": None}, EINVAL), ({"ids": None}, EINVAL), ({"A": None}, EINVAL), ({"B": None}, EINVAL), ({"base": None}, EINVAL),
    ({"out": None}, EINVAL), ({"ws": None}, EINVAL), ({"M": -1}, EINVAL), ({"M": 1 << 31}, EINVAL), ({"K": 0}, EINVAL),
    ({"K": -8}, EINVAL), ({"K": 252}, EINVAL), ({"K": (1 << 20) + 8, "ldx": 1 << 21}, EINVAL), ({"ldx": 255}, EINVAL),
    ({"L": 0}, EINVAL), ({"L": 65537}, EINVAL), ({"R": 0}, EINVAL), ({"R": 12}, EINVAL), ({"R": 264}, EINVAL),
    ({"R": -8}, EINVAL), ({"N": 0}, EINVAL), ({"N": (1 << 23) + 1, "ldb": (1 << 24) - 1, "ldo": (1 << 24) - 1}, EINVAL), ({"ldb": 39}, EINVAL),
    ({"ldo": 39}, EINVAL), ({"ldo": 41}, EINVAL), ({"ldx": 1 << 24}, EINVAL), ({"ldb": 1 << 24, "ldo": 1 << 24}, EINVAL), ({"x_type": 3}, EUNSUPPORTED), ({"ab": 0}, EUNSUPPORTED),
    ({"ab": 3}, EUNSUPPORTED), ({"out_type": -1}, EUNSUPPORTED), ({"A": off(8)}, EINVAL), ({"B": off(8)}, EINVAL),
    ({"ws": off(8)}, EINVAL), ({"x": off(2)}, EINVAL), ({"x": off(1), "x_type": 1}, EINVAL), ({"base": off(2)}, EINVAL),
    ({"out": off(2)}, EINVAL), ({"out": off(1), "out_type": 2, "base": off(1)}, EINVAL), ({"ids": off(2)}, EINVAL),
    ({"ranks": off(2)}, EINVAL), ({"scale": off(2)}, EINVAL), ({"ws_bytes": 16}, EWORKSPACE),
    ({"ws_bytes": 0}, EWORKSPACE), ({"M": 0, "x": None, "ids": None, "base": None, "out": None, "ws": None, "ws_bytes": 0}, 0)])
def test_lora_refusals(change, status):
    lib = w4.load()
    assert lib.w4a8_lora_add(*{**LORA, **change}.values()) == status
    if status:
        assert lib.w4a8_last_error()


def test_lora_workspace():
    size = w4.load().w4a8_lora_workspace_size
    assert size(0, 256, 8, 16) == 0 and size(4, 252, 8, 16) == 0 and size(4, 256, 0, 16) == 0 and size(4, 256, 8, 12) == 0
    assert size(-1, 256, 8, 16) == 0
    for M in (1, 5, 64, 100, 1000, 32768, 32769, 1 << 30):
        for R in (8, 16, 256):
            for K in (8, 4096, 1 << 20):
                assert 4 * min(M, 32768) * R <= size(M, K, 8, R) < 1 << 30
    # the largest workspace is taken to the byte
    lib, need = w4.load(), size(4, 256, 8, 16)
    assert lib.w4a8_lora_add(*{**LORA, "ws_bytes": need - 1}.values()) == EWORKSPACE


NORM = dict(res=F, rt=0, ldr=64, y=F, yt=0, ldy=64, M=4, H=64, post=1, pw=None, pb=None, gate=None, gt=0, ldg=0, rs=1.0, ys=1.0,
            ro=off(65536), ldro=64, pre=1, qw=None, qb=None, eps=1e-6, z=off(131072), zt=0, ldz=64, qa=F, sc=F, stream=None)


@pytest.mark.parametrize("change,status", [
    ({"M": -1}, EINVAL), ({"M": 1 << 31}, EINVAL), ({"H": 0}, EINVAL), ({"H": 32769}, EINVAL), ({"res": None, "y": None, "post": 0}, EINVAL),
    ({"y": None}, EINVAL), ({"y": None, "post": 0, "gate": F}, EINVAL), ({"post": 3}, EUNSUPPORTED), ({"post": -1}, EUNSUPPORTED),
    ({"pre": 3}, EUNSUPPORTED), ({"rt": 3}, EUNSUPPORTED), ({"yt": -1}, EUNSUPPORTED), ({"zt": 3}, EUNSUPPORTED),
    ({"gate": F, "gt": 5}, EUNSUPPORTED), ({"post": 0, "pw": F}, EINVAL), ({"pre": 0, "qb": F}, EINVAL),
    ({"ro": None, "z": None, "qa": None, "sc": None}, EINVAL), ({"sc": None}, EINVAL), ({"qa": None}, EINVAL),
    ({"ldr": 63}, EINVAL), ({"ldy": 63}, EINVAL), ({"ldro": 63}, EINVAL), ({"ldz": 63}, EINVAL), ({"gate": F, "ldg": 63}, EINVAL),
    ({"gate": F, "ldg": -1}, EINVAL), ({"res": off(2)}, EINVAL), ({"y": off(1), "yt": 1}, EINVAL), ({"ro": off(2)}, EINVAL),
    ({"z": off(2)}, EINVAL), ({"gate": off(2)}, EINVAL), ({"qa": off(8)}, EINVAL), ({"sc": off(2)}, EINVAL), ({"pw": off(2)}, EINVAL),
    ({"qw": off(1)}, EINVAL), ({"eps": 0.0}, EINVAL), ({"eps": 1e-41}, EINVAL), ({"eps": -1e-6}, EINVAL), ({"eps": float("nan")}, EINVAL),
    ({"rs": float("inf")}, EINVAL), ({"ys": float("nan")}, EINVAL), ({"z": off(65536)}, EINVAL),
    ({"ro": F, "ldro": 65}, EINVAL), ({"ro": F, "rt": 0, "yt": 1}, EINVAL), ({"z": F, "zt": 2}, EINVAL), ({"z": F, "ldz": 72}, EINVAL),
    ({"M": 0, "res": None, "y": None, "ro": None, "z": None, "qa": None, "sc": None, "post": 0}, 0)])
def test_norm_refusals(change, status):
    lib = w4.load()
    assert lib.w4a8_residual_norm_quantize(*{**NORM, **change}.values()) == status
    if status:
        assert lib.w4a8_last_error()


def test_python_checks():
    torch = pytest.importorskip("torch")
    z = torch.zeros
    ids, ws = z(2, dtype=torch.int32), z(1024, dtype=torch.uint8)
    A, B = z(3, 8, 16, dtype=torch.bfloat16), z(3, 9, 8, dtype=torch.bfloat16)
    bad = [dict(), dict(out=z(2, 8)), dict(ids=z(2)), dict(ids=z(3, dtype=torch.int32)), dict(B=z(3, 9, 16, dtype=torch.bfloat16)),
           dict(B=z(3, 9, 8, dtype=torch.float16)), dict(scale=z(2)), dict(ranks=z(3)), dict(base=z(2, 9, dtype=torch.float16)),
           dict(x=z(2, 16, dtype=torch.float64))]  # the first: host tensors, there is no CPU fallback
    for change in bad:
        c = dict(dict(out=z(2, 9), x=z(2, 16), ids=ids, A=A, B=B, scale=None, ranks=None, base=None), **change)
        with pytest.raises(AssertionError):
            w4.prepare_lora_add(c["out"], c["x"], c["ids"], c["A"], c["B"], ws, scale=c["scale"], ranks=c["ranks"], base=c["base"])
    outs = (z(2, 16), None, z(2, 16, dtype=torch.int8), z(2))
    for change in (dict(), dict(y=z(2, 8)), dict(pre="batch"), dict(pre_w=z(8)), dict(gate=z(3, 16)), dict(outs=(z(2, 16, dtype=torch.float16),) + outs[1:]),
                   dict(outs=(None, None, z(2, 16, dtype=torch.int8), z(3)))):
        c = dict(dict(y=z(2, 16), outs=outs, pre="rms", pre_w=None, gate=None), **change)
        with pytest.raises(AssertionError):
            w4.prepare_residual_norm_quantize(z(2, 16), c["y"], c["outs"], pre=c["pre"], pre_w=c["pre_w"], gate=c["gate"])


def test_oracle_worked_examples():
    """The 64-bit forms on numbers that can be checked by hand."""
    v, _ = o.norm(np.array([[3.0, 4.0]]), "rms", None, None, 0.5)           # mean square 12.5, + 0.5 = 13
    assert np.allclose(v, [[3 / 13 ** 0.5, 4 / 13 ** 0.5]], rtol=1e-15)
    v, _ = o.norm(np.array([[1.0, 3.0]]), "layer", np.array([2.0, 1.0]), np.array([0.0, 5.0]), 3.0)  # mean 2, var 1
    assert np.allclose(v, [[-1.0, 5.5]], rtol=1e-15)
    q, s = o.quantized(np.array([[1.27, -0.635, 0.0]]))
    assert q.tolist() == [[127, -64, 0]] or q.tolist() == [[127, -63, 0]]
    x, A, B = np.array([[1.0, 2.0]]), np.array([[[3.0, 4.0], [100.0, 100.0]]]), np.array([[[0.5, 9.0], [-1.0, 9.0]]])
    v, _ = o.lora(x, [0], A, B, [1], [2.0], np.array([[10.0, 20.0]]), "f32", True)  # v = 11
    assert v.tolist() == [[21.0, -2.0]]
    v, bound = o.lora(x, [1], A, B, None, None, np.array([[10.0, 20.0]]), "f32", True)  # no such adapter
    assert v.tolist() == [[10.0, 20.0]] and not bound.any()
