"""Refusals of the 8-bit product and of the scored router, on the CPU: a rejected call launches nothing."""
import ctypes

import numpy as np
import pytest

import w4a8_quantized_gemm_token_amd as w4
from tests import w8_oracle as o

EINVAL, EUNSUPPORTED = 1, 2
F = ctypes.c_void_p(4096)


def off(n):
    return ctypes.c_void_p(4096 + n)


GEMM = dict(qa=F, sa=F, M=4, K=256, qw=F, sw=F, N=40, bias=None, out=F, type=0, ldo=40, stream=None)


@pytest.mark.parametrize("change,status", [
    ({"qa": None}, EINVAL), ({"sa": None}, EINVAL), ({"qw": None}, EINVAL), ({"sw": None}, EINVAL),
    ({"out": None}, EINVAL), ({"M": -1}, EINVAL), ({"M": 1 << 31}, EINVAL), ({"K": 0}, EINVAL), ({"K": -16}, EINVAL),
    ({"K": 24}, EINVAL), ({"K": 1 << 17}, EINVAL), ({"N": 0}, EINVAL), ({"N": 1 << 31, "ldo": 1 << 31}, EINVAL),
    ({"ldo": 39}, EINVAL), ({"type": 3}, EUNSUPPORTED), ({"type": -1}, EUNSUPPORTED), ({"qa": off(8)}, EINVAL),
    ({"qw": off(8)}, EINVAL), ({"out": off(2)}, EINVAL), ({"out": off(1), "type": 1}, EINVAL),
    ({"M": 0, "qa": None, "sa": None, "out": None}, 0)])
def test_gemm_refusals(change, status):
    lib = w4.load()
    assert lib.w4a8_gemm_w8a8(*{**GEMM, **change}.values()) == status
    if status:
        assert lib.w4a8_last_error()


GROUPED = dict(qa=F, sa=F, R=8, rows=F, off=F, E=4, K=256, qw=F, sw=F, N=40, slots=16, out=F, stream=None)


@pytest.mark.parametrize("change,status", [
    ({"qa": None}, EINVAL), ({"sa": None}, EINVAL), ({"off": None}, EINVAL), ({"qw": None}, EINVAL),
    ({"sw": None}, EINVAL), ({"out": None}, EINVAL), ({"R": -1}, EINVAL), ({"R": 1 << 31}, EINVAL), ({"E": 0}, EINVAL),
    ({"E": 1025}, EINVAL), ({"K": 40}, EINVAL), ({"K": 1 << 17}, EINVAL), ({"N": 0}, EINVAL), ({"slots": -1}, EINVAL),
    ({"slots": 1 << 31}, EINVAL), ({"qa": off(8)}, EINVAL), ({"qw": off(4)}, EINVAL), ({"out": off(4)}, EINVAL),
    ({"slots": 0}, 0), ({"R": 0}, 0)])
def test_grouped_refusals(change, status):
    lib = w4.load()
    assert lib.w4a8_moe_grouped_gemm_w8a8(*{**GROUPED, **change}.values()) == status


ROUTE = dict(logits=F, type=0, ldl=64, bias=None, T=4, E=64, k=8, shared=0, score=0, n=8, keep=4, lead=2, renorm=1,
             scale=1.0, ids=F, w=F, off=F, perm=F, rows=None, sop=F, stream=None)


@pytest.mark.parametrize("change,status", [
    ({"logits": None}, EINVAL), ({"ids": None}, EINVAL), ({"w": None}, EINVAL), ({"off": None}, EINVAL),
    ({"perm": None}, EINVAL), ({"sop": None}, EINVAL), ({"T": -1}, EINVAL), ({"T": 1 << 28}, EINVAL), ({"T": 1 << 62}, EINVAL),
    ({"E": 0}, EINVAL), ({"E": 1025, "ldl": 1025, "n": 1, "keep": 1}, EINVAL), ({"ldl": 63}, EINVAL), ({"k": 0}, EINVAL),
    ({"k": 33}, EINVAL), ({"E": 4, "n": 1, "keep": 1, "k": 5}, EINVAL), ({"shared": 2}, EINVAL), ({"type": 3}, EUNSUPPORTED),
    ({"score": 2}, EUNSUPPORTED), ({"n": 0}, EINVAL), ({"n": 7}, EINVAL), ({"E": 130, "ldl": 130, "n": 65, "keep": 9}, EINVAL),
    ({"keep": 0}, EINVAL), ({"keep": 9}, EINVAL), ({"k": 9, "keep": 1}, EINVAL), ({"lead": 0}, EINVAL), ({"lead": 3}, EINVAL),
    ({"n": 64, "keep": 8, "lead": 2}, EINVAL), ({"renorm": 2}, EINVAL), ({"scale": float("nan")}, EINVAL),
    ({"scale": float("inf")}, EINVAL), ({"logits": off(2)}, EINVAL), ({"logits": off(1), "type": 2}, EINVAL)])
def test_route_refusals(change, status):
    lib = w4.load()
    assert lib.w4a8_moe_route_scored(*{**ROUTE, **change}.values()) == status
    assert lib.w4a8_last_error()


def test_python_checks():
    torch = pytest.importorskip("torch")
    z = torch.zeros
    with pytest.raises(AssertionError):
        w4.prepare_gemm_w8a8(z(2, 16, dtype=torch.int8), z(2), z(8, 16, dtype=torch.int8), z(8), z(2, 9))
    with pytest.raises(AssertionError):
        w4.prepare_gemm_w8a8(z(2, 16, dtype=torch.int8), z(2), z(8, 16, dtype=torch.int8), z(8, dtype=torch.float64), z(2, 8))
    with pytest.raises(AssertionError):  # host tensors: there is no CPU fallback
        w4.prepare_gemm_w8a8(z(2, 16, dtype=torch.int8), z(2), z(8, 16, dtype=torch.int8), z(8), z(2, 8))
    with pytest.raises(AssertionError):
        w4.prepare_moe_grouped_gemm_w8a8(z(2, 16, dtype=torch.int8), z(2), None, z(3, dtype=torch.int32),
                                         z(2, 8, 16, dtype=torch.int8), z(2, 8), 5, z(5, 8))


# ------------------------------------------------------------------ the oracle itself
def test_oracle_route_by_hand():
    x = np.array([[0.0, np.log(3.0), -np.inf, np.log(2.0)]])
    ids, w = o.route(x, 2)                                 # softmax 1/6, 3/6, 0, 2/6
    assert ids.tolist() == [[1, 3]] and np.allclose(w, [[0.6, 0.4]])
    ids, w = o.route(x, 2, renorm=False, scale=2.0)
    assert np.allclose(w, [[1.0, 2 / 3]])
    ids, w = o.route(x, 2, score="sigmoid", bias=np.array([0.6, 0.0, 9.0, 0.0]))   # 1.1, .75, -inf, 2/3
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[0.4, 0.6]])
    ids, _ = o.route(x, 2, n_groups=2, topk_groups=1, group_lead=2)                # groups 4/6 and 2/6
    assert ids.tolist() == [[1, 0]]
    ids, w = o.route(np.full((1, 4), -np.inf), 2)
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]


def test_oracle_mistakes_are_caught():
    """A planted mistake in the oracle's inputs is outside the stated bounds: one code off by one, the bias left out,
    a sum rounded to bfloat16."""
    rng = np.random.default_rng(0)
    qa, qw = rng.integers(-127, 128, (3, 64), dtype=np.int8), rng.integers(-127, 128, (5, 64), dtype=np.int8)
    sa, sw, b = np.full(3, 0.01, np.float32), np.full(5, 0.02, np.float32), np.full(5, 0.5, np.float32)
    ref, bound = o.product(qa, sa, qw, sw, b)
    o.close(ref.astype(np.float32), ref, bound, 0.0, 0.0)
    wrong = qa.copy()
    wrong[1, 7] += 1 if wrong[1, 7] < 0 else -1
    for bad in (o.product(wrong, sa, qw, sw, b)[0], o.product(qa, sa, qw, sw)[0], ref * (1 + 2.0 ** -9)):
        with pytest.raises(AssertionError):
            o.close(bad, ref, bound, 0.0, 0.0)


# ------------------------------------------------------------------ devices
def test_calls_run_on_their_tensors_device(monkeypatch):
    """Each call makes its tensors' device the current one while it launches: the library launches on the
    current device."""
    torch = pytest.importorskip("torch")
    entered, launched = [], []

    class Guard:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            entered.append(self.device)

        def __exit__(self, *_):
            entered.pop()

    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(w4, "_call", lambda name, *args: launched.append((name, list(entered))))
    monkeypatch.setattr(w4, "_dev_ptr", lambda t: None)
    monkeypatch.setattr(w4, "_dev_rows_ptr", lambda t: None)
    monkeypatch.setattr(w4, "_stream", lambda device=None: None)
    z, i8, i32 = torch.zeros, torch.int8, torch.int32
    w4.quantize_weights_w8(z(8, 16))
    w4.gemm_w8a8(z(2, 16, dtype=i8), z(2), z(8, 16, dtype=i8), z(8))
    w4.moe_route_scored(z(2, 8), 3)
    w4.moe_grouped_gemm_w8a8(z(2, 16, dtype=i8), z(2), None, z(3, dtype=i32), z(2, 8, 16, dtype=i8), z(2, 8), 2)
    assert [name for name, _ in launched] == ["w4a8_quantize_act", "w4a8_gemm_w8a8", "w4a8_moe_route_scored",
                                              "w4a8_moe_grouped_gemm_w8a8"]
    assert all(devices == [torch.device("cpu")] for _, devices in launched), launched


# ------------------------------------------------------------------ which sizes the GPU tests run
def split_of_k(K, max_waves=16, max_nw=4):
    """(windows per wave, more than one pass) of the few-row loop: the launcher's rule, written again."""
    windows = -(-K // 128)
    passes = -(-windows // (max_waves * max_nw))
    per = -(-windows // passes)
    if passes > 1:
        return max_nw, True
    fits = [nw for nw in range(1, max_nw + 1) if -(-per // nw) <= max_waves]
    return min(fits, key=lambda nw: (-(-per // nw) * nw - per, nw)), False


def test_gpu_tests_reach_every_split_of_k():
    pytest.importorskip("torch")
    from tests.test_gpu_w8a8_forms import FEW_ROW_K
    every = {(1, False), (2, False), (3, False), (4, False), (4, True)}
    assert {split_of_k(K) for K in FEW_ROW_K} == every
    assert {split_of_k(K) for K in FEW_ROW_K if K % 128} == every  # with a part window too
    assert {split_of_k(16 * c) for c in range(1, 8192)} == every   # there are no others
