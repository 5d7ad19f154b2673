"""GPU tests of the norms, gate and residual between blocks against their 64-bit form (blocks_oracle)."""
from __future__ import annotations

import numpy as np
import pytest

from tests import blocks_oracle as o
from tests.gpu_common import cuda, to_dev, to_host

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
    M, W = values.shape
    ld = ld or W
    flat = torch.full((shift + M * ld + 8,), SENTINEL, dtype=TYPES[kind], device=cuda())
    view = flat[shift:shift + M * ld].view(M, ld)[:, :W]
    view.copy_(torch.as_tensor(values))
    return view, flat


def host64(t):
    return None if t is None else to_host(t.double())


def as_type(v, kind):
    """float64 through fp32 to the type, back in float64."""
    with np.errstate(over="ignore", invalid="ignore"):
        t = torch.as_tensor(np.asarray(v).astype(np.float32)).to(TYPES[kind])
    return t.double().numpy()


def between(got, value, size, kind, what):
    """got is value rounded to its type, for a value within the 64-bit slack."""
    slack = o.SLACK * size + 2.0 ** -1040
    lo, hi = as_type(value - slack, kind), as_type(value + slack, kind)
    ok = (lo <= got) & (got <= hi) | (np.isnan(got) & np.isnan(value))
    assert ok.all(), (f"{what}: {int((~ok).sum())} of {ok.size} outside, first at {np.argwhere(~ok)[0].tolist()}: "
                      f"{got[~ok][0]!r} for {value[~ok][0]!r}")


class Case:
    def __init__(self, seed, M, H, post="rms", pre="rms", gate="none", weights=True, bias=False, res="f32", y="f32", z="f32",
                 g="f32", codes=True, ld=None, shift=0, res_scale=0.75, y_scale=1.5, eps=1e-5, stream=True):
        rng = np.random.default_rng(seed)
        self.M, self.H, self.post, self.pre, self.codes, self.eps = M, H, post, pre, codes, eps
        self.res_scale, self.y_scale, self.ld, self.shift, self.z, self.stream = res_scale, y_scale, ld, shift, z, stream
        self.res_type = res or "f32"
        spread = np.exp(rng.uniform(-2, 2, (M, 1)))
        self.res = rows(rng.standard_normal((M, H)) * spread, res, ld, shift)[0] if res else None
        self.y = rows((rng.standard_normal((M, H)) + 0.5) * spread[::-1], y, ld, shift)[0] if y else None
        if not y:
            self.post = post = "none"
            gate = "none"
        self.gate = None
        if gate == "channel":
            self.gate = to_dev(rng.standard_normal(H)).to(TYPES[g])
        elif gate == "row":
            self.gate = rows(rng.standard_normal((M, H)), g, ld, shift)[0]

        def vector(live):
            return rng.uniform(0.5, 1.5, H).astype(np.float32) if live else None

        self.post_w, self.post_b = vector(weights and post != "none"), vector(bias and post != "none")
        self.pre_w, self.pre_b = vector(weights and pre != "none"), vector(bias and pre != "none")
        self.vectors = {n: None if getattr(self, n) is None else to_dev(getattr(self, n))
                        for n in ("post_w", "post_b", "pre_w", "pre_b")}

    def outputs(self):
        out, flat = rows(np.zeros((self.M, self.H)), self.res_type, self.ld, self.shift) if self.stream else (None, None)
        z, zflat = rows(np.zeros((self.M, self.H)), self.z, self.ld, self.shift) if self.z else (None, None)
        qa = torch.full((self.M + 1, self.H), 99, dtype=torch.int8, device=cuda()) if self.codes else None
        sc = torch.full((self.M + 1,), -1.0, device=cuda()) if self.codes else None
        return out, flat, z, zflat, qa, sc

    def launch(self, outs):
        w4 = w4mod()
        return w4.prepare_residual_norm_quantize(self.res, self.y, outs, post=self.post, gate=self.gate, res_scale=self.res_scale,
                                                 y_scale=self.y_scale, pre=self.pre, eps=self.eps, **self.vectors)

    def call(self):
        out, flat, z, zflat, qa, sc = self.outputs()
        M = self.M
        self.launch((out, z, None if qa is None else qa[:M], None if sc is None else sc[:M]))()
        for f in (flat, zflat):
            if f is not None:
                keep = torch.ones_like(f, dtype=torch.bool)
                ld = self.ld or self.H
                keep[self.shift:self.shift + M * ld].view(M, ld)[:, :self.H] = False
                assert bool((f[keep] == SENTINEL).all()), "elements between or behind the rows were written"
        if qa is not None:
            assert bool((qa[M] == 99).all()) and float(sc[M]) == -1.0
            qa, sc = qa[:M], sc[:M]
        return out, z, qa, sc

    def check(self, what=""):
        out, z, qa, sc = self.call()
        value, size = o.joined(host64(self.res), host64(self.y), self.post, self.post_w, self.post_b, host64(self.gate),
                               self.res_scale, self.y_scale, self.eps)
        if out is not None:
            stream = host64(out)
            between(stream, value, size, self.res_type, what + " stream")
        else:
            stream = as_type(value, self.res_type)
        zv, zsize = o.norm(stream, self.pre, self.pre_w, self.pre_b, self.eps)
        if z is not None:
            between(host64(z), zv, zsize, self.z, what + " z")
        if qa is not None:
            slack = o.SLACK * zsize
            lo, hi = (zv - slack).astype(np.float32), (zv + slack).astype(np.float32)
            if z is not None and self.z == "f32":  # the codes are of the z that is returned
                lo = hi = to_host(z)
            qlo, slo = o.quantized(lo)
            qhi, shi = o.quantized(hi)
            top = np.abs(zv).max(1)
            got, gs = to_host(qa), to_host(sc)
            sure = (lo == hi).all(1)
            assert sure.mean() > 0.5 or self.M < 4 or not 64 <= self.H <= 9000  # most rows are compared exactly
            assert np.array_equal(got[sure], qlo[sure]), what + " codes"
            assert np.array_equal(gs[sure], slo[sure]), what + " scales"
            # rows with a z that the slack lets round to two fp32 values: q = rint(z / s) in fp32 has |z / s - q| <= 1/2 + 127 2^-24,
            # and s is max |z| / 127 with three roundings at most
            step = gs.astype(np.float64)[:, None]
            assert (np.abs(got * step - zv) <= step * (0.5 + 2.0 ** -17) + slack)[~sure].all(), what + " codes"
            assert (np.abs(gs - top / 127) <= 2.0 ** -22 * top / 127 + slack.max(1) + 2.0 ** -149).all(), what + " scales"


HS = [1, 2, 7, 8, 9, 63, 64, 65, 100, 128, 513, 1000, 1024, 2048, 2056, 4104, 5003, 8192, 8200, 9001, 16384, 16392, 30011, 32760, 32768]


@pytest.mark.parametrize("H", HS)
@pytest.mark.parametrize("M", [1, 5])
def test_sizes(M, H):
    Case(H + M, M, H, bias=True, gate="channel", z="f32").check(f"M={M} H={H}")
    Case(H + M, M, H, post="layer", pre="layer", res="bf16", z="f16").check(f"M={M} H={H} layer")


@pytest.mark.parametrize("z", [None, "f32", "f16", "bf16"])
@pytest.mark.parametrize("y", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("res", ["f32", "f16", "bf16"])
def test_types(res, y, z):
    for g in TYPES:
        Case(3, 7, 264, gate="row", res=res, y=y, z=z, g=g).check(g)
    Case(4, 7, 1003, gate="channel", res=res, y=y, z=z, g=y, pre="layer").check()


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("gate", ["none", "channel", "row"])
@pytest.mark.parametrize("H", [96, 2050])
def test_forms(post, pre, gate, H):
    for weights, bias in ((True, False), (False, False), (True, True), (False, True)):
        Case(H, 6, H, post, pre, gate, weights, bias, res="bf16", z="bf16").check(f"{weights} {bias}")


@pytest.mark.parametrize("H", [80, 4097])
def test_parts_left_out(H):
    for stream, z, codes in ((True, None, False), (False, "f32", False), (False, None, True), (True, "f16", False), (True, None, True),
                             (False, "bf16", True)):
        for res, y in (("f32", "f32"), ("bf16", None), (None, "f16"), ("f32", None), (None, "f32")):
            Case(H, 4, H, res=res, y=y, stream=stream, z=z, codes=codes).check(f"{stream} {z} {codes} {res} {y}")


@pytest.mark.parametrize("shift", [0, 1, 2, 3, 4, 5, 8])
def test_strides_and_alignment(shift):
    for H in (64, 75, 1032, 8200):
        for kind in TYPES:
            Case(shift, 3, H, gate="row", g=kind, res=kind, y=kind, z=kind, ld=H + shift, shift=shift).check(f"{H} {kind}")
            Case(shift, 3, H, res=kind, y="f32", z=kind, ld=H + 8 * shift, shift=0).check(f"{H} {kind}")


@pytest.mark.parametrize("M,H", [(33, 1024), (300, 512), (300, 77), (1000, 264), (2100, 2048), (70000, 24), (4100, 130)])
def test_many_rows(M, H):
    Case(M, M, H, res="bf16", y="f16", z="f32", gate="channel").check()


def test_values_at_the_ends():
    """Rows of zeros, of one value, of fp32's ends, and streams past a 16-bit type's range."""
    w4 = w4mod()
    H = 520
    x = np.zeros((6, H), np.float32)
    x[1] = 2.5
    x[2] = 3e38
    x[2, ::2] *= -1
    x[3] = 1e-42
    x[4, 17] = 1e30
    x[5] = np.linspace(-7e4, 7e4, H)
    for post in ("none", "rms", "layer"):
        c = Case(1, 6, H, post=post, pre="rms", weights=False, res=None, y="f32", z="f32", y_scale=1.0, eps=1e-12)
        c.y.copy_(to_dev(x))
        c.check(post)
    c = Case(1, 6, H, post="none", pre="none", res="f16", y="f32", z=None, codes=False, y_scale=1.0, res_scale=0.0)
    c.y.copy_(to_dev(x))
    out = to_host(c.call()[0].float())
    with np.errstate(over="ignore"):
        assert np.array_equal(out, x.astype(np.float16).astype(np.float32) + 0.0)
    zero = w4.residual_norm_quantize(torch.zeros(3, H, device=cuda()), z_dtype=torch.float32)
    assert not any(bool(t.any()) for t in zero)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite_rows_stay_alone(bad):
    c = Case(8, 9, 1031, post="rms", pre="rms", gate="row", res="f32", y="f32", z="f32")
    ref = [t.clone() for t in c.call()]
    c.y[4, 100] = bad
    got = c.call()
    keep = [m for m in range(9) if m != 4]
    for r, t in zip(ref, got):
        assert torch.equal(r[keep], t[keep])
    assert not bool(torch.isfinite(got[0][4]).all())


def test_codes_beside_the_quantizers():
    """qa and a_scale beside w4a8_quantize_act of the fp32 z, whose scale is a quotient: the scales within a step of each
    other (one rounding each, and that of 1/127: 2^-22), the codes the same but next to a border of rint."""
    w4 = w4mod()
    for H in (16, 1024, 7168, 9008):
        c = Case(H, 20, H, gate="channel", res="bf16", z="f32")
        _, z, qa, sc = c.call()
        q, s = w4.quantize_act(z.contiguous())
        assert bool(((sc - s).abs() <= 2.0 ** -22 * s).all())
        border = (z / s[:, None]).abs()
        border = (border - border.floor() - 0.5).abs() < 127 * 2.0 ** -21
        assert torch.equal(qa[~border], q[~border]) and float(border.float().mean()) < 1e-3


@pytest.mark.parametrize("H", [64, 1003, 8192])
@pytest.mark.parametrize("kind", sorted(TYPES))
def test_in_place(H, kind):
    """The stream over the residual, z over y, and the stream over y give the same bytes."""
    c = Case(H, 5, H, res=kind, y=kind, z=kind, gate="row", g=kind)
    out, z, qa, sc = [t.clone() for t in c.call()]
    keep_res, keep_y, keep_gate = c.res.clone(), c.y.clone(), c.gate.clone()
    for so, zo in ((c.res, c.y), (c.y, c.res), (c.gate, c.y), (c.res, c.gate)):
        qa2, sc2 = torch.zeros_like(qa), torch.zeros_like(sc)
        c.launch((so, zo, qa2, sc2))()
        assert torch.equal(so, out) and torch.equal(zo, z) and torch.equal(qa2, qa) and torch.equal(sc2, sc)
        c.res.copy_(keep_res)
        c.y.copy_(keep_y)
        c.gate.copy_(keep_gate)


def test_rows_do_not_depend_on_the_batch():
    c = Case(2, 700, 1032, res="bf16", y="f32", z="f32")
    whole = [t.clone() for t in c.call()]
    for m in (1, 3, 64, 300):
        d = Case(2, 700, 1032, res="bf16", y="f32", z="f32")
        d.M, d.res, d.y = m, d.res[:m], d.y[:m]
        for a, b in zip(d.call(), whole):
            assert torch.equal(a, b[:m])


def test_offsets_past_32_bits():
    """Rows whose last elements lie past 2^31."""
    M, H, ld = 40000, 64, 60000
    res = torch.zeros(M, ld, dtype=torch.bfloat16, device=cuda())
    gen = torch.Generator(device=cuda()).manual_seed(3)
    vals = torch.randn(M, H, generator=gen, device=cuda()).to(torch.bfloat16)
    res[:, :H] = vals
    view = res[:, :H]
    w4 = w4mod()
    a = w4.residual_norm_quantize(view, y=vals, post="rms", z_dtype=torch.float32, res_out=view)
    b = w4.residual_norm_quantize(vals, y=vals, post="rms", z_dtype=torch.float32)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    assert not bool(res[:, H:H + 100].any())


def test_streams_and_graphs():
    c = Case(6, 64, 4104, gate="row", res="bf16", z="bf16")
    d = Case(7, 300, 520, gate="channel", res="f32", z="f32", pre="layer")
    launches, outs = [], []
    side = [torch.cuda.Stream() for _ in (c, d)]
    for case, s in zip((c, d), side):
        out, _, z, _, qa, sc = case.outputs()
        outs.append((out, z, qa[:case.M], sc[:case.M]))
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            launches.append(case.launch(outs[-1]))
    want = [[t.clone() for t in case.call()] for case in (c, d)]
    torch.cuda.synchronize()
    for _ in range(4):
        for one in launches:
            one()
    torch.cuda.synchronize()
    for w, g in zip(want, outs):
        assert all(torch.equal(p, q) for p, q in zip(w, g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for case, o_ in zip((c, d), outs):
            case.launch(o_)()
    for _ in range(4):
        for case in (c, d):
            case.y.mul_(0.5)
            case.res.add_(1.0)
        want = [[t.clone() for t in case.call()] for case in (c, d)]
        for g in outs:
            for t in g:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for w, g in zip(want, outs):
            assert all(torch.equal(p, q) for p, q in zip(w, g))


def test_empty():
    out = w4mod().residual_norm_quantize(torch.zeros(0, 40, device=cuda()), z_dtype=torch.float16)
    assert [tuple(t.shape) for t in out] == [(0, 40), (0, 40), (0, 40), (0,)]
