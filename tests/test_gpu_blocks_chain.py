"""A run of the operators as a served block uses them: norm and codes, the shared 4-bit projection, the requests' adapters on
its output, and the join with the stream, stage by stage against the 64-bit forms; then the run captured into a graph."""
from __future__ import annotations

import numpy as np
import pytest

import synthetic
from tests import blocks_oracle as o
from tests.gpu_common import check_close, cuda, device_layer, oracle_columns, to_dev, to_host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def host64(t):
    return to_host(t.double())


class Block:
    """x -> norm -> codes -> W x + adapters -> stream of H; a square projection, so that blocks can follow each other."""

    def __init__(self, M, H, L, R, seed=3):
        import w4a8_quantized_gemm_token_amd as w4
        rng = np.random.default_rng(seed)
        dev = cuda()
        self.M, self.H, self.seed = M, H, seed
        self.stream = to_dev(rng.standard_normal((M, H)).astype(np.float32)).to(torch.bfloat16)
        self.w_pre = to_dev(rng.uniform(0.5, 1.5, H).astype(np.float32))
        self.w_post = to_dev(rng.uniform(0.5, 1.5, H).astype(np.float32))
        self.gate = to_dev(rng.uniform(0.1, 0.5, H).astype(np.float32))
        self.layer = device_layer(seed, synthetic.TAG_W, 0, H, H)
        self.ids = rng.integers(-1, L, M).astype(np.int32)
        self.A = to_dev((rng.standard_normal((L, R, H)) / np.sqrt(H)).astype(np.float32)).to(torch.bfloat16)
        self.B = to_dev((0.3 * rng.standard_normal((L, H, R))).astype(np.float32)).to(torch.bfloat16)
        self.scale = rng.uniform(0.5, 2, L).astype(np.float32)
        e = lambda *shape, t=torch.float32: torch.zeros(*shape, dtype=t, device=dev)  # noqa: E731
        self.z, self.qa, self.sa = e(M, H, t=torch.bfloat16), e(M, H, t=torch.int8), e(M)
        self.out, self.raw = e(M, H), e(M, H)
        self.joined = e(M, H, t=torch.bfloat16)
        self.z2, self.qa2, self.sa2 = e(M, H, t=torch.float32), e(M, H, t=torch.int8), e(M)
        self.space = torch.empty(w4.lora_workspace(M, H, L, R), dtype=torch.uint8, device=dev)
        self.ids_dev, self.scale_dev = to_dev(self.ids), to_dev(self.scale)

    def run(self):
        import w4a8_quantized_gemm_token_amd as w4
        w4.prepare_residual_norm_quantize(self.stream, None, (None, self.z, self.qa, self.sa), pre_w=self.w_pre)()
        w4.gemm(self.qa, self.sa, *self.layer, out=self.out)
        self.raw.copy_(self.out)
        w4.lora_add(self.out, self.z, self.ids_dev, self.A, self.B, workspace=self.space, scale=self.scale_dev)
        w4.prepare_residual_norm_quantize(self.stream, self.out, (self.joined, self.z2, self.qa2, self.sa2), post="rms",
                                          post_w=self.w_post, gate=self.gate, pre="layer", pre_w=self.w_pre)()

    def outputs(self):
        return (self.z, self.qa, self.sa, self.out, self.joined, self.z2, self.qa2, self.sa2)


@pytest.mark.parametrize("M", [1, 20, 150])
def test_block_stage_by_stage(orc, M):
    H, L, R = 512, 6, 16
    b = Block(M, H, L, R)
    b.run()
    torch.cuda.synchronize()
    # the first norm: codes of the fp32 z
    z, size = o.norm(host64(b.stream), "rms", to_host(b.w_pre), None, 1e-6)
    lo, hi = (z - o.SLACK * size).astype(np.float32), (z + o.SLACK * size).astype(np.float32)
    sure = (lo == hi).all(1)
    q, s = o.quantized(lo)
    assert sure.any() and np.array_equal(to_host(b.qa)[sure], q[sure]) and np.array_equal(to_host(b.sa)[sure], s[sure])
    assert (np.abs(host64(b.z) - z) <= 2.0 ** -8 * np.abs(z) * 1.001).all()
    # the shared projection, of the codes the kernel made
    codes, scale, zp = oracle_columns(orc, b.seed, synthetic.TAG_W, 0, H, np.arange(H))
    ref, mag = orc.gemm(to_host(b.qa), to_host(b.sa), codes, scale, zp)
    check_close(to_host(b.raw), ref, mag)
    # the adapters on its output
    value, bound = o.lora(host64(b.z), b.ids, host64(b.A), host64(b.B), None, b.scale, host64(b.raw), "f32", True)
    o.close(host64(b.out), value, bound, "f32")
    # the join and the next norm
    value, size = o.joined(host64(b.stream), host64(b.out), "rms", to_host(b.w_post), None, host64(b.gate), 1.0, 1.0, 1e-6)
    assert (np.abs(host64(b.joined) - value) <= 2.0 ** -8 * np.abs(value) * 1.001 + o.SLACK * size).all()
    z2, size = o.norm(host64(b.joined), "layer", to_host(b.w_pre), None, 1e-6)
    assert (np.abs(host64(b.z2) - z2) <= 2.0 ** -24 * np.abs(z2) * 1.001 + o.SLACK * size + 2.0 ** -149).all()
    q, s = o.quantized(to_host(b.z2))
    assert np.array_equal(to_host(b.qa2), q) and np.array_equal(to_host(b.sa2), s)


def test_block_in_a_graph():
    b = Block(70, 512, 6, 16)
    b.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    for turn in range(4):
        b.stream.add_(0.25)
        b.ids_dev.copy_(torch.roll(b.ids_dev, 1))
        b.run()
        torch.cuda.synchronize()
        want = [t.clone() for t in b.outputs()]
        for t in b.outputs():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(b.outputs(), want)), turn
