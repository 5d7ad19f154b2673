"""Argument checks of the adapters' and the norms' binding that need no device: a clear refusal, not an error of Python's own."""
import pytest

import w4a8_quantized_gemm_token_amd as w4

torch = pytest.importorskip("torch")


def test_prepared_adapters_need_a_workspace():
    z = torch.zeros
    A, B = z(3, 8, 16, dtype=torch.bfloat16), z(3, 9, 8, dtype=torch.bfloat16)
    with pytest.raises(AssertionError, match="workspace"):
        w4.prepare_lora_add(z(2, 9), z(2, 16), z(2, dtype=torch.int32), A, B, None)


def test_norms_need_an_input():
    outs = (torch.zeros(2, 16), None, None, None)
    with pytest.raises(AssertionError, match="res or y"):
        w4.prepare_residual_norm_quantize(None, None, outs)
    with pytest.raises(AssertionError, match="res or y"):
        w4.residual_norm_quantize(None)
