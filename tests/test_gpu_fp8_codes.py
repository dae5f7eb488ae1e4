"""e4m3 codes as float8_e4m3fn tensors, as FP8 checkpoints hold them."""
import pytest
import torch

from test_gpu_fp8_block import BF, DEV, inputs
from w8a8_quantized_linear_channel_amd import ops as q8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 20, 200])
def test_float8_codes(M):
    x, w, bias = inputs(M, M, 300, 400, BF)
    x, w, b = x.to(DEV), w.to(DEV), torch.from_numpy(bias).to(DEV)
    wq, ws = q8.q8_quantize_weight_block(w)
    w8 = wq.view(torch.float8_e4m3fn)
    want = q8.q8_linear_fp8_block(x, wq, ws, bias=b)
    assert torch.equal(q8.q8_linear_fp8_block(x, w8, ws, bias=b), want)
    assert isinstance(q8._fast().linear_fp8_block(x, w8, ws, b, None, None), torch.Tensor)
    need = q8.q8_workspace_bytes("fp8_block", M, 300, 400)
    assert torch.equal(q8.q8_linear_fp8_block(x, w8, ws, bias=b, workspace=torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)), want)
    xq, xs = q8.q8_quantize_act_block(x)
    want = q8.q8_gemm_fp8_block(xq, xs, wq, ws)
    assert torch.equal(q8.q8_gemm_fp8_block(xq.view(torch.float8_e4m3fn), xs, w8, ws), want)
    for bad in (wq.view(torch.int8), wq.view(torch.float8_e5m2)):
        with pytest.raises(TypeError):
            q8.q8_linear_fp8_block(x, bad, ws)
        with pytest.raises(TypeError):
            q8.q8_gemm_fp8_block(xq, xs, bad, ws)
