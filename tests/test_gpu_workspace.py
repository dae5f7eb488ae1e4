"""A caller's workspace that is not plain memory of the device is refused before anything is launched."""
import pytest
import torch

from w8a8_quantized_linear_channel_amd import ops as q8

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def calls():
    x = torch.randn(64, 256, device=DEV, dtype=torch.bfloat16)
    w = torch.randn(128, 256, device=DEV)
    wq, ws, wz = q8.q8_quantize_weight(w)
    w8, s8, _ = q8.q8_quantize_weight(w, "fp8_e4m3")
    wb, sb = q8.q8_quantize_weight_block(w)
    yield "fp8_block", lambda t: q8.q8_linear_fp8_block(x, wb, sb, workspace=t)
    yield "linear", lambda t: q8.q8_linear(x, wq, ws, wz, workspace=t)
    yield "fp8", lambda t: q8.q8_linear_fp8(x, w8, s8, workspace=t)
    yield "decomp", lambda t: q8.q8_linear_int8_decomp(x.half(), wq, ws, wz, 6.0, workspace=t)


def test_workspaces():
    for op, call in calls():
        need = q8.q8_workspace_bytes(op, 64, 128, 256)
        assert need > 0
        with pytest.raises(TypeError):
            call(torch.empty(need, dtype=torch.uint8))
        with pytest.raises(TypeError):
            call(need)
        with pytest.raises(ValueError):
            call(torch.empty(1, dtype=torch.uint8, device=DEV).expand(need))       # one byte of memory
        with pytest.raises(ValueError):
            call(torch.empty(2 * need, dtype=torch.uint8, device=DEV)[::2])
        want = call(None)
        assert torch.equal(call(torch.empty(need, dtype=torch.uint8, device=DEV)), want)
        assert torch.equal(call(torch.empty(-(-need // 4), dtype=torch.float32, device=DEV)), want)
