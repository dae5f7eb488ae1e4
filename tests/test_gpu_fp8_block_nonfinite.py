"""NaN and infinities into the block-scaled FP8 linear: what they touch is not finite, the rest as without them."""
import pytest
import torch

from test_gpu_fp8_block import BF, DEV, F32, HF, inputs
from w8a8_quantized_linear_channel_amd import ops as q8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 4, 5, 40, 300])
@pytest.mark.parametrize("K", [128, 400, 1040])
@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("value", [float("nan"), -float("nan"), float("inf"), -float("inf")])
def test_activations(M, K, dt, value):
    N = 200
    x, w, _ = inputs(M + K, M, N, K, dt)
    x, w = x.to(DEV), w.to(DEV)
    wq, ws = q8.q8_quantize_weight_block(w)
    clean_q, clean_s = q8.q8_quantize_act_block(x)
    clean = q8.q8_linear_fp8_block(x, wq, ws)
    for row, at in {(0, 0), (M - 1, K - 1), (M // 2, K // 2)}:
        bad = x.clone()
        bad[row, at] = value
        xq, xs = q8.q8_quantize_act_block(bad)
        assert not xs[at // 128, row].isfinite() and xs[at // 128, row].isnan() == bad[row, at].isnan()
        keep = torch.ones_like(clean_s, dtype=torch.bool)
        keep[at // 128, row] = False
        assert torch.equal(xs[keep], clean_s[keep])
        codes = keep.t().repeat_interleave(128, 1)[:, :K]
        assert torch.equal(xq[codes], clean_q[codes])
        rows = [m for m in range(M) if m != row]
        for y in (q8.q8_linear_fp8_block(bad, wq, ws), q8.q8_gemm_fp8_block(xq, xs, wq, ws, out_dtype=clean.dtype)):
            assert not y[row].isfinite().any()
            if value != value:
                assert y[row].isnan().all()
            if y.shape == clean.shape and M > 4:
                assert torch.equal(y[rows], clean[rows])
        assert torch.equal(q8.q8_linear_fp8_block(bad, wq, ws)[rows], clean[rows])


@pytest.mark.parametrize("value", [float("nan"), -float("inf")])
def test_weights(value):
    x, w, _ = inputs(7, 20, 300, 400, BF)
    x, w = x.to(DEV), w.to(DEV)
    wq, ws = q8.q8_quantize_weight_block(w)
    clean = q8.q8_linear_fp8_block(x, wq, ws)
    w[130, 399] = value
    bq, bs = q8.q8_quantize_weight_block(w)
    assert not bs[1, 3].isfinite()
    keep = torch.ones_like(ws, dtype=torch.bool)
    keep[1, 3] = False
    assert torch.equal(bs[keep], ws[keep])
    y = q8.q8_linear_fp8_block(x, bq, bs)
    assert not y[:, 130].isfinite().any() and not y[:, 128:256].isfinite().any()
    assert torch.equal(y[:, :128], clean[:, :128]) and torch.equal(y[:, 256:], clean[:, 256:])
