"""Argument checks of the cache and block-FP8 calls, before any device work
(fake pointers, never dereferenced), and the plain forms the GPU tests use."""
import os

import numpy as np
import pytest
import torch

import kv8_plain as PL
from w8a8_quantized_linear_channel_amd import _lib as E

needs_lib = pytest.mark.skipif(not os.path.exists(E.LIB_PATH), reason="libq8.so not built")
P, MIS = 0x10000, 0x10004


def append(**kw):
    a = dict(q=P, qs=1024, k=P, ks=512, v=P, vs=512, dt=E.Q8_BF16, T=4, Hq=8, Hkv=4, D=128, cos=P, sin=P, pos=100, rot=128,
             il=0, start=P, len=P, table=P, S=2, mp=10, mq=4, kc=P, ke=P, vc=P, ve=P, np=50, page=64, out=P, st=None)
    a.update(kw)
    return E.lib().q8_kv_append(*a.values())


def attend(**kw):
    a = dict(q=P, qs=1024, dt=E.Q8_BF16, T=4, Hq=8, Hkv=4, D=128, start=P, len=P, table=P, S=2, mp=10, mq=4, mkv=640,
             kc=P, ke=P, vc=P, ve=P, np=50, page=64, scale=0.1, causal=1, window=0, out=P, lse=None, ws=P, wsn=1 << 30,
             st=None)
    a.update(kw)
    return E.lib().q8_attention_kv8(*a.values())


@needs_lib
@pytest.mark.parametrize("call", [append, attend])
def test_sizes_pointers_alignment(call):
    for kw in (dict(T=-1), dict(S=0), dict(S=40000), dict(Hkv=0), dict(D=96), dict(D=0), dict(page=16), dict(page=100),
               dict(np=0), dict(mp=0), dict(mp=1 << 31), dict(mq=-1), dict(qs=1000), dict(qs=1028), dict(Hq=0),
               dict(T=1 << 31)):
        assert call(**kw) == 2, kw
    for name in ("start", "len", "table", "kc", "ke", "vc", "ve", "q", "out"):
        assert call(**{name: None}) == 1, name
    for name in ("q", "kc", "vc", "out"):
        assert call(**{name: MIS}) == 6, name
    assert call(start=P + 1) == 6
    assert call(dt=7) == 3


@needs_lib
def test_append_arguments():
    assert append(k=None) == 1 and append(v=None) == 1 and append(cos=None) == 1 and append(sin=None) == 1
    for kw in (dict(rot=8), dict(rot=24), dict(rot=144), dict(pos=0), dict(ks=500), dict(vs=508)):
        assert append(**kw) == 2, kw
    assert append(k=MIS) == 6 and append(cos=MIS) == 6


@needs_lib
def test_attention_arguments_and_workspace():
    L = E.lib()
    assert attend(dt=E.Q8_F32) == 3
    assert attend(Hq=9) == 2 and attend(mkv=-1) == 2
    for kw in (dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1)):
        assert attend(**kw) == 5, kw
    need = L.q8_attention_workspace_bytes(2, 32, 8, 128, 2, 1, 120000, 0)
    assert need > 0
    many = dict(T=2, Hq=32, qs=4096, Hkv=8, mq=1, mkv=120000, mp=4000)
    assert attend(**many, ws=None) == 7 and attend(**many, wsn=need - 1) == 7 and attend(**many, ws=MIS) == 6
    # no split: no workspace
    assert L.q8_attention_workspace_bytes(1, 8, 8, 64, 1, 1, 128, 0) == 0
    for bad in ((-1, 8, 8, 64, 1, 1, 128, 0), (1, 9, 8, 64, 1, 1, 128, 0), (1, 8, 8, 65, 1, 1, 128, 0), (1, 8, 8, 64, 1, 1, 128, -1)):
        assert L.q8_attention_workspace_bytes(*bad) == 0


@needs_lib
def test_block_fp8_arguments():
    L = E.lib()
    f = lambda x=P, dt=E.Q8_BF16, M=20, K=256, wq=P, ws=P, N=64, b=None, y=P, yd=E.Q8_BF16, w=P, n=1 << 20: L.q8_linear_fp8_block(  # noqa: E731
        x, dt, M, K, wq, ws, N, b, y, yd, w, n, None)
    assert f(dt=9) == 3 and f(yd=E.Q8_F32) == 3
    assert f(M=-1) == 2 and f(K=24) == 2 and f(N=0) == 2 and f(K=65552) == 2
    assert f(x=None) == 1 and f(wq=None) == 1 and f(ws=None) == 1 and f(y=None) == 1
    assert f(x=MIS) == 6 and f(b=MIS) == 6 and f(w=MIS) == 6
    need = L.q8_workspace_bytes(E.Q8_OP_FP8_BLOCK, 2000, 64, 256)
    assert need >= 2000 * 256 + 2000 * 2 * 4
    assert f(M=2000, w=None) == 7 and f(M=2000, n=need - 1) == 7
    assert L.q8_quantize_act_block(None, E.Q8_BF16, 4, 128, P, P, None) == 1
    assert L.q8_quantize_act_block(P, E.Q8_BF16, 4, 100, P, P, None) == 2
    assert L.q8_quantize_weight_block(P, 5, 4, 128, P, P, None) == 3
    assert L.q8_quantize_weight_block(P, E.Q8_F32, 0, 128, P, P, None) == 2
    assert L.q8_gemm_fp8_block(P, P, 4, 128, P, P, 16, None, P, E.Q8_F32, None) == 3
    assert L.q8_gemm_fp8_block(P, None, 4, 128, P, P, 16, None, P, E.Q8_F16, None) == 1


def test_plain_codes_are_torch_codes():
    """The oracle's e4m3 rounding against torch's cast, every bf16 value up to 448."""
    x = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    x = x[torch.isfinite(x) & (x.abs() <= 448)]
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(PL.e4m3_codes(x.numpy()), want)


def test_plain_append_then_attention():
    """The cache's plain form: what was appended, in one go or token by token, is what attention reads."""
    rng = np.random.default_rng(0)
    k, v = (rng.standard_normal((50, 2, 64)).astype(np.float32) for _ in range(2))
    table = np.array([[2, 0]], np.int32)
    zero = lambda: {"k": np.zeros((3, 2, 32, 64), np.uint8), "ke": np.zeros((3, 2), np.uint8),  # noqa: E731
                    "v": np.zeros((3, 2, 64, 32), np.uint8), "ve": np.zeros((3, 2), np.uint8)}
    one, each = zero(), zero()
    PL.append(one, table, [0, 50], [50], k, v)
    for i in range(50):
        PL.append(each, table, [0, 1], [i + 1], k[i:i + 1], v[i:i + 1])
    for cache in (one, each):
        got = PL.gathered(cache, table[0], 50, "k").transpose(1, 0, 2)
        assert np.abs(got - k).max() <= 2.0 ** -4 * np.abs(k).max()
        q = rng.standard_normal((1, 4, 64))
        out, lse, _, _ = PL.attention(cache, table, [0, 1], [50], q)
        kk, vv = (PL.gathered(cache, table[0], 50, n) for n in "kv")
        s = torch.from_numpy(kk[1] @ q[0, 3] / 8)
        assert np.allclose(out[0, 3], torch.softmax(s, 0).numpy() @ vv[1])
        assert np.isclose(lse[0, 3], torch.logsumexp(s, 0).item())
