"""Argument checks of the calls for drafted tokens and branching sequences, before
any device work (fake pointers, never dereferenced), and their plain forms."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import kv8_more_plain as M
import kv8_plain as P
from w8a8_quantized_linear_channel_amd import _lib as E

needs_lib = pytest.mark.skipif(not os.path.exists(E.LIB_PATH), reason="libq8.so not built")
A, MIS = 0x10000, 0x10004


def append(**kw):
    a = dict(q=A, qs=1024, k=A, ks=512, v=A, vs=512, dt=E.Q8_BF16, T=4, Hq=8, Hkv=4, D=128, qw=A, kw=A, wdt=E.Q8_BF16,
             eps=1e-6, cos=A, sin=A, pos=100, rot=128, il=0, tp=A, start=A, len=A, table=A, S=2, mp=10, mq=4, kc=A, ke=A,
             vc=A, ve=A, np=50, page=64, out=A, st=None)
    a.update(kw)
    return E.lib().q8_kv_append_norm(*a.values())


def attend(**kw):
    a = dict(q=A, qs=1024, dt=E.Q8_BF16, T=4, Hq=8, Hkv=4, D=128, start=A, len=A, table=A, S=2, mp=10, mq=4, mkv=640,
             kc=A, ke=A, vc=A, ve=A, np=50, page=64, mask=A, words=1, tp=A, scale=0.1, window=0, out=A, lse=None, ws=A,
             wsn=1 << 30, st=None)
    a.update(kw)
    return E.lib().q8_attention_kv8_tree(*a.values())


def layers(*pointers):
    return (ctypes.c_void_p * len(pointers))(*pointers)


def compact(n=2, **kw):
    a = dict(k=layers(A, A + 4096), ke=layers(A, A), v=layers(A, A), ve=layers(A, A), layers=n, Hkv=4, D=128, start=A,
             len=A + 512, table=A + 1024, S=2, mp=10, np=50, page=64, keep=A + 2048, width=5, kept=A + 2560, out=A + 4096,
             st=None)
    a.update(kw)
    return E.lib().q8_kv_compact(*a.values())


def fork(n=2, **kw):
    a = dict(k=layers(A, A + 4096), ke=layers(A, A), v=layers(A, A), ve=layers(A, A), layers=n, Hkv=4, D=128, np=50, page=64,
             table=A, len=A + 512, refs=A + 1024, S=2, mp=10, parent=A + 2048, outs=3, room=1, tout=A + 4096, lout=A + 8192,
             rout=A + 12288, missing=A + 16384, ws=A + 65536, wsn=1 << 20, st=None)
    a.update(kw)
    return E.lib().q8_kv_fork(*a.values())


@needs_lib
@pytest.mark.parametrize("call", [append, attend])
def test_token_calls(call):
    for kw in (dict(T=-1), dict(S=0), dict(S=40000), dict(Hkv=0), dict(D=96), dict(page=16), dict(np=0), dict(mp=0),
               dict(mp=1 << 31), dict(mq=-1), dict(qs=1000), dict(Hq=0), dict(T=1 << 31)):
        assert call(**kw) == 2, kw
    for name in ("start", "len", "table", "kc", "ke", "vc", "ve", "q", "out"):
        assert call(**{name: None}) == 1, name
    for name in ("q", "kc", "vc", "out"):
        assert call(**{name: MIS}) == 6, name
    assert call(start=A + 1) == 6 and call(tp=A + 2) == 6
    assert call(dt=7) == 3


@needs_lib
def test_append_norm_arguments():
    assert append(k=None) == 1 and append(v=None) == 1 and append(cos=None) == 1
    for kw in (dict(rot=8), dict(rot=144), dict(pos=0), dict(ks=500), dict(vs=508)):
        assert append(**kw) == 2, kw
    assert append(wdt=5) == 3
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert append(eps=eps) == 5, eps
        assert append(eps=eps, qw=None) == 5
    assert append(qw=MIS) == 6 and append(kw=MIS) == 6


@needs_lib
def test_tree_arguments_and_workspace():
    assert attend(dt=E.Q8_F32) == 3
    for kw in (dict(Hq=9), dict(mkv=-1), dict(words=0), dict(words=32769), dict(words=-1)):
        assert attend(**kw) == 2, kw
    for kw in (dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1)):
        assert attend(**kw) == 5, kw
    assert attend(mask=None) == 1 and attend(mask=MIS) == 6
    many = dict(T=40, Hq=32, qs=4096, Hkv=8, mq=20, mkv=120000, mp=4000)
    need = E.lib().q8_attention_tree_workspace_bytes(40, 32, 8, 128, 2, 20, 120000, 0)
    assert need > 0
    assert E.lib().q8_attention_tree_workspace_bytes(40, 31, 8, 128, 2, 20, 120000, 0) == 0
    assert attend(**many, ws=None) == 7 and attend(**many, wsn=need - 1) == 7 and attend(**many, ws=MIS) == 6


@needs_lib
def test_layers_arguments():
    for call in (compact, fork):
        for kw in (dict(n=0), dict(n=513), dict(Hkv=0), dict(D=100), dict(S=0), dict(S=40000), dict(mp=0), dict(np=0), dict(page=48)):
            assert call(**kw) == 2, kw
        for name in ("k", "ke", "v", "ve", "table", "len"):
            assert call(**{name: None}) == 1, name
        assert call(v=layers(A, None)) == 1 and call(ke=layers(None, A)) == 1
        assert call(k=layers(A, MIS)) == 6 and call(v=layers(MIS, A)) == 6
        assert call(k=layers(A, A)) == 5                  # a layer twice
        assert call(len=A + 2) == 6
    assert compact(start=None) == 1 and compact(keep=None) == 1 and compact(kept=None) == 1 and compact(out=None) == 1
    assert compact(width=-1) == 2 and compact(keep=A + 2050) == 6 and compact(out=A + 4098) == 6
    for same in (A, A + 8, A + 508, A + 512, A + 1024 + 76, A + 2048 + 36, A + 2564):      # the outputs over an input
        assert compact(out=same) == 5, hex(same)


@needs_lib
def test_fork_arguments():
    for name in ("refs", "parent", "tout", "lout", "rout", "missing"):
        assert fork(**{name: None}) == 1, name
        assert fork(**{name: A + 20002}) == 6, name
    for kw in (dict(outs=0), dict(outs=40000), dict(room=-1), dict(room=(1 << 30) + 1)):
        assert fork(**kw) == 2, kw
    need = E.lib().q8_kv_fork_workspace_bytes(2, 3, 50)
    assert need > 0 and fork(ws=None) == 7 and fork(wsn=need - 1) == 7 and fork(ws=A + 65540) == 6
    for kw in (dict(tout=A), dict(lout=A + 512), dict(rout=A + 1024), dict(missing=A + 2056), dict(lout=A + 4100),
               dict(rout=A + 8196), dict(missing=A + 12288), dict(ws=A), dict(tout=A + 65536)):
        assert fork(**kw) == 5, kw
    for bad in ((0, 3, 50), (2, 0, 50), (2, 3, 0), (40000, 3, 50), (2, 40000, 50)):
        assert E.lib().q8_kv_fork_workspace_bytes(*bad) == 0


def test_plain_norm_and_tree():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 64)).astype(np.float32)
    y = M.normalised(x, np.ones(64, np.float32), 1e-6)
    assert np.allclose(np.square(y).mean(2), 1.0, atol=1e-5)
    up, sees = M.tree_of(rng, 80)
    assert (sees.sum(1) >= 1).all() and all(sees[i, u] for i, u in enumerate(up) if u >= 0)
    w = M.words_of(sees, 2)
    assert all(((int(w[i, j // 64]) >> (j % 64)) & 1) == sees[i, j] for i in range(80) for j in range(80))
    # a chain is causal attention
    table = np.array([[1, 0, 2]], np.int32)
    cache = {"k": P.e4m3_codes(rng.standard_normal((3, 2, 32, 64)) * 60), "ke": np.full((3, 2), 120, np.uint8),
             "v": P.e4m3_codes(rng.standard_normal((3, 2, 64, 32)) * 60), "ve": np.full((3, 2), 120, np.uint8)}
    q = rng.standard_normal((9, 4, 64))
    chain = [np.tril(np.ones((9, 9), bool))]
    for window in (0, 20):
        a = P.attention(cache, table, [0, 9], [70], q, None, True, window)
        b = M.tree_attention(cache, table, [0, 9], [70], q, chain, None, None, window)
        assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])


def test_plain_compact_and_fork():
    rng = np.random.default_rng(1)
    # all kept in place: nothing changes; the same values appended afresh: compact gives the append's codes
    table = np.array([[2, 0, 1]], np.int32)
    zero = lambda: {"k": np.zeros((3, 1, 32, 64), np.uint8), "ke": np.zeros((3, 1), np.uint8),  # noqa: E731
                    "v": np.zeros((3, 1, 64, 32), np.uint8), "ve": np.zeros((3, 1), np.uint8)}
    cache = zero()
    x = rng.standard_normal((80, 1, 64)).astype(np.float32)
    P.append(cache, table, [0, 80], [80], x, x)
    was = {n: a.copy() for n, a in cache.items()}
    assert M.compact(cache, table, [0, 20], [80], np.array([[0, 1, 2]]), [3]).tolist() == [63]
    assert all(np.array_equal(cache[n], was[n]) for n in cache)
    keep = [1, 4, 7, 9, 12, 19]
    k, v = (P.gathered(cache, table[0], 80, n)[0] for n in "kv")
    assert M.compact(cache, table, [0, 20], [80], np.array([keep]), [6]).tolist() == [66]
    ref = {n: a.copy() for n, a in was.items()}
    rows = lambda a: a[[60 + u for u in keep]][:, None].astype(np.float32)  # noqa: E731
    P.append(ref, table, [0, 6], [66], rows(k), rows(v))
    assert all(np.array_equal(cache[n], ref[n]) for n in cache)
    assert M.path([0, 2, 2, 5], 9) == [0, 2] and M.path([1, 2, 9], 9) == [1, 2] and M.path([0, 0], 9) == [0]
    # forks: counts are what the tables hold, new pages hold what their parents' did
    pages = 12
    cache = {"k": rng.integers(0, 127, (pages, 2, 32, 64)).astype(np.uint8), "ke": rng.integers(0, 255, (pages, 2)).astype(np.uint8),
             "v": rng.integers(0, 127, (pages, 2, 64, 32)).astype(np.uint8), "ve": rng.integers(0, 255, (pages, 2)).astype(np.uint8)}
    table = np.array([[5, 3, -1], [7, -1, -1]], np.int32)
    refs = np.zeros(pages, np.int32)
    refs[[5, 3, 7]] = 1
    out, lens, count, missing = M.fork([cache], table, [40, 32], refs, [0, 0, 1, -1, 0], 1)
    assert lens.tolist() == [40, 40, 32, 0, 40] and missing == 0
    assert out.tolist() == [[5, 3, -1], [5, 0, -1], [7, 1, -1], [-1, -1, -1], [5, 2, -1]]
    assert count.tolist() == [1, 1, 1, 1, 0, 3, 0, 1, 0, 0, 0, 0]
    assert all(np.array_equal(cache[n][0], cache[n][3]) and np.array_equal(cache[n][2], cache[n][3]) for n in cache)


def test_every_launch_is_within_its_limits(tmp_path):
    here = os.path.dirname(os.path.abspath(__file__))
    csrc = os.path.join(os.path.dirname(here), "w8a8_quantized_linear_channel_amd", "csrc")
    exe = str(tmp_path / "tree_plan_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", f"-I{csrc}",
                    os.path.join(here, "native", "tree_plan_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


@needs_lib
def test_rows_past_32_bits_are_refused():
    for T, Hq, want in ((1 << 26, 32, 2), (1 << 30, 2, 2), ((1 << 26) - 64, 32, 5)):
        assert attend(T=T, Hq=Hq, Hkv=1, D=64, qs=Hq * 64, window=-1) == want, (T, Hq)
        assert (E.lib().q8_attention_tree_workspace_bytes(T, Hq, 1, 64, 1, 1, 100000, 0) == 0) == (want == 2)
