"""Caches of several layers that share memory are refused (fake pointers, never dereferenced: every call here is)."""
import os

import pytest

from test_kv8_more_abi import A, compact, fork, layers
from w8a8_quantized_linear_channel_amd import _lib as E

pytestmark = pytest.mark.skipif(not os.path.exists(E.LIB_PATH), reason="libq8.so not built")

HEADS, D, PAGES, PAGE = 4, 128, 50, 64                   # as compact() and fork() have them
CODES, EXPS = PAGES * HEADS * PAGE * D, PAGES * HEADS
NAMES = ("k", "ke", "v", "ve")
SIZE = {"k": CODES, "v": CODES, "ke": EXPS, "ve": EXPS}


def apart(n=3):
    """Pointers of n layers, each array behind the one before it."""
    at, out = A + (1 << 24), {}
    for name in NAMES:
        out[name] = []
        for _ in range(n):
            out[name].append(at)
            at += -(-SIZE[name] // 16) * 16
    return out


def call(f, p):
    return f(n=len(p["k"]), **{name: layers(*p[name]) for name in NAMES})


@pytest.mark.parametrize("f", [compact, fork])
def test_memory_of_two_arrays(f):
    for name in NAMES:
        for other in NAMES:
            for i, j in ((0, 1), (1, 2), (0, 2), (2, 0), (1, 1)):
                if (name, i) == (other, j):
                    continue
                for off in (0, SIZE[other] - 16, 16 - SIZE[name]):
                    p = apart()
                    p[name][i] = p[other][j] + off // 16 * 16      # the same, or the ends in each other
                    assert call(f, p) == E.Q8_ERR_BAD_ARG, (name, i, other, j, off)


@pytest.mark.parametrize("f", [compact, fork])
def test_one_layer_whose_values_are_its_keys(f):
    p = apart(1)
    p["v"] = p["k"]
    assert call(f, p) == E.Q8_ERR_BAD_ARG
    p = apart(1)
    p["ve"] = p["ke"]
    assert call(f, p) == E.Q8_ERR_BAD_ARG


@pytest.mark.parametrize("f", [compact, fork])
def test_many_layers(f):
    for i, j in ((0, 511), (3, 4), (100, 64)):
        p = apart(512)
        p["ve"][i] = p["ve"][j] + EXPS - 1
        assert call(f, p) == E.Q8_ERR_BAD_ARG


def test_memory_of_tables_and_caches():
    """Arrays that a call reads or writes in the memory of a cache."""
    base = apart(2)
    for f, arrays in ((compact, ("start", "len", "table", "keep", "kept", "out")),
                      (fork, ("table", "len", "refs", "parent", "tout", "lout", "rout", "missing", "ws"))):
        for name in arrays:
            for cache, end in (("k", CODES - 16), ("ve", EXPS // 16 * 16 - 16)):
                kw = {n: layers(*base[n]) for n in NAMES}
                assert f(**kw, **{name: base[cache][1] + end}) == E.Q8_ERR_BAD_ARG, (f.__name__, name, cache)
