"""q8_kv_compact and q8_kv_fork against their definitions, byte for byte."""
import numpy as np
import pytest
import torch

import kv8_more_plain as M
from test_gpu_kv8 import DEV, batch_of, device, host, random_cache, table_of
from test_gpu_kv8_drafts import interpreted, up
from w8a8_quantized_linear_channel_amd import _lib
from w8a8_quantized_linear_channel_amd import ops as q8

pytestmark = pytest.mark.gpu


def same(got, want, what=""):
    for i, (g, w) in enumerate(zip(got, want)):
        g = host(g)
        for name in ("ke", "ve", "k", "v"):
            bad = np.argwhere(g[name] != w[name])
            assert len(bad) == 0, (what, i, name, len(bad), bad[:3])


# ---------------------------------------------------------------- compact
def run_compact(rng, news, lens, Hk, D, page, keeps, layers=1, width=None, spread=6, table=None, pages=None, caches=None, n_keep=None):
    if table is None:
        table, pages = table_of(rng, [max(n, 1) for n in lens], page)
    if caches is None:
        caches = [random_cache(rng, pages, Hk, page, D, spread) for _ in range(layers)]
    width = max([len(k) for k in keeps] + [1]) if width is None else width
    keep = np.full((len(keeps), width), -1, np.int32)
    for s, k in enumerate(keeps):
        keep[s, :len(k)] = k
    n_keep = np.array([len(k) for k in keeps] if n_keep is None else n_keep, np.int32)
    start, batch = batch_of(news, lens, table)
    got = [device(c) for c in caches]
    out = q8.q8_kv_compact(got if len(got) > 1 else got[0], batch, up(keep), up(n_keep))
    want = [M.compact(c, table, start, lens, keep, n_keep) for c in caches]
    assert np.array_equal(out.cpu().numpy(), want[0])
    same(got, caches)


def some_path(rng, n, share):
    return np.flatnonzero(rng.random(n) < share).tolist()


@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_compact_shapes(page, D):
    rng = np.random.default_rng(page + D)
    news, lens = [12, 1, 40, 0, 9, 2 * page + 7], [70, 33, 45, 20, page + 4, 3 * page + 1]
    for share in (0.1, 0.4, 0.9):
        run_compact(rng, news, lens, 2, D, page, [some_path(rng, n, share) for n in news], layers=2)


def test_compact_places():
    """Every first token and every place of the drafts in a page; nothing kept, all kept, only the last."""
    rng = np.random.default_rng(3)
    for past in range(0, 34):
        run_compact(rng, [5, 40, 4], [past + 5, past + 40, past + 4], 1, 64, 32,
                    [[past % 5], some_path(rng, 40, 0.3), [[], [0, 1, 2, 3], [3], [0, 2]][past % 4]])


def test_compact_long_paths():
    rng = np.random.default_rng(4)
    for page in (32, 128):
        run_compact(rng, [300, 150], [333, 151], 1, 64, page, [some_path(rng, 300, 0.7), list(range(1, 150))])
        run_compact(rng, [400], [413], 1, 128, page, [list(range(0, 100)) + list(range(130, 400, 3))])


def test_compact_lists_that_are_none():
    rng = np.random.default_rng(5)
    lists = [[3, 2, 5], [-1, 4], [2, 2, 3], [0, 9, 12], [1, 5, 20, 21], [0, 0], [4, 6]]
    for n in ([9] * 7, [2] * 7, [22] * 7):
        run_compact(rng, n, [50 + x for x in n], 1, 64, 32, lists)
    # counts that are not the lists' lengths, below zero, beyond the width; a width of none
    run_compact(rng, [9, 9, 9], [60, 61, 62], 1, 64, 32, [[1, 3, 5], [2, 4, 5], [0, 2, 7]], n_keep=[2, -5, 99])
    run_compact(rng, [9, 9], [60, 61], 1, 64, 32, [[], []], width=0)
    run_compact(rng, [9, 9], [60, 61], 1, 64, 32, [[], []], width=0, n_keep=[3, 3])


def test_compact_slots_and_pages_that_are_not_there():
    rng = np.random.default_rng(6)
    # more drafts than tokens, a sequence past its table, lengths of zero
    run_compact(rng, [9, 6, 3], [4, 70, 0], 1, 64, 32, [[1, 6, 7, 8], [1, 3, 5], [1, 2]])
    table = np.array([[0, 99, 2], [-1, 3, -7], [4, 5, 6]], np.int32)
    news, lens = [50, 40, 30], [90, 60, 130]
    run_compact(rng, news, lens, 1, 64, 32, [some_path(rng, n, 0.5) for n in news], table=table, pages=8)


def test_compact_codes_and_scales():
    """NaN codes, zeros, subnormal codes, exponent bytes at their ends."""
    rng = np.random.default_rng(7)
    for lo, hi in ((0, 3), (0, 255), (250, 255), (100, 140)):
        table, pages = table_of(rng, [100, 70], 32)
        c = random_cache(rng, pages, 2, 32, 64)
        c["k"], c["v"] = (rng.integers(0, 256, c[n].shape).astype(np.uint8) for n in "kv")
        c["k"][rng.random(c["k"].shape) < 0.3] = 0
        c["ke"], c["ve"] = (rng.integers(lo, hi, c["ke"].shape).astype(np.uint8) for _ in range(2))
        c["v"][table[0, 2]] &= 0x87                       # subnormals and zeros only
        run_compact(rng, [60, 50], [100, 70], 2, 64, 32, [some_path(rng, 60, 0.4), some_path(rng, 50, 0.5)], caches=[c], table=table)


def test_compact_many_layers_and_sequences():
    rng = np.random.default_rng(8)
    run_compact(rng, [5, 9], [40, 70], 1, 64, 32, [[1, 4], [2, 5, 8]], layers=65)
    news = [int(rng.integers(1, 12)) for _ in range(200)]
    run_compact(rng, news, [n + int(rng.integers(0, 60)) for n in news], 3, 64, 32, [some_path(rng, n, 0.5) for n in news])


# ---------------------------------------------------------------- fork
def tables_in_use(rng, S, width, page, pages, shared=0.2, reserve=1):
    """Tables, lengths and counts of a batch, some full pages shared, some rows with pages for later tokens."""
    order, at = rng.permutation(pages), 0
    table, lens = np.full((S, width), -1, np.int32), np.zeros(S, np.int32)
    for s in range(S):
        lens[s] = rng.integers(0, (width - reserve) * page + 1)
        need = min(width, -(-int(lens[s]) // page) + int(rng.integers(0, reserve + 1)))
        for j in range(need):
            up_to = [int(table[p, j]) for p in range(s) if lens[p] // page > j]
            if j < lens[s] // page and up_to and rng.random() < shared:
                table[s, j] = up_to[int(rng.integers(len(up_to)))]
            else:
                table[s, j] = order[at]
                at += 1
    refs = np.bincount(table[table >= 0], minlength=pages).astype(np.int32)
    return table, lens, refs


def run_fork(rng, table, lens, refs, parent, room, Hk=1, D=64, page=32, layers=1, caches=None):
    caches = [random_cache(rng, len(refs), Hk, page, D) for _ in range(layers)] if caches is None else caches
    got = [device(c) for c in caches]
    f = q8.q8_kv_fork(got if len(got) > 1 else got[0], up(table), up(lens), up(refs), up(np.array(parent, np.int32)), room=room)
    out, length, count, missing = M.fork(caches, table, lens, refs, parent, room)
    assert np.array_equal(f.block_table.cpu().numpy(), out)
    assert np.array_equal(f.kv_len.cpu().numpy(), length)
    assert np.array_equal(f.refs.cpu().numpy(), count)
    assert f.missing.item() == missing
    same(got, caches)
    return out, length, count, missing


@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("D,Hk", [(64, 1), (128, 3), (256, 2)])
def test_fork_shapes(page, D, Hk):
    rng = np.random.default_rng(page + D)
    for S, outs, room in ((1, 1, 0), (1, 9, 1), (5, 5, 1), (7, 3, 40), (4, 20, 300)):
        table, lens, refs = tables_in_use(rng, S, 6, page, 200)
        run_fork(rng, table, lens, refs, rng.integers(-1, S, outs).tolist(), room, Hk, D, page, layers=2)


def test_fork_free_pages_run_out():
    rng = np.random.default_rng(2)
    for pages in (12, 14, 16, 18, 30):
        for room in (0, 1, 33, 200):
            table, lens, refs = tables_in_use(rng, 3, 4, 32, pages)
            run_fork(rng, table, lens, refs, rng.integers(0, 3, 8).tolist(), room)
    # a full batch that goes on as it is, one that is let go, one whose freed pages serve the others
    table, lens, refs = tables_in_use(rng, 3, 4, 32, 12, shared=0)
    run_fork(rng, table, lens, refs, [0, 1, 2], 0)
    out = run_fork(rng, table, lens, refs, [-1, 99, -7], 50)
    assert (out[2] == 0).all() and (out[0] == -1).all()
    run_fork(rng, table, lens, refs, [1, 1, 1, 1], 20)


def test_fork_tables_that_are_not_in_order():
    rng = np.random.default_rng(3)
    pages = 20
    # entries outside, holes, an open page that two rows hold (copied for both), counts that others hold too
    table = np.array([[3, 99, -5, 7], [4, 5, 5, -1], [6, 8, -1, -1], [9, 8, -1, -1]], np.int32)
    lens = np.array([100, 70, 40, 45], np.int32)
    refs = np.bincount(table[(table >= 0) & (table < pages)], minlength=pages).astype(np.int32)
    for parent in ([0, 0, 1, 2, 3], [2, 3, 2, 3], [1, 0], [3, 2, 1, 0]):
        for extra in (0, 1):
            r = refs.copy()
            r[[3, 8]] += extra
            run_fork(rng, table, lens, r, parent, 20)
    # lengths below zero and past the table
    run_fork(rng, table, np.array([-4, 1000, 0, 128], np.int32), refs, [0, 1, 2, 3, 1, 3], 1)


def test_fork_many():
    """More sequences than threads, more pages than a pass looks at, wide rows, more layers than a launch."""
    rng = np.random.default_rng(4)
    table, lens, refs = tables_in_use(rng, 1500, 2, 32, 6000, shared=0)
    run_fork(rng, table, lens, refs, rng.integers(-1, 1500, 2500).tolist(), 20, D=64)
    table, lens, refs = tables_in_use(rng, 3, 150, 32, 700)
    run_fork(rng, table, lens, refs, [2, 2, 1, 0, 2], 700)
    table, lens, refs = tables_in_use(rng, 3, 3, 32, 30)
    run_fork(rng, table, lens, refs, [2, 2, 1], 1, layers=65)


def test_fork_steps_keep_the_books():
    """Beams that grow by a token a step: after each the counts are what the table holds, and codes are the parents'."""
    rng = np.random.default_rng(5)
    page, pages, S = 32, 60, 4
    cache = device(random_cache(rng, pages, 1, page, 64))
    table = np.full((S, 8), -1, np.int32)
    table[0, 0] = 11
    refs = np.zeros(pages, np.int32)
    refs[11] = 1
    text = [[]] * S                                       # the first feature's codes of every sequence
    text[0] = [7] * 20
    cache.k[11, 0, :20, 0] = 7
    f = q8.KvFork(up(table), up(np.array([20, 0, 0, 0], np.int32)), up(refs), None)
    for step in range(80):
        parent = [0] * S if step == 0 else rng.integers(0, S, S).tolist()
        f = q8.q8_kv_fork(cache, f.block_table, f.kv_len, f.refs, up(np.array(parent, np.int32)), room=1)
        text = [text[p] + [int(rng.integers(1, 100))] for p in parent]
        t, n = f.block_table.cpu().numpy(), f.kv_len.cpu().numpy()
        assert np.array_equal(np.bincount(t[t >= 0], minlength=pages), f.refs.cpu().numpy()) and f.missing.item() == 0
        for s in range(S):
            assert n[s] == len(text[s]) - 1
            cache.k[int(t[s, n[s] // page]), 0, int(n[s]) % page, 0] = text[s][-1]
        f = f._replace(kv_len=f.kv_len + 1)
        codes = cache.k[:, 0, :, 0].cpu().numpy()
        for s in range(S):
            assert codes[t[s, :-(-len(text[s]) // page)]].flatten()[:len(text[s])].tolist() == text[s], (step, s)


# ---------------------------------------------------------------- streams, graphs, the binding
def test_other_stream_and_graph():
    rng = np.random.default_rng(9)
    table, lens, refs = tables_in_use(rng, 4, 5, 64, 60, shared=0)
    lens = np.maximum(lens, 12).astype(np.int32)
    refs[:] = 0
    table[:] = rng.permutation(60)[:20].reshape(4, 5)
    refs[table.flatten()] = 1
    base = [random_cache(rng, 60, 2, 64, 128) for _ in range(3)]
    start = up(np.array([0, 6, 12, 18, 24], np.int32))
    keep, kept = np.array([[1, 3], [0, 5], [2, -1], [0, 1]], np.int32), up(np.array([2, 2, 1, 2], np.int32))
    parents = [[0, 0, 3, 1], [2, 2, 2, 2], [1, 0, 3, 2], [3, 3, 1, -1]]

    def step(caches, keep, parent, out):
        batch = q8.KvBatch(start, up_lens, up_table, 6, 320)
        n = q8.q8_kv_compact(caches, batch, keep, kept, out=out[0])
        return q8.q8_kv_fork(caches, up_table, n, up_refs, parent, room=6, out=out[1], workspace=out[2])

    up_lens, up_table, up_refs = up(lens), up(table), up(refs)
    i32 = lambda *n: torch.empty(*n, dtype=torch.int32, device=DEV)  # noqa: E731
    outs = lambda: (i32(4), q8.KvFork(i32(4, 5), i32(4), i32(60), i32(1)),  # noqa: E731
                    torch.empty(q8.q8_kv_fork_workspace_bytes(4, 4, 60), dtype=torch.uint8, device=DEV))
    eager_caches, eager = [device(c) for c in base], []
    for p in parents:
        eager.append([t.clone() for t in step(eager_caches, up(keep), up(np.array(p, np.int32)), outs())])
    want = [[t.clone() for t in c] for c in eager_caches]
    side = torch.cuda.Stream()
    caches, parent, out = [device(c) for c in base], up(np.array(parents[0], np.int32)), outs()
    held = up(keep)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f = step(caches, held, parent, out)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(f, eager[0]))
    caches = [device(c) for c in base]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = step(caches, held, parent, out)
    for i, p in enumerate(parents):
        parent.copy_(torch.tensor(p, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(f, eager[i])), i
        (torch.randn(256, 256, device=DEV) @ torch.randn(256, 256, device=DEV)).sum().item()
    for a, b in zip(caches, want):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_compiled_and_interpreted_calls_agree():
    rng = np.random.default_rng(11)
    table, lens, refs = tables_in_use(rng, 3, 4, 32, 40, shared=0)
    lens = np.maximum(lens, 9).astype(np.int32)
    table[:] = rng.permutation(40)[:12].reshape(3, 4)
    refs[:] = 0
    refs[table.flatten()] = 1
    base = [random_cache(rng, 40, 2, 32, 64) for _ in range(2)]
    batch = q8.KvBatch(up(np.array([0, 8, 16, 24], np.int32)), up(lens), up(table), 8, 128)
    keep, kept = up(np.array([[1, 3], [0, 5], [2, 7]], np.int32)), up(np.array([2, 2, 2], np.int32))
    parent = up(np.array([1, 1, 0, 2], np.int32))

    def both(caches):
        n = q8.q8_kv_compact(tuple(tuple(c) for c in caches), batch, keep, kept)
        return [n, *q8.q8_kv_fork(caches, batch.block_table, n, up(refs), parent, room=3), *caches[0], *caches[1]]

    for a, b in zip(both([device(c) for c in base]), interpreted(lambda: both([device(c) for c in base]))):
        assert torch.equal(a, b)
    fast, one = q8._fast(), device(base[0])
    assert isinstance(fast.kv_compact(one, batch, keep, kept, None), torch.Tensor)
    assert fast.kv_compact([one, one], batch, keep, kept, None) == _lib.Q8_ERR_BAD_ARG
    assert fast.kv_compact([], batch, keep, kept, None) is NotImplemented
    assert fast.kv_fork(one, batch.block_table, batch.kv_len, up(refs), parent, -1, None, None) == 2
    assert fast.kv_fork(one, batch.block_table, batch.kv_len, up(refs).long(), parent, 0, None, None) is NotImplemented


def test_binding_refusals():
    cache, other = (q8.q8_kv_cache(4, 2, 64, page=32, device=DEV) for _ in range(2))
    _, batch = batch_of([2], [2], [[0, 1]])
    keep, kept = torch.zeros(1, 2, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    refs, parent = torch.ones(4, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    com = lambda **kw: q8.q8_kv_compact(**{**dict(caches=[cache, other], batch=batch, keep=keep, n_keep=kept), **kw})  # noqa: E731
    frk = lambda **kw: q8.q8_kv_fork(**{**dict(caches=[cache, other], block_table=batch.block_table, kv_len=batch.kv_len, refs=refs,  # noqa: E731
                                               parent=parent), **kw})
    for call in (com, frk):
        with pytest.raises(_lib.Q8Error):
            call(caches=[cache, cache])
        with pytest.raises(ValueError):
            call(caches=[])
        with pytest.raises(ValueError):
            call(caches=[cache, q8.q8_kv_cache(5, 2, 64, page=32, device=DEV)])
        with pytest.raises(TypeError):
            call(caches=[cache, other._replace(k=other.k.float())])
        with pytest.raises(TypeError):
            call(caches=[cache, other._replace(v_exp=other.v_exp.cpu())])
    with pytest.raises(TypeError):
        com(keep=keep.long())
    with pytest.raises(ValueError):
        com(n_keep=parent)
    with pytest.raises(_lib.Q8Error):
        com(out=batch.kv_len)
    with pytest.raises(TypeError):
        frk(refs=refs.long())
    with pytest.raises(ValueError):
        frk(refs=refs[:3])
    with pytest.raises(_lib.Q8Error):
        frk(room=-1)
    with pytest.raises(_lib.Q8Error):
        frk(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    out = frk()
    with pytest.raises(_lib.Q8Error):
        frk(out=out._replace(refs=refs))
    with pytest.raises(ValueError):
        frk(out=out._replace(kv_len=out.refs))
