"""The page operators against their sequential restatement: books, holders,
info and the bytes of every page, which have to be equal."""
import random

import numpy as np
import pytest
import torch

from kv_cache_vector_gb300 import abi
from oracle import pages as OP

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_cache_vector_gb300 import build
    build.build()
    abi.lib()
    abi.tq_device_status(reset=True)


def make_pool(seed, n_pages, L=2, Hkv=2, page=32, d=32, kb=4, vb=2):
    g = torch.Generator().manual_seed(seed)
    layers = []
    for _ in range(L):
        byte = lambda bits: torch.randint(0, 256, (n_pages, Hkv, page, d * bits // 8), generator=g,  # noqa: E731
                                          dtype=torch.uint8).cuda()
        norm = lambda: torch.randn(n_pages, Hkv, page, generator=g).cuda()  # noqa: E731
        layers.append(abi.PagedCache(byte(kb), norm(), byte(vb), norm(), kb, vb))
    return abi.PagedLayers(layers)


def contents(pool):
    return [[t.cpu().numpy().copy() for t in (c.k_packed, c.k_norm, c.v_packed, c.v_norm)] for c in pool.layers]


def check_contents(pool, before, pairs, before_dst=None):
    want = before_dst or before
    for layer, (got, old) in enumerate(zip(contents(pool), before)):
        for a in range(4):
            w = want[layer][a].copy()
            for s, t in pairs:
                w[t] = old[a][s]
            wrong = np.flatnonzero((got[a] != w).reshape(len(w), -1).any(1))
            assert wrong.size == 0, (layer, a, wrong[:20], pairs[:20])


def random_table(rng, n, max_pages, n_pages, page, fill=0.7):
    """Rows with shared beginnings, some cut back into a shared page, on shuffled page ids."""
    ids = list(range(n_pages))
    rng.shuffle(ids)
    table = np.full((n, max_pages), -1, np.int32)
    lens = np.zeros(n, np.int32)
    refs = np.zeros(n_pages, np.int32)
    used = 0
    for i in range(n):
        length = rng.choice((0, 1, page, page * max_pages, rng.randrange(0, page * max_pages + 1)))
        need, row = -(-length // page), []
        if i and rng.random() < 0.6:
            j = rng.randrange(i)
            have = -(-int(lens[j]) // page)
            row = list(table[j, :rng.randrange(0, min(have, need) + 1)])
            if row and rng.random() < 0.5:
                length = len(row) * page - rng.randrange(page)
                need = len(row)
        more = need - len(row)
        if used + more > fill * n_pages:
            length, need, more = len(row) * page, len(row), 0
        row += ids[used:used + more]
        used += more
        table[i, :need], lens[i] = row, length
        for e in row:
            refs[e] += 1
    return table, lens, refs


def on_gpu(table, lens, refs):
    return abi.PageTable(*(torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (table, lens, refs)))


def check_books(out, info, want):
    torch.cuda.synchronize()
    assert tuple(info.tolist()) == want[-1]
    assert np.array_equal(out.lens.cpu().numpy(), want[1])
    assert np.array_equal(out.refs.cpu().numpy(), want[2])
    assert np.array_equal(out.block_table.cpu().numpy(), want[0])


SHAPES = [  # n_seqs, max_pages, n_pages, page, layers, Hkv, d, kb, vb
    (1, 1, 1, 32, 1, 1, 32, 2, 2),
    (5, 4, 23, 32, 2, 2, 64, 3, 4),
    (33, 9, 300, 64, 3, 1, 128, 4, 3),
    (130, 7, 1031, 32, 1, 3, 32, 2, 3),
    (400, 70, 20011, 32, 1, 1, 32, 2, 2),   # eight CTAs plan
    (9, 6, 60, 256, 66, 1, 32, 4, 2),       # more layers than one copy launch takes
]


def setup(shape, seed, fill=0.7):
    n, mp, N, page, L, Hkv, d, kb, vb = shape
    rng = random.Random(seed)
    return rng, random_table(rng, n, mp, N, page, fill), make_pool(seed, N, L, Hkv, page, d, kb, vb), page


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("seed", range(3))
def test_fork(shape, seed):
    rng, (table, lens, refs), pool, page = setup(shape, 10 + seed)
    n = len(lens)
    parents = np.array([rng.choice((i, rng.randrange(-1, n))) for i in range(n)], np.int32)
    if seed == 2:
        parents[:] = rng.randrange(n)  # every row a branch of one
    want = OP.fork(table, lens, refs, parents, page)
    before, t = contents(pool), on_gpu(table, lens, refs)
    out, info = abi.tq_pages_fork(t, torch.from_numpy(parents).cuda(), pool)
    check_books(out, info, want)
    check_contents(pool, before, want[3])
    check_books(t, info, (table, lens, refs, want[-1]))  # the input is as it was
    assert abi.tq_device_status(reset=True) == 0


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seed", range(3))
def test_resize(shape, seed, in_place):
    rng, (table, lens, refs), pool, page = setup(shape, 20 + seed, 0.6)
    top = page * table.shape[1]
    to = np.array([rng.choice((-1, 0, min(top, int(k) + 1), min(top, int(k) + rng.randrange(page)),
                               rng.randrange(0, int(k) + 1))) for k in lens], np.int32)
    want = OP.resize(table, lens, refs, to, page)
    before, t = contents(pool), on_gpu(table, lens, refs)
    out, info = abi.tq_pages_resize(t, torch.from_numpy(to).cuda(), pool, out=t if in_place else None)
    assert (out is t) == in_place
    check_books(out, info, want)
    check_contents(pool, before, want[3])
    assert abi.tq_device_status(reset=True) == 0


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(shape, in_place):
    _, (table, lens, refs), pool, page = setup(shape, 31, 0.5)
    want = OP.compact(table, lens, refs, page)
    before, t = contents(pool), on_gpu(table, lens, refs)
    out, moved, info = abi.tq_pages_compact(t, pool, out=t if in_place else None)
    check_books(out, info, want)
    assert np.array_equal(moved.cpu().numpy(), want[4])
    check_contents(pool, before, want[3])
    # once closed up there is nothing to move
    out2, moved2, info2 = abi.tq_pages_compact(out, pool)
    check_books(out2, info2, (*want[:3], (want[-1][0], 0)))
    check_contents(pool, before, want[3])


def test_compact_keeps_pages_that_no_row_holds():
    """A page held by something other than a row (refs set by the caller) stays and moves like the others."""
    _, (table, lens, refs), pool, page = setup(SHAPES[2], 32, 0.4)
    spare = [p for p in range(len(refs)) if refs[p] == 0][-3:]
    refs[spare] = 2
    want = OP.compact(table, lens, refs, page)
    before = contents(pool)
    out, moved, info = abi.tq_pages_compact(on_gpu(table, lens, refs), pool)
    check_books(out, info, want)
    assert np.array_equal(moved.cpu().numpy(), want[4])
    check_contents(pool, before, want[3])


def test_too_few_pages_changes_nothing():
    page, pool = 32, make_pool(5, 8)
    table = np.full((3, 6), -1, np.int32)
    table[0, :3], table[1, :2] = [7, 1, 4], [7, 2]
    lens, refs = np.array([70, 64, 0], np.int32), np.array([0, 1, 1, 0, 1, 0, 0, 2], np.int32)
    before, t = contents(pool), on_gpu(table, lens, refs)
    to = np.array([190, 190, -1], np.int32)
    want = OP.resize(table, lens, refs, to, page)
    assert want[-1] == (0, 3)
    for out in (None, t):
        got, info = abi.tq_pages_resize(t, torch.from_numpy(to).cuda(), pool, out=out)
        check_books(got, info, want)
    refs[:] += (refs == 0)  # every page held
    parents = np.array([0, 0, 0], np.int32)
    want = OP.fork(table, lens, refs, parents, page)
    got, info = abi.tq_pages_fork(on_gpu(table, lens, refs), torch.from_numpy(parents).cuda(), pool)
    assert want[-1] == (0, 1)  # row 1's page 2 is given back, two copies are owed
    check_books(got, info, want)
    check_contents(pool, before, [])


@pytest.mark.parametrize("what", ["id", "negative id", "length", "negative length", "argument"])
def test_books_out_of_range_change_nothing(what):
    page, pool = 32, make_pool(6, 8)
    table, lens = np.full((2, 3), -1, np.int32), np.array([40, 10], np.int32)
    table[0, :2], table[1, 0] = [3, 5], 0
    refs = np.array([1, 0, 0, 1, 0, 1, 0, 0], np.int32)
    parents, to = np.array([1, 0], np.int32), np.array([50, 12], np.int32)
    if what == "id":
        table[0, 1] = 8
    elif what == "negative id":
        table[1, 0] = -2
    elif what == "length":
        lens[1] = 97
    elif what == "negative length":
        lens[0] = -1
    else:
        parents[1], to[0] = 2, 97
    before = contents(pool)
    for fn, arg in (("fork", parents), ("resize", to), ("compact", None)):
        if what == "argument" and arg is None:
            continue
        t = on_gpu(table, lens, refs)
        args = (t, pool) if arg is None else (t, torch.from_numpy(arg).cuda(), pool)
        got = getattr(abi, f"tq_pages_{fn}")(*args)
        check_books(got[0], got[-1], (table, lens, refs, (0, -1)))
        assert abi.tq_device_status(reset=True) == 61
    check_contents(pool, before, [])


@pytest.mark.parametrize("same", [True, False])
@pytest.mark.parametrize("n_pages,n", [(1, 1), (40, 13), (3000, 1400), (20000, 9000)])
def test_copy(n_pages, n, same):
    rng = np.random.default_rng(n)
    src = make_pool(7, n_pages, L=2, Hkv=1, d=64, kb=3, vb=4)
    dst = src if same else make_pool(8, n_pages + 5, L=2, Hkv=1, d=64, kb=3, vb=4)
    ids = rng.permutation(n_pages).astype(np.int32)
    s = ids[:n]
    t = (ids[n:2 * n] if same else rng.permutation(n_pages + 5).astype(np.int32)[:n]).copy()
    s = s[:len(t)].copy()
    if n > 10:
        s[3], t[5] = -1, -7                    # no pairs
    before, before_dst = contents(src), contents(dst)
    abi.tq_pages_copy(src, dst, torch.from_numpy(s).cuda(), torch.from_numpy(t).cuda())
    torch.cuda.synchronize()
    check_contents(dst, before, OP.copy_pairs(s, t, n_pages, dst.n_pages, same), before_dst)
    assert abi.tq_device_status(reset=True) == 0


@pytest.mark.parametrize("s,t,same,status", [
    ([0, 1, 2], [5, 5, 6], True, 62),      # one destination twice: the first pair has it
    ([0, 1, 2], [5, 0, 6], True, 62),      # a destination that is a source
    ([3], [3], True, 62),                  # a page onto itself
    ([3, 4], [3, 4], False, 0),            # the same ids of two pools
    ([0, 12, 2], [5, 6, 7], True, 61),     # past the pool
    ([0, 1, 2], [5, 6, 12], False, 61),
    ([-1, -1], [-1, -1], True, 0),
])
def test_copy_conflicts_are_refused_by_pair(s, t, same, status):
    src = make_pool(9, 12)
    dst = src if same else make_pool(10, 12)
    before, before_dst = contents(src), contents(dst)
    ids = [torch.tensor(x, dtype=torch.int32).cuda() for x in (s, t)]
    abi.tq_pages_copy(src, dst, *ids)
    assert abi.tq_device_status(reset=True) == status
    check_contents(dst, before, OP.copy_pairs(s, t, 12, 12, same), before_dst)


@pytest.mark.parametrize("same", [True, False])
@pytest.mark.parametrize("n", [2, 31, 127, 128, 129, 200, 3000])
def test_copy_of_random_pairs(n, same):
    """Ids out of range, skipped pairs, destinations given twice and destinations that are
    sources, with as many pairs as one kernel looks over by itself and with more."""
    rng = np.random.default_rng(n)
    N = max(40, n + 3)
    src = make_pool(12, N, L=3, Hkv=1)
    dst = src if same else make_pool(13, N + 2, L=3, Hkv=1)
    s = rng.integers(0, N, n).astype(np.int32)
    t = rng.integers(0, dst.n_pages, n).astype(np.int32)
    s[rng.random(n) < 0.1], t[rng.random(n) < 0.1] = -3, -1
    s[0] = N                                   # past the pool
    before, before_dst = contents(src), contents(dst)
    want = OP.copy_pairs(s, t, N, dst.n_pages, same)
    assert n < 20 or 0 < len(want) < n
    abi.tq_pages_copy(src, dst, torch.from_numpy(s).cuda(), torch.from_numpy(t).cuda())
    assert abi.tq_device_status(reset=True) in (61, 62)
    check_contents(dst, before, want, before_dst)


@pytest.mark.parametrize("L", [1, 4, 5, 64, 65, 130])
@pytest.mark.parametrize("n", [3, 150])
def test_copy_of_many_layers(L, n):
    """As many layers as a launch takes and more, with few pairs and many."""
    N = 310
    src = make_pool(16, N, L=L, Hkv=1)
    ids = np.random.default_rng(L).permutation(N).astype(np.int32)
    s, t = ids[:n].copy(), ids[n:2 * n].copy()
    before = contents(src)
    abi.tq_pages_copy(src, src, torch.from_numpy(s).cuda(), torch.from_numpy(t).cuda())
    assert abi.tq_device_status(reset=True) == 0
    check_contents(src, before, list(zip(s.tolist(), t.tolist())))


def test_what_a_call_says_stays_with_the_table_it_wrote():
    page, N = 32, 12
    pool = make_pool(14, N)
    t = on_gpu(np.full((2, 4), -1, np.int32), np.zeros(2, np.int32), np.zeros(N, np.int32))
    grow = lambda *k: torch.tensor(k, dtype=torch.int32).cuda()  # noqa: E731
    out, info = abi.tq_pages_resize(t, grow(40, 10), pool)
    assert info is out.info and out is not t and t.info is None and info.tolist() == [3, 0]
    other, info2 = abi.tq_pages_resize(out, grow(100, 0), pool)
    assert info2.tolist() == [2, 0] and info.tolist() == [3, 0]    # another table's
    mine = torch.full((2,), 7, dtype=torch.int32, device="cuda")
    same, info3 = abi.tq_pages_resize(other, grow(0, 0), pool, out=other, info=mine)
    assert same is other and info3 is mine and mine.tolist() == [0, 0] and other.info.tolist() == [2, 0]
    moved = torch.empty(N, dtype=torch.int32, device="cuda")
    done, m, i = abi.tq_pages_compact(out, pool, moved_to=moved)
    assert m is moved and i is done.info and done.moved_to is None and i.tolist() == [3, 0]
    done2, m2, _ = abi.tq_pages_compact(out, pool, out=done)
    assert done2 is done and m2 is done.moved_to and torch.equal(m2, moved)


def test_a_refused_call_leaves_the_table_as_it_was():
    pool = make_pool(15, 12)
    t = on_gpu(np.full((2, 4), -1, np.int32), np.zeros(2, np.int32), np.zeros(12, np.int32))
    to = torch.tensor([40, 10], dtype=torch.int32).cuda()
    out = on_gpu(np.zeros((2, 4), np.int32), np.zeros(2, np.int64), np.zeros(12, np.int32))
    with pytest.raises(TypeError):
        abi.tq_pages_resize(t, to, pool, out=out)
    assert out.info is None
    for bad in (dict(info=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(out=abi.PageTable(
            t.block_table[:, :3].contiguous(), t.lens, t.refs)), dict(workspace=torch.zeros(1 << 20))):
        with pytest.raises(ValueError):
            abi.tq_pages_resize(t, to, pool, **bad)
    with pytest.raises(ValueError):
        abi.tq_pages_resize(t, to[:1], pool)
    with pytest.raises(abi.TQError):     # a workspace that is too small
        abi.tq_pages_resize(t, to, pool, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert t.info is None and not t.lens.any() and not t.refs.any()


def test_captured_and_replayed_on_another_stream():
    """One decode step's books in a graph: the row lengths move on between replays."""
    page, n, mp, N = 32, 4, 5, 30
    pool = make_pool(11, N)
    t = on_gpu(np.full((n, mp), -1, np.int32), np.zeros(n, np.int32), np.zeros(N, np.int32))
    new_lens, info = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = torch.empty(abi.tq_pages_workspace_bytes(n, mp, N), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        abi.tq_pages_resize(t, new_lens, pool, out=t, info=info, workspace=ws)  # warm-up: nothing to do
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        abi.tq_pages_resize(t, new_lens, pool, out=t, info=info, workspace=ws)
    books = tuple(x.cpu().numpy() for x in (t.block_table, t.lens, t.refs))
    rng = random.Random(3)
    for _ in range(6):
        to = np.array([min(page * mp, int(k) + rng.choice((0, 1, 31, 40))) if rng.random() < 0.8 else 0
                       for k in books[1]], np.int32)
        new_lens.copy_(torch.from_numpy(to))
        want = OP.resize(*books, to, page)
        g.replay()
        check_books(t, info, want)
        books = want[:3]


@pytest.mark.parametrize("n,holders", [(1 << 17, 0), (40000, 3), (257, 0), (257, 1)])
def test_many_rows_go_on_in_one_shared_page(n, holders):
    """All rows are branches of one prompt: all but the last take a private copy (all of them where
    something else holds the page too), in a time that grows with the rows, not with their square."""
    page, N = 32, n + 9
    pool = make_pool(17, N, L=1, Hkv=1, d=32, kb=2, vb=2)
    table, lens, refs = np.full((n, 3), -1, np.int32), np.full(n, 40, np.int32), np.zeros(N, np.int32)
    table[:, 0], table[:, 1] = 4, 2
    refs[4], refs[2] = n, n + holders
    to = np.full(n, 41, np.int32)
    to[5::7] = -1                              # some stay as they are
    want = OP.resize(table, lens, refs, to, page)
    grows = int((to > 0).sum())
    assert want[-1] == (min(grows, n + holders - 1), 0)
    before, t, new = contents(pool), on_gpu(table, lens, refs), torch.from_numpy(to).cuda()
    out, info = abi.tq_pages_resize(t, new, pool)
    check_books(out, info, want)
    check_contents(pool, before, want[3])
    assert abi.tq_device_status(reset=True) == 0
    alone = table.copy()                       # the same rows with last pages of their own
    alone[:, 1] = np.delete(np.arange(n + 1), 4)
    refs2 = np.zeros(N, np.int32)
    refs2[:n + 1] = 1
    refs2[4] = n
    t2, ws = on_gpu(alone, lens, refs2), torch.empty(abi.tq_pages_workspace_bytes(n, 3, N), dtype=torch.uint8, device="cuda")

    def ms(table):
        best = 1e9
        for _ in range(3):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            abi.tq_pages_resize(table, new, pool, out=out, workspace=ws)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    assert ms(t) <= 4 * ms(t2) + 1.0


def test_what_a_call_said_is_not_written_again():
    """Steps of a loop in place: what each said stays as it was, on whichever stream it is read, and
    in a graph of several steps too."""
    page, N = 32, 12
    pool = make_pool(18, N)
    t = on_gpu(np.full((2, 4), -1, np.int32), np.zeros(2, np.int32), np.zeros(N, np.int32))
    grow = lambda *k: torch.tensor(k, dtype=torch.int32).cuda()  # noqa: E731
    said = []
    for step in (grow(40, 10), grow(100, 0), grow(128, 128), grow(0, 0)):
        said.append(abi.tq_pages_resize(t, step, pool, out=t)[1])
        assert t.info is said[-1]
    moved = [abi.tq_pages_compact(t, pool, out=t)[1:]]
    abi.tq_pages_resize(t, grow(60, 60), pool, out=t)
    moved.append(abi.tq_pages_compact(t, pool, out=t)[1:])
    assert [x.tolist() for x in said] == [[3, 0], [2, 0], [4, 0], [0, 0]]
    assert moved[0][1].tolist() == [0, 0] and (moved[0][0] == -1).all()
    assert moved[1][1].tolist() == [4, 0] and moved[1][0].tolist() == [0, 1, 2, 3] + [-1] * 8
    assert t.moved_to is moved[1][0] and t.info is moved[1][1]
    # captured: each step of the graph has its own, and a call outside of it another
    abi.tq_pages_resize(t, grow(0, 0), pool, out=t)
    a, b = grow(40, 10), grow(100, 0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        i1 = abi.tq_pages_resize(t, a, pool, out=t)[1]
        i2 = abi.tq_pages_resize(t, b, pool, out=t)[1]
    g.replay()
    torch.cuda.synchronize()
    assert i1.tolist() == [3, 0] and i2.tolist() == [2, 0]
    abi.tq_pages_resize(t, grow(0, 0), pool, out=t)
    assert i1.tolist() == [3, 0] and i2.tolist() == [2, 0] and t.info.tolist() == [0, 0]


def test_layers_keep_the_tensors_whose_addresses_they_pass():
    """A PagedCache may get other tensors later: the pool's calls go on with the ones that it was made of."""
    import gc
    import weakref
    c = abi.PagedCache.empty(12, 1, 32, 64, 4, 3)
    c.k_packed.copy_(torch.arange(12, dtype=torch.uint8).view(12, 1, 1, 1).expand_as(c.k_packed))
    pool, was = abi.PagedLayers(c), c.k_packed.data_ptr()
    kept = [weakref.ref(t) for t in (c.k_packed, c.k_norm, c.v_packed, c.v_norm)]
    c.k_packed, c.k_norm, c.v_packed, c.v_norm = (torch.zeros_like(t) for t in (c.k_packed, c.k_norm, c.v_packed, c.v_norm))
    gc.collect()
    assert all(k() is not None for k in kept) and kept[0]().data_ptr() == was
    ids = lambda *k: torch.tensor(k, dtype=torch.int32).cuda()  # noqa: E731
    abi.tq_pages_copy(pool, pool, ids(3), ids(7))
    assert (kept[0]()[7] == 3).all() and not c.k_packed.any()
