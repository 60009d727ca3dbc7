"""The sequential restatement of the page operators keeps a page table sound:
random sequences of fork, resize and compaction, with each row's positions
holding values of their own, checked against plain Python lists of what every
row has written.  And the entry points' refusals, which come before any launch."""
import ctypes
import random

import numpy as np
import pytest

from kv_cache_vector_gb300 import abi
from oracle import pages as OP


def _apply(pool, pairs):
    """Copies of a call read the pages as they were before it."""
    new = pool.copy()
    for s, t in pairs:
        new[t] = pool[s]
    return new


@pytest.mark.parametrize("seed", range(6))
def test_books_stay_sound(seed):
    rng = random.Random(seed)
    page, n, max_pages, n_pages = 32, 7, 6, 40
    table = np.full((n, max_pages), -1, np.int32)
    lens, refs = np.zeros(n, np.int32), np.zeros(n_pages, np.int32)
    pool = np.zeros((n_pages, page), np.int64)
    rows, stamp = [[] for _ in range(n)], 0
    for _ in range(150):
        op = rng.choice(("fork", "resize", "resize", "compact"))
        if op == "fork":
            parents = np.array([rng.choice((i, i, rng.randrange(-1, n))) for i in range(n)], np.int32)
            t, l, r, pairs, info = OP.fork(table, lens, refs, parents, page)
            if info[1] == 0:
                rows = [list(rows[p]) if p >= 0 else [] for p in parents]
        elif op == "resize":
            to = np.array([rng.choice((-1, 0, rng.randrange(0, max_pages * page + 1),
                                       min(max_pages * page, int(k) + rng.randrange(20)))) for k in lens], np.int32)
            t, l, r, pairs, info = OP.resize(table, lens, refs, to, page)
        else:
            t, l, r, pairs, _, info = OP.compact(table, lens, refs, page)
        assert info[1] >= 0
        pool = _apply(pool, pairs)
        if op == "resize" and info[1] == 0:  # the rows write their new positions
            for i in range(n):
                rows[i] = rows[i][:l[i]]
                for p in range(len(rows[i]), l[i]):
                    stamp += 1
                    rows[i].append(stamp)
                    pool[t[i, p // page], p % page] = stamp
        table, lens, refs = t, l, r
        count = np.zeros(n_pages, np.int32)
        for i in range(n):
            used = -(-int(lens[i]) // page)
            assert (table[i, used:] == -1).all()
            for e in table[i, :used]:
                count[e] += 1
            assert [pool[table[i, p // page], p % page] for p in range(lens[i])] == rows[i]
        assert np.array_equal(count, refs)


@pytest.fixture(scope="module")
def L():
    from kv_cache_vector_gb300 import build
    build.build()
    return abi.lib()


def _cache(at=1 << 32, n_pages=4, page_size=64):
    return abi.PagedCacheView(at, at + (1 << 24), at + (2 << 24), at + (3 << 24), n_pages, page_size)


def _layers(*caches):
    return (abi.PagedCacheView * len(caches))(*caches)


def test_refusals_of_the_books(L):
    A, W = 1 << 20, 1 << 28
    tab = lambda a, t=None: abi.PageTableView(a, a + 4096, a + 8192 if t is None else t)  # noqa: E731
    a, b, arg, info = tab(A), tab(A + (1 << 16)), A + (1 << 18), A + (1 << 19)
    ly = _layers(_cache())
    need = L.tq_pages_workspace_bytes(4, 8, 4)
    assert need >= 4 * (5 * 4 + 3 * 4)
    assert L.tq_pages_workspace_bytes(-1, 8, 4) == 0
    assert L.tq_pages_workspace_bytes(4, 8, 0) == 0
    assert L.tq_pages_workspace_bytes(4, 8, 1 << 31) == 0

    def fork(i=a, p=arg, o=b, n=4, mp=8, layers=ly, nl=1, hkv=2, d=128, kb=4, vb=3, inf=info, ws=W, size=need):
        return L.tq_pages_fork(i, p, o, n, mp, layers, nl, hkv, d, kb, vb, inf, ws, size, None)

    assert fork(n=0) == 1
    assert fork(mp=0) == 1
    assert fork(layers=None) == 1
    assert fork(nl=0) == 1
    assert fork(hkv=0) == 1
    assert fork(d=96) == 2
    assert fork(d=16) == 2
    assert fork(kb=5) == 2
    assert fork(vb=1) == 2
    assert fork(layers=_layers(_cache(page_size=48))) == 2
    assert fork(layers=_layers(_cache(page_size=16))) == 2
    assert fork(mp=1 << 26) == 2                                   # lengths past int32
    assert fork(layers=_layers(_cache(n_pages=0))) == 1
    assert fork(layers=_layers(_cache(n_pages=1 << 31))) == 1
    assert fork(layers=_layers(_cache(), _cache(1 << 36, 5)), nl=2) == 1    # another geometry
    assert fork(layers=_layers(abi.PagedCacheView(1 << 32, (1 << 33) + 4, 1 << 34, 1 << 35, 4, 64))) == 3
    assert fork(p=None) == 1
    assert fork(inf=None) == 1
    assert fork(i=abi.PageTableView(A, None, A + 8192)) == 1
    assert fork(p=arg + 2) == 3
    assert fork(ws=None) == 5
    assert fork(size=need - 1) == 5
    assert fork(ws=W + 4) == 3
    assert fork(o=a) == 1                                          # rows exchange places: not in place
    assert fork(o=tab(A, A + (1 << 17))) == 1                      # partly the input
    assert fork(inf=A + 4) == 1                                    # info inside the table
    assert fork(p=A + (1 << 16) + 4) == 1                          # parents inside the output
    resize = lambda o: L.tq_pages_resize(a, arg, o, 4, 8, ly, 1, 2, 128, 4, 3, info, W, need, None)  # noqa: E731
    assert resize(tab(A + 4)) == 1                                 # neither in place nor apart
    assert L.tq_pages_resize(a, None, b, 4, 8, ly, 1, 2, 128, 4, 3, info, W, need, None) == 1
    assert L.tq_pages_compact(a, b, None, 4, 8, ly, 1, 2, 128, 4, 3, info, W, need, None) == 1
    assert L.tq_pages_compact(a, b, A + 8192, 4, 8, ly, 1, 2, 128, 4, 3, info, W, need, None) == 1  # moved_to on refs


def test_most_rows_of_a_table(L):
    a, b = abi.PageTableView(1 << 32, 1 << 33, 1 << 34), abi.PageTableView(1 << 35, 1 << 36, 1 << 37)
    ly, n = _layers(_cache(1 << 40)), (1 << 18) + 1
    assert L.tq_pages_workspace_bytes(n, 8, 4) == 0
    need, W = 1 << 30, 1 << 38
    assert L.tq_pages_fork(a, 1 << 39, b, n, 8, ly, 1, 2, 128, 4, 3, 1 << 20, W, need, None) == 2
    assert L.tq_pages_resize(a, 1 << 39, b, n, 8, ly, 1, 2, 128, 4, 3, 1 << 20, W, need, None) == 2
    assert L.tq_pages_compact(a, b, 1 << 39, n, 8, ly, 1, 2, 128, 4, 3, 1 << 20, W, need, None) == 2
    # the most rows: refused for the workspace only
    assert L.tq_pages_fork(a, 1 << 39, b, n - 1, 8, ly, 1, 2, 128, 4, 3, 1 << 20, None, 0, None) == 5


def test_refusals_of_the_copy(L):
    ids, W = 1 << 20, 1 << 28
    one, two = _layers(_cache()), _layers(_cache(1 << 36))
    need = L.tq_pages_workspace_bytes(0, 0, 4)

    def copy(s=one, t=two, nl=1, hkv=2, d=128, kb=4, vb=3, si=ids, ti=ids + 4096, n=2, ws=W, size=need):
        return L.tq_pages_copy(s, t, nl, hkv, d, kb, vb, si, ti, n, ws, size, None)

    assert copy(n=0) == 0 and copy(n=0, si=None, ti=None, ws=None) == 0   # nothing to copy
    assert copy(n=-1) == 1
    assert copy(n=5) == 1                                                  # more than the pool has
    assert copy(s=None) == 1 and copy(t=None) == 1
    assert copy(t=_layers(_cache(1 << 36, 4, 128))) == 1                   # another page size
    assert copy(t=_layers(_cache((1 << 32) + 4096))) == 1                  # overlapping pools
    assert copy(s=_layers(_cache(), _cache(1 << 36)), t=_layers(_cache(1 << 36), _cache(1 << 40)), nl=2) == 1
    assert copy(s=_layers(_cache(), _cache(1 << 36)), t=_layers(_cache(), _cache(1 << 40)), nl=2) == 1
    # a K array of one pool over a V array of the other, a few layers on
    far = [_cache((40 + i) << 32) for i in range(70)]
    assert copy(s=_layers(*far[:69], abi.PagedCacheView(1 << 32, 1 << 33, 1 << 34, (109 << 32) + (1 << 24), 4, 64)),
                t=_layers(*[_cache((200 + i) << 32) for i in range(69)], far[69]), nl=70) == 1
    assert copy(s=_layers(*far), t=_layers(*[_cache((200 + i) << 32) for i in range(70)]), nl=70, ti=ids + 2) == 3
    # many pairs: with a workspace, and the ids outside of it
    many = dict(s=_layers(_cache(n_pages=200)), t=_layers(_cache(1 << 36, 200)), n=129,
                size=L.tq_pages_workspace_bytes(0, 0, 200))
    assert copy(**{**many, "si": W + 64}) == 1 and copy(**{**many, "ti": W + many["size"] - 4}) == 1
    assert copy(**{**many, "ws": None}) == 5 and copy(**{**many, "size": many["size"] - 1}) == 5
    assert copy(**{**many, "ws": W + 8}) == 3
    assert copy(d=48) == 2 and copy(kb=1) == 2
    assert copy(si=None) == 1 and copy(ti=ids + 2) == 3


def test_python_layer_refusals():
    import torch
    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError):
        abi.PagedLayers([])
    with pytest.raises(ValueError):  # host tensors
        abi.PagedLayers(abi.PagedCache(z(4, 2, 32, 64), z(4, 2, 32, dt=torch.float32), z(4, 2, 32, 48),
                                       z(4, 2, 32, dt=torch.float32), 4, 3))
    assert ctypes.sizeof(abi.PageTableView) == 24


def test_prefill_paged_refusals(L):
    """tq_attn_prefill_paged checks its arguments on the host before any launch."""
    p128, p16 = abi.Plan(128, 42), abi.Plan(16, 42)
    A, W = 1 << 20, 1 << 28
    f = ctypes.c_float
    need = L.tq_attn_prefill_paged_workspace_bytes(8, 2, 128)
    assert need > 0
    for bad in ((0, 2, 128), (8, 3, 128), (8, 0, 128), (8, 2, 16), (8, 2, 96)):
        assert L.tq_attn_prefill_paged_workspace_bytes(*bad) == 0

    def call(plan=p128.handle, q=A, n_q=10, B=2, Hq=8, Hkv=2, cache=_cache(), bt=A, mp=4, cu=A, ctx=A, window=0,
             kb=4, vb=3, scale=1.0, out=A, dt=1, ws=W, size=need):
        return L.tq_attn_prefill_paged(plan, q, n_q, B, Hq, Hkv, cache, bt, mp, cu, ctx, window, kb, vb, f(scale), out,
                                       dt, ws, size, None)

    assert call(plan=None) == 1
    assert call(plan=p16.handle) == 2
    assert call(B=-1) == 1 and call(n_q=-1) == 1 and call(Hq=7) == 1 and call(Hkv=0) == 1 and call(mp=0) == 1
    assert call(window=-1) == 1 and call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(kb=1) == 2 and call(vb=5) == 2 and call(dt=2) == 2
    assert call(Hq=258, Hkv=2) == 2                                  # 129 heads a group
    assert call(cache=_cache(page_size=48)) == 2
    assert call(cache=_cache(n_pages=0)) == 1
    assert call(mp=1 << 25) == 2                                     # positions past 2^30
    assert call(n_q=1 << 30) == 2                                    # rows past int32
    assert call(B=0, q=None, out=None, ws=None) == 0 and call(n_q=0, q=None) == 0
    for name in ("q", "out", "bt", "cu", "ctx"):
        assert call(**{name: None}) == 1
        assert call(**{name: A + 2}) == 3
    assert call(q=A + 8) == 3 and call(out=A + 8) == 3
    assert call(cache=abi.PagedCacheView(1 << 32, (1 << 33) + 4, 1 << 34, 1 << 35, 4, 64)) == 3  # norms: 16 bytes
    assert call(ws=None) == 5 and call(size=need - 1) == 5 and call(ws=W + 8) == 3
    # q, out and the workspace lie apart
    assert call(out=A) == 1 and call(out=A + 10 * 8 * 128 * 2 - 16) == 1 and call(q=W + need - 16) == 1
    assert call(out=W - 16, q=1 << 40) == 1 and call(out=W + 16, q=1 << 40) == 1


def test_prefill_paged_python_refusals():
    """Shapes and ranges that would not fit into the call are refused before it."""
    import torch
    plan = abi.Plan(128, 42)
    q, i32 = torch.zeros(3, 4, 128, dtype=torch.bfloat16), lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    norm = lambda *s: torch.zeros(*s, dtype=torch.float32)  # noqa: E731
    byte = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    good = abi.PagedCache(byte(4, 2, 32, 64), norm(4, 2, 32), byte(4, 2, 32, 48), norm(4, 2, 32), 4, 3)

    def call(cache=good, window=0, q=q, cu=i32(3), table=i32(2, 4), ctx=i32(2)):
        return abi.tq_attn_prefill_paged(plan, q, cu, cache, table, ctx, 0.1, window=window)

    for bad in (abi.PagedCache(byte(4, 2, 32, 64), norm(4, 2, 32), byte(4, 2, 32, 64), norm(4, 2, 32), 4, 3),
                abi.PagedCache(byte(4, 2, 32, 64), norm(4, 2, 32), byte(3, 2, 32, 48), norm(3, 2, 32), 4, 3),
                abi.PagedCache(byte(4, 2, 32, 48), norm(4, 2, 32), byte(4, 2, 32, 48), norm(4, 2, 32), 4, 3),
                abi.PagedCache(byte(4, 2, 32, 64), norm(4, 2, 32), byte(4, 2, 32, 48), norm(4, 2, 31), 4, 3)):
        with pytest.raises(ValueError):
            call(bad)
    for window in (-1, 1 << 31, (1 << 32) + 5):
        with pytest.raises(ValueError):
            call(window=window)
    for kw in (dict(cu=i32(2)), dict(table=i32(3, 4)), dict(q=q[..., :64])):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(TypeError):
        call(q=q.float())
    with pytest.raises(TypeError):
        call(abi.PagedCache(good.k_packed, good.k_norm.half(), good.v_packed, good.v_norm, 4, 3))


def test_pages_and_pools_past_the_kernels_counters_are_refused(L):
    """Sizes whose products leave 64 bits, and pools whose page numbers leave 32 bits in a loop's step."""
    A, W = 1 << 20, 1 << 28
    tab = lambda a: abi.PageTableView(a, a + 4096, a + 8192)  # noqa: E731

    def fork(cache, hkv, d=128, kb=4, vb=3):
        return L.tq_pages_fork(tab(A), A + (1 << 18), tab(A + (1 << 16)), 4, 1, _layers(cache), 1, hkv, d, kb, vb,
                               A + (1 << 19), W, 64, None)

    def copy(cache, hkv, d=128):
        return L.tq_pages_copy(_layers(cache), _layers(cache), 1, hkv, d, 4, 3, A, A + 4096, 0, None, 0, None)

    for hkv, page in ((1 << 30, 1 << 30), ((1 << 31) - 1, 1 << 30), (1 << 29, 1 << 30), (1 << 24, 1 << 5), (1, 1 << 24)):
        for d in (32, 64, 128, 256):
            if hkv * page * (d + 16) <= 1 << 31:
                continue
            assert fork(_cache(page_size=page), hkv, d) == 2, (hkv, page, d)
            assert copy(_cache(page_size=page), hkv, d) == 2, (hkv, page, d)
    assert copy(_cache(page_size=64), 8) == 0
    # the largest page of 32-bit counters passes, a size further does not
    most = (1 << 31) // ((128 + 16) * 64)
    assert copy(_cache(page_size=64), most) == 0 and copy(_cache(page_size=64), most + 1) == 2
    for n in ((1 << 30) + 1, (1 << 31) - 8000, (1 << 31) - 1):
        assert fork(_cache(n_pages=n), 2) == 1
        assert copy(_cache(n_pages=n), 2) == 1
        assert L.tq_pages_workspace_bytes(4, 8, n) == 0
    assert L.tq_pages_workspace_bytes(4, 8, 1 << 30) > 0 and copy(_cache(n_pages=1 << 30), 2) == 0


def test_reported_values_from_many_threads(monkeypatch):
    """No two calls get one tensor, and none finds the list empty that another thread emptied."""
    import threading

    import torch
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False, raising=False)
    monkeypatch.setattr(abi, "_FRESH", {})
    dev, out, wrong = torch.device("cpu"), [], []

    def take(n):
        try:
            for _ in range(700):
                out.append(abi._fresh(dev, 0, n))
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=take, args=(n,)) for n in (2, 2, 2, 2, 5, 70000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and len({t.data_ptr() for t in out}) == len(out) == 6 * 700

    class Emptied(list):  # between the look and the taking
        def __bool__(self):
            return True

    abi._FRESH[dev.index, 0, 2] = Emptied()
    assert abi._fresh(dev, 0, 2).shape == (2,)
