"""The step operators' restatement on worked examples, and the refusals of their
C entries (no kernel is launched here)."""
import ctypes

import numpy as np
import pytest

from kv_cache_vector_gb300 import abi
from oracle import steps

TABLE = np.array([[3, 1, -1], [0, -1, -1], [2, 4, 5]], np.int32)


def test_slots_of_a_worked_example():
    cu, pos, slot, mask, status = steps.slots(TABLE, [40, 0, 96], [10, 0, 2], 32, 6, 14)
    assert status == 0 and mask is None
    assert cu.tolist() == [0, 10, 10, 12]
    assert pos.tolist() == [*range(30, 40), 94, 95, 0, 0]
    assert slot.tolist() == [3 * 32 + 30, 3 * 32 + 31, *range(32, 40), 5 * 32 + 30, 5 * 32 + 31, -1, -1]


def test_masks_of_a_worked_tree():
    #  0 - 1 - 3        row 2: two roots
    #   \- 2
    cu, pos, slot, mask, status = steps.slots(TABLE, [20, 0, 50], [4, 0, 2], 32, 6, 6, [-1, 0, 0, 1, -1, -1], 1)
    assert status == 0
    assert mask[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b1, 0b10]
    assert pos.tolist() == [16, 17, 17, 18, 48, 48]


@pytest.mark.parametrize("lens,counts,status", [([5, 0, 0], [6, 0, 0], 63), ([5, 0, 0], [-1, 0, 0], 63),
                                                ([97, 0, 0], [1, 0, 0], 63), ([50, 0, 0], [41, 0, 0], 63),
                                                ([70, 0, 0], [3, 0, 0], 64)])
def test_slots_out_of_range(lens, counts, status):
    cu, pos, slot, _, got = steps.slots(TABLE, lens, counts, 32, 6, 40)
    assert got == status
    if status == 63:
        assert not cu.any() and not pos.any() and (slot == -1).all()
    else:
        assert slot[:3].tolist() == [-1] * 3


def test_keep_of_a_worked_example():
    x = np.arange(6 * 32).reshape(6, 1, 32)
    new, (y,), status = steps.keep(TABLE, [40, 0, 96], [1] * 6, [10, 0, 4], np.array([[0, 3, 9], [0, 0, 0], [1, 2, 3]]),
                                   [3, 0, 3], 32, [x])
    assert status == 0 and new.tolist() == [33, 0, 95]
    assert y[3, 0, 30] == x[3, 0, 30] and y[3, 0, 31] == x[1, 0, 1] and y[1, 0, 0] == x[1, 0, 7]
    assert y[5, 0, 28:31].tolist() == x[5, 0, 29:32].tolist() and y[5, 0, 31] == x[5, 0, 31]


@pytest.mark.parametrize("kept,n_keep", [([1, 1], 2), ([2, 1], 2), ([0, 10], 2), ([-1, 3], 2), ([0, 1], 3), ([0, 1], -1)])
def test_keep_refuses_lists_out_of_order(kept, n_keep):
    x = np.arange(6 * 32).reshape(6, 1, 32)
    new, (y,), status = steps.keep(TABLE[:1], [40], [1] * 6, [10], np.array([kept]), [n_keep], 32, [x])
    assert status == 66 and new.tolist() == [40] and (x == y).all()


def test_keep_refuses_shared_pages():
    x = np.arange(6 * 32).reshape(6, 1, 32)
    new, (y,), status = steps.keep(TABLE[:1], [40], [1, 2, 1, 1, 1, 1], [10], np.array([[0, 4]]), [2], 32, [x])
    assert status == 66 and new.tolist() == [40] and (x == y).all()


# ---------------------------------------------------------------- C refusals

A16 = 1 << 20  # an aligned address that no call here reads


@pytest.fixture(scope="module")
def L():
    from kv_cache_vector_gb300 import build
    build.build()
    return abi.lib()


def _cache(**kw):
    c = abi.PagedCacheView(A16, 2 * A16, 3 * A16, 4 * A16, 8, 64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _table(**kw):
    t = abi.PageTableView(5 * A16, 6 * A16, 7 * A16)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _slots(L, **kw):
    a = dict(table=_table(), n_seqs=4, max_pages=8, n_pages=8, page=64, counts=8 * A16, parents=None, words=1, n=16,
             cu=9 * A16, pos=10 * A16, slots=11 * A16, mask=12 * A16)
    a.update(kw)
    return L.tq_pages_slots(a["table"], a["n_seqs"], a["max_pages"], a["n_pages"], a["page"], a["counts"], a["parents"],
                            a["words"], a["n"], a["cu"], a["pos"], a["slots"], a["mask"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=0), 1), (dict(max_pages=0), 1), (dict(n_pages=0), 1), (dict(n=-1), 1), (dict(counts=None), 1),
    (dict(cu=None), 1), (dict(pos=None), 1), (dict(slots=None), 1), (dict(table=_table(lens=None)), 1),
    (dict(parents=13 * A16, mask=None), 1), (dict(parents=13 * A16, words=0), 1), (dict(parents=13 * A16, words=33), 2),
    (dict(page=48), 2), (dict(page=16), 2), (dict(n_seqs=(1 << 18) + 1), 2), (dict(n=1 << 31), 2),
    (dict(max_pages=1 << 26), 2), (dict(slots=11 * A16 + 4), 3), (dict(cu=9 * A16 + 2), 3), (dict(cu=8 * A16), 1),
    (dict(pos=6 * A16 + 8), 1), (dict(slots=10 * A16 + 32), 1), (dict(parents=12 * A16 + 32), 1)])
def test_slots_refusals(L, kw, code):
    assert _slots(L, **kw) == code


def _keep(L, **kw):
    a = dict(table=_table(), n_seqs=4, max_pages=8, counts=8 * A16, keep=9 * A16, max_keep=8, n_keep=10 * A16,
             new=11 * A16, layer=_cache(), layers=1, Hkv=2, d=128, kb=4, vb=3)
    a.update(kw)
    return L.tq_pages_keep(a["table"], a["n_seqs"], a["max_pages"], a["counts"], a["keep"], a["max_keep"], a["n_keep"],
                           a["new"], ctypes.byref(a["layer"]), a["layers"], a["Hkv"], a["d"], a["kb"], a["vb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=0), 1), (dict(max_keep=0), 1), (dict(counts=None), 1), (dict(keep=None), 1), (dict(n_keep=None), 1),
    (dict(new=None), 1), (dict(layers=0), 1), (dict(Hkv=0), 1), (dict(table=_table(refs=None)), 1),
    (dict(layer=_cache(k_packed=None)), 1), (dict(d=16), 2), (dict(d=96), 2), (dict(kb=5), 2), (dict(vb=1), 2),
    (dict(layer=_cache(page_size=48)), 2), (dict(layer=_cache(k_norm=2 * A16 + 4)), 3), (dict(new=11 * A16 + 2), 3),
    (dict(new=6 * A16), 1), (dict(new=9 * A16 + 16), 1), (dict(new=7 * A16 + 4), 1)])
def test_keep_refusals(L, kw, code):
    assert _keep(L, **kw) == code


def test_keep_refuses_a_layer_given_twice(L):
    two = (abi.PagedCacheView * 2)(_cache(), _cache())
    a = (_table(), 4, 8, 8 * A16, 9 * A16, 8, 10 * A16, 11 * A16, two)
    assert L.tq_pages_keep(*a, 2, 2, 128, 4, 3, None) == 1


def _append(L, owner, **kw):
    a = dict(plan=owner.handle, kb=4, vb=3, k=8 * A16, ks=256, v=9 * A16, vs=256, dt=1, n=4, Hkv=2, cache=_cache(),
             slots=10 * A16)
    a.update(kw)
    return L.tq_append_slots(a["plan"], a["kb"], a["vb"], a["k"], a["ks"], a["v"], a["vs"], a["dt"], a["n"], a["Hkv"],
                             a["cache"], a["slots"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(plan=None), 1), (dict(n=-1), 1), (dict(Hkv=0), 1), (dict(k=None), 1), (dict(slots=None), 1), (dict(ks=255), 1),
    (dict(vs=0), 1), (dict(vs=-256), 1), (dict(kb=1), 2), (dict(dt=2), 2), (dict(cache=_cache(page_size=40)), 2),
    (dict(cache=_cache(n_pages=0)), 1), (dict(ks=257), 3), (dict(k=8 * A16 + 8), 3), (dict(slots=10 * A16 + 4), 3),
    (dict(n=0, k=None, v=None), 0)])
def test_append_slots_refusals(L, kw, code):
    assert _append(L, abi.Plan(128, 42), **kw) == code
    assert _append(L, abi.Plan(16, 42), ks=32, vs=32) == 2


def _tokens(L, owner, fn, sees, **kw):
    ws = getattr(L, fn + "_workspace_bytes")(8, 2, 128)
    a = dict(plan=owner.handle, q=20 * A16, n=4, B=2, Hq=8, Hkv=2, cache=_cache(), bt=5 * A16, mp=8, cu=6 * A16, ctx=7 * A16,
             kb=4, vb=3, scale=0.1, out=21 * A16, dt=1, ws=1 << 40, size=ws, seen=sees)
    a.update(kw)
    return getattr(L, fn)(a["plan"], a["q"], a["n"], a["B"], a["Hq"], a["Hkv"], a["cache"], a["bt"], a["mp"], a["cu"],
                          a["ctx"], *a["seen"], a["kb"], a["vb"], a["scale"], a["out"], a["dt"], a["ws"], a["size"], None)


COMMON = [
    (dict(plan=None), 1), (dict(q=None), 1), (dict(cu=None), 1), (dict(n=-1), 1), (dict(B=-1), 1), (dict(Hq=7), 1),
    (dict(scale=float("nan")), 1), (dict(mp=0), 1), (dict(kb=5), 2), (dict(dt=2), 2), (dict(Hq=129, Hkv=1), 2),
    (dict(cache=_cache(page_size=16)), 2), (dict(mp=1 << 25), 2), (dict(q=20 * A16 + 8), 3),
    (dict(cache=_cache(k_norm=2 * A16 + 4)), 3), (dict(size=64), 5), (dict(ws=None), 5), (dict(out=20 * A16), 1),
    (dict(n=0), 0), (dict(B=0), 0)]


@pytest.mark.parametrize("kw,code", COMMON + [(dict(seen=(-1, 4)), 1), (dict(seen=(16, -1)), 1)])
def test_sinks_refusals(L, kw, code):
    assert _tokens(L, abi.Plan(128, 42), "tq_attn_sinks_paged", (16, 4), **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(seen=(None, 1)), 1), (dict(seen=(22 * A16, 0)), 1), (dict(seen=(22 * A16, 33)), 2),
    (dict(seen=(22 * A16 + 2, 1)), 3), (dict(seen=(21 * A16 + 64, 1)), 1), (dict(seen=((1 << 40) + 64, 1)), 1)])
def test_tree_refusals(L, kw, code):
    assert _tokens(L, abi.Plan(128, 42), "tq_attn_tree_paged", (22 * A16, 1), **kw) == code


def test_head_dimensions(L):
    for fn, seen in (("tq_attn_sinks_paged", (16, 4)), ("tq_attn_tree_paged", (22 * A16, 1))):
        assert _tokens(L, abi.Plan(16, 42), fn, seen) == 2
        size = getattr(L, fn + "_workspace_bytes")
        assert size(8, 2, 96) == 0 and size(7, 2, 128) == 0 and size(0, 2, 128) == 0
