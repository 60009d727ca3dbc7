"""tq_pages_keep refuses layers that share memory, and arguments inside the layers'
arrays: rows would be moved twice, or the lists moved over.  (No kernel is launched
here: `counts` is misaligned, which is refused later and with another code.)"""
import pytest

from kv_cache_vector_gb300 import abi

AT = 1 << 20          # a layer's arrays start so far apart: 8 pages of 2 x 64 rows of 64 bytes take 64 KB
BOOKS = 1 << 40


@pytest.fixture(scope="module")
def L():
    from kv_cache_vector_gb300 import build
    build.build()
    return abi.lib()


def layer(i, **kw):
    a = dict(k_packed=(4 * i + 1) * AT, k_norm=(4 * i + 2) * AT, v_packed=(4 * i + 3) * AT, v_norm=(4 * i + 4) * AT)
    a.update(kw)
    return abi.PagedCacheView(a["k_packed"], a["k_norm"], a["v_packed"], a["v_norm"], 8, 64)


def keep(L, layers, **kw):
    a = dict(bt=BOOKS, lens=BOOKS + AT, refs=BOOKS + 2 * AT, counts=BOOKS + 3 * AT + 2, keep=BOOKS + 4 * AT,
             n_keep=BOOKS + 5 * AT, new=BOOKS + 6 * AT)
    a.update(kw)
    views = (abi.PagedCacheView * len(layers))(*layers)
    return L.tq_pages_keep(abi.PageTableView(a["bt"], a["lens"], a["refs"]), 4, 8, a["counts"], a["keep"], 8,
                           a["n_keep"], a["new"], views, len(layers), 2, 128, 4, 4, None)


@pytest.mark.parametrize("n", [1, 2, 3, 64, 65, 130, 300])
def test_layers_apart_are_not_refused_for_that(L, n):
    layers = [layer(i) for i in range(n)]
    assert keep(L, layers) == 3 and keep(L, layers[::-1]) == 3
    # side by side, as slices of one tensor for each kind
    rows = [layer(0, k_packed=AT + 65536 * i, k_norm=64 * AT + 4096 * i, v_packed=128 * AT + 65536 * i,
                  v_norm=256 * AT + 4096 * i) for i in range(n)]
    assert keep(L, rows) == 3


@pytest.mark.parametrize("n", [2, 3, 65, 130, 300])
@pytest.mark.parametrize("name,size", [("k_packed", 65536), ("k_norm", 4096), ("v_packed", 65536), ("v_norm", 4096)])
def test_an_array_of_two_layers(L, name, size, n):
    layers = [layer(i) for i in range(n)]
    at = getattr(layers[0], name)
    for shift in (0, 16, size - 16, -(size - 16)):
        for other in {1, n // 2, n - 1} - {0}:
            some = list(layers)
            some[other] = layer(other, **{name: at + shift})
            assert keep(L, some) == 1 and keep(L, some[::-1]) == 1
    some = list(layers)
    some[n - 1] = layer(n - 1, **{name: at + size})
    assert keep(L, some) == 3


def test_arrays_of_one_layer(L):
    assert keep(L, [layer(0, v_packed=AT)]) == 1
    assert keep(L, [layer(0), layer(1, v_norm=5 * AT + 32)]) == 1
    assert keep(L, [layer(0, k_norm=AT + 65536)]) == 3


@pytest.mark.parametrize("which", ["bt", "lens", "refs", "counts", "keep", "n_keep", "new"])
def test_arguments_inside_the_layers(L, which):
    odd = 2 if which == "counts" else 0
    for n, at in ((1, AT), (3, 7 * AT), (200, 799 * AT)):
        layers = [layer(i) for i in range(n)]
        for inside in (at, at + 40, at - 8):
            assert keep(L, layers, **{which: inside + odd}) == 1
        assert keep(L, layers, **{which: at + 65536 + odd}) == 3
