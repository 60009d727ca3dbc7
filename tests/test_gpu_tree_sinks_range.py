"""tq_attn_sinks_paged and tq_attn_tree_paged within the accuracy that the header
states, which knows what each token attends to and how much: the tolerance of
test_gpu_prefill_paged_range.py.

Batches of few rows round three factors of a product to fp16, not four: the query,
the level and P = p |V norm|; K's norm stays out of the products.  P of a position
whose p |V norm| is far below the row's largest is off by 2^-25 where the largest
is at least 2^7."""
import math

import numpy as np
import pytest
import torch

from kv_cache_vector_gb300 import abi, synth
from test_gpu_prefill_paged import SIGMA, Batch
from test_gpu_prefill_paged_range import set_rows
from test_gpu_tree_sinks import pack, random_trees, sinks_seen, tree_seen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_cache_vector_gb300 import build
    build.build()
    abi.lib()
    abi.tq_device_status(reset=True)


def reference(bt, scale, seen):
    """(attention in 64 bits, its tolerance), both [rows of q, Hq, d]."""
    q = bt.q.double().numpy()
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    G, rd = bt.Hq // bt.Hkv, math.sqrt(bt.d)
    for b, (n, c) in enumerate(bt.lens):
        k, v = bt.decoded(b) if n and c else (None, None)
        for t in range(n):
            on = seen[b][t]
            if not on.any():
                continue
            for h in range(bt.Hq):
                kk, vv, qq = k[h // G, on], v[h // G, on], q[bt.cu[b] + t, h]
                s = kk @ qq * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                o = p @ vv
                S = abs(scale) * np.linalg.norm(qq) * np.linalg.norm(kk, axis=1) / rd
                out[bt.cu[b] + t, h] = o
                tol[bt.cu[b] + t, h] = 6 * SIGMA * ((p * S) @ np.abs(vv - o) + (p @ np.linalg.norm(vv, axis=1)) / rd) + \
                    3 * 2.0 ** -11 * (p @ np.abs(vv))
    return out, tol


def compare(bt, scale, seen, fn, *more):
    args = bt.gpu()
    want, tol = reference(bt, scale, seen)
    for dt in (torch.float32, torch.bfloat16):
        got = fn(*args, *more, out_dtype=dt).double().cpu().numpy()
        assert abi.tq_device_status(reset=True) == 0
        over = np.abs(got - want) - tol - (np.abs(want) * 2.0 ** -8 if dt == torch.bfloat16 else 0.0)
        over = np.where(np.isnan(got), np.inf, over)
        at = np.unravel_index(np.argmax(over), over.shape)
        assert over[at] <= 0, (at, got[at], want[at], tol[at])
    return want


def both(bt, scale, window, sinks):
    want = compare(bt, scale, sinks_seen(bt, window, sinks), abi.tq_attn_sinks_paged, scale, window, sinks)
    sees = random_trees(np.random.default_rng(3), bt.lens)[1]
    words = 1 + (max(n for n, _ in bt.lens) - 1) // 32
    compare(bt, scale, tree_seen(bt, sees), abi.tq_attn_tree_paged, pack(sees, words, bt.q.shape[0]).cuda(), scale)
    return want


# 8 and 16 rows of a KV head in the kernel for few rows, and more than it takes
LENS = [[(1, 700), (2, 1900), (1, 130)], [(4, 700), (3, 300)], [(40, 700), (7, 300)]]


@pytest.mark.parametrize("lens", LENS, ids=["one tile", "two tiles", "many rows"])
@pytest.mark.parametrize("d,kb,vb", [(32, 4, 4), (64, 4, 4), (128, 4, 3), (256, 4, 4)])
def test_rows_with_outlier_channels(d, kb, vb, lens):
    """Correlated rows with a few channels eight times as large: sharp softmaxes over large values."""
    bt = Batch(81, lens, 8, 2, d, 64, kb, vb)
    for b, (_, c) in enumerate(lens):
        set_rows(bt, b, *(np.stack([synth.lowrank_rows(40 + which, c, d, stream=10 * b + h).double().numpy()
                                    for h in range(2)]) for which in (0, 1)))
    n = int(bt.cu[-1])
    bt.q = torch.stack([synth.lowrank_rows(42, n, d, stream=h) for h in range(8)], 1)
    want = both(bt, 1 / math.sqrt(d), 400, 4)
    assert np.abs(want).max() > 10


@pytest.mark.parametrize("seed", range(24))
def test_seeded_norms(seed):
    """Lengths, heads, pages, windows, widths and spreads of norms drawn together."""
    g = np.random.default_rng(2000 + seed)
    d = int(g.choice([32, 64, 128, 256]))
    Hkv, G = int(g.integers(1, 4)), int(g.choice([1, 2, 3, 4, 8]))
    most = int(g.choice([1, 2, 4, 16, 60]))
    lens = [(int(g.integers(1, most + 1)), 0) for _ in range(int(g.integers(1, 8)))]
    lens = [(n, n + int(g.choice([0, 1, 130, int(g.integers(0, 900))]))) for n, _ in lens]
    bt = Batch(seed, lens, Hkv * G, Hkv, d, int(g.choice([32, 64, 128])), int(g.integers(2, 5)), int(g.integers(2, 5)),
               flags=int(g.integers(0, 4)))
    ks, vs = (float(g.choice([0, 2, 9, 14, 30, 60])) for _ in range(2))
    vbase = float(g.integers(-30, 30))
    for b, (_, c) in enumerate(lens):
        for h in range(Hkv):
            for p in range(c):
                bt.set_norm(b, "k", h, p, math.sqrt(d) * 2.0 ** -(g.random() * ks))
                bt.set_norm(b, "v", h, p, 0.0 if g.random() < 0.05 else 2.0 ** (vbase + vs * (g.random() - 0.5)))
    both(bt, float(g.choice([1.0, -0.7, 0.3])) / math.sqrt(d), int(g.choice([0, 1, int(g.integers(1, 300)), 5000])),
         int(g.choice([0, 1, 4, int(g.integers(0, 200))])))
