"""Trees and sinks over rows of V norm 0, in batches of few query rows: a row
whose best score belongs to a position without a value, far above every position
with one, and whole chunks without values after that.  The weights of the values
that are left are below 2^-128 of the best one's; the result is finite, and
nearly 0.

Against the attention in 64 bits, with the tolerance of test_gpu_tree_sinks.py."""
import math

import numpy as np
import pytest
import torch

from kv_cache_vector_gb300 import abi
from oracle import oracle as O
from test_gpu_prefill_paged import Batch
from test_gpu_tree_sinks import run_sinks, run_tree

pytestmark = pytest.mark.gpu
LEAD = 150 * math.log(2.0)  # of the best score, in nats


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_cache_vector_gb300 import build
    build.build()
    abi.lib()
    abi.tq_device_status(reset=True)


def put(bt, b, i, values):
    """Entries (0 packed K, 1 K norms, 2 packed V, 3 V norms) of all positions of sequence b, [Hkv, ctx, ..]."""
    bt.rows[b][i][:] = values
    pos = np.arange(values.shape[1])
    pages, off = bt.bt_host[b, pos // bt.page][:, None], (pos % bt.page)[:, None]
    bt.arrays[("kp", "kn", "vp", "vn")[i]][pages, np.arange(bt.Hkv)[None], off] = np.swapaxes(bt.rows[b][i], 0, 1)


def leading(lens, Hkv, d, best, v_norms):
    """A batch whose rows all share one query, with the scale under which position `best`
    (K along the query) leads by LEAD; v_norms: a norm for each position."""
    bt = Batch(61, lens, Hkv, Hkv, d, 128, 4, 4)
    q = bt.q.float()
    q[:] = q[:1, :1]
    bt.q = q.to(torch.bfloat16)
    along = bt.q[0, 0].double().numpy()
    row, _ = O.encode(bt.s, 4, along[None])
    gap = math.inf
    for b, (_, c) in enumerate(lens):
        packed, norms = bt.rows[b][0].copy(), np.full((Hkv, c), 0.01, np.float32)
        packed[:, best], norms[:, best] = row[0], 0.3
        put(bt, b, 0, packed)
        put(bt, b, 1, norms)
        put(bt, b, 3, np.broadcast_to(np.asarray(v_norms(c), np.float32), (Hkv, c)))
        s = bt.decoded(b)[0] @ along
        gap = min(gap, float((s[:, best] - np.delete(s, best, axis=1).max(1)).min()))
    return bt, LEAD / gap


def values_until(first, best):
    """V norms of 2^-60 at positions below `first` other than `best`, 0 at the others."""
    return lambda c: [2.0 ** -60 if j < first and j != best else 0.0 for j in range(c)]


def chain(lens):
    return [np.tril(np.ones((n, n), bool)) for n, _ in lens]


# one sequence, whose items are taken whole, and batches of which a CTA takes several items
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("lens,Hkv", [([(1, 600)], 1), ([(4, 380)], 2), ([(1, 900)] * 24, 8), ([(10, 900)] * 24, 8)])
def test_chunks_without_values_behind_a_lead(lens, Hkv, d):
    bt, scale = leading(lens, Hkv, d, 5, values_until(128, 5))
    run_sinks(bt, scale, 0, 0)
    run_sinks(bt, scale, 220, 64)
    run_tree(bt, scale, chain(lens))


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("many,base", [(False, 256), (False, 384), (True, 256), (True, 672)])
def test_nodes_without_values_that_are_not_attended_to(many, base, d):
    """The draft's own rows have no values, and some tokens or all attend to none of them; the
    pages' tails are rows of norm 0."""
    lens = [(6, base + 6)] * (24 if many else 1)
    bt, scale = leading(lens, 8 if many else 1, d, 5, values_until(base, 5))
    for norms in (bt.arrays["kn"], bt.arrays["vn"]):
        norms[np.isnan(norms)] = 0.0
    some = np.eye(6, dtype=bool)
    some[1] = some[4] = False
    for sees in (some, np.zeros((6, 6), bool)):
        run_tree(bt, scale, [sees] * len(lens))


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("many,best", [(False, 260), (False, 390), (True, 260), (True, 390)])
def test_a_lead_that_comes_in_a_chunk_without_values(many, best, d):
    lens = [(3, 560)] * (24 if many else 1)
    bt, scale = leading(lens, 8 if many else 1, d, best, values_until(128, best))
    run_sinks(bt, scale, 0, 0)
    run_tree(bt, scale, chain(lens))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_pages_out_of_range_behind_a_lead(d):
    """They count as rows of norm 0."""
    lens = [(2, 600)] * 24
    bt, scale = leading(lens, 8, d, 5, values_until(600, 5))
    for j in (3, 4):
        bt.bt_host[:, j] = bt.n_pages + j
    out = abi.tq_attn_sinks_paged(*bt.gpu(), scale, 0, 0, out_dtype=torch.float32)
    assert abi.tq_device_status(reset=True) == 72
    assert out.isfinite().all() and out.abs().max() < 2.0 ** -60


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("many", [False, True])
def test_a_value_behind_chunks_without_any(many, d):
    """Of 2^-150 of the weight, but 2^150 of the others' values."""
    lens = [(2, 560)] * (24 if many else 1)
    bt, scale = leading(lens, 8 if many else 1, d, 5,
                        lambda c: [2.0 ** 80 if j == 520 else 2.0 ** -70 if j < 128 and j != 5 else 0.0 for j in range(c)])
    run_sinks(bt, scale, 0, 0)
    run_tree(bt, scale, chain(lens))
