"""tq_attn_tree_paged and tq_attn_sinks_paged against the attention in 64 bits
over the oracle's decoded rows.

Tolerance: that of tq_attn_prefill_paged (test_gpu_prefill_paged.py): the kernels
round at most the same four factors of every product to fp16."""
import math

import numpy as np
import pytest
import torch

from kv_cache_vector_gb300 import abi
from test_gpu_prefill_paged import Batch, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_cache_vector_gb300 import build
    build.build()
    abi.lib()
    abi.tq_device_status(reset=True)


def random_trees(rng, lens):
    """Parents of each sequence's nodes, and the masks that follow from them."""
    parents = [[-1 if i == 0 or rng.random() < 0.1 else int(rng.integers(max(0, i - 6), i)) for i in range(n)]
               for n, _ in lens]
    sees = []
    for tree in parents:
        m = np.zeros((len(tree), len(tree)), bool)
        for i, p in enumerate(tree):
            if p >= 0:
                m[i] = m[p]
            m[i, i] = True
        sees.append(m)
    return parents, sees


def pack(sees, words, n_q):
    """[n_q, words] int32 mask rows, random bits past each sequence's nodes."""
    rng = np.random.default_rng(5)
    bits = rng.random((n_q, 32 * words)) < 0.5
    at = 0
    for m in sees:
        bits[at:at + len(m), :len(m)] = m
        at += len(m)
    return torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy())


def want(bt, scale, seen):
    """(attention, per-row S, per-row V) with seen[b] [n, ctx]."""
    q = bt.q.double().numpy()
    out, S, V = np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    G = bt.Hq // bt.Hkv
    for b, (n, c) in enumerate(bt.lens):
        if not n or not c:
            continue
        k, v = bt.decoded(b)
        some = seen[b].any(1)
        rows = slice(bt.cu[b], bt.cu[b + 1])
        for h in range(bt.Hq):
            kk, vv, qq = k[h // G], v[h // G], q[rows, h]
            bad = ~(np.isfinite(kk).all(1) & np.isfinite(vv).all(1))
            s = np.where(seen[b], qq @ np.where(np.isfinite(kk), kk, 0.0).T * scale, -np.inf)
            p = np.exp(s - np.where(some, s.max(1, initial=-np.inf), 0.0)[:, None])
            p /= np.where(some, p.sum(1), 1.0)[:, None]
            o = p @ np.where(np.isfinite(vv), vv, 0.0)
            o[(seen[b] & bad).any(1)] = np.nan
            out[rows, h] = o
            kn, vn = (np.where(bad, 0.0, np.linalg.norm(x, axis=1)) for x in (kk, vv))
            S[rows, h] = abs(scale) * np.linalg.norm(qq, axis=1) * np.where(seen[b], kn, 0.0).max(1, initial=0.0) / \
                math.sqrt(bt.d)
            V[rows, h] = np.where(seen[b], vn, 0.0).max(1, initial=0.0) / math.sqrt(bt.d)
    return out, S, V


def tree_seen(bt, sees):
    return [np.concatenate([np.ones((n, c - n), bool), m], 1) if c >= n else np.zeros((n, c), bool)
            for (n, c), m in zip(bt.lens, sees)]


def sinks_seen(bt, window, sinks):
    seen = []
    for n, c in bt.lens:
        p, j = np.arange(c - n, c)[:, None], np.arange(c)
        seen.append((j <= p) & ((j > p - (window or 1 << 40)) | (j < sinks)))
    return seen


def run(bt, scale, seen, fn, *more):
    """Both output types against the reference; they are the same values, rounded."""
    args = bt.gpu()
    n = int(bt.cu[-1])
    ref = want(bt, scale, seen)
    o32 = fn(*args, *more, out_dtype=torch.float32)
    o16 = fn(*args, *more)
    torch.cuda.synchronize()
    assert abi.tq_device_status(reset=True) == 0
    check(o32, *ref, n, bf16=False)
    check(o16, *ref, n)
    assert torch.equal(o32.to(torch.bfloat16).nan_to_num(7.0), o16.nan_to_num(7.0))
    return o16


def run_tree(bt, scale, sees, words=None):
    words = words or 1 + (max([len(m) for m in sees] + [1]) - 1) // 32
    mask = pack(sees, words, bt.q.shape[0]).cuda()
    return run(bt, scale, tree_seen(bt, sees), abi.tq_attn_tree_paged, mask, scale)


def run_sinks(bt, scale, window, sinks):
    return run(bt, scale, sinks_seen(bt, window, sinks), abi.tq_attn_sinks_paged, scale, window, sinks)


TREES = [
    # (nodes, context) lengths, Hq, Hkv, page, kb, vb, words
    ([(1, 1)], 1, 1, 32, 4, 4, 1),
    ([(7, 300), (3, 33), (1, 129), (0, 64)], 32, 8, 64, 4, 3, None),
    ([(5, 5), (31, 40), (32, 32), (33, 161)], 8, 2, 64, 3, 2, 3),        # hardly any context, nodes in two blocks
    ([(24, 1024), (16, 1000), (9, 2060)], 32, 8, 256, 4, 3, None),
    ([(64, 700), (65, 131), (20, 128)], 12, 4, 32, 2, 4, None),          # three heads a group
    ([(40, 290), (3, 1000)], 40, 2, 32, 4, 2, None),                     # twenty
    ([(128, 500), (2, 77)], 8, 1, 128, 3, 3, 7),                         # many rows, mask rows with room
    ([(300, 600)], 4, 1, 64, 4, 4, None),
    ([(3, 9000)], 8, 1, 256, 4, 3, None),                                # one item over all SMs
]


@pytest.mark.parametrize("d", [128, 64, 256, 32])
@pytest.mark.parametrize("lens,Hq,Hkv,page,kb,vb,words", TREES)
def test_trees(lens, Hq, Hkv, page, kb, vb, words, d):
    bt = Batch(21, lens, Hq, Hkv, d, page, kb, vb)
    run_tree(bt, 1 / math.sqrt(d), random_trees(np.random.default_rng(3), lens)[1], words)


@pytest.mark.parametrize("d", [128, 256])
def test_any_mask_and_rows_that_attend_to_nothing(d):
    """Bits need not be a tree's; a token need not see itself; with nothing in
    front of the tokens an empty row is zero."""
    lens = [(20, 20), (40, 170), (130, 130), (3, 3)]
    bt = Batch(22, lens, 8, 2, d, 32, 4, 3)
    rng = np.random.default_rng(4)
    sees = [rng.random((n, n)) < 0.3 for n, _ in lens]
    for m in sees:
        m[1] = False
    sees[3][:] = False
    out = run_tree(bt, 0.1, sees)
    assert not out[1].any() and not out[190:193].any() and not out[61].any() and out[21].any()


def test_a_chain_is_the_causal_attention():
    bt = Batch(23, [(17, 400), (64, 64), (1, 2000)], 8, 2, 128, 64, 4, 3)
    sees = [np.tril(np.ones((n, n), bool)) for n, _ in bt.lens]
    out = run_tree(bt, 0.1, sees)
    args = bt.gpu()
    full = want(bt, 0.1, tree_seen(bt, sees))
    check(abi.tq_attn_prefill_paged(*args, 0.1), *full, int(bt.cu[-1]))
    assert (out.float() - abi.tq_attn_prefill_paged(*args, 0.1).float()).abs().max() <= 0.02 * out.float().abs().max()


SINKS = [
    # (query, context) lengths, Hq, Hkv, page, kb, vb, window, sinks
    ([(1, 1)], 1, 1, 32, 4, 4, 16, 4),
    ([(1, 129), (1, 128), (1, 127), (1, 2300)], 8, 2, 64, 4, 3, 100, 4),     # single tokens
    ([(1, 5000)] * 20, 32, 8, 256, 4, 3, 1000, 4),
    ([(5, 700), (3, 33), (0, 64), (7, 7)], 32, 8, 64, 4, 3, 50, 1),
    ([(130, 130), (64, 1200), (257, 900)], 8, 2, 256, 3, 2, 200, 37),
    ([(100, 600), (1, 2000)], 12, 4, 32, 2, 4, 128, 128),                    # sinks of whole blocks
    ([(33, 395), (200, 500)], 5, 1, 128, 3, 3, 5, 131),
    ([(40, 700), (3, 290)], 40, 2, 32, 4, 2, 1, 3),                          # a window of one position
    ([(300, 1000), (1, 513), (20, 20)], 4, 4, 64, 4, 4, 100, 600),           # sinks into and past the window
    ([(9, 4), (4, 4), (3, 0)], 4, 2, 32, 4, 3, 3, 2),                        # more tokens than positions
    ([(129, 1290), (2, 640)], 2, 1, 64, 2, 2, 64, 0),                        # no sinks
    ([(129, 1290), (2, 640)], 2, 1, 64, 2, 2, 0, 9),                         # no window
    ([(3, 400), (2, 640)], 8, 2, 64, 4, 3, 4000, 2 ** 31 - 1),
    ([(1, 9000), (1, 8000)], 8, 1, 256, 4, 3, 7000, 4),                      # over all SMs
]


@pytest.mark.parametrize("d", [128, 64, 256, 32])
@pytest.mark.parametrize("lens,Hq,Hkv,page,kb,vb,window,sinks", SINKS)
def test_sinks(lens, Hq, Hkv, page, kb, vb, window, sinks, d):
    run_sinks(Batch(24, lens, Hq, Hkv, d, page, kb, vb), 1 / math.sqrt(d), window, sinks)


@pytest.mark.parametrize("seed", range(6))
def test_seeded_sweep(seed):
    rng = np.random.default_rng(seed)
    d = int(rng.choice([32, 64, 128, 256]))
    Hkv = int(rng.choice([1, 2, 3]))
    G, page = int(rng.choice([1, 2, 3, 4, 7, 8])), int(rng.choice([32, 64, 128]))
    B = int(rng.integers(1, 30))
    n = np.minimum(rng.integers(0, 50, B), rng.integers(1, 60, B))
    lens = [(int(x), int(x + c)) for x, c in zip(n, (10 ** rng.uniform(0, 3.2, B)).astype(int))]
    kb, vb = int(rng.integers(2, 5)), int(rng.integers(2, 5))
    bt = Batch(seed + 30, lens, G * Hkv, Hkv, d, page, kb, vb)
    run_sinks(bt, 1 / math.sqrt(d), int(rng.integers(1, 400)), int(rng.integers(0, 200)))
    run_tree(bt, 1 / math.sqrt(d), random_trees(rng, lens)[1])


# Batches of few query rows (16 and fewer per sequence and KV head) and of more
# go to different kernels.
few_and_more = pytest.mark.parametrize("lens", [[(9, 700), (2, 1300)], [(40, 700), (2, 1300)]], ids=["few", "more"])


@few_and_more
@pytest.mark.parametrize("flags", [1, 2, 3])
@pytest.mark.parametrize("d", [32, 128, 256])
def test_plan_variants(d, flags, lens):
    bt = Batch(25, lens, 8, 4, d, 64, 3, 3, flags=flags)
    run_sinks(bt, 1 / math.sqrt(d), 70, 5)
    run_tree(bt, 1 / math.sqrt(d), random_trees(np.random.default_rng(1), bt.lens)[1])


@few_and_more
@pytest.mark.parametrize("scale", [-0.3, 0.0, 0.02, 0.5])
def test_scales(scale, lens):
    bt = Batch(26, lens, 4, 2, 128, 64, 4, 4)
    run_sinks(bt, scale, 70, 5)
    run_tree(bt, scale, random_trees(np.random.default_rng(1), bt.lens)[1])


@pytest.mark.parametrize("name,norm,qmul,scale", [
    ("log normal", lambda r, n: np.exp(2 * r.standard_normal(n)), 1.0, 0.01),
    ("tiny", lambda r, n: np.full(n, 2.0 ** -70), 1.0, 2.0 ** 67),
    ("huge", lambda r, n: np.full(n, 2.0 ** 70), 1.0, 2.0 ** -73),
    ("small queries", lambda r, n: np.ones(n), 2.0 ** -60, 2.0 ** 57),
    ("large queries", lambda r, n: np.ones(n), 2.0 ** 80, 2.0 ** -83),
    ("spread wide", lambda r, n: 2.0 ** r.integers(-80, 90, n), 1.0, 2.0 ** -90),
    ("falling blocks", lambda r, n: 2.0 ** (-(np.arange(n) // 64 % 40) / 4.0), 1.0, 0.1),
    ("zeros", lambda r, n: (r.random(n) < 0.5) * 1.0, 1.0, 0.1),
    ("all zero", lambda r, n: np.zeros(n), 1.0, 0.1),
])
@few_and_more
@pytest.mark.parametrize("d", [64, 128, 256])
def test_norms_of_all_sizes(name, norm, qmul, scale, d, lens):
    bt = Batch(27, lens, 4, 2, d, 64, 4, 4, norm=norm, qmul=qmul)
    run_sinks(bt, scale, 300, 6)
    run_tree(bt, scale, random_trees(np.random.default_rng(1), bt.lens)[1])


@pytest.mark.parametrize("n", [3, 40])
def test_sinks_and_window_of_very_different_norms(n):
    """Neither side's size takes bits from the other's, wherever a row's weight lies."""
    bt = Batch(28, [(n, 900)], 4, 1, 128, 64, 4, 4)
    for pos in range(4):
        bt.set_norm(0, "v", 0, pos, 2.0 ** 40)
        bt.set_norm(0, "k", 0, pos, 2.0 ** -40)
    run_sinks(bt, 0.5, 100, 4)
    for pos in range(4, 900):  # far larger ones that no row attends to
        if 4 <= pos < 700:
            bt.set_norm(0, "v", 0, pos, 2.0 ** 90)
            bt.set_norm(0, "k", 0, pos, 2.0 ** 90)
    run_sinks(bt, 0.5, 100, 4)


@pytest.mark.parametrize("which,value", [("k", np.nan), ("k", np.inf), ("v", np.nan), ("v", -np.inf), ("v", np.inf)])
@pytest.mark.parametrize("d", [128, 256])
def test_non_finite_norms_reach_only_the_tokens_that_attend(which, value, d):
    """Few rows: the last 5 tokens of one sequence and single ones of others."""
    lens = [(5, 200), (1, 300), (1, 90)]
    bt = Batch(40, lens, 4, 2, d, 64, 4, 3)
    bt.set_norm(0, which, 1, 134, value)  # leaves the window between the third and the fourth token
    bt.set_norm(1, which, 0, 200, value)  # between the sinks and the window
    bt.set_norm(2, which, 0, 3, value)    # a sink
    run_sinks(bt, 1 / math.sqrt(d), 64, 7)
    bt = Batch(40, lens, 4, 2, d, 64, 4, 3)
    bt.set_norm(0, which, 1, 197, value)  # node 2: its descendants alone
    run_tree(bt, 1 / math.sqrt(d), random_trees(np.random.default_rng(2), lens)[1])


@pytest.mark.parametrize("which,value", [("k", np.nan), ("k", np.inf), ("v", np.nan), ("v", -np.inf), ("v", np.inf)])
@pytest.mark.parametrize("d", [128, 256])
def test_non_finite_norms_reach_only_rows_that_attend(which, value, d):
    bt = Batch(29, [(60, 200), (14, 300)], 4, 2, d, 64, 4, 3)
    bt.set_norm(0, which, 1, 170, value)
    bt.set_norm(1, which, 0, 130, value)  # between the sinks and the window
    bt.set_norm(1, which, 0, 299, value)
    run_sinks(bt, 1 / math.sqrt(d), 64, 7)
    bt = Batch(29, [(60, 200), (14, 300)], 4, 2, d, 64, 4, 3)
    bt.set_norm(0, which, 1, 150, value)  # node 10: its descendants alone
    bt.set_norm(1, which, 1, 299, value)
    run_tree(bt, 1 / math.sqrt(d), random_trees(np.random.default_rng(2), bt.lens)[1])


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("d", [32, 128, 256])
def test_non_finite_queries_stay_in_their_row(value, d):
    bt = Batch(31, [(6, 200), (3, 500), (20, 260)], 4, 2, d, 64, 4, 3)
    args = bt.gpu()
    clean = abi.tq_attn_sinks_paged(*args, 0.1, 90, 4)
    bad = torch.zeros(clean.shape[:2], dtype=torch.bool)
    for row, h in ((0, 0), (7, 1), (8, 3), (20, 2), (28, 3)):
        args[1][row, h, d // 2 + 1] = value
        bad[row, h] = True
    out = abi.tq_attn_sinks_paged(*args, 0.1, 90, 4)
    assert abi.tq_device_status(reset=True) == 0
    assert out[bad.cuda()].isnan().all()
    assert torch.equal(out[~bad.cuda()], clean[~bad.cuda()])


def test_rows_outside_every_sequence_keep_their_values():
    bt = Batch(32, [(3, 90), (0, 0), (5, 5)], 4, 2, 128, 32, 4, 3, tail=4)
    bt.cu = bt.cu + 2
    args = bt.gpu()
    mask = torch.full((12, 1), -1, dtype=torch.int32, device="cuda")
    for dt in (torch.bfloat16, torch.float32):
        for call in (lambda o: abi.tq_attn_sinks_paged(*args, 0.1, 20, 2, out=o),
                     lambda o: abi.tq_attn_tree_paged(*args, mask, 0.1, out=o)):
            out = torch.full(bt.q.shape, 3.5, dtype=dt, device="cuda")
            assert call(out).data_ptr() == out.data_ptr()
            assert (out[:2] == 3.5).all() and (out[10:] == 3.5).all() and not (out[2:10] == 3.5).any()


def test_lengths_out_of_range_leave_the_sequence_out():
    bt = Batch(33, [(4, 60), (40, 60), (4, 60)], 4, 2, 128, 32, 4, 3)
    plan, q, cu, cache, table, ctx = bt.gpu()
    seen = sinks_seen(bt, 30, 3)
    ref = want(bt, 0.1, seen)
    keep = [*range(4), *range(44, 48)]
    x = torch.tensor([60, 97, 60], dtype=torch.int32).cuda()
    out = abi.tq_attn_sinks_paged(plan, q, cu, cache, table, x, 0.1, 30, 3, out=torch.full(q.shape, 3.5, device="cuda"))
    assert abi.tq_device_status(reset=True) == 71
    assert (out[4:44] == 3.5).all()
    check(out[keep], *(r[keep] for r in ref), 8, bf16=False)
    # trees: more nodes than bits, more nodes than positions
    sees = [np.eye(n, dtype=bool) for n, _ in bt.lens]
    ref = want(bt, 0.1, tree_seen(bt, sees))
    for words, lens in ((1, [60, 60, 60]), (2, [60, 39, 60])):
        mask = pack(sees, 2, 48)[:, :words].contiguous().cuda()
        x = torch.tensor(lens, dtype=torch.int32).cuda()
        out = abi.tq_attn_tree_paged(plan, q, cu, cache, table, x, mask, 0.1, out=torch.full(q.shape, 3.5, device="cuda"))
        assert abi.tq_device_status(reset=True) == 75
        assert (out[4:44] == 3.5).all()
        check(out[keep], *(r[keep] for r in ref), 8, bf16=False)


@pytest.mark.parametrize("n", [5, 20])
@pytest.mark.parametrize("d", [128, 256])
def test_bad_pages_count_as_zero_rows_and_pages_between_are_not_read(n, d):
    bt = Batch(34, [(6, 300), (n, 900)], 4, 2, d, 64, 4, 3)
    for b, j, page in ((0, 1, -5), (1, 13, bt.n_pages), (1, 0, -1)):
        bt.bt_host[b, j] = page
        for which in "kv":
            bt.rows[b][1 if which == "k" else 3][:, 64 * j:64 * j + 64] = 0.0
    bt.bt_host[1, 2:10] = 1 << 30  # between the sinks and the window
    args = bt.gpu()
    out = abi.tq_attn_sinks_paged(*args, 0.1, 200, 70, out_dtype=torch.float32)
    assert abi.tq_device_status(reset=True) == 72
    check(out, *want(bt, 0.1, sinks_seen(bt, 200, 70)), 6 + n, bf16=False)
    bt.bt_host[1, 2:10] = bt.bt_host[1, 11]
    bt.bt_host[1, 0] = bt.bt_host[1, 11]
    bt.bt_host[1, 13] = bt.bt_host[1, 11]
    bt.bt_host[0, 1] = bt.bt_host[0, 2]
    args = bt.gpu()
    abi.tq_attn_sinks_paged(*args, 0.1, 200, 70)
    assert abi.tq_device_status(reset=True) == 0


@pytest.mark.parametrize("nodes", [(30, 1, 17), (5, 1, 6)])
def test_repeats_streams_and_graphs_give_the_same_bits(nodes):
    bt = Batch(35, list(zip(nodes, (900, 3000, 64))), 8, 2, 128, 64, 4, 3)
    args = bt.gpu()
    sees = random_trees(np.random.default_rng(1), bt.lens)[1]
    mask = pack(sees, 1, sum(nodes)).cuda()
    ws = [torch.empty(abi.tq_attn_tree_paged_workspace_bytes(8, 2, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    for call in (lambda **k: abi.tq_attn_tree_paged(*args, mask, 0.1, **k),
                 lambda **k: abi.tq_attn_sinks_paged(*args, 0.1, 500, 4, **k)):
        first = call()
        for _ in range(3):
            assert torch.equal(call(), first)
        outs = [torch.empty_like(first) for _ in range(2)]
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(5):  # two calls at once, a workspace each
            call(out=outs[0], workspace=ws[0])
            with torch.cuda.stream(side):
                call(out=outs[1], workspace=ws[1])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], first) and torch.equal(outs[1], first)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call(out=outs[0], workspace=ws[0])
        for lens in ([900, 3000, 64], [800, 2000, 63]):  # the captured call follows the lengths
            args[5].copy_(torch.tensor(lens, dtype=torch.int32))
            eager = call()
            outs[0].zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[0], eager)
        args[5].copy_(torch.tensor([900, 3000, 64], dtype=torch.int32))
    assert abi.tq_device_status(reset=True) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 12])
def test_values_lost_in_a_probability_that_count(d, n):
    """A score far below the largest whose V norm makes it count: 2^-140 of the weight, 2^150 of
    the value; and beside it a row whose largest weight has no value at all."""
    bt = Batch(41, [(n, 400), (1, 100)], 2, 1, d, 32, 4, 4, qmul=1.0)
    q = bt.q.float()
    q[:] = q[:1, :1]  # one query: the keys below are along it or against it
    bt.q = q.to(torch.bfloat16)
    k = bt.decoded(0)[0][0] @ bt.q[0, 0].double().numpy()
    for j in range(400):
        bt.set_norm(0, "k", 0, j, 0.1)
        bt.set_norm(0, "v", 0, j, 2.0 ** -60)
    top, low = int(np.argmax(k[:380])), int(np.argmin(k[:380]))
    bt.set_norm(0, "k", 0, top, 30.0)
    bt.set_norm(0, "k", 0, low, 30.0)
    k = bt.decoded(0)[0][0] @ bt.q[0, 0].double().numpy()
    scale = 97.0 / (k[top] - k[low])  # nats: 2^-140
    bt.set_norm(0, "v", 0, low, 2.0 ** 90)
    run_sinks(bt, scale, 390, 400)
    bt.set_norm(0, "v", 0, top, 0.0)
    run_sinks(bt, scale, 390, 400)
    bt.set_norm(0, "v", 0, low, 0.0)
    run_sinks(bt, scale, 390, 400)


def test_a_window_past_every_length_and_none():
    """Of few rows too, up to the largest window."""
    bt = Batch(42, [(1, 700), (3, 129), (1, 40)], 8, 2, 128, 64, 4, 3)
    out = run_sinks(bt, 0.1, 0, 4)
    for window in (700, 2 ** 20, 2 ** 30 + 5, 2 ** 31 - 1):
        assert torch.equal(run_sinks(bt, 0.1, window, 4), out)
        assert torch.equal(run_sinks(bt, 0.1, window, 0), out)


def test_arrays_of_more_than_4_gib():
    """Pages at the end of a pool whose arrays pass 2^32 bytes: appended to, attended to, kept."""
    page, Hkv, d, n_pages = 256, 8, 128, 36000
    c = abi.PagedCache.empty(n_pages, Hkv, page, d, 4, 4)
    assert c.k_packed.numel() > 2 ** 32 and c.v_packed.numel() > 2 ** 32
    small = abi.PagedCache.empty(4, Hkv, page, d, 4, 4)
    plan, g = abi.Plan(d, 42), torch.Generator(device="cuda").manual_seed(3)
    k, v = torch.randn(2, 700, Hkv, d, generator=g, device="cuda")
    q = torch.randn(5, 32, d, generator=g, device="cuda").to(torch.bfloat16)
    cu, ctx = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 5], [700]))
    mask = torch.full((5, 1), 29, dtype=torch.int32, device="cuda")
    outs = []
    for cache, first in ((c, n_pages - 4), (small, 0)):
        bt = torch.arange(first, first + 3, dtype=torch.int32, device="cuda")[None]
        refs = torch.ones(cache.n_pages, dtype=torch.int32, device="cuda")
        table = abi.PageTable(bt, ctx, refs)
        m = abi.tq_pages_slots(table, ctx, 700, page)
        abi.tq_append_slots(plan, cache, k, v, m.slots)
        a = abi.tq_attn_tree_paged(plan, q, cu, cache, bt, ctx, mask, 0.1)
        b = abi.tq_attn_sinks_paged(plan, q[:1], cu.clamp(max=1), cache, bt, ctx, 0.1, 300, 4)
        five, keep = torch.tensor([5], dtype=torch.int32, device="cuda"), torch.tensor([[1, 3]], dtype=torch.int32, device="cuda")
        new = abi.tq_pages_keep(table, five, keep, keep[0, :1] + 1, cache)
        e = abi.tq_attn_sinks_paged(plan, q[:1], cu.clamp(max=1), cache, bt, new, 0.1, 300, 4)
        outs.append((m.positions, a, b, new, e))
    assert int(outs[0][3]) == 697 and abi.tq_device_status(reset=True) == 0
    assert all(torch.equal(x, y) for x, y in zip(*outs))


def test_refusals():
    bt = Batch(36, [(4, 60)], 4, 2, 128, 32, 4, 3)
    args = bt.gpu()
    mask = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        abi.tq_attn_tree_paged(*args, mask[:3], 0.1)
    with pytest.raises(ValueError):
        abi.tq_attn_tree_paged(*args, mask[:, 0], 0.1)
    with pytest.raises(TypeError):
        abi.tq_attn_tree_paged(*args, mask.long(), 0.1)
    with pytest.raises(ValueError):
        abi.tq_attn_tree_paged(*args, mask.cpu(), 0.1)
    with pytest.raises(ValueError):
        abi.tq_attn_tree_paged(*args, torch.zeros(4, 2, dtype=torch.int32, device="cuda")[:, :1], 0.1)
    with pytest.raises(abi.TQError):
        abi.tq_attn_tree_paged(*args, mask[:, :0], 0.1)
    with pytest.raises(ValueError):
        abi.tq_attn_sinks_paged(*args, 0.1, -1, 4)
    with pytest.raises(ValueError):
        abi.tq_attn_sinks_paged(*args, 0.1, 16, -4)
    with pytest.raises(TypeError):
        abi.tq_attn_sinks_paged(args[0], args[1].float(), *args[2:], 0.1, 16, 4)
    with pytest.raises(abi.TQError):
        abi.tq_attn_sinks_paged(*args, float("inf"), 16, 4)
    with pytest.raises(ValueError):
        abi.tq_attn_sinks_paged(*args, 0.1, 16, 4, out=torch.empty(3, 4, 128, device="cuda"))


@pytest.mark.parametrize("d", [128, 64, 256, 32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (130, 0), (250, 5), (200, 130), (256, 0)])
@pytest.mark.parametrize("lens,Hq,Hkv", [
    ([(1, 700)], 4, 1), ([(1, 3000), (1, 1), (1, 0), (1, 129), (0, 50)], 32, 8), ([(4, 900), (1, 256), (3, 3)], 32, 8),
    ([(1, 300 + 60 * i) for i in range(19)], 8, 8)])
def test_short_windows_of_few_rows(lens, Hq, Hkv, window, sinks, d):
    """Items that one CTA takes whole."""
    run_sinks(Batch(51, lens, Hq, Hkv, d, 64, 4, 3), 0.1, window, sinks)


@pytest.mark.parametrize("d", [128, 64, 256])
@pytest.mark.parametrize("lens,Hq,Hkv", [([(2, 9)], 2, 1), ([(7, 200), (1, 1), (0, 0), (3, 400), (5, 4 * 32)], 8, 8), ([(16, 300)], 1, 1)])
def test_trees_over_small_tables(lens, Hq, Hkv, d):
    rng = np.random.default_rng(52)
    bt = Batch(52, lens, Hq, Hkv, d, 32, 3, 4)
    run_tree(bt, 0.1, random_trees(rng, lens)[1])


@pytest.mark.parametrize("window", [100, 0])
def test_sequences_between_lengths_that_step_back(window):
    """cu_q 0 10 0 10 ...: every second sequence is out of range, and the others, of the same rows,
    are more items than the number of rows lets one expect; the first is there at least."""
    bt = Batch(53, [(10, 200)], 8, 2, 128, 32, 4, 3)
    plan, q, cu, cache, table, ctx = bt.gpu()
    ref = want(bt, 0.1, sinks_seen(bt, window, 3))
    n = 7
    cu = torch.tensor([0, 10] * ((n + 1) // 2), dtype=torch.int32).cuda()
    out = abi.tq_attn_sinks_paged(plan, q, cu, cache, table.repeat(n, 1), ctx.repeat(n), 0.1, window, 3,
                                  out_dtype=torch.float32)
    assert abi.tq_device_status(reset=True) == 71
    check(out, *ref, 10, bf16=False)
