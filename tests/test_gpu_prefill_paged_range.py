"""tq_attn_prefill_paged over norms of every size, with a tolerance that comes
from what each token attends to and how much.

Tolerance.  Four roundings to fp16 per product, SIGMA = 2 * 2^-11 / sqrt(3) in
the root mean square (each at most eps / 2 = 2^-11 relative).  A score's error
has at most the standard deviation SIGMA S_j, S_j = scale |q| |k_j| / sqrt(d),
and moves element i of the output by p_j S_j SIGMA |v_ji - out_i|; the second
product's roundings by SIGMA p_j |v_j| / sqrt(d), as the rotation spreads them
over the row.  The deviations are added up as if they were all of one sign, and
taken six times:
  6 SIGMA sum_j p_j (S_j |v_ji - out_i| + |v_j| / sqrt(d)).
Three of the second product's roundings may be the same for all coordinates of a
position, and then scale it instead: of the probability, of the norm, and of the
levels, which at 2 bits are of only two sizes.  Each is at most half a step, 2^-11:
  + 3 * 2^-11 sum_j p_j |v_ji|.
(A row of a single position, d = 64, 2 bits: all its elements off by 9.1e-4 of
themselves, of which the first sum allows 3.4e-3 |v| / sqrt(d), less than that for an
element of four times the mean size.)
Probabilities that leave fp16's normal range are off by 2^-25 where the largest
is at least 2^-8, less than a thousandth of the second term at these lengths.
No term knows a position that the token does not attend to."""
import math

import numpy as np
import pytest
import torch

from kv_cache_vector_gb300 import abi, synth
from oracle import oracle as O
from test_gpu_prefill_paged import SIGMA, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_cache_vector_gb300 import build
    build.build()
    abi.lib()
    abi.tq_device_status(reset=True)


# Sequences that fill the GPU: with few items each is cut into parts of about a block, with these
# behind them items are mostly whole and their blocks follow one another in one running softmax.
CROWD = [(1, 20)] * 400
both_ways = pytest.mark.parametrize("crowd", [[], CROWD], ids=["few", "many"])


def reference(bt, scale, window=0):
    """(attention in 64 bits, its tolerance), both [rows of q, Hq, d]; zero for a crowd's rows."""
    q = bt.q.double().numpy()
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    G, rd = bt.Hq // bt.Hkv, math.sqrt(bt.d)
    for b, (n, c) in enumerate(bt.lens[:-len(CROWD)] if bt.lens[-len(CROWD):] == CROWD else bt.lens):
        k, v = bt.decoded(b) if n and c else (None, None)
        for t in range(n):
            p1 = c - n + t + 1
            lo = max(0, p1 - window) if window else 0
            if p1 <= 0:
                continue
            for h in range(bt.Hq):
                kk, vv, qq = k[h // G, lo:p1], v[h // G, lo:p1], q[bt.cu[b] + t, h]
                s = kk @ qq * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                o = p @ vv
                S = abs(scale) * np.linalg.norm(qq) * np.linalg.norm(kk, axis=1) / rd
                out[bt.cu[b] + t, h] = o
                tol[bt.cu[b] + t, h] = 6 * SIGMA * ((p * S) @ np.abs(vv - o) + (p @ np.linalg.norm(vv, axis=1)) / rd) + \
                    3 * 2.0 ** -11 * (p @ np.abs(vv))
    return out, tol


def compare(bt, scale, window=0, rows=None):
    """Both output types against the reference; rows [rows of q, Hkv]: the ones that are compared."""
    args = bt.gpu()
    want, tol = reference(bt, scale, window)
    on = np.ones(want.shape[:2], bool) if rows is None else np.repeat(rows, bt.Hq // bt.Hkv, 1)
    if bt.lens[-len(CROWD):] == CROWD:
        on[-len(CROWD):] = False
    for dt in (torch.float32, torch.bfloat16):
        got = abi.tq_attn_prefill_paged(*args, scale, window=window, out_dtype=dt)
        assert abi.tq_device_status(reset=True) == 0
        got = got.double().cpu().numpy()
        err = np.abs(got - want)
        over = np.where(on[..., None], err - tol - (np.abs(want) * 2.0 ** -8 if dt == torch.bfloat16 else 0.0), -np.inf)
        over = np.where(np.isnan(got) & on[..., None], np.inf, over)
        at = np.unravel_index(np.argmax(over), over.shape)
        assert over[at] <= 0, (at, got[at], want[at], tol[at])
    return got, want, tol


def attends(bt, marks, window=0):
    """Which rows of q, per KV head, attend to one of the (sequence, head, position) marks."""
    hit = np.zeros((bt.q.shape[0], bt.Hkv), bool)
    for b, h, pos in marks:
        n, c = bt.lens[b]
        p = np.arange(c - n, c)
        hit[bt.cu[b]:bt.cu[b + 1], h] |= (p >= pos) & (p - pos < (window or 1 << 40))
    return hit


OUTSIDE = [
    # lengths, window, marked (sequence, head, position): behind the causal mask of most
    # tokens, in front of the window of most, and in an earlier block than theirs
    ([(40, 200), (1, 70)], 0, [(0, 0, 199), (0, 1, 170)]),
    ([(150, 300), (3, 90)], 0, [(0, 1, 299), (0, 0, 260), (1, 0, 89)]),
    ([(180, 420)], 64, [(0, 0, 180), (0, 1, 230), (0, 1, 240)]),
    ([(20, 500), (130, 700)], 100, [(0, 0, 381), (1, 1, 471), (1, 0, 560)]),
]


@both_ways
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("ratio", [4, 9, 12, 15, 18, 24, 40, 90])
@pytest.mark.parametrize("d,kb,vb", [(32, 4, 4), (64, 3, 4), (128, 4, 3), (256, 4, 4)])
def test_a_large_norm_does_not_reach_rows_that_do_not_attend_to_it(d, kb, vb, ratio, which, crowd):
    for i, (lens, window, marks) in enumerate(OUTSIDE):
        bt = Batch(20 + i, lens + crowd, 4, 2, d, 64, kb, vb)
        for b, h, pos in marks:
            bt.set_norm(b, which, h, pos, math.sqrt(d) * 2.0 ** ratio)
        # a token that attends to so large a key has a softmax of steps: any rounding of a
        # score may turn it, so those rows are left out (a large value changes no score)
        rows = ~attends(bt, marks, window) if which == "k" else None
        assert rows is None or 0.2 < rows.mean() < 1
        compare(bt, 1 / math.sqrt(d), window, rows)


@both_ways
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [[(1, 3000)], [(300, 900)], [(9, 400), (2, 1100)]])
@pytest.mark.parametrize("name,vnorm", [
    ("blocks far apart", lambda p: 2.0 ** np.array([60, -60, 3, -75, 80, 0])[p // 128 % 6]),
    ("growing far", lambda p: 2.0 ** np.minimum(80, -80 + p / 3)),
    ("falling far", lambda p: 2.0 ** np.maximum(-80, 80 - p / 3)),
    ("zeros, then tiny", lambda p: np.where(p < 150, 0.0, 2.0 ** -60)),
    ("tiny, then zeros", lambda p: np.where(p < 150, 2.0 ** -60, 0.0)),
    ("mixed within blocks", lambda p: 2.0 ** ((p * 37 % 121) - 60.0)),
])
def test_values_of_all_sizes(name, vnorm, lens, d, crowd):
    """Scores of all sizes too: where the values are small they take most of the weight."""
    bt = Batch(30, lens + crowd, 4, 2, d, 64, 4, 4)
    for b, (_, c) in enumerate(lens):
        v = vnorm(np.arange(c)).astype(np.float32)
        for h in range(2):
            for p in range(c):
                bt.set_norm(b, "v", h, p, v[p])
    compare(bt, 0.2)


@both_ways
@pytest.mark.parametrize("d", [128, 256])
def test_small_values_with_all_the_weight(d, crowd):
    """Sharp softmaxes whose winners have far smaller V norms than the rest."""
    bt = Batch(31, [(40, 900)] + crowd, 4, 1, d, 64, 4, 4)
    for pos in (0, 200, 511, 850):
        bt.set_norm(0, "k", 0, pos, 60.0 * d / 128)
        bt.set_norm(0, "v", 0, pos, 1e-3)
    got, want, tol = compare(bt, 0.5)
    got, want, tol = (x[:40] for x in (got, want, tol))
    won = np.linalg.norm(want, axis=-1) < 2e-3
    assert won.mean() > 0.3
    # rows of zeros in their place would not pass, nor rows 5% off
    assert (np.abs(want[won]) > tol[won]).any(-1).all()
    assert (0.05 * np.abs(want[won]) > tol[won] + np.abs(want[won]) * 2.0 ** -8).any(-1).mean() > 0.5


@both_ways
@pytest.mark.parametrize("d", [64, 128, 256])
def test_values_spread_over_many_powers(d, crowd):
    """Norms with a log-normal spread of four powers of two, judged row by row."""
    bt = Batch(32, [(60, 500), (1, 700), (140, 140)] + crowd, 4, 2, d, 32, 4, 4,
               norm=lambda r, n: np.exp(3 * r.standard_normal(n)))
    compare(bt, 0.002)


@pytest.mark.parametrize("lens", [[(40, 200), (1, 70)], [(150, 300)]])
@pytest.mark.parametrize("d", [32, 128, 256])
@pytest.mark.parametrize("scale", [0.1, -0.1, 1e-38])
def test_scores_below_the_smallest_number_are_zero(scale, d, lens):
    """Tiny queries over tiny keys: the product of their powers of two is no fp32 number, and all
    that a token attends to has the same weight."""
    bt = Batch(33, lens, 4, 2, d, 64, 4, 4, qmul=2.0 ** -70)
    for b, (_, c) in enumerate(lens):
        for h in range(2):
            for pos in range(c):
                bt.set_norm(b, "k", h, pos, 2.0 ** -85)
    compare(bt, scale)


@pytest.mark.parametrize("entry", ["gone", "another's"])
@pytest.mark.parametrize("page,window", [(32, 1), (32, 40), (64, 100), (256, 300)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_pages_in_front_of_the_window_are_not_read(d, page, window, entry):
    """A cache that keeps only a window's pages has given the ones before it back: their entries are
    -1, or hold rows of something else."""
    lens = [(1, 500), (40, 700), (300, 1000), (3, 3)]
    bt = Batch(34, lens, 4, 2, d, page, 4, 3)
    want, tol = reference(bt, 0.1, window)
    for b, (n, c) in enumerate(lens):
        for j in range(max(0, c - n - window + 1) // page):
            if entry == "gone":
                bt.bt_host[b, j] = -1
            else:
                for a in ("kn", "vn"):
                    bt.arrays[a][bt.bt_host[b, j]] = 2.0 ** 60
    out = abi.tq_attn_prefill_paged(*bt.gpu(), 0.1, window=window, out_dtype=torch.float32)
    assert abi.tq_device_status(reset=True) == 0
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    if entry == "gone":  # the same bits as with the pages there
        full = abi.tq_attn_prefill_paged(*Batch(34, lens, 4, 2, d, page, 4, 3).gpu(), 0.1, window=window,
                                         out_dtype=torch.float32)
        assert torch.equal(out, full)


def set_rows(bt, b, k, v):
    """Sequence b's positions hold the rows k and v [Hkv, positions, d]."""
    pos, page = np.arange(bt.lens[b][1]), bt.page
    pg, off, hh = bt.bt_host[b, pos // page][:, None], (pos % page)[:, None], np.arange(bt.Hkv)[None]
    enc = []
    for x, bits in ((k, bt.kb), (v, bt.vb)):
        p, n = O.encode(bt.s, bits, x.reshape(-1, bt.d), s2=bt.s2, kind=bt.kind)
        enc += [p.reshape(bt.Hkv, len(pos), -1), n.reshape(bt.Hkv, len(pos))]
    bt.rows[b] = enc
    for a, src in zip(("kp", "kn", "vp", "vn"), enc):
        bt.arrays[a][pg, hh, off] = src.swapaxes(0, 1)


@pytest.mark.parametrize("d,kb,vb", [(64, 4, 4), (128, 4, 3), (256, 4, 4)])
def test_rows_with_outlier_channels(d, kb, vb):
    """Correlated rows with a few channels eight times as large: sharp softmaxes over large values,
    where the fp16 operands show most.  The decode attention of the same tokens is closer."""
    lens = [(120, 120), (40, 700)]
    bt = Batch(35, lens, 8, 2, d, 64, kb, vb)
    for b, (_, c) in enumerate(lens):
        set_rows(bt, b, *(np.stack([synth.lowrank_rows(40 + which, c, d, stream=10 * b + h).double().numpy()
                                    for h in range(2)]) for which in (0, 1)))
    bt.q = torch.stack([synth.lowrank_rows(42, 160, d, stream=h) for h in range(8)], 1)
    got, want, _ = compare(bt, 1 / math.sqrt(d))
    assert np.abs(want).max() > 10
    plan, q, _, cache, table, ctx = bt.gpu()
    last = torch.tensor([119, 159]).cuda()
    one = abi.tq_attn_decode_paged(plan, q[last].contiguous(), cache, table, ctx, 700, 1 / math.sqrt(d))
    assert np.abs(one.double().cpu().numpy() - want[[119, 159]]).max() <= 2e-3


@both_ways
@pytest.mark.parametrize("seed", range(40))
def test_seeded_sweep(seed, crowd):
    """Lengths, heads, pages, windows, widths and spreads of norms drawn together; slots without a
    position hold NaN norms, as in all of these batches."""
    g = np.random.default_rng(1000 + seed)
    d = int(g.choice([32, 64, 128, 256]))
    Hkv, G = int(g.integers(1, 4)), int(g.choice([1, 2, 3, 5, 8]))
    lens = []
    for _ in range(int(g.integers(1, 6))):
        n = int(g.choice([0, 1, 2, int(g.integers(1, 40)), int(g.integers(1, 150))]))
        lens.append((n, max(0, n - int(g.integers(0, 3))) + int(g.choice([0, 1, 130, int(g.integers(0, 900))]))))
    if not sum(n for n, _ in lens):
        lens.append((3, 200))
    window = int(g.choice([0, 0, 1, int(g.integers(1, 300)), 5000]))
    bt = Batch(seed, lens + crowd, Hkv * G, Hkv, d, int(g.choice([32, 64, 128, 512])), int(g.integers(2, 5)),
               int(g.integers(2, 5)), flags=int(g.integers(0, 4)))
    ks, vs = (float(g.choice([0, 2, 9, 14, 30, 60])) for _ in range(2))
    vbase = float(g.integers(-30, 30))
    for b, (_, c) in enumerate(lens):
        for h in range(Hkv):
            for p in range(c):
                bt.set_norm(b, "k", h, p, math.sqrt(d) * 2.0 ** -(g.random() * ks))
                bt.set_norm(b, "v", h, p, 0.0 if g.random() < 0.05 else 2.0 ** (vbase + vs * (g.random() - 0.5)))
    compare(bt, float(g.choice([1.0, -0.7, 0.3])) / math.sqrt(d), window)


@both_ways
@pytest.mark.parametrize("ratio", [8, 20, 40, 90])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_zero_values_beside_a_large_one_that_is_not_attended(d, ratio, crowd):
    """Tokens that attend, in one block, to positions with a V norm of 0 only, while the block holds a
    large one in front of their window or behind the causal mask."""
    for lens, window, marks in (([(120, 260), (20, 150)], 0, [(0, 128, 256, 252), (1, 128, 149, 149)]),
                                ([(180, 420), (300, 900)], 150, [(0, 128, 256, 130), (1, 640, 768, 641)])):
        bt = Batch(36, lens + crowd, 4, 2, d, 64, 4, 4)
        for b, z0, z1, large in marks:
            for h in range(2):
                for p in range(z0, z1):
                    bt.set_norm(b, "v", h, p, 0.0)
                bt.set_norm(b, "v", h, large, math.sqrt(d) * 2.0 ** ratio)
        compare(bt, 1 / math.sqrt(d), window)
