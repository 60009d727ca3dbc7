"""tq_attn_prefill_paged against the attention in 64 bits over the oracle's
decoded rows.

Tolerance.  The kernel rounds four factors of every product to fp16 (query,
level, norm, level times norm; for the output P in the query's place), each off
by at most 2^-11 relative, 2^-11 / sqrt(3) in the root mean square: 2 * 2^-11 /
sqrt(3) = 5.64e-4 for the four.  A score q . k then has an error of standard
deviation 5.64e-4 * S, S = scale |q| |k| / sqrt(d) (the rotation spreads both
over all d coordinates), which changes the output by at most that part of the
values' root mean square V; the second product adds 5.64e-4 V.  Six standard
deviations: 6 * 5.64e-4 (1 + S) V per element, and the output's own rounding
on top (bf16: 2^-8 relative).  Over all elements the root mean square error
stays below 1.5 standard deviations."""
import math

import numpy as np
import pytest
import torch

from kv_cache_vector_gb300 import abi, synth
from oracle import oracle as O

pytestmark = pytest.mark.gpu
SIGMA = 2 * 2.0 ** -11 / math.sqrt(3)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_cache_vector_gb300 import build
    build.build()
    abi.lib()
    abi.tq_device_status(reset=True)


class Batch:
    """Sequences of given (query, context) lengths in shuffled pages; slots that
    hold no position have NaN norms and random bytes, table entries past a
    sequence's pages are -1."""

    def __init__(self, seed, lens, Hq, Hkv, d, page, kb, vb, flags=0, norm=None, tail=0, qmul=1.0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.s = O.signs(42, d)
        self.s2 = O.signs2(42, d) if flags & abi.PLAN_TWO_SIDED_SIGNS else None
        self.kind = "gauss" if flags & abi.PLAN_GAUSSIAN_CODEBOOK else "sphere"
        self.plan = abi.Plan(d, 42, flags)
        self.lens, self.Hq, self.Hkv, self.d, self.page, self.kb, self.vb = lens, Hq, Hkv, d, page, kb, vb
        need = [-(-c // page) for _, c in lens]
        n_pages, max_pages = sum(need) + 2, max(max(need), 1) + 1
        perm = rng.permutation(n_pages).astype(np.int32)
        bt, at = np.full((len(lens), max_pages), -1, np.int32), 0
        kp = torch.randint(0, 256, (n_pages, Hkv, page, d * kb // 8), generator=g, dtype=torch.uint8).numpy()
        vp = torch.randint(0, 256, (n_pages, Hkv, page, d * vb // 8), generator=g, dtype=torch.uint8).numpy()
        kn = np.full((n_pages, Hkv, page), np.nan, np.float32)
        vn = np.full((n_pages, Hkv, page), np.nan, np.float32)
        self.rows = []
        for b, (_, c) in enumerate(lens):
            bt[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
            k, v = rng.standard_normal((2, Hkv * c, d))
            if norm is not None:
                k, v = k * norm(rng, Hkv * c)[:, None], v * norm(rng, Hkv * c)[:, None]
            enc = []
            for x, bits in ((k, kb), (v, vb)):
                p, n = O.encode(self.s, bits, x, s2=self.s2, kind=self.kind) if c else \
                    (np.zeros((0, d * bits // 8), np.uint8), np.zeros(0, np.float32))
                enc += [p.reshape(Hkv, c, d * bits // 8), n.reshape(Hkv, c)]
            self.rows.append(enc)
            pos = np.arange(c)
            pg, off, hh = bt[b, pos // page][:, None], (pos % page)[:, None], np.arange(Hkv)[None]
            for dst, src in zip((kp, kn, vp, vn), enc):
                dst[pg, hh, off] = src.swapaxes(0, 1)
        self.arrays = dict(kp=kp, kn=kn, vp=vp, vn=vn)
        self.bt_host, self.n_pages = bt, n_pages
        n_q = sum(n for n, _ in lens)
        self.q = (torch.randn(n_q + tail, Hq, d, generator=g) * qmul).to(torch.bfloat16)
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)

    def set_norm(self, b, which, h, pos, value):
        """One position's K or V norm, in the pages and in the reference's rows."""
        pg = self.bt_host[b, pos // self.page]
        self.arrays["kn" if which == "k" else "vn"][pg, h, pos % self.page] = value
        self.rows[b][1 if which == "k" else 3][h, pos] = value

    def gpu(self):
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        a = self.arrays
        self.cache = abi.PagedCache(t(a["kp"]), t(a["kn"]), t(a["vp"]), t(a["vn"]), self.kb, self.vb)
        return (self.plan, self.q.cuda(), t(self.cu), self.cache, t(self.bt_host),
                torch.tensor([c for _, c in self.lens], dtype=torch.int32).cuda())

    def decoded(self, b):
        kp, kn, vp, vn = self.rows[b]
        out = []
        for p, n, bits in ((kp, kn, self.kb), (vp, vn, self.vb)):
            x = O.decode(self.s, bits, p.reshape(-1, p.shape[-1]), np.ones(n.size, np.float32), s2=self.s2, kind=self.kind)
            with np.errstate(invalid="ignore"):
                out.append(x.reshape(*n.shape, self.d) * n.astype(np.float64)[..., None])
        return out

    def want(self, scale, window=0):
        """(attention, per-row S, per-row V): both from the rows that each token attends to."""
        q = self.q.double().numpy()
        out, S, V = np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
        G = self.Hq // self.Hkv
        for b, (n, c) in enumerate(self.lens):
            if not n or not c:
                continue
            k, v = self.decoded(b)
            pos = np.arange(c - n, c)[:, None]
            seen = (np.arange(c) <= pos) & (np.arange(c) > pos - (window or 1 << 40))
            some = seen.any(1)
            for h in range(self.Hq):
                kk, vv = k[h // G], v[h // G]
                qq = q[self.cu[b]:self.cu[b + 1], h]
                s = np.where(seen, qq @ np.where(np.isfinite(kk), kk, 0.0).T * scale, -np.inf)
                bad = ~(np.isfinite(kk).all(1) & np.isfinite(vv).all(1))
                p = np.exp(s - np.where(some, s.max(1, initial=-np.inf), 0.0)[:, None])
                p /= np.where(some, p.sum(1), 1.0)[:, None]
                o = p @ np.where(np.isfinite(vv), vv, 0.0)
                o[(seen & bad).any(1)] = np.nan
                out[self.cu[b]:self.cu[b + 1], h] = o
                kn = np.where(bad, 0.0, np.linalg.norm(kk, axis=1))
                vn = np.where(bad, 0.0, np.linalg.norm(vv, axis=1))
                S[self.cu[b]:self.cu[b + 1], h] = abs(scale) * np.linalg.norm(qq, axis=1) * \
                    np.where(seen, kn, 0.0).max(1, initial=0.0) / math.sqrt(self.d)
                V[self.cu[b]:self.cu[b + 1], h] = np.where(seen, vn, 0.0).max(1, initial=0.0) / math.sqrt(self.d)
        return out, S, V


def check(got, want, S, V, n_q, bf16=True):
    got = got.double().cpu().numpy()[:n_q]
    want, S, V = want[:n_q], S[:n_q], V[:n_q]
    bad = np.isnan(want)
    assert np.array_equal(np.isnan(got), bad)
    err = np.where(bad, 0.0, np.abs(np.where(bad, 0.0, got) - np.where(bad, 0.0, want)))
    unit = (SIGMA * (1 + S) * V)[..., None]
    own = np.where(bad, 0.0, np.abs(want)) * 2.0 ** -8 if bf16 else 0.0
    over = err - 6 * unit - own
    at = np.unravel_index(np.argmax(over), over.shape)
    assert over[at] <= 0, (at, got[at], want[at], err[at], unit[at[:-1]])
    if not bf16:
        use = np.broadcast_to(unit, err.shape) > 0
        if use.any():
            rms = math.sqrt(np.mean((err / np.where(use, np.broadcast_to(unit, err.shape), 1.0))[use] ** 2))
            assert rms <= 1.5, rms


def run_both(bt, scale, window=0):
    """Both output types; they are the same values, rounded."""
    args = bt.gpu()
    n = int(bt.cu[-1])
    want, S, V = bt.want(scale, window)
    o32 = abi.tq_attn_prefill_paged(*args, scale, window=window, out_dtype=torch.float32)
    o16 = abi.tq_attn_prefill_paged(*args, scale, window=window)
    torch.cuda.synchronize()
    assert abi.tq_device_status(reset=True) == 0
    check(o32, want, S, V, n, bf16=False)
    check(o16, want, S, V, n)
    assert torch.equal(o32.to(torch.bfloat16).nan_to_num(7.0), o16.nan_to_num(7.0))
    assert not o16[n:].any()
    return o16


CASES = [
    # (query, context) lengths, Hq, Hkv, page, kb, vb, window
    ([(1, 1)], 1, 1, 32, 4, 4, 0),
    ([(1, 129), (1, 128), (1, 127), (1, 300)], 8, 2, 64, 4, 3, 0),       # single tokens
    ([(5, 700), (3, 33), (0, 64), (7, 7)], 32, 8, 64, 4, 3, 0),          # drafts; a sequence without queries
    ([(130, 130), (64, 200), (257, 900)], 8, 2, 256, 3, 2, 0),           # split and paired tiles
    ([(100, 100), (1, 2000)], 12, 4, 32, 2, 4, 0),                       # three heads a group
    ([(33, 95), (200, 500)], 5, 1, 128, 3, 3, 0),                        # five
    ([(40, 40), (3, 290)], 40, 2, 32, 4, 2, 0),                          # twenty
    ([(300, 1000), (1, 513), (20, 20)], 4, 4, 64, 4, 4, 100),            # windows
    ([(150, 400)], 8, 4, 32, 4, 4, 1),                                   # of one position: itself
    ([(129, 129), (2, 640)], 2, 1, 64, 2, 2, 4096),                      # past every length
    ([(9, 4), (4, 4), (3, 0)], 4, 2, 32, 4, 3, 0),                       # more tokens than positions: zero rows
    ([(1, 9000)], 8, 1, 256, 4, 3, 0),                                   # one row tile over all SMs
]


@pytest.mark.parametrize("d", [128, 64, 256, 32])
@pytest.mark.parametrize("lens,Hq,Hkv,page,kb,vb,window", CASES)
def test_parity(lens, Hq, Hkv, page, kb, vb, window, d):
    run_both(Batch(1, lens, Hq, Hkv, d, page, kb, vb), 1 / math.sqrt(d), window)


@pytest.mark.parametrize("d", [128, 256])
def test_many_sequences(d):
    rng = np.random.default_rng(d)
    lens = [(int(n), int(n + c)) for n, c in zip(rng.integers(0, 9, 150), rng.integers(0, 200, 150))]
    run_both(Batch(2, lens, 4, 2, d, 32, 4, 3), 1 / math.sqrt(d))


def test_more_sequences_than_threads():
    lens = [(1, 1 + i % 40) if i % 3 else (0, 5) for i in range(1500)]
    run_both(Batch(3, lens, 2, 1, 64, 32, 3, 4), 0.125)


@pytest.mark.parametrize("lens", [
    [(1, 5000)],                                    # one item over all CTAs
    [(1, 100), (1, 3000), (1, 90), (1, 129)],       # unequal items: few shares and many
    [(200, 700), (1, 4000), (70, 70)],              # several tiles, paired and split
    [(4, 1), (2, 0), (1, 128), (0, 500)],           # items of one block and of none
    [(1, 900)] * 18,                                # nearly an item per CTA
    [(1, 2000)] * 19 + [(1, 40)] * 19,              # as many items as CTAs, and more
    [(0, 0)] * 700 + [(3, 1000), (1, 1)],           # empty sequences before a few items
])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_few_items(lens, d):
    """Shares that are parts of one item each, and the sizes about which that ends."""
    run_both(Batch(16, lens, 16, 8 if len(lens) < 100 else 2, d, 64, 4, 3), 1 / math.sqrt(d))


@pytest.mark.parametrize("flags", [1, 2, 3])
@pytest.mark.parametrize("d", [32, 128, 256])
def test_plan_variants(d, flags):
    run_both(Batch(4, [(70, 300), (1, 40)], 8, 4, d, 64, 3, 3, flags=flags), 1 / math.sqrt(d))


@pytest.mark.parametrize("scale", [-0.3, 0.0, 0.02, 0.5])
def test_scales(scale):
    run_both(Batch(5, [(20, 400), (200, 333)], 4, 2, 128, 64, 4, 4), scale)


@pytest.mark.parametrize("name,norm,qmul,scale", [
    ("log normal", lambda r, n: np.exp(2 * r.standard_normal(n)), 1.0, 0.01),
    ("tiny", lambda r, n: np.full(n, 2.0 ** -70), 1.0, 2.0 ** 67),
    ("huge", lambda r, n: np.full(n, 2.0 ** 70), 1.0, 2.0 ** -73),
    ("small queries", lambda r, n: np.ones(n), 2.0 ** -60, 2.0 ** 57),
    ("large queries", lambda r, n: np.ones(n), 2.0 ** 80, 2.0 ** -83),
    ("growing blocks", lambda r, n: 2.0 ** (np.arange(n) // 64 % 40 / 4.0), 1.0, 2e-5),
    ("falling blocks", lambda r, n: 2.0 ** (-(np.arange(n) // 64 % 40) / 4.0), 1.0, 0.1),
    ("zeros", lambda r, n: (r.random(n) < 0.5) * 1.0, 1.0, 0.1),
    ("all zero", lambda r, n: np.zeros(n), 1.0, 0.1),
])
@pytest.mark.parametrize("d", [128, 256])
def test_norms_of_all_sizes(name, norm, qmul, scale, d):
    run_both(Batch(6, [(150, 700), (2, 1300)], 4, 2, d, 64, 4, 4, norm=norm, qmul=qmul), scale)


def test_a_few_rows_take_all_the_weight():
    """Sharp softmaxes whose winner has a far smaller V norm than the rest."""
    bt = Batch(7, [(40, 900)], 4, 1, 128, 64, 4, 4, qmul=1.0)
    for pos in (0, 200, 511, 850):
        bt.set_norm(0, "k", 0, pos, 60.0)
        bt.set_norm(0, "v", 0, pos, 1e-3)
    run_both(bt, 0.5)


@pytest.mark.parametrize("which,value", [("k", np.nan), ("k", np.inf), ("v", np.nan), ("v", -np.inf), ("v", np.inf)])
@pytest.mark.parametrize("d", [128, 256])
def test_non_finite_norms_reach_only_rows_that_attend(which, value, d):
    bt = Batch(8, [(60, 200), (140, 300)], 4, 2, d, 64, 4, 3)
    bt.set_norm(0, which, 1, 170, value)   # attended by the last 30 tokens of sequence 0
    bt.set_norm(1, which, 0, 130, value)   # outside the window of most
    bt.set_norm(1, which, 0, 299, value)   # the last token's own position
    run_both(bt, 1 / math.sqrt(d), window=64)


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("d", [32, 128, 256])
def test_non_finite_queries_stay_in_their_row(value, d):
    bt = Batch(14, [(60, 200), (3, 500), (200, 260)], 4, 2, d, 64, 4, 3)
    args = bt.gpu()
    clean = abi.tq_attn_prefill_paged(*args, 0.1)
    bad = torch.zeros(clean.shape[:2], dtype=torch.bool)
    for row, h in ((0, 0), (7, 1), (61, 2), (100, 3), (262, 0)):
        args[1][row, h, d // 2 + 1] = value
        bad[row, h] = True
    out = abi.tq_attn_prefill_paged(*args, 0.1)
    assert abi.tq_device_status(reset=True) == 0
    assert out[bad.cuda()].isnan().all()
    assert torch.equal(out[~bad.cuda()], clean[~bad.cuda()])


@pytest.mark.parametrize("window", [400, 4000, 2 ** 30 + 5, 2 ** 31 - 1])
def test_a_window_past_every_length_is_none(window):
    """Also for tokens before the first position (a position minus the window stays in 32 bits)."""
    bt = Batch(15, [(300, 40), (5, 200), (140, 300)], 4, 2, 128, 64, 4, 3)
    out = run_both(bt, 0.1, window)
    assert torch.equal(out, abi.tq_attn_prefill_paged(*bt.gpu(), 0.1))


def test_rows_outside_every_sequence_keep_their_values():
    bt = Batch(9, [(3, 90), (0, 0), (5, 5)], 4, 2, 128, 32, 4, 3, tail=4)
    bt.cu = bt.cu + 2  # two rows before the first sequence, two behind the last
    args = bt.gpu()
    for dt in (torch.bfloat16, torch.float32):
        out = torch.full(bt.q.shape, 3.5, dtype=dt, device="cuda")
        got = abi.tq_attn_prefill_paged(*args, 0.1, out=out)
        assert got.data_ptr() == out.data_ptr()
        assert (out[:2] == 3.5).all() and (out[10:] == 3.5).all() and not (out[2:10] == 3.5).any()
    want, S, V = bt.want(0.1)
    check(out[2:], want[2:], S[2:], V[2:], 8, bf16=False)


def test_lengths_out_of_range_leave_the_sequence_out():
    bt = Batch(10, [(4, 60), (4, 60), (4, 60)], 4, 2, 128, 32, 4, 3)
    plan, q, cu, cache, table, ctx = bt.gpu()
    want, S, V = bt.want(0.1)
    for bad_cu, bad_ctx, out_rows in (([0, 4, 8, 13], None, (8, 12)), ([0, 4, 3, 12], None, (4, 12)),
                                      ([-1, 4, 8, 12], None, (0, 4)), (None, [60, -1, 60], (4, 8)),
                                      (None, [60, 60, 97], (8, 12))):
        c = torch.tensor(bad_cu, dtype=torch.int32).cuda() if bad_cu else cu
        x = torch.tensor(bad_ctx, dtype=torch.int32).cuda() if bad_ctx else ctx
        out = torch.full(q.shape, 3.5, device="cuda")
        abi.tq_attn_prefill_paged(plan, q, c, cache, table, x, 0.1, out=out)
        assert abi.tq_device_status(reset=True) == 71
        lo, hi = out_rows
        if bad_cu != [0, 4, 3, 12]:  # there the third sequence's rows are others
            assert (out[lo:hi] == 3.5).all()
            keep = [r for r in range(12) if not lo <= r < hi]
            check(out[keep], want[keep], S[keep], V[keep], len(keep), bf16=False)
        else:
            check(out, want, S, V, 3, bf16=False)


def test_bad_pages_count_as_zero_rows():
    bt = Batch(11, [(6, 300), (200, 400)], 4, 2, 128, 64, 4, 3)
    for b, j, page in ((0, 1, -5), (1, 3, bt.n_pages)):
        bt.bt_host[b, j] = page
        for which in "kv":
            bt.rows[b][1 if which == "k" else 3][:, 64 * j:64 * j + 64] = 0.0
    args = bt.gpu()
    out = abi.tq_attn_prefill_paged(*args, 0.1, out_dtype=torch.float32)
    assert abi.tq_device_status(reset=True) == 72
    check(out, *bt.want(0.1), int(bt.cu[-1]), bf16=False)


def test_same_as_the_decode_attention_for_single_tokens():
    bt = Batch(12, [(1, 50), (1, 1000), (1, 64)], 8, 2, 128, 64, 4, 3)
    plan, q, cu, cache, table, ctx = bt.gpu()
    scale = 1 / math.sqrt(128)
    a = abi.tq_attn_prefill_paged(plan, q, cu, cache, table, ctx, scale, out_dtype=torch.float32)
    b = abi.tq_attn_decode_paged(plan, q, cache, table, ctx, 1000, scale)
    _, S, V = bt.want(scale)
    assert ((a - b).abs().cpu().numpy() <= 6 * (SIGMA * (1 + S) * V)[..., None] + 2e-3).all()


def test_repeats_streams_and_graphs_give_the_same_bits():
    bt = Batch(13, [(300, 900), (1, 3000), (17, 64)], 8, 2, 128, 64, 4, 3)
    args = bt.gpu()
    scale = 1 / math.sqrt(128)
    first = abi.tq_attn_prefill_paged(*args, scale)
    for _ in range(3):
        assert torch.equal(abi.tq_attn_prefill_paged(*args, scale), first)
    need = abi.tq_attn_prefill_paged_workspace_bytes(8, 2, 128)
    side = torch.cuda.Stream()
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(first) for _ in range(2)]
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):  # two calls at once, a workspace each
        abi.tq_attn_prefill_paged(*args, scale, out=outs[0], workspace=ws[0])
        with torch.cuda.stream(side):
            abi.tq_attn_prefill_paged(*args, scale, out=outs[1], workspace=ws[1])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        abi.tq_attn_prefill_paged(*args, scale, out=outs[0], workspace=ws[0])
    # other lengths in the same buffers: the captured call follows them
    outs[0].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first)
    args[2].copy_(torch.tensor([0, 10, 11, 318], dtype=torch.int32))
    args[5].copy_(torch.tensor([800, 2000, 63], dtype=torch.int32))
    eager = abi.tq_attn_prefill_paged(*args, scale)
    outs[0].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], eager)
    assert abi.tq_device_status(reset=True) == 0
