"""The paged operators together, as a serving loop uses them: pages taken for
prompts, the prompts' rows appended and attended to in chunks, rows branched,
decode steps, drafted tokens checked and some cut off again, rows freed and
the pool closed up.  Two layers share the books.  After every attention the
output is compared with the attention in 64 bits over each row's own history
of (oracle-encoded) keys and values."""
import math
import random

import numpy as np
import pytest
import torch

from kv_cache_vector_gb300 import abi
from oracle import oracle as O

pytestmark = pytest.mark.gpu
SIGMA = 2 * 2.0 ** -11 / math.sqrt(3)  # four fp16 roundings, as in the attention's own tests


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_cache_vector_gb300 import build
    build.build()
    abi.lib()
    abi.tq_device_status(reset=True)


class Server:
    def __init__(self, seed, d=128, page=32, Hq=8, Hkv=2, kb=4, vb=3, L=2, rows=6, max_pages=8, n_pages=34):
        self.rng, self.g = random.Random(seed), np.random.default_rng(seed)
        self.d, self.page, self.Hq, self.Hkv, self.kb, self.vb, self.L, self.rows = d, page, Hq, Hkv, kb, vb, L, rows
        self.plan, self.s = abi.Plan(d, 42), O.signs(42, d)
        self.pool = abi.PagedLayers([abi.PagedCache.empty(n_pages, Hkv, page, d, kb, vb) for _ in range(L)])
        self.books = abi.PageTable.empty(rows, max_pages, n_pages)
        self.top = max_pages * page
        self.hist = [[] for _ in range(rows)]  # per row a list of token numbers
        self.tokens = []                       # per token number, per layer (k, v): [Hkv, d] rows

    def new_tokens(self, n):
        at = len(self.tokens)
        kv = torch.from_numpy(self.g.standard_normal((n, self.L, 2, self.Hkv, self.d))).to(torch.bfloat16)
        self.tokens += list(kv)
        return list(range(at, at + n))

    def resize(self, lens):
        to = torch.tensor(lens, dtype=torch.int32).cuda()
        _, info = abi.tq_pages_resize(self.books, to, self.pool, out=self.books)
        assert info.tolist()[1] == 0
        for r, n in enumerate(lens):
            if n >= 0:
                self.hist[r] = self.hist[r][:n]

    def append(self, counts, attend="prefill"):
        """counts[r] new tokens at the end of row r: pages, rows of K and V, attention."""
        lens = [len(h) for h in self.hist]
        self.resize([lens[r] + n if n else -1 for r, n in enumerate(counts)])
        who = [(r, lens[r] + i) for r, n in enumerate(counts) for i in range(n)]
        if not who:
            return
        for r, n in enumerate(counts):
            self.hist[r] += self.new_tokens(n)
        row = torch.tensor([r for r, _ in who]).cuda()
        pos = torch.tensor([p for _, p in who]).cuda()
        slot = self.books.block_table[row, pos // self.page][:, None].contiguous()
        off = (pos % self.page).to(torch.int32)
        kv = torch.stack([self.tokens[self.hist[r][p]] for r, p in who]).cuda()  # [T, L, 2, Hkv, d]
        q = torch.from_numpy(self.g.standard_normal((len(who), self.Hq, self.d))).to(torch.bfloat16).cuda()
        scale = 1 / math.sqrt(self.d)
        for layer, cache in enumerate(self.pool.layers):
            k, v = kv[:, layer, 0].contiguous(), kv[:, layer, 1].contiguous()
            if attend == "step":  # one token per row, appended by the decode call itself
                n = len(who)
                out = abi.tq_attn_decode_append_paged(self.plan, q, k, v, cache, self.books.block_table[row].contiguous(),
                                                      pos.to(torch.int32), self.top, scale)
                tol = 2e-3
            else:
                abi.tq_append_paged(self.plan, cache, k, v, slot, off)
                cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()
                out = abi.tq_attn_prefill_paged(self.plan, q, cu, cache, self.books.block_table, self.books.lens, scale,
                                                out_dtype=torch.float32)
                tol = 0.0
            self.check(layer, who, q, out, scale, tol)

    def decoded(self, layer, toks):
        kv = torch.stack([self.tokens[t][layer] for t in toks]).double().numpy()  # [n, 2, Hkv, d]
        out = []
        for i, bits in ((0, self.kb), (1, self.vb)):
            x = kv[:, i].reshape(-1, self.d)
            p, n = O.encode(self.s, bits, x)
            out.append(O.decode(self.s, bits, p, n).reshape(len(toks), self.Hkv, self.d))
        return out

    def check(self, layer, who, q, out, scale, tol):
        q, out = q.double().cpu().numpy(), out.double().cpu().numpy()
        G = self.Hq // self.Hkv
        cache = {}
        for i, (r, p) in enumerate(who):
            if r not in cache:
                cache[r] = self.decoded(layer, self.hist[r])
            k, v = (x[:p + 1].repeat(G, 1) for x in cache[r])  # [n, Hq, d]
            s = np.einsum("hd,nhd->hn", q[i], k) * scale
            w = np.exp(s - s.max(1, keepdims=True))
            want = np.einsum("hn,nhd->hd", w / w.sum(1, keepdims=True), v)
            S = scale * np.linalg.norm(q[i], axis=1) * np.linalg.norm(k, axis=2).max(0) / math.sqrt(self.d)
            V = np.linalg.norm(v, axis=2).max(0) / math.sqrt(self.d)
            # a key or value whose normalised coordinate lies within 1e-6 of a codebook
            # boundary may be encoded to the next level: at most one in 1e5 coordinates, a
            # level apart by at most 2 |x| / sqrt(d), so its part in the output is far below
            bound = (6 * SIGMA * (1 + S) * V + tol)[:, None]
            assert (np.abs(out[i] - want) <= bound).all(), (layer, r, p, np.abs(out[i] - want).max())

    def fork(self, parents):
        out, info = abi.tq_pages_fork(self.books, torch.tensor(parents, dtype=torch.int32).cuda(), self.pool)
        assert info.tolist()[1] == 0
        self.books = out
        self.hist = [list(self.hist[p]) if p >= 0 else [] for p in parents]

    def compact(self):
        out, moved, info = abi.tq_pages_compact(self.books, self.pool, out=self.books)
        held = int((self.books.refs > 0).sum())
        assert info.tolist()[0] == held and (self.books.refs[:held] > 0).all()

    def sound(self):
        lens = self.books.lens.tolist()
        assert lens == [len(h) for h in self.hist]
        table, count = self.books.block_table.cpu().numpy(), np.zeros(self.pool.n_pages, np.int64)
        for r, n in enumerate(lens):
            used = -(-n // self.page)
            assert (table[r, used:] == -1).all()
            np.add.at(count, table[r, :used], 1)
        assert np.array_equal(count, self.books.refs.cpu().numpy())


@pytest.mark.parametrize("d,kb,vb", [(128, 4, 3), (64, 3, 4), (256, 4, 4)])
def test_a_serving_loop(d, kb, vb):
    sv = Server(d, d=d, kb=kb, vb=vb)
    sv.append([70, 33, 0, 1, 0, 0])                     # prompts
    sv.append([40, 0, 64, 0, 0, 0])                     # a second chunk beside a new prompt
    sv.sound()
    sv.fork([0, 1, 2, 3, 0, 0])                         # two branches of row 0
    sv.sound()
    for _ in range(3):
        sv.append([1, 1, 1, 1, 1, 1], attend="step")    # decode steps, each branch its own
    sv.append([4, 2, 0, 5, 3, 1])                       # drafted tokens, checked together
    sv.resize([len(sv.hist[0]) - 3, -1, -1, len(sv.hist[3]) - 5, -1, -1])  # some are rejected
    sv.sound()
    sv.append([1, 0, 1, 1, 1, 1])
    sv.resize([-1, 0, -1, -1, 100, -1])                 # one ended, one cut back into a shared page
    sv.compact()
    sv.sound()
    sv.append([0, 20, 0, 0, 2, 7])                      # goes on inside the shared page: a private copy
    sv.fork([5, 4, -1, 2, 4, 0])                        # beams reordered, one dropped
    sv.compact()
    sv.append([1, 1, 3, 1, 1, 1])
    sv.sound()
    assert abi.tq_device_status(reset=True) == 0


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes an array: pages at its end are copied, attended to and moved as
    those at its start."""
    n_pages, Hkv, page, d = 140000, 8, 64, 128
    pool = abi.PagedLayers(abi.PagedCache.empty(n_pages, Hkv, page, d, 4, 4))
    c = pool.layers[0]
    assert c.k_packed.numel() > 2 ** 32 and c.v_packed.numel() > 2 ** 32
    g = torch.Generator().manual_seed(3)
    low, high = torch.arange(1, 8), torch.arange(n_pages - 7, n_pages)
    for t in (c.k_packed, c.v_packed):
        t[1:8] = torch.randint(0, 256, t[1:8].shape, generator=g, dtype=torch.uint8).cuda()
    for t in (c.k_norm, c.v_norm):
        t[1:8] = 5 + 5 * torch.rand(t[1:8].shape, generator=g).cuda()
    ids = lambda x: x.to(torch.int32).cuda()  # noqa: E731
    abi.tq_pages_copy(pool, pool, ids(low), ids(high))
    for t in (c.k_packed, c.k_norm, c.v_packed, c.v_norm):
        assert torch.equal(t[1:8], t[n_pages - 7:]) and t[1:8].any()
    n, ctx = 130, 7 * page - 5
    q = torch.randn(n + 1, 32, d, generator=g).to(torch.bfloat16).cuda()
    cu, lens = ids(torch.tensor([0, n, n + 1])), ids(torch.tensor([ctx, ctx]))
    outs = [abi.tq_attn_prefill_paged(abi.Plan(d, 42), q, cu, c, ids(torch.stack([x, x])), lens, 0.1) for x in (low, high)]
    assert torch.equal(*outs) and outs[0].any()
    books = abi.PageTable.empty(2, 7, n_pages)
    books.block_table[0], books.lens[0] = ids(high), ctx
    books.refs[n_pages - 7:] = 1
    books, info = abi.tq_pages_fork(books, ids(torch.tensor([0, 0])), pool)
    assert info.tolist() == [1, 0] and books.block_table[1].tolist() == high.tolist()[:6] + [0]
    for t in (c.k_packed, c.k_norm, c.v_packed, c.v_norm):
        assert torch.equal(t[0], t[n_pages - 1])
    books, moved, info = abi.tq_pages_compact(books, pool, out=books)
    assert info.tolist() == [8, 7] and books.block_table[0].tolist() == list(range(1, 8))
    for t in (c.k_packed, c.k_norm, c.v_packed, c.v_norm):
        assert torch.equal(t[1:8], t[n_pages - 7:])
    assert abi.tq_device_status(reset=True) == 0
