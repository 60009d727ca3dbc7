"""A step's slot map, the append at slots and the keeping of drafted rows: books
and bytes equal to the sequential restatement's; and a speculative step from the
pages to the kept rows."""
import math

import numpy as np
import pytest
import torch

from kv_cache_vector_gb300 import abi, synth
from oracle import oracle as O
from oracle import steps
from parity import compare_encode
from test_gpu_prefill_paged import check
from test_gpu_tree_sinks import random_trees, want

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_cache_vector_gb300 import build
    build.build()
    abi.lib()
    abi.tq_device_status(reset=True)


def t32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def books(rng, n, max_new, max_ctx, page, spare=3):
    """Rows of `counts` new tokens behind up to max_ctx positions, shuffled pages."""
    counts = rng.integers(0, max_new + 1, n)
    lens = counts + rng.integers(0, max_ctx + 1, n)
    need = -(-lens // page)
    n_pages = int(need.sum()) + spare
    table = np.full((n, max(1, need.max()) + 1), -1, np.int32)
    ids, at = rng.permutation(n_pages), 0
    for b in range(n):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    refs = np.zeros(n_pages, np.int32)
    refs[ids[:at]] = 1
    return table, lens.astype(np.int32), refs, counts.astype(np.int32)


def gpu_table(table, lens, refs):
    return abi.PageTable(t32(table), t32(lens), t32(refs))


def same_slots(m, ref, status):
    cu, pos, slot, mask, said = ref
    assert abi.tq_device_status(reset=True) == said == status
    assert np.array_equal(m.cu_q.cpu().numpy(), cu)
    assert np.array_equal(m.positions.cpu().numpy(), pos)
    assert np.array_equal(m.slots.cpu().numpy(), slot)
    if mask is not None:
        assert np.array_equal(m.mask.cpu().numpy().view(np.uint32), mask)


@pytest.mark.parametrize("n,max_new,max_ctx,page,pad", [
    (1, 1, 0, 32, 0), (1, 700, 300, 32, 5), (64, 1, 2000, 64, 0), (64, 0, 500, 64, 7), (300, 9, 700, 128, 100),
    (512, 3, 90, 32, 1), (513, 3, 90, 32, 0), (3000, 4, 60, 32, 9), (7, 9000, 100, 256, 1000)])
def test_slots(n, max_new, max_ctx, page, pad):
    rng = np.random.default_rng(n + max_new)
    table, lens, refs, counts = books(rng, n, max_new, max_ctx, page)
    T = int(counts.sum()) + pad
    m = abi.tq_pages_slots(gpu_table(table, lens, refs), t32(counts), T, page)
    assert m.mask is None
    same_slots(m, steps.slots(table, lens, counts, page, len(refs), T), 0)


@pytest.mark.parametrize("n,max_new,words,pad", [(1, 1, 1, 0), (3, 32, 1, 4), (40, 33, 2, 0), (5, 200, 7, 50), (2, 1024, 32, 3)])
def test_slots_of_trees(n, max_new, words, pad):
    rng = np.random.default_rng(words)
    table, lens, refs, counts = books(rng, n, max_new, 300, 64)
    T = int(counts.sum()) + pad
    parents = sum(random_trees(rng, [(int(c), 0) for c in counts])[0], []) + [7] * pad
    m = abi.tq_pages_slots(gpu_table(table, lens, refs), t32(counts), T, 64, parents=t32(parents), mask_words=words)
    same_slots(m, steps.slots(table, lens, counts, 64, len(refs), T, parents, words), 0)


def test_slots_of_chains_stars_and_roots():
    table, lens, refs, counts = np.array([[0, 1], [2, 3], [5, 4]]), np.array([64, 40, 33]), np.ones(6, int), np.array([40, 33, 33])
    parents = [*range(-1, 39), -1, *([0] * 32), *([-1] * 33)]
    m = abi.tq_pages_slots(gpu_table(table, lens, refs), t32(counts), 106, 32, parents=t32(parents), mask_words=2)
    same_slots(m, steps.slots(table, lens, counts, 32, 6, 106, parents, 2), 0)
    assert m.positions[40:73].tolist() == [7] + [8] * 32


@pytest.mark.parametrize("change,status", [
    (dict(counts=[1, -1, 2]), 63), (dict(counts=[1, 41, 2]), 63), (dict(lens=[40, 65, 40]), 63), (dict(T=4), 63),
    (dict(counts=[1, 33, 2], lens=[40, 40, 40], T=40, tree=True), 63), (dict(page_at=(1, 1, 9)), 64),
    (dict(page_at=(1, 1, -1)), 64), (dict(tree=True, parents=[-1, -2, 0, -1, 1]), 65),
    (dict(tree=True, parents=[-1, -1, 1, -1, 5]), 65)])
def test_slots_out_of_range(change, status):
    table = np.array([[0, 1], [2, 3], [5, 4]])
    lens, counts, T = np.array(change.get("lens", [40, 40, 40])), np.array(change.get("counts", [1, 2, 2])), change.get("T", 5)
    if "page_at" in change:
        b, j, p = change["page_at"]
        table[b, j] = p
    tree = change.get("tree", False)
    parents = change.get("parents", [-1] * T) if tree else None
    m = abi.tq_pages_slots(gpu_table(table, lens, np.ones(6)), t32(counts), T, 32,
                           parents=t32(parents) if tree else None, mask_words=1)
    same_slots(m, steps.slots(table, lens, counts, 32, 6, T, parents, 1), status)


def test_results_of_steps_are_their_own():
    """Steps of the sizes of the one before, of others and of no tokens."""
    rng = np.random.default_rng(8)
    made = []
    for n, new, words in [(5, 6, 0)] * 40 + [(5, 6, 1), (9, 6, 0), (9, 6, 1), (9, 6, 1), (5, 6, 1)] * 8 + [(5, 0, 0), (5, 0, 1)] * 3 + [(100, 100, 4)] * 6:
        table, lens, refs, counts = books(rng, n, new, 200, 32)
        T = n * new
        parents = [-1] * T if words else None
        m = abi.tq_pages_slots(gpu_table(table, lens, refs), t32(counts), T, 32,
                               parents=t32(parents) if words else None, mask_words=max(1, words))
        made.append((m, steps.slots(table, lens, counts, 32, len(refs), T, parents, words)))
    for m, ref in made:
        same_slots(m, ref, 0)
    at = [t.data_ptr() for m, _ in made for t in (m.cu_q, m.positions, m.slots, m.mask) if t is not None and t.numel()]
    assert len(set(at)) == len(at)


def test_slots_into_given_tensors_and_graphs():
    rng = np.random.default_rng(8)
    table, lens, refs, counts = books(rng, 30, 6, 200, 32)
    tb, c, T = gpu_table(table, lens, refs), t32(counts), 200
    out = abi.TokenSlots(*(torch.full((k,), 99, dtype=dt, device="cuda") for k, dt in
                           ((31, torch.int32), (T, torch.int32), (T, torch.int64))))
    assert abi.tq_pages_slots(tb, c, T, 32, out=out) is out
    same_slots(out, steps.slots(table, lens, counts, 32, len(refs), T), 0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m = abi.tq_pages_slots(tb, c, T, 32)
    less = np.maximum(counts - 1, 0)
    c.copy_(t32(less))
    g.replay()
    same_slots(m, steps.slots(table, lens, less, 32, len(refs), T), 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m = abi.tq_pages_slots(tb, c, T, 32)
    side.synchronize()
    same_slots(m, steps.slots(table, lens, less, 32, len(refs), T), 0)
    empty = abi.tq_pages_slots(tb, torch.zeros_like(c), 0, 32)
    assert empty.slots.numel() == 0 and not empty.cu_q.any()


def test_slots_refusals():
    tb, c = gpu_table(np.zeros((2, 2)), np.array([3, 3]), np.ones(2)), t32([1, 1])
    for bad in (c.long(), c.float()):
        with pytest.raises(TypeError):
            abi.tq_pages_slots(tb, bad, 2, 32)
    for bad in (c.cpu(), t32([1, 1, 1]), t32([1, 1, 1, 1])[::2]):
        with pytest.raises(ValueError):
            abi.tq_pages_slots(tb, bad, 2, 32)
    with pytest.raises(ValueError):
        abi.tq_pages_slots(tb, c, 2, 32, parents=t32([-1]))
    with pytest.raises(ValueError):
        abi.tq_pages_slots(tb, c, 2, 32, parents=t32([-1, -1]), mask_words=0)
    with pytest.raises(abi.TQError):
        abi.tq_pages_slots(tb, c, 2, 48)
    with pytest.raises(ValueError):
        abi.tq_pages_slots(tb, c, 2, 32, out=abi.TokenSlots(c, c, c.long()))


# ------------------------------------------------------------ append at slots

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,Hkv,kb,vb", [(32, 1, 2, 3), (64, 3, 4, 2), (128, 8, 4, 3), (256, 2, 3, 4)])
def test_append_slots(d, Hkv, kb, vb, dtype):
    """Bytes of tq_append_paged where there is a slot, nothing anywhere else; K
    and V as slices of a fused projection."""
    rng = np.random.default_rng(d)
    T, page, n_pages = 41, 32, 5
    slots = rng.permutation(n_pages * page)[:T]
    slots[[3, 17]] = [-1, -7]
    x = synth.normal_rows(5, T * (2 * Hkv + 1), d, dtype).reshape(T, (2 * Hkv + 1), d).cuda()
    k, v = x[:, 1:1 + Hkv], x[:, 1 + Hkv:]
    plan = abi.Plan(d, 42)
    caches = []
    for _ in range(2):
        c = abi.PagedCache.empty(n_pages, Hkv, page, d, kb, vb)
        for a in (c.k_packed, c.k_norm, c.v_packed, c.v_norm):
            a.fill_(77)
        caches.append(c)
    abi.tq_append_slots(plan, caches[0], k, v, torch.from_numpy(slots).cuda())
    real = slots >= 0
    abi.tq_append_paged(plan, caches[1], k[real].contiguous(), v[real].contiguous(),
                        t32(slots[real] // page)[:, None].contiguous(), t32(slots[real] % page))
    assert abi.tq_device_status(reset=True) == 0
    for a in ("k_packed", "k_norm", "v_packed", "v_norm"):
        assert torch.equal(getattr(caches[0], a), getattr(caches[1], a)), a
    pg, off = slots[real] // page, slots[real] % page
    compare_encode(O.signs(42, d), kb, k[real].double().cpu().numpy().reshape(-1, d),
                   caches[0].k_packed.cpu().numpy()[pg, :, off].reshape(-1, d * kb // 8),
                   caches[0].k_norm.cpu().numpy()[pg, :, off].reshape(-1))


def test_append_slots_past_the_pool_and_refusals():
    plan, c = abi.Plan(128, 42), abi.PagedCache.empty(2, 2, 32, 128, 4, 3)
    x = torch.randn(3, 6, 128, device="cuda")
    k, v = x[:, :2], x[:, 2:4]
    s = torch.tensor([64, 5, 1 << 40], device="cuda")
    abi.tq_append_slots(plan, c, k, v, s)
    assert abi.tq_device_status(reset=True) == 42
    assert (c.k_norm != 0).sum() == 2 and (c.k_norm[0, :, 5] != 0).all()
    abi.tq_append_slots(plan, c, k[:0], v[:0], s[:0])
    for bad in ((k, v[:2], s), (k, v.bfloat16(), s), (x[:, ::3], x[:, 1::3], s), (k, v, s[:2]), (k, v, s.int()),
                (k, v, s.cpu()), (x[:, :3], x[:, 3:], s), (k[..., :64], v[..., :64], s)):
        with pytest.raises(ValueError):
            abi.tq_append_slots(plan, c, *bad, )
    odd = torch.randn(3 * 257 + 8, device="cuda")[:3 * 257].reshape(3, 257)[:, :256].reshape(3, 2, 128)
    with pytest.raises((abi.TQError, ValueError)):
        abi.tq_append_slots(plan, c, odd.as_strided((3, 2, 128), (257, 128, 1)), v, s)


# ------------------------------------------------------------------ kept rows

def pool(rng, L, n_pages, Hkv, page, d, kb, vb):
    t = lambda *s: torch.from_numpy(rng.integers(0, 256, s, dtype=np.uint8)).cuda()  # noqa: E731
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
    lead = (n_pages, Hkv, page)
    return [abi.PagedCache(t(*lead, d * kb // 8), f(*lead), t(*lead, d * vb // 8), f(*lead), kb, vb) for _ in range(L)]


def arrays(layers):
    return [a.cpu().numpy() for c in layers for a in (c.k_packed, c.k_norm, c.v_packed, c.v_norm)]


def kept_lists(rng, counts, most):
    kept = rng.integers(-5, 1 << 20, (len(counts), most)).astype(np.int32)  # past a list: anything
    n_keep = np.zeros(len(counts), np.int32)
    for b, n in enumerate(counts):
        k = int(rng.integers(0, min(n, most) + 1))
        kept[b, :k] = np.sort(rng.permutation(n)[:k])
        n_keep[b] = k
    return kept, n_keep


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("n,max_new,most,L,Hkv,page,kb,vb", [
    (1, 5, 3, 1, 1, 32, 4, 4), (9, 40, 12, 3, 2, 32, 4, 3), (40, 12, 12, 5, 3, 64, 3, 2), (3, 300, 200, 2, 2, 32, 2, 3)])
def test_keep(n, max_new, most, L, Hkv, page, kb, vb, d):
    rng = np.random.default_rng(d + n)
    table, lens, refs, counts = books(rng, n, max_new, 200, page)
    kept, n_keep = kept_lists(rng, counts, most)
    layers = pool(rng, L, len(refs), Hkv, page, d, kb, vb)
    new, after, status = steps.keep(table, lens, refs, counts, kept, n_keep, page, arrays(layers))
    tb = gpu_table(table, lens, refs)
    got = abi.tq_pages_keep(tb, t32(counts), t32(kept), t32(n_keep), layers)
    assert abi.tq_device_status(reset=True) == status == 0
    assert np.array_equal(got.cpu().numpy(), new)
    for a, b in zip(arrays(layers), after):
        assert np.array_equal(a, b, equal_nan=True)
    assert np.array_equal(tb.block_table.cpu().numpy(), table) and np.array_equal(tb.lens.cpu().numpy(), lens)


def test_keep_of_more_layers_than_a_launch_takes():
    rng = np.random.default_rng(2)
    table, lens, refs, counts = books(rng, 6, 10, 60, 32)
    kept, n_keep = kept_lists(rng, counts, 6)
    layers = pool(rng, 130, len(refs), 1, 32, 32, 4, 2)
    new, after, _ = steps.keep(table, lens, refs, counts, kept, n_keep, 32, arrays(layers))
    got = abi.tq_pages_keep(gpu_table(table, lens, refs), t32(counts), t32(kept), t32(n_keep), abi.PagedLayers(layers))
    assert np.array_equal(got.cpu().numpy(), new)
    assert all(np.array_equal(a, b) for a, b in zip(arrays(layers), after))


@pytest.mark.parametrize("change", [
    dict(counts=-1), dict(counts=90), dict(n_keep=-1), dict(n_keep=11), dict(n_keep=5, most=4), dict(kept=[0, 3, 3]),
    dict(kept=[1, 0, 3]), dict(kept=[0, 2, 10]), dict(kept=[-1, 2, 3]), dict(kept=[0, 2, 1 << 30]), dict(lens=65),
    dict(page=-1), dict(page=6), dict(refs=2)])
def test_keep_leaves_a_row_out(change):
    rng = np.random.default_rng(3)
    table, lens, counts = np.array([[3, 1], [0, 5], [2, 4]], np.int32), np.array([40, 40, 40], np.int32), np.array([10, 10, 10], np.int32)
    refs, n_keep, most = np.ones(6, np.int32), np.array([3, 3, 3], np.int32), change.get("most", 12)
    kept = np.tile(np.array([0, 2, 9] + [0] * 9, np.int32)[:most], (3, 1))
    for name, x in (("counts", counts), ("n_keep", n_keep), ("lens", lens)):
        x[1] = change.get(name, x[1])
    kept[1, :3] = change.get("kept", kept[1, :3])
    table[1, 1] = change.get("page", 5)
    refs[0] = change.get("refs", 1)
    layers = pool(rng, 2, 6, 2, 32, 64, 4, 3)
    new, after, status = steps.keep(table, lens, refs, counts, kept, n_keep, 32, arrays(layers))
    got = abi.tq_pages_keep(gpu_table(table, lens, refs), t32(counts), t32(kept), t32(n_keep), layers)
    assert abi.tq_device_status(reset=True) == status == 66
    assert got.tolist() == new.tolist() == [33, int(lens[1]), 33]
    assert all(np.array_equal(a, b) for a, b in zip(arrays(layers), after))


def test_keep_refusals():
    layers = pool(np.random.default_rng(1), 1, 4, 1, 32, 64, 4, 3)
    tb = gpu_table(np.zeros((2, 2)), np.array([5, 5]), np.ones(4))
    c, k, n = t32([3, 3]), t32(np.zeros((2, 4))), t32([1, 1])
    for bad in ((c[:1], k, n), (c, k[0], n), (c, k, n[:1]), (c.cpu(), k, n), (c, k.T, n)):
        with pytest.raises(ValueError):
            abi.tq_pages_keep(tb, *bad, layers)
    with pytest.raises(TypeError):
        abi.tq_pages_keep(tb, c.long(), k, n, layers)
    with pytest.raises(abi.TQError):
        abi.tq_pages_keep(tb, c, k, n, layers, out=tb.lens)
    with pytest.raises(abi.TQError):
        abi.tq_pages_keep(tb, c, k[:, :0], n, layers)


# ------------------------------------------------------------- all of a step

@pytest.mark.parametrize("graph", [False, True])
def test_a_speculative_step(graph):
    """Pages for the drafts, the slot map, the append in every layer, the trees'
    attention, the accepted paths kept, the left-over pages given back -- then a
    step of single tokens with sinks: captured or not, everything on the device."""
    rng = np.random.default_rng(9)
    n, page, d, Hkv, Hq, kb, vb, L, n_pages, words = 5, 32, 128, 2, 8, 4, 3, 2, 60, 1
    plan, scale = abi.Plan(d, 42), 1 / math.sqrt(d)
    s = O.signs(42, d)
    layers = [abi.PagedCache.empty(n_pages, Hkv, page, d, kb, vb) for _ in range(L)]
    held = abi.PagedLayers(layers)
    draft = np.array([7, 0, 12, 1, 30])
    ctx = np.array([40, 33, 100, 0, 64])
    T, parents = 56, sum(random_trees(rng, [(int(x), 0) for x in draft])[0], []) + [0] * 6
    par = [parents[i:i + k] for i, k in zip(np.concatenate([[0], np.cumsum(draft)[:-1]]), draft)]
    # accepted: a path down each tree
    kept, n_keep = np.zeros((n, 8), np.int32), np.zeros(n, np.int32)
    for b, tree in enumerate(par):
        at = -1
        while n_keep[b] < 6:
            kids = [i for i, p in enumerate(tree) if p == at and i > at]
            if not kids:
                break
            at = int(rng.choice(kids))
            kept[b, n_keep[b]] = at
            n_keep[b] += 1
    g = torch.Generator().manual_seed(4)
    ctx_rows = torch.randn(L, 2, int(ctx.sum()), Hkv, d, generator=g).to(torch.bfloat16)
    new_rows = torch.randn(L, 2, T, Hkv, d, generator=g).to(torch.bfloat16)
    last_rows = torch.randn(L, 2, n, Hkv, d, generator=g).to(torch.bfloat16)
    q = torch.randn(T, Hq, d, generator=g).to(torch.bfloat16)
    q1 = torch.randn(n, Hq, d, generator=g).to(torch.bfloat16)
    dev = dict(new=new_rows.cuda(), last=last_rows.cuda(), q=q.cuda(), q1=q1.cuda(), draft=t32(draft), par=t32(parents),
               kept=t32(kept), n_keep=t32(n_keep), one=t32(np.ones(n)), ctx=t32(ctx))

    table = abi.PageTable.empty(n, 8, n_pages)
    table, info = abi.tq_pages_resize(table, dev["ctx"], held)
    m = abi.tq_pages_slots(table, table.lens, int(ctx.sum()), page)
    for l, c in enumerate(layers):
        abi.tq_append_slots(plan, c, ctx_rows[l, 0].cuda(), ctx_rows[l, 1].cuda(), m.slots)

    def step(table):
        grown, _ = abi.tq_pages_resize(table, dev["ctx"] + dev["draft"], held)
        m = abi.tq_pages_slots(grown, dev["draft"], T, page, parents=dev["par"], mask_words=words)
        outs = []
        for l, c in enumerate(layers):
            abi.tq_append_slots(plan, c, dev["new"][l, 0], dev["new"][l, 1], m.slots)
            outs.append(abi.tq_attn_tree_paged(plan, dev["q"], m.cu_q, c, grown.block_table, grown.lens, m.mask, scale))
        lens = abi.tq_pages_keep(grown, dev["draft"], dev["kept"], dev["n_keep"], held)
        cut, _ = abi.tq_pages_resize(grown, lens, held)
        last, info = abi.tq_pages_resize(cut, cut.lens + 1, held)
        m1 = abi.tq_pages_slots(last, dev["one"], n, page)
        for l, c in enumerate(layers):
            abi.tq_append_slots(plan, c, dev["last"][l, 0], dev["last"][l, 1], m1.slots)
            outs.append(abi.tq_attn_sinks_paged(plan, dev["q1"], m1.cu_q, c, last.block_table, last.lens, scale, 20, 3))
        return m, outs, last, info

    if graph:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            m, outs, last, info = step(table)
        gr.replay()
    else:
        m, outs, last, info = step(table)
    torch.cuda.synchronize()
    assert abi.tq_device_status(reset=True) == 0
    assert info.tolist()[1] == 0 and last.lens.tolist() == (ctx + n_keep + 1).tolist()
    assert int((last.refs > 0).sum()) == int((-(-(ctx + n_keep + 1) // page)).sum())

    # the same from the rows themselves, encoded by the oracle
    def decoded(x, bits):
        p, nm = O.encode(s, bits, x.double().numpy().reshape(-1, d))
        return O.decode(s, bits, p, nm).reshape(*x.shape[:-1], d)

    starts = np.concatenate([[0], np.cumsum(ctx)])
    cu = np.concatenate([[0], np.cumsum(draft)])

    class Rows:
        pass

    for l in range(L):
        for phase in (0, 1):
            bt = Rows()
            bt.Hq, bt.Hkv, bt.d = Hq, Hkv, d
            old = [decoded(ctx_rows[l, i], (kb, vb)[i]) for i in (0, 1)]
            new = [decoded(new_rows[l, i], (kb, vb)[i]) for i in (0, 1)]
            end = [decoded(last_rows[l, i], (kb, vb)[i]) for i in (0, 1)]
            rows, seen, lens = [], [], []
            for b in range(n):
                pick = np.arange(draft[b]) if phase == 0 else kept[b, :n_keep[b]]
                rows.append([np.concatenate([o[starts[b]:starts[b + 1]], w[cu[b] + pick]] + ([e[b:b + 1]] if phase else []))
                             .swapaxes(0, 1) for o, w, e in zip(old, new, end)])
                c = rows[-1][0].shape[1]
                k = int(draft[b]) if phase == 0 else 1
                lens.append((k, c))
                if phase == 0:
                    see = np.zeros((k, c), bool)
                    see[:, :ctx[b]] = True
                    for i, p in enumerate(par[b]):
                        if p >= 0:
                            see[i, ctx[b]:] = see[p, ctx[b]:]
                        see[i, ctx[b] + i] = True
                else:
                    j = np.arange(c)
                    see = ((j > c - 1 - 20) | (j < 3))[None]
                seen.append(see)
            bt.lens, bt.q = lens, q if phase == 0 else q1
            bt.cu = cu if phase == 0 else np.arange(n + 1)
            bt.decoded = lambda b: rows[b]
            check(outs[l + L * phase], *want(bt, scale, seen), int(bt.cu[-1]))
