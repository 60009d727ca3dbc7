"""Cases for speculative and long-running serving over the paged packed cache:
attention of the nodes of drafted trees, attention over a sliding window with a
few first positions that stay visible, a step's slot map, and the keeping of an
accepted path of drafted rows.

`run` computes an operator in plain torch, or (with `own`) through the
package's entry points.  The page contents are rows of the codec's format: a
fp32 norm and 2-, 3- or 4-bit indices of the Lloyd-Max codebook per
coordinate, in the rotated domain.
"""
from __future__ import annotations

import functools
import math
import random

import numpy as np
import torch

own = False

SEED = 42  # of the plan's sign diagonal


# ------------------------------------------------------------------ the cases

def listed():
    llama = {"Hq": 32, "Hkv": 8, "d": 128, "kb": 4, "vb": 3}
    return [
        # one draft of a few nodes for two short conversations: latency counts
        {"name": "tree few", "op": "tree", "B": 2, "q_lo": 6, "q_hi": 8, "c_lo": 200, "c_hi": 900, "page": 64, "mix": 1,
         **llama},
        # a serving step in which every conversation has a small tree to be checked
        {"name": "tree batch", "op": "tree", "B": 32, "q_lo": 10, "q_hi": 24, "c_lo": 1000, "c_hi": 8000, "page": 256,
         "mix": 2, **llama},
        # wide trees over long contexts
        {"name": "tree long", "op": "tree", "B": 8, "q_lo": 40, "q_hi": 64, "c_lo": 16000, "c_hi": 32000, "page": 256,
         "mix": 3, **llama},
        # a d = 256 model, odd numbers of nodes
        {"name": "tree d256", "op": "tree", "B": 5, "q_lo": 5, "q_hi": 33, "c_lo": 700, "c_hi": 6000, "page": 32,
         "mix": 4, "Hq": 8, "Hkv": 4, "d": 256, "kb": 4, "vb": 4},
        # single tokens of a few short conversations: latency counts
        {"name": "sinks few", "op": "sinks", "B": 4, "q_lo": 1, "q_hi": 1, "c_lo": 300, "c_hi": 2000, "page": 64,
         "window": 256, "sinks": 4, "mix": 5, **llama},
        # a decode step of many long-running conversations
        {"name": "sinks decode", "op": "sinks", "B": 64, "q_lo": 1, "q_hi": 1, "c_lo": 5000, "c_hi": 30000, "page": 256,
         "window": 4096, "sinks": 4, "mix": 6, **llama},
        # two long prompts taken in chunks of 4096 tokens
        {"name": "sinks chunk", "op": "sinks", "B": 2, "q_lo": 4096, "q_hi": 4096, "c_lo": 8000, "c_hi": 12000,
         "page": 256, "window": 4096, "sinks": 4, "mix": 7, **llama},
        # single tokens and odd chunks in one step, a d = 64 model with three heads a group
        {"name": "sinks mixed d64", "op": "sinks", "B": 9, "q_lo": 1, "q_hi": 300, "c_lo": 50, "c_hi": 5000, "page": 32,
         "window": 777, "sinks": 37, "mix": 8, "Hq": 12, "Hkv": 4, "d": 64, "kb": 3, "vb": 2},
        # where the tokens of a decode step go
        {"name": "slots step", "op": "slots", "n_seqs": 64, "q_lo": 1, "q_hi": 1, "len_hi": 2000, "max_pages": 64,
         "page": 64, "pad": 0, "words": 0, "mix": 9},
        # the drafted trees of many conversations, in buffers with room for more
        {"name": "slots trees", "op": "slots", "n_seqs": 256, "q_lo": 10, "q_hi": 64, "len_hi": 8000, "max_pages": 64,
         "page": 256, "pad": 500, "words": 2, "mix": 10},
        # the accepted tokens of a few conversations
        {"name": "keep few", "op": "keep", "n_seqs": 4, "q_lo": 6, "q_hi": 8, "len_hi": 900, "most": 4, "L": 2,
         "page": 64, "mix": 52, "Hkv": 8, "d": 128, "kb": 4, "vb": 3},
        # the accepted paths of a serving step, 32 layers
        {"name": "keep batch", "op": "keep", "n_seqs": 64, "q_lo": 10, "q_hi": 60, "len_hi": 2000, "most": 8, "L": 32,
         "page": 64, "mix": 16, "Hkv": 8, "d": 128, "kb": 4, "vb": 3},
    ]


def draw(rng):
    def logint(lo, hi):
        return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))

    d = rng.choice((64, 128, 128, 256))
    heads = {"Hkv": rng.choice((1, 2, 3, 4, 8)), "d": d, "kb": rng.choice((2, 3, 4)), "vb": rng.choice((2, 3, 4)),
             "page": rng.choice((32, 64, 128, 256)), "mix": rng.randrange(1 << 20)}
    op = rng.choice(("tree", "tree", "sinks", "sinks", "slots", "keep"))
    if op in ("tree", "sinks"):
        tree = op == "tree"
        q_hi, c_hi, B = logint(1, 128 if tree else 4096), logint(1, 32000), logint(1, 64)
        if not tree and rng.random() < 0.4:
            q_hi = 1  # a decode step
        Hq = heads["Hkv"] * rng.choice((1, 2, 3, 4, 5, 8))
        # the plain form's scores and rows stay under half of the longest listed cases'
        while B * q_hi * (q_hi + c_hi) * Hq > 2e9 or B * (q_hi + c_hi) * heads["Hkv"] * d > 8e8:
            q_hi, B, c_hi = max(1, q_hi - q_hi // 4), max(1, B - B // 3), max(1, c_hi - c_hi // 8)
        case = {"op": op, "B": B, "q_lo": logint(1, q_hi), "q_hi": q_hi, "c_lo": logint(1, c_hi), "c_hi": c_hi, "Hq": Hq,
                **heads}
        return case if tree else {**case, "window": logint(16, 8192), "sinks": rng.choice((0, 1, 4, 4, logint(1, 300)))}
    if op == "slots":
        words = rng.choice((0, 0, 1, 2, 4))
        q_hi = logint(1, 32 * words if words else 2000)
        n_seqs, len_hi = min(logint(1, 2000), 200000 // q_hi), logint(max(40, q_hi), 30000)
        return {"op": op, "n_seqs": n_seqs, "q_lo": rng.choice((0, logint(1, q_hi))), "q_hi": q_hi, "len_hi": len_hi,
                "max_pages": -(-len_hi // heads["page"]) + rng.randrange(5), "page": heads["page"],
                "pad": rng.choice((0, logint(1, 1000))), "words": words, "mix": heads["mix"]}
    n_seqs, q_hi = logint(1, 200), logint(1, 128)
    len_hi = logint(max(40, q_hi), 2500)
    page_bytes = heads["Hkv"] * heads["page"] * (d * (heads["kb"] + heads["vb"]) // 8 + 8)
    n_seqs = max(1, min(n_seqs, int(1.8e9 / (page_bytes * (len_hi // heads["page"] + 2)))))
    case = {"op": op, "n_seqs": n_seqs, "q_lo": logint(1, q_hi), "q_hi": q_hi, "len_hi": len_hi, "most": logint(1, 16),
            **heads}
    n_pages = _books(case)[4]
    return {**case, "L": max(1, min(logint(1, 32), int(2.0e9 / (page_bytes * n_pages))))}


# ------------------------------------------------------- shapes behind a case

def _spread(rng, lo, hi):
    lo, hi = min(lo, hi), max(lo, hi)
    if lo < 1:
        return rng.randint(lo, hi)
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _lengths(case):
    """The numbers of new tokens and the context lengths of a batch."""
    rng = random.Random(case["mix"])
    q = [_spread(rng, case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    return q, [n + _spread(rng, case["c_lo"], case["c_hi"]) for n in q]


def _trees(case, counts):
    """Parents of drafted nodes, each in front of its children (-1: a child of
    the last token before the draft): a few candidates per node, best first."""
    rng = random.Random(case["mix"] + 1)
    out = []
    for n in counts:
        reach = rng.randint(1, max(1, n // 3))
        out.append([-1 if i == 0 or rng.random() < 0.05 else rng.randrange(max(0, i - reach), i) for i in range(n)])
    return out


def _masks(parents, words):
    """[nodes, words] int32: bit j of row t: node t sees node j."""
    rows = []
    for tree in parents:
        seen = []
        for t, p in enumerate(tree):
            seen.append((seen[p] if p >= 0 else 0) | 1 << t)
        rows += seen
    return np.array([[r >> 32 * w & 0xFFFFFFFF for w in range(words)] for r in rows],
                    dtype=np.uint32).reshape(-1, words).view(np.int32)


def _books(case):
    """(new tokens, lengths, pages needed, longest row's pages, pages of the pool)"""
    rng = random.Random(case["mix"])
    counts = [_spread(rng, case["q_lo"], case["q_hi"]) for _ in range(case["n_seqs"])]
    lens = [n + rng.randrange(0, max(1, case["len_hi"] - n + 1)) for n in counts]
    need = [-(-n // case["page"]) for n in lens]
    return counts, lens, need, max(need + [1]), sum(need) + 3


def _paths(case, counts):
    """The accepted nodes of each row, root first: a walk down its tree."""
    rng = random.Random(case["mix"] + 2)
    out = []
    for tree in _trees(case, counts):
        want, path, at = rng.randint(0, case["most"]), [], -1
        while len(path) < want:
            children = [i for i, p in enumerate(tree) if p == at and i > at]
            if not children:
                break
            at = rng.choice(children)
            path.append(at)
        out.append(path)
    return out


def work(case):
    if case["op"] in ("tree", "sinks"):
        row = case["d"] * (case["kb"] + case["vb"]) // 8 + 8  # packed K and V and their norms
        q, ctx = _lengths(case)
        pairs = read = 0
        if case["op"] == "tree":
            masks = _masks(_trees(case, q), 1 + (max(q) - 1) // 32)
            pairs = sum(n * (c - n) for n, c in zip(q, ctx)) + int(np.unpackbits(masks.view(np.uint8)).sum())
            read = sum(ctx)
        else:
            w, s = case["window"], case["sinks"]
            for n, c in zip(q, ctx):
                at = np.arange(c - n, c)
                pairs += int((np.minimum(at + 1, w) + np.minimum(s, np.maximum(at + 1 - w, 0))).sum())
                read += min(c, n - 1 + w) + min(s, max(0, c - (n - 1 + w)))
        return {"bytes": read * case["Hkv"] * row + sum(q) * case["Hq"] * case["d"] * 4,
                "flops": 4 * case["Hq"] * case["d"] * pairs}
    counts, lens, need, longest, n_pages = _books(case)
    if case["op"] == "slots":
        total, page = sum(counts), case["page"]
        pages = sum(-(-n // page) - (n - k) // page for k, n in zip(counts, lens) if k)
        return {"bytes": 4 * (3 * len(lens) + 1) + 4 * pages + (total + case["pad"]) * (12 + 4 * case["words"])
                + (4 * total if case["words"] else 0), "flops": 0}
    row = case["d"] * (case["kb"] + case["vb"]) // 8 + 8
    moved = sum(i != j for path in _paths(case, counts) for i, j in enumerate(path))
    return {"bytes": 2 * moved * case["L"] * case["Hkv"] * row + 16 * len(lens), "flops": 0}


# ------------------------------------------------------------------ the codec

@functools.lru_cache(maxsize=None)
def _codebook(d, bits):
    """(centroids, boundaries), float32: the Lloyd-Max codebook of one
    coordinate of a uniform unit vector in R^d, density ~ (1 - x^2)^((d-3)/2)."""
    H = 1 << (bits - 1)

    def cumulative(x):  # int_0^asin(x) cos^(d-2), by the reduction formula
        t = np.arcsin(x)
        s, c2 = np.sin(t), np.cos(t) ** 2
        w, power = (t, np.cos(t)) if d % 2 == 0 else (s, c2)
        for k in range(2 + d % 2, d - 1, 2):
            w = power * s / k + (k - 1) / k * w
            power = power * c2
        return w

    edges = np.linspace(0.0, min(1.0, 2.5 / math.sqrt(d)), H + 1)
    edges[-1] = 1.0
    centres = np.zeros(H)
    for _ in range(20000):
        m = (1.0 - edges ** 2) ** (0.5 * (d - 1)) / (d - 1)
        new = (m[:-1] - m[1:]) / np.diff(cumulative(edges))
        moved, centres = np.max(np.abs(new - centres)), new
        if moved < 1e-14:
            break
        edges[1:-1] = 0.5 * (centres[1:] + centres[:-1])
    inner = edges[1:-1]
    return (np.concatenate([-centres[::-1], centres]).astype(np.float32),
            np.concatenate([-inner[::-1], [0.0], inner]).astype(np.float32))


@functools.lru_cache(maxsize=None)
def _signs(d):
    """The seeded sign diagonal: top bits of the splitmix64 stream."""
    out, state, mask = [], SEED, (1 << 64) - 1
    for _ in range(d):
        state = (state + 0x9E3779B97F4A7C15) & mask
        z = ((state ^ (state >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        out.append(-1.0 if (z ^ (z >> 31)) >> 63 else 1.0)
    return np.array(out)


def _rotation(d, dtype):
    """R = H diag(s) / sqrt(d), H the Sylvester Hadamard matrix."""
    H = np.ones((1, 1))
    while H.shape[0] < d:
        H = np.block([[H, H], [H, -H]])
    return torch.from_numpy(H * _signs(d) / math.sqrt(d)).to("cuda", dtype)


def _pack(idx, bits):
    """[..., d] indices -> [..., d * bits / 8] bytes, a dense LSB-first bit stream."""
    at = torch.arange(8, device=idx.device)
    word = (idx.reshape(*idx.shape[:-1], -1, 8).to(torch.int64) << (bits * at)).sum(-1, keepdim=True)
    return ((word >> (8 * at[:bits])) & 255).to(torch.uint8).reshape(*idx.shape[:-1], -1)


def _unpack(packed, bits):
    at = torch.arange(8, device=packed.device)
    word = (packed.reshape(*packed.shape[:-1], -1, bits).to(torch.int64) << (8 * at[:bits])).sum(-1, keepdim=True)
    return ((word >> (bits * at)) & ((1 << bits) - 1)).reshape(*packed.shape[:-1], -1)


def _rows(g, shape, d, bits):
    """Encoded rows (packed, norms): rotated activations are near normal, their norms vary."""
    y = torch.randn(*shape, d, generator=g, device="cuda")
    norm = y.norm(dim=-1) * torch.exp(0.25 * torch.randn(*shape, generator=g, device="cuda"))
    bounds = torch.from_numpy(_codebook(d, bits)[1]).cuda()
    return _pack(torch.bucketize(y / y.norm(dim=-1, keepdim=True), bounds, right=True), bits), norm


# ---------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    st = {"case": case}
    {"tree": _prepare_attn, "sinks": _prepare_attn, "slots": _prepare_slots, "keep": _prepare_keep}[case["op"]](case, g, st)
    return st


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(g, need, n_pages, max_pages):
    """Block table of rows with pages in shuffled order, -1 past each row's."""
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor(np.concatenate([[0], np.cumsum(need)[:-1]]), device="cuda")
    col = torch.arange(max_pages, device="cuda")
    at = (first[:, None] + col).clamp(max=n_pages - 1)
    return torch.where(col < torch.tensor(need, device="cuda")[:, None], ids[at], -1).to(torch.int32)


def _prepare_attn(case, g, st):
    d, Hkv, page = case["d"], case["Hkv"], case["page"]
    q_lens, ctx = _lengths(case)
    need = [-(-c // page) for c in ctx]
    n_pages = sum(need) + 3
    st["table"] = _table(g, need, n_pages, max(need) + 1)
    k, kn = _rows(g, (n_pages, Hkv, page), d, case["kb"])
    v, vn = _rows(g, (n_pages, Hkv, page), d, case["vb"])
    total = sum(q_lens)
    st.update(k=k, kn=kn, v=v, vn=vn, ctx=_ints(ctx), cu=_ints([0] + list(np.cumsum(q_lens))),
              max_q=max(q_lens), max_ctx=max(ctx), scale=1.0 / math.sqrt(d),
              q=torch.randn(total, case["Hq"], d, generator=g, device="cuda").to(torch.bfloat16),
              out=torch.zeros(total, case["Hq"], d, dtype=torch.bfloat16, device="cuda"))
    if case["op"] == "tree":
        st["mask"] = torch.from_numpy(_masks(_trees(case, q_lens), 1 + (max(q_lens) - 1) // 32)).cuda()
    if own:
        from kv_cache_vector_gb300 import abi
        st["plan"] = abi.Plan(d, SEED)
        st["cache"] = abi.PagedCache(k, kn, v, vn, case["kb"], case["vb"])
        size = abi.tq_attn_tree_paged_workspace_bytes if case["op"] == "tree" else abi.tq_attn_sinks_paged_workspace_bytes
        st["ws"] = torch.empty(size(case["Hq"], Hkv, d), dtype=torch.uint8, device="cuda")


def _prepare_slots(case, g, st):
    counts, lens, need, longest, n_pages = _books(case)
    st["table"] = _table(g, need, n_pages, max(longest, case["max_pages"]))
    st.update(lens=_ints(lens), counts=_ints(counts), n_pages=n_pages, n_tokens=sum(counts) + case["pad"])
    if case["words"]:
        st["parents"] = _ints(sum(_trees(case, counts), []) + [0] * case["pad"])
        st["max_q"] = max(max(counts), 1)
    if own:
        from kv_cache_vector_gb300 import abi
        st["pages"] = abi.PageTable(st["table"], st["lens"], torch.zeros(n_pages, dtype=torch.int32, device="cuda"))


def _prepare_keep(case, g, st):
    counts, lens, need, longest, n_pages = _books(case)
    paths = _paths(case, counts)
    st["table"] = _table(g, need, n_pages, longest)
    keep = np.full((len(paths), case["most"]), -1, dtype=np.int32)
    for i, path in enumerate(paths):
        keep[i, :len(path)] = path
    st.update(lens=_ints(lens), counts=_ints(counts), keep=torch.from_numpy(keep).cuda(),
              n_keep=_ints([len(p) for p in paths]))
    lead = (case["L"], n_pages, case["Hkv"], case["page"])

    def data(bits):
        n = math.prod(lead) * case["d"] * bits // 8
        x = torch.randint(-2 ** 31, 2 ** 31 - 1, (n // 4,), generator=g, device="cuda", dtype=torch.int32)
        return x.view(torch.uint8).reshape(*lead, -1)

    def norms():
        return torch.randn(*lead, generator=g, device="cuda").abs_() + 8.0

    st["pool"] = {"k": data(case["kb"]), "kn": norms(), "v": data(case["vb"]), "vn": norms()}
    if own:
        from kv_cache_vector_gb300 import abi
        p = st["pool"]
        st["layers"] = abi.PagedLayers([abi.PagedCache(p["k"][i], p["kn"][i], p["v"][i], p["vn"][i], case["kb"],
                                                       case["vb"]) for i in range(case["L"])])
        refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        refs[st["table"][st["table"] >= 0].long()] = 1
        st["pages"] = abi.PageTable(st["table"], st["lens"], refs)


# -------------------------------------------------------------------- a pass

def run(st):
    return {"tree": _attn, "sinks": _attn, "slots": _slots, "keep": _keep}[st["case"]["op"]](st)


def _attn(st):
    case = st["case"]
    if own:
        from kv_cache_vector_gb300 import abi
        where = (st["plan"], st["q"], st["cu"], st["cache"], st["table"], st["ctx"])
        if case["op"] == "tree":
            return abi.tq_attn_tree_paged(*where, st["mask"], st["scale"], out=st["out"], workspace=st["ws"])
        return abi.tq_attn_sinks_paged(*where, st["scale"], case["window"], case["sinks"], out=st["out"],
                                       workspace=st["ws"])
    d, G, page, dev = case["d"], case["Hq"] // case["Hkv"], case["page"], st["q"].device
    cu, ctx = st["cu"].long(), st["ctx"].long()
    n = cu[1:] - cu[:-1]
    at = torch.arange(st["max_ctx"], device=dev)
    ids = st["table"][:, at // page].long().clamp(min=0)  # [B, C]
    off = (at % page).expand_as(ids)

    def rows(packed, norm, bits):  # [B, Hkv, C, d] in the rotated domain
        cen = torch.from_numpy(_codebook(d, bits)[0]).to(dev)
        x = cen[_unpack(packed[ids, :, off], bits)] * norm[ids, :, off][..., None]
        return x.permute(0, 2, 1, 3)

    k, v = rows(st["k"], st["kn"], case["kb"]), rows(st["v"], st["vn"], case["vb"])
    R = _rotation(d, torch.float32)
    t = torch.arange(st["max_q"], device=dev)
    take = (cu[:-1, None] + t).clamp(max=st["q"].shape[0] - 1)
    q = (st["q"].float() @ R.T)[take]  # [B, T, Hq, d]
    q = q.reshape(*take.shape, case["Hkv"], G, d).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, Hkv, G T, d]
    s = (q @ k.transpose(2, 3)).unflatten(2, (G, -1)).mul_(st["scale"])  # [B, Hkv, G, T, C]
    base = (ctx - n)[:, None]
    if case["op"] == "tree":
        node = (at - base)[:, None]  # [B, 1, C]: the node at a position
        word = st["mask"][take].gather(2, (node.clamp(0, st["max_q"] - 1) // 32).expand(-1, t.numel(), -1))
        seen = (node < 0) | ((node < n[:, None, None]) & ((word >> node.clamp(min=0) % 32) & 1 > 0))
    else:
        pos = (base + t)[..., None]  # [B, T, 1]
        seen = (at <= pos) & ((at > pos - case["window"]) | (at < case["sinks"]))
    s.masked_fill_(~seen[:, None, None], -torch.inf)
    s.sub_(s.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)).exp_()
    total = s.sum(-1, keepdim=True).clamp(min=1e-30)
    o = (s.flatten(2, 3) @ v).unflatten(2, (G, -1)) / total
    o = (o @ R).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B, T, Hq, d]
    real = (t < n[:, None]).flatten()
    st["out"][take.flatten()[real]] = o.flatten(0, 1)[real].to(torch.bfloat16)
    return st["out"]


def _slots(st):
    case, T = st["case"], st["n_tokens"]
    if own:
        from kv_cache_vector_gb300 import abi
        m = abi.tq_pages_slots(st["pages"], st["counts"], T, case["page"], parents=st.get("parents"),
                               mask_words=case["words"])
        return {"cu_q": m.cu_q, "positions": m.positions, "slots": m.slots, "mask": m.mask}
    cu = torch.cat([st["counts"].new_zeros(1), torch.cumsum(st["counts"], 0, dtype=torch.int32)])
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    real = t < cu[-1]
    row = torch.searchsorted(cu[1:], t, right=True).clamp(max=cu.numel() - 2)
    i = t - cu[row]  # of the row's new tokens
    base = (st["lens"] - st["counts"])[row]
    at = torch.where(real, base + i, 0)
    page = st["table"][row, at // case["page"]].long()
    out = {"cu_q": cu, "slots": torch.where(real, page * case["page"] + at % case["page"], -1), "positions": at,
           "mask": None}
    if not case["words"]:
        return out
    # who sees whom, by squaring: [rows, nodes, nodes], node t of a row sees node j
    n = st["max_q"]
    sees = torch.eye(n, device="cuda").repeat(cu.numel() - 1, 1, 1)
    child = real & (st["parents"] >= 0)
    sees[row[child], i[child].long(), st["parents"][child].long()] = 1.0
    for _ in range((n - 1).bit_length()):
        sees = (sees @ sees).clamp_(max=1.0)
    j = torch.arange(32 * case["words"], device="cuda")
    bits = torch.zeros(T, j.numel(), dtype=torch.int64, device="cuda")
    bits[:, :n] = torch.where(real[:, None], sees[row, i.long().clamp(max=n - 1)], 0.0).long()
    words = (bits.unflatten(1, (-1, 32)) << (j[:32])).sum(-1)
    out["mask"] = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    depth = bits.sum(1) - 1
    out["positions"] = torch.where(real, base + depth, 0).to(torch.int32)
    return out


def _keep(st):
    pool = st["pool"]
    if own:
        from kv_cache_vector_gb300 import abi
        new = abi.tq_pages_keep(st["pages"], st["counts"], st["keep"], st["n_keep"], st["layers"])
        return {"lens": new, "pool": pool}
    page = st["case"]["page"]
    i = torch.arange(st["keep"].shape[1], device="cuda")
    base = (st["lens"] - st["counts"])[:, None]
    moves = i < st["n_keep"][:, None]
    row = torch.arange(base.shape[0], device="cuda")[:, None].expand_as(moves)[moves]
    src, dst = (base + st["keep"])[moves].long(), (base + i)[moves].long()
    ps, pd = st["table"][row, src // page].long(), st["table"][row, dst // page].long()
    for x in pool.values():  # every row is read before one is written
        x[:, pd, :, dst % page] = x[:, ps, :, src % page]
    return {"lens": st["lens"] - st["counts"] + st["n_keep"], "pool": pool}


# --------------------------------------------------------------- 64-bit values

def exact(case, seed):
    """The attention from its definition in 64 bits: rows decoded to the
    original domain, one (sequence, query head) at a time.  The other operators
    give whole values or move them and have none."""
    if case["op"] not in ("tree", "sinks"):
        return None
    st = prepare(case, seed)
    d, G, page = case["d"], case["Hq"] // case["Hkv"], case["page"]
    R = _rotation(d, torch.float64)
    cu, ctx = st["cu"].tolist(), st["ctx"].tolist()
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")

    def decoded(packed, norm, bits, pages, n, h):
        cen = torch.from_numpy(_codebook(d, bits)[0].astype(np.float64)).cuda()
        y = cen[_unpack(packed[pages, h], bits)] * norm[pages, h].double()[..., None]
        return y.flatten(0, 1)[:n] @ R

    for b, n in enumerate(ctx):
        lo, hi = cu[b], cu[b + 1]
        m = hi - lo
        pages = st["table"][b, :-(-n // page)].long()
        j = torch.arange(n, device="cuda")
        if case["op"] == "tree":
            seen = torch.ones(m, n, dtype=torch.bool, device="cuda")
            x = torch.arange(m, device="cuda")
            seen[:, n - m:] = ((st["mask"][lo:hi].long()[:, x // 32] >> (x % 32)) & 1).bool()
        else:
            pos = torch.arange(n - m, n, device="cuda")[:, None]
            seen = (j <= pos) & ((pos - j < case["window"]) | (j < case["sinks"]))
        for h in range(case["Hkv"]):
            k = decoded(st["k"], st["kn"], case["kb"], pages, n, h)
            v = decoded(st["v"], st["vn"], case["vb"], pages, n, h)
            for r in range(h * G, (h + 1) * G):
                s = (st["q"][lo:hi, r].double() @ k.T) * st["scale"]
                out[lo:hi, r] = torch.softmax(s.masked_fill(~seen, -torch.inf), -1) @ v
    return out
