"""Cases for the paged cache's operators: multi-token attention over the packed
pages, and the upkeep of the pages themselves (copy, fork, resize, compact).

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
        # checking a few drafted tokens of a handful of conversations: latency counts
        {"name": "attn verify", "op": "attn", "B": 4, "q_lo": 3, "q_hi": 6, "c_lo": 400, "c_hi": 2000,
         "page": 64, "window": 0, "mix": 1, **llama},
        # a serving step that mixes single tokens, short prompts and prompt chunks
        {"name": "attn mixed batch", "op": "attn", "B": 32, "q_lo": 1, "q_hi": 512, "c_lo": 200, "c_hi": 7600,
         "page": 256, "window": 0, "mix": 2, **llama},
        # two long prompts taken in chunks of 4096 tokens
        {"name": "attn long chunk", "op": "attn", "B": 2, "q_lo": 4096, "q_hi": 4096, "c_lo": 8000, "c_hi": 12000,
         "page": 256, "window": 0, "mix": 3, **llama},
        # a sliding-window layer of a d = 256 model, odd chunk lengths
        {"name": "attn window d256", "op": "attn", "B": 5, "q_lo": 700, "q_hi": 1500, "c_lo": 900, "c_hi": 5000,
         "page": 32, "window": 1024, "mix": 4, "Hq": 8, "Hkv": 4, "d": 256, "kb": 4, "vb": 4},
        # a few pages of a prefix moved inside a small pool
        {"name": "copy few", "op": "copy", "n": 5, "n_pages": 64, "same": True, "L": 2, "Hkv": 8, "page": 64,
         "d": 128, "kb": 4, "vb": 3, "mix": 5},
        # near half of a 32-layer pool taken out to another one
        {"name": "copy pool", "op": "copy", "n": 473, "n_pages": 1000, "same": False, "L": 32, "Hkv": 8, "page": 64,
         "d": 128, "kb": 4, "vb": 3, "mix": 6},
        # one conversation branched
        {"name": "fork one", "op": "fork", "n_seqs": 8, "max_pages": 32, "len_hi": 1500, "family": 2, "L": 2,
         "Hkv": 8, "page": 64, "d": 128, "kb": 4, "vb": 3, "change": 0.4, "spare": 16, "mix": 7},
        # the rows of a beam search reordered, 16 layers
        {"name": "fork beams", "op": "fork", "n_seqs": 256, "max_pages": 64, "len_hi": 2000, "family": 8, "L": 16,
         "Hkv": 8, "page": 64, "d": 128, "kb": 4, "vb": 3, "change": 0.7, "spare": 260, "mix": 8},
        # the pages of one decode step
        {"name": "resize step", "op": "resize", "n_seqs": 64, "max_pages": 64, "len_hi": 2000, "family": 1, "L": 2,
         "Hkv": 8, "page": 64, "d": 128, "kb": 4, "vb": 3, "grow": 1, "change": 1.0, "spare": 100, "mix": 9},
        # many requests at once: ended ones freed, prompts started, shared tails made private
        {"name": "resize many", "op": "resize", "n_seqs": 512, "max_pages": 96, "len_hi": 1200, "family": 4, "L": 10,
         "Hkv": 4, "page": 32, "d": 256, "kb": 4, "vb": 4, "grow": 700, "change": 0.8, "spare": 600, "mix": 10},
        # a small pool closed up
        {"name": "compact small", "op": "compact", "n_seqs": 16, "max_pages": 32, "len_hi": 700, "family": 2, "L": 2,
         "Hkv": 8, "page": 64, "d": 128, "kb": 4, "vb": 3, "spare": 90, "mix": 11},
        # a half-empty 32-layer pool closed up
        {"name": "compact pool", "op": "compact", "n_seqs": 64, "max_pages": 64, "len_hi": 2600, "family": 2, "L": 32,
         "Hkv": 8, "page": 64, "d": 128, "kb": 4, "vb": 3, "spare": 400, "mix": 12},
    ]


def draw(rng):
    def logint(lo, hi):
        return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))

    d = rng.choice((64, 128, 128, 256))
    heads = {"Hkv": rng.choice((1, 2, 3, 4, 8)), "d": d, "kb": rng.choice((2, 3, 4)), "vb": rng.choice((2, 3, 4)),
             "page": rng.choice((32, 64, 128, 256)), "mix": rng.randrange(1 << 20)}
    op = rng.choice(("attn", "attn", "attn", "copy", "fork", "resize", "compact"))
    if op == "attn":
        q_hi, c_hi, B = logint(1, 4096), logint(1, 16000), logint(1, 48)
        Hq = heads["Hkv"] * rng.choice((1, 2, 3, 4, 5, 8))
        while B * q_hi * (q_hi + c_hi) * Hq > 2e9:  # under half of the longest listed case
            q_hi, B = max(1, q_hi // 2 + q_hi % 2 - 1), max(1, B - B // 4)
        return {"op": op, "B": B, "q_lo": logint(1, q_hi), "q_hi": q_hi, "c_lo": logint(1, c_hi), "c_hi": c_hi,
                "window": rng.choice((0, 0, logint(1, 4096))), "Hq": Hq, **heads}
    page_bytes = heads["Hkv"] * heads["page"] * (d * (heads["kb"] + heads["vb"]) // 8 + 8)
    if op == "copy":
        n_pages = logint(8, 1000)
        L = max(1, min(logint(1, 32), int(2.0e9 / (page_bytes * n_pages))))
        same = rng.random() < 0.5
        return {"op": op, "n": logint(1, n_pages // 2), "n_pages": n_pages, "same": same, "L": L, **heads}
    n_seqs, len_hi = logint(2, 400), logint(40, 2500)
    max_pages = -(-2 * len_hi // heads["page"]) + rng.randrange(5)
    case = {"op": op, "n_seqs": n_seqs, "max_pages": max_pages, "len_hi": len_hi, "family": rng.choice((1, 2, 3, 6)),
            "spare": n_seqs + logint(4, 300), **heads}
    if op != "compact":
        case["change"] = round(rng.uniform(0.1, 1.0), 3)
    if op == "resize":
        case["grow"] = logint(1, len_hi)
    _, _, n_pages = _table_of(case)
    if n_pages * page_bytes > 2.0e9:  # too large a pool for one layer: fewer rows
        case["n_seqs"] = max(2, int(n_seqs * 1.8e9 / (n_pages * page_bytes)))
        _, _, n_pages = _table_of(case)
    case["L"] = max(1, min(logint(1, 32), int(2.0e9 / (page_bytes * n_pages))))
    return case


# ------------------------------------------------------- shapes behind a case

def _lengths(case):
    """The chunk and context lengths of a batch, spread over their logarithms."""
    rng = random.Random(case["mix"])

    def spread(lo, hi):
        lo, hi = min(lo, hi), max(lo, hi)
        return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    q = [spread(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    return q, [n + spread(case["c_lo"], case["c_hi"]) for n in q]


def _table_of(case):
    """(lens, pages of each row as numbers 0 .. used - 1, pages of the pool):
    families of rows that share the pages of a common beginning, some of them
    cut back into a shared page."""
    rng = random.Random(case["mix"])
    page, lens, rows, used = case["page"], [], [], 0
    while len(rows) < case["n_seqs"]:
        first = None
        for _ in range(min(case["family"], case["n_seqs"] - len(rows))):
            n = rng.randrange(0, case["len_hi"] + 1)
            need, row = -(-n // page), []
            if first:
                row = first[:rng.randrange(0, min(len(first), need) + 1)]
                if row and rng.random() < 0.3:  # cut back into the shared beginning
                    n = len(row) * page - rng.randrange(page)
                    need = len(row)
            row = row + list(range(used, used + need - len(row)))
            used = max(used, row[-1] + 1 if row else 0)
            first = first or row
            lens.append(n)
            rows.append(row)
    return lens, rows, used + case["spare"]


def _parents(case):
    rng = random.Random(case["mix"] + 1)
    n = case["n_seqs"]
    return [rng.randrange(-1, n) if rng.random() < case["change"] else i for i in range(n)]


def _new_lens(case, lens, rows, n_pages):
    """New lengths that the pool has pages for: some rows freed, some cut, most grown."""
    rng = random.Random(case["mix"] + 2)
    left = case["spare"] - len(lens)  # a page for every row's shared tail
    top = case["max_pages"] * case["page"]
    new = []
    for n in lens:
        to = n
        if rng.random() < case["change"]:
            kind = rng.random()
            if case["grow"] == 1 or kind > 0.35:
                to = min(top, n + rng.randint(1, case["grow"]))
            else:
                to = 0 if kind < 0.2 else rng.randint(0, n)
        more = -(-to // case["page"]) - -(-n // case["page"])
        if more > left:
            to, more = n, 0
        left -= max(0, more)
        new.append(to)
    return new


def _copied(case):
    """How many pages the pass copies: what the operator cannot do without."""
    lens, rows, n_pages = _table_of(case)
    page = case["page"]
    if case["op"] == "fork":
        parents = _parents(case)
        firsts = {p: (p if parents[p] == p else i) for i, p in reversed(list(enumerate(parents))) if p >= 0}
        return sum(p >= 0 and lens[p] % page != 0 and firsts[p] != i for i, p in enumerate(parents))
    refs = [0] * n_pages
    for row in rows:
        for p in row:
            refs[p] += 1
    new = _new_lens(case, lens, rows, n_pages)
    for n, row in zip(new, rows):
        for p in row[-(-n // page):]:
            refs[p] -= 1
    k = 0
    for n, old, row in zip(new, lens, rows):
        if n > old and old % page and refs[row[-1]] > 1:
            refs[row[-1]] -= 1
            k += 1
    return k


def work(case):
    row = case["d"] * (case["kb"] + case["vb"]) // 8 + 8  # packed K and V and their norms
    if case["op"] == "attn":
        q, ctx = _lengths(case)
        pairs = read = 0
        for n, c in zip(q, ctx):
            w = case["window"] or c
            pairs += sum(min(p + 1, w) for p in range(c - n, c))
            read += min(c, n - 1 + w)
        return {"bytes": read * case["Hkv"] * row + sum(q) * case["Hq"] * case["d"] * 4,
                "flops": 4 * case["Hq"] * case["d"] * pairs}
    page_bytes = case["L"] * case["Hkv"] * case["page"] * row
    if case["op"] == "copy":
        return {"bytes": 2 * case["n"] * page_bytes + 8 * case["n"], "flops": 0}
    lens, rows, n_pages = _table_of(case)
    books = 4 * (2 * n_pages + 2 * case["n_seqs"] * (case["max_pages"] + 1))
    if case["op"] == "compact":
        live = len({p for r in rows for p in r})
        # of the live pages, those with ids past the live count move; ids are a random permutation
        return {"bytes": books + 2 * page_bytes * round(live * (1 - live / n_pages)), "flops": 0}
    return {"bytes": books + 2 * page_bytes * _copied(case), "flops": 0}


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
    if case["op"] == "attn":
        _prepare_attn(case, g, st)
    else:
        _prepare_pages(case, g, st)
    return st


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_attn(case, g, st):
    d, Hkv, page = case["d"], case["Hkv"], case["page"]
    q_lens, ctx = _lengths(case)
    need = [-(-c // page) for c in ctx]
    n_pages, max_pages = sum(need) + 3, max(need) + 1
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((case["B"], max_pages), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    k, kn = _rows(g, (n_pages, Hkv, page), d, case["kb"])
    v, vn = _rows(g, (n_pages, Hkv, page), d, case["vb"])
    total = sum(q_lens)
    st.update(k=k, kn=kn, v=v, vn=vn, table=table, ctx=_ints(ctx), cu=_ints([0] + list(np.cumsum(q_lens))),
              max_q=max(q_lens), max_ctx=max(ctx), scale=1.0 / math.sqrt(d),
              q=torch.randn(total, case["Hq"], d, generator=g, device="cuda").to(torch.bfloat16),
              out=torch.zeros(total, case["Hq"], d, dtype=torch.bfloat16, device="cuda"))
    if own:
        from kv_cache_vector_gb300 import abi
        st["plan"] = abi.Plan(d, SEED)
        st["cache"] = abi.PagedCache(k, kn, v, vn, case["kb"], case["vb"])
        st["ws"] = torch.empty(abi.tq_attn_prefill_paged_workspace_bytes(case["Hq"], Hkv, d), dtype=torch.uint8,
                               device="cuda")


def _pool(case, g, n_pages):
    """The stacked arrays of a pool of L layers: k, kn, v, vn."""
    lead = (case["L"], n_pages, case["Hkv"], case["page"])

    def data(bits):
        n = math.prod(lead) * case["d"] * bits // 8
        x = torch.randint(-2 ** 31, 2 ** 31 - 1, (n // 4,), generator=g, device="cuda", dtype=torch.int32)
        return x.view(torch.uint8).reshape(*lead, -1)

    def norms():
        return torch.randn(*lead, generator=g, device="cuda").abs_() + 8.0

    return {"k": data(case["kb"]), "kn": norms(), "v": data(case["vb"]), "vn": norms()}


def _layers(case, pool):
    from kv_cache_vector_gb300 import abi
    return abi.PagedLayers([abi.PagedCache(pool["k"][i], pool["kn"][i], pool["v"][i], pool["vn"][i], case["kb"],
                                           case["vb"]) for i in range(case["L"])])


def _prepare_pages(case, g, st):
    if case["op"] == "copy":
        n, n_pages = case["n"], case["n_pages"]
        st["src"] = _pool(case, g, n_pages)
        st["dst"] = st["src"] if case["same"] else _pool(case, g, n_pages)
        ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        st["src_ids"], st["dst_ids"] = ids[:n].contiguous(), ids[n:2 * n].contiguous()
        if own:
            st["src_layers"] = _layers(case, st["src"])
            st["dst_layers"] = st["src_layers"] if case["same"] else _layers(case, st["dst"])
        return
    lens, rows, n_pages = _table_of(case)
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    flat = torch.full((case["n_seqs"], case["max_pages"]), -1, dtype=torch.int64)
    for i, row in enumerate(rows):
        flat[i, :len(row)] = torch.tensor(row, dtype=torch.int64)
    flat = flat.cuda()
    st["table"] = torch.where(flat >= 0, ids[flat.clamp(min=0)], -1).to(torch.int32)
    st["lens"] = _ints(lens)
    st["refs"] = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    used = st["table"][flat >= 0].long()
    st["refs"].index_add_(0, used, torch.ones_like(used, dtype=torch.int32))
    if case["op"] == "fork":
        st["parents"] = _ints(_parents(case))
    elif case["op"] == "resize":
        st["new_lens"] = _ints(_new_lens(case, lens, rows, n_pages))
    st["pool"] = _pool(case, g, n_pages)
    if own:
        from kv_cache_vector_gb300 import abi
        st["layers"] = _layers(case, st["pool"])
        st["pages"] = abi.PageTable(st["table"], st["lens"], st["refs"])
        st["out"] = abi.PageTable(*(torch.empty_like(st[k]) for k in ("table", "lens", "refs")))
        st["ws"] = torch.empty(abi.tq_pages_workspace_bytes(case["n_seqs"], case["max_pages"], n_pages),
                               dtype=torch.uint8, device="cuda")


# -------------------------------------------------------------------- a pass

def run(st):
    return {"attn": _attn, "copy": _copy, "fork": _fork, "resize": _resize, "compact": _compact}[st["case"]["op"]](st)


def _attn(st):
    case = st["case"]
    if own:
        from kv_cache_vector_gb300 import abi
        return abi.tq_attn_prefill_paged(st["plan"], st["q"], st["cu"], st["cache"], st["table"], st["ctx"],
                                         st["scale"], window=case["window"], out=st["out"], workspace=st["ws"])
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
    pos = (ctx - n)[:, None] + t  # [B, T]
    off_mask = at > pos[..., None]
    if case["window"]:
        off_mask |= at <= pos[..., None] - case["window"]
    s.masked_fill_(off_mask[:, None, None], -torch.inf)
    s.sub_(s.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)).exp_()
    total = s.sum(-1, keepdim=True).clamp(min=1e-30)
    o = (s.flatten(2, 3) @ v).unflatten(2, (G, -1)) / total
    o = (o @ R).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [B, T, Hq, d]
    real = (t < n[:, None]).flatten()
    st["out"][take.flatten()[real]] = o.flatten(0, 1)[real].to(torch.bfloat16)
    return st["out"]


def _move(src, dst, src_ids, dst_ids):
    dst["k"][:, dst_ids] = src["k"][:, src_ids]
    dst["kn"][:, dst_ids] = src["kn"][:, src_ids]
    dst["v"][:, dst_ids] = src["v"][:, src_ids]
    dst["vn"][:, dst_ids] = src["vn"][:, src_ids]


def _copy(st):
    if own:
        from kv_cache_vector_gb300 import abi
        abi.tq_pages_copy(st["src_layers"], st["dst_layers"], st["src_ids"], st["dst_ids"])
    else:
        _move(st["src"], st["dst"], st["src_ids"].long(), st["dst_ids"].long())
    return st["dst"]


def _books(table, info, st):
    return {"table": table.block_table, "lens": table.lens, "refs": table.refs, "info": info, "pool": st["pool"]}


def _counts(refs, entries, mask, sign):
    """refs with `sign` added for every entry under the mask."""
    more = torch.zeros(refs.numel() + 1, dtype=refs.dtype, device=refs.device)
    at = torch.where(mask, entries, refs.numel()).flatten().long()
    more.index_add_(0, at, torch.full_like(at, sign, dtype=refs.dtype))
    return refs + more[:-1]


def _fork(st):
    if own:
        from kv_cache_vector_gb300 import abi
        return _books(*abi.tq_pages_fork(st["pages"], st["parents"], st["layers"], out=st["out"], workspace=st["ws"]), st)
    page, n = st["case"]["page"], st["lens"].numel()
    i = torch.arange(n, device="cuda")
    col = torch.arange(st["table"].shape[1], device="cuda")
    parents = st["parents"].long()
    there, p = parents >= 0, parents.clamp(min=0)
    lens = torch.where(there, st["lens"][p], 0)
    used, was = (lens + page - 1) // page, (st["lens"] + page - 1) // page
    rank = torch.where(p == i, 0, i + 1)
    first = torch.full((n + 1,), n + 1, device="cuda").scatter_reduce(0, torch.where(there, p, n), rank, "amin")
    needs = there & (lens % page != 0) & (rank != first[p])  # a last page of its own
    table = torch.where(col < used[:, None], st["table"][p], -1)
    last = (used - 1).clamp(min=0)[:, None].long()
    shared = (col < used[:, None]) & ~(needs[:, None] & (col == last))
    refs = _counts(_counts(st["refs"], st["table"], col < was[:, None], -1), table, shared, 1)
    kth = torch.cumsum(needs, 0)
    fresh = torch.searchsorted(torch.cumsum(refs == 0, 0), kth)
    old = table.gather(1, last)[:, 0].long()
    table = torch.where(needs[:, None] & (col == last), fresh[:, None].to(torch.int32), table)
    refs = _counts(refs, fresh, needs, 1)
    _move(st["pool"], st["pool"], old[needs], fresh[needs])
    info = torch.stack([kth[-1], torch.zeros_like(kth[-1])]).to(torch.int32)
    return {"table": table, "lens": lens, "refs": refs, "info": info, "pool": st["pool"]}


def _resize(st):
    if own:
        from kv_cache_vector_gb300 import abi
        return _books(*abi.tq_pages_resize(st["pages"], st["new_lens"], st["layers"], out=st["out"],
                                           workspace=st["ws"]), st)
    page, n = st["case"]["page"], st["lens"].numel()
    col = torch.arange(st["table"].shape[1], device="cuda")
    lens, was = st["new_lens"], st["lens"]
    used, had = (lens + page - 1) // page, (was + page - 1) // page
    refs = _counts(st["refs"], st["table"], (col >= used[:, None]) & (col < had[:, None]), -1)
    free = torch.cumsum(refs == 0, 0)
    last = (had - 1).clamp(min=0)
    tail = st["table"].gather(1, last[:, None].long())[:, 0].long().clamp(min=0)
    writes = (lens > was) & (was % page != 0)  # rows that go on inside their last page
    before = ((tail[:, None] == tail) & writes & writes[:, None]).tril(-1).sum(1)
    private = writes & (refs[tail] - before > 1)
    takes = private + (used - had).clamp(min=0)
    start = torch.cumsum(takes, 0) - takes
    kth = start[:, None] + 1 + torch.where(col == last[:, None], 0, private[:, None] + col - had[:, None])
    new = ((col >= had[:, None]) & (col < used[:, None])) | (private[:, None] & (col == last[:, None]))
    fresh = torch.searchsorted(free, kth.clamp(min=1))
    table = torch.where(new, fresh.to(torch.int32), torch.where(col < used[:, None], st["table"], -1))
    refs = _counts(_counts(refs, tail, private, -1), table, new, 1)
    _move(st["pool"], st["pool"], tail[private], table.gather(1, last[:, None].long())[:, 0].long()[private])
    total = takes.sum()
    info = torch.stack([total, torch.zeros_like(total)]).to(torch.int32)
    return {"table": table, "lens": lens, "refs": refs, "info": info, "pool": st["pool"]}


def _compact(st):
    if own:
        from kv_cache_vector_gb300 import abi
        table, moved, info = abi.tq_pages_compact(st["pages"], st["layers"], out=st["out"], workspace=st["ws"])
        return {"moved": moved, **_books(table, info, st)}
    refs, N = st["refs"], st["refs"].numel()
    page = st["case"]["page"]
    ids = torch.arange(N, device="cuda")
    live = refs > 0
    count = live.sum()
    holes = ~live & (ids < count)
    high = live & (ids >= count)
    to = torch.searchsorted(torch.cumsum(holes, 0), torch.cumsum(high, 0).clamp(min=1))
    moved = torch.where(high, to, torch.where(live, ids, -1)).to(torch.int32)
    used = (st["lens"] + page - 1) // page
    col = torch.arange(st["table"].shape[1], device="cuda")
    table = torch.where(col < used[:, None], moved[st["table"].long().clamp(min=0)], -1)
    out = torch.zeros(N + 1, dtype=refs.dtype, device="cuda")
    out[torch.where(live, moved.long(), N)] = refs
    _move(st["pool"], st["pool"], ids[high], to[high])
    info = torch.stack([count, high.sum()]).to(torch.int32)
    return {"moved": moved, "table": table, "lens": st["lens"], "refs": out[:-1], "info": info, "pool": st["pool"]}


# --------------------------------------------------------------- 64-bit values

def exact(case, seed):
    """The attention from its definition in 64 bits: rows decoded to the
    original domain, one (sequence, KV head) at a time.  The page operators
    move whole values and have none."""
    if case["op"] != "attn":
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
        pages = st["table"][b, :-(-n // page)].long()
        pos = torch.arange(n - (hi - lo), n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")
        seen = (j <= pos) & (j > pos - (case["window"] or n + 1))
        for h in range(case["Hkv"]):
            k = decoded(st["k"], st["kn"], case["kb"], pages, n, h)
            v = decoded(st["v"], st["vn"], case["vb"], pages, n, h)
            for r in range(h * G, (h + 1) * G):
                s = (st["q"][lo:hi, r].double() @ k.T) * st["scale"]
                out[lo:hi, r] = torch.softmax(s.masked_fill(~seen, -torch.inf), -1) @ v
    return out
