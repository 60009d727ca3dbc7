// tq_paged_parts.cuh -- how the paged attention kernels cut their work into
// shares: items (row tile of a sequence, KV head) on one line, weighted by their
// blocks of positions; which blocks an item reads; which positions a query row
// attends to.  Z: a kernel's geometry (kN positions a block, kRows query rows an
// item, kCost* its costs).
//
// MODE says what a query row attends to:
//   kPpCausal  positions max(0, p - window + 1) .. p of the token at position p
//   kPpSinks   the same and positions 0 .. sinks - 1 up to p
//   kPpTree    every position in front of the sequence's tokens, and of those the
//              ones whose bit is set in the token's row of a mask
#pragma once

#include <cfloat>
#include <climits>

#include "tq_async.cuh"
#include "tq_device.cuh"
#include "tq_tmem.cuh"
#include "tq_umma.cuh"

namespace tq {
namespace dev {

constexpr int kPpStatusRange = 71;  // cu_q or ctx_lens outside their ranges
constexpr int kPpStatusPage = 72;   // a page id outside [0, n_pages)
constexpr int kPpStatusWait = 73;   // a wait gave up
constexpr int kPpStatusAlign = 74;  // shared memory not 1024-byte aligned
constexpr int kPpStatusTree = 75;   // more tokens than positions or than bits of a mask row

struct PpArgs {
    const __nv_bfloat16* q;
    void* out;
    const int32_t* cu;
    const int32_t* ctx;
    const int32_t* bt;
    tq_paged_cache c;
    float* part;   // [shares][2] parts
    int32_t* meta;  // [shares][kPpMeta]
    int64_t n_q;
    int B, Hq, Hkv, max_pages, shift, window, k_bits, v_bits, out_bf16;
    int sinks;             // kPpSinks
    const uint32_t* mask;  // kPpTree: [n_q][words]
    int words;
    int whole;             // (kernel for few rows) a share is an item
    uint32_t khi[4], klo[4], vhi[4], vlo[4];  // level bytes (see expand)
};
// what a share left: bit 0 a part of the item it starts in, bit 1 one of the
// item it owns (which starts in this share and ends in the share kMetaLast;
// -1: none), that item's first row of q, KV head, rows.  kShareFailed: a wait
// gave up in the share, and its parts may be missing
enum { kMetaHas = 0, kMetaLast, kMetaQ0, kMetaH, kMetaRow0, kMetaRows, kPpMeta = 8 };
constexpr int kShareFailed = 4;

// Where a share starts or goes on: sequence, row tile, KV head, and the units
// (or, where the share is one part of an item, the parts) of the item that
// belong to earlier shares.
struct PpCursor {
    int b, i, h;
    int64_t off;
    int64_t left;  // units of this share from here on
    int n, ctx, q0;  // the sequence's lengths and first row of q
    int parts;       // > 0: the share is part `off` of so many of one item
};

// Weights and ranges of sequence b's items.  A unit line position is only an
// estimate of cost: any consistent weight gives a correct cut.
template <class Z, int MODE>
struct PpSeq {
    int n, ctx, q0, tiles = 0, rows;
    int64_t base, cap, kstar, over;
    int G;

    __device__ void load(const PpArgs& A, int b, int* status) {
        const int64_t c0 = A.cu[b], c1 = A.cu[b + 1];
        const int len = A.ctx[b];
        if (c0 < 0 || c1 < c0 || c1 > A.n_q || len < 0 || len > ((int64_t)A.max_pages << A.shift) ||
            (c1 - c0) * (A.Hq / A.Hkv) > INT32_MAX) {
            if (status) report_timeout(status, kPpStatusRange);
            set(A, 0, 0, 0);
        } else if (MODE == kPpTree && (c1 - c0 > len || c1 - c0 > 32ll * A.words)) {
            if (status) report_timeout(status, kPpStatusTree);
            set(A, 0, 0, 0);
        } else {
            set(A, (int)(c1 - c0), len, (int)c0);
        }
    }
    __device__ void set(const PpArgs& A, int tokens, int len, int first) {
        n = tokens;
        ctx = len;
        q0 = first;
        G = A.Hq / A.Hkv;
        rows = n * G;
        tiles = (rows + Z::kRows - 1) / Z::kRows;
        base = ctx > n ? (int64_t)(ctx - n) * G : 0;
        cap = A.window > 0 ? (int64_t)A.window * G + Z::kRows : INT64_MAX;
        if (MODE == kPpSinks && A.window > 0) cap += (int64_t)A.sinks * G;
        if (MODE == kPpTree) base = cap = (int64_t)ctx * G;  // every tile reads all positions
        // tiles before the window's cap binds: base + (k + 1) kRows < cap
        kstar = cap == INT64_MAX ? INT32_MAX : (cap - base - 1) / Z::kRows;
        if (cap - base - 1 < 0) kstar = 0;
        over = (int64_t)Z::kCostItem * Z::kN * G;
    }
    __device__ int factor(int i) const {
        return rows - (int64_t)i * Z::kRows > 128 ? Z::kCostPair : Z::kCostSplit;
    }
    __device__ int64_t weight(int i) const { return work(i) + over; }
    __device__ int64_t work(int i) const {  // without the item's own cost
        const int64_t e = base + min((int64_t)(i + 1) * Z::kRows, (int64_t)rows);
        return factor(i) * min(e, cap);
    }
    // sum of the weights of tiles 0 .. i - 1
    __device__ int64_t before(int i) const {
        if (i <= 0) return 0;
        if (i == tiles) return before(i - 1) + weight(i - 1);
        const int64_t m = min((int64_t)i, kstar);
        int64_t s = m * base + (int64_t)Z::kRows * (m * (m + 1) / 2);
        if (i > m) s += (i - m) * cap;
        return Z::kCostPair * s + i * over;
    }
};

// One part of an item: blocks [blk0, blk1) of the item's nblk, its first
// position and the share's bookkeeping.
struct PpPart {
    int b, i, h;
    int row0, rows;      // first row within (sequence, KV head); valid rows
    int lo_blk;          // first block of the item
    int blk0, blk1, nblk;
    int kv_lo, kv_end;   // the positions that some row attends to
    int pair;            // the two streams take two row tiles
    bool head, whole;    // part starts the item; covers it
};

// The block at which a cut `off` units into an item of w units falls.  The
// item's own cost lies in front of its blocks: a share that starts inside an
// item pays it once more, nearly every share does, and so the shares stay
// equal.  Any rounding will do that never decreases and is the same for every
// CTA.
__device__ __forceinline__ int pp_cut(int nblk, int64_t off, int64_t w, int64_t over) {
    return off >= w ? nblk
                    : off <= over ? 0 : min(nblk, (int)((float)nblk * __fdividef((float)(off - over), (float)(w - over))));
}

// kPpSinks: blocks between the sinks' last and the window's first of an item
// that reads positions [0, sinks) and [kv_lo, kv_end); its block number j.
template <class Z>
__device__ __forceinline__ int pp_skipped(const PpArgs& A, int kv_lo, int kv_end) {
    return max(0, kv_lo / Z::kN - (min(A.sinks, kv_end) + Z::kN - 1) / Z::kN);
}
template <class Z, int MODE>
__device__ __forceinline__ int pp_block_at(const PpArgs& A, int kv_lo, int kv_end, int j) {
    if constexpr (MODE != kPpSinks) return j;
    return j < (min(A.sinks, kv_end) + Z::kN - 1) / Z::kN ? j : j + pp_skipped<Z>(A, kv_lo, kv_end);
}

// Blocks of row tile i, the first of them, and its first position and their end.
template <class Z, int MODE>
__device__ __forceinline__ int pp_blocks(const PpArgs& A, const PpSeq<Z, MODE>& q, int i, int* lo_blk = nullptr,
                                         int* kv_lo = nullptr, int* kv_end = nullptr) {
    if constexpr (MODE == kPpTree) {
        if (lo_blk) *lo_blk = 0;
        if (kv_lo) *kv_lo = 0;
        if (kv_end) *kv_end = q.ctx;
        return (q.ctx + Z::kN - 1) / Z::kN;
    }
    const int row0 = i * Z::kRows, rows = min(Z::kRows, q.rows - row0);
    const int first_pos = q.ctx - q.n + row0 / q.G;
    const int end = max(0, q.ctx - q.n + (row0 + rows - 1) / q.G + 1);
    const int at = A.window > 0 ? max(0, first_pos - A.window + 1) : 0, lo = at / Z::kN;
    if (kv_lo) *kv_lo = at;
    if (kv_end) *kv_end = end;
    if constexpr (MODE == kPpSinks) {  // numbered from 0: pp_block_at
        if (lo_blk) *lo_blk = 0;
        return (end + Z::kN - 1) / Z::kN - pp_skipped<Z>(A, at, end);
    }
    if (lo_blk) *lo_blk = lo;
    return max(0, (end + Z::kN - 1) / Z::kN - lo);
}

// Rows and blocks of item p.b, p.i, p.h.
template <class Z, int MODE>
__device__ __forceinline__ void pp_rows(const PpArgs& A, const PpSeq<Z, MODE>& q, PpPart& p) {
    p.row0 = p.i * Z::kRows;
    p.rows = min(Z::kRows, q.rows - p.row0);
    p.pair = Z::kStreams == 2 && p.rows > 128;
    p.nblk = pp_blocks(A, q, p.i, &p.lo_blk, &p.kv_lo, &p.kv_end);
}

// The share's next part with work in it; advances the cursor.  False at the
// end of the share.  Items without blocks (no position to attend to) come as
// a whole part with blk0 == blk1, to the share that holds their start.
template <class Z, int MODE>
__device__ bool pp_next(const PpArgs& A, PpCursor& c, PpSeq<Z, MODE>& q, PpPart& p) {
    while (c.left > 0) {
        while (c.i >= q.tiles) {  // next sequence with rows
            if (++c.b >= A.B) {
                c.left = 0;
                return false;
            }
            q.load(A, c.b, nullptr);
            c.i = 0;
            c.h = 0;
        }
        const int64_t w = q.weight(c.i);
        const int64_t end = min(w, c.off + c.left);
        p.b = c.b;
        p.i = c.i;
        p.h = c.h;
        pp_rows(A, q, p);
        p.blk0 = pp_cut(p.nblk, c.off, w, q.over);
        p.blk1 = pp_cut(p.nblk, end, w, q.over);
        p.head = c.off == 0;
        p.whole = p.nblk == 0 ? p.head : (p.blk0 == 0 && p.blk1 == p.nblk);
        c.left -= end - c.off;
        c.off = end;
        if (c.off >= w) {  // on to the next item
            c.off = 0;
            if (++c.h >= A.Hkv) {
                c.h = 0;
                ++c.i;
            }
        }
        if (p.whole || p.blk1 > p.blk0) return true;
    }
    return false;
}

// A part as the copy warp hands it to the others, through shared memory.
struct PpJob {
    int nb;        // blocks, -1: no more parts
    int flags;     // kJob*
    int q0;        // the sequence's first row of q
    int h;         // KV head
    int row0, rows;  // first row within (sequence, KV head); valid rows
    int blk;       // first block
    int kv_lo, kv_end;  // positions before the one and from the other on are not read
    int pos0;      // position of the sequence's token 0
    int tok0, rest;  // row0 / G and row0 % G
};
enum { kJobPair = 1, kJobWhole = 2, kJobHead = 4 };

// The share's next part: the one part of a share that is a part of an item
// (first: it has not been handed out), or the next along the line.
template <class Z, int MODE>
__device__ __forceinline__ bool pp_next_part(const PpArgs& A, PpCursor& cur, PpSeq<Z, MODE>& seq, PpPart& u, bool first) {
    if (cur.parts == 0) return pp_next(A, cur, seq, u);
    u.b = cur.b, u.i = cur.i, u.h = cur.h;
    pp_rows(A, seq, u);
    const uint32_t nb = u.nblk, at = (uint32_t)cur.off, of = cur.parts;  // nb of < 2^32
    u.blk0 = nb * at / of;
    u.blk1 = nb * (at + 1) / of;
    u.head = cur.off == 0;
    u.whole = u.nblk == 0 ? u.head : (u.blk0 == 0 && u.blk1 == u.nblk);
    return first && (u.whole || u.blk1 > u.blk0);
}
template <class Z, int MODE>
__device__ __forceinline__ void pp_write_job(volatile PpJob* m, bool more, const PpPart& u, const PpSeq<Z, MODE>& seq) {
    m->nb = more ? u.blk1 - u.blk0 : -1;
    if (!more) return;
    m->flags = (u.pair ? kJobPair : 0) | (u.whole ? kJobWhole : 0) | (u.head ? kJobHead : 0);
    m->q0 = seq.q0;
    m->h = u.h;
    m->row0 = u.row0;
    m->rows = u.rows;
    m->blk = u.lo_blk + u.blk0;
    m->kv_lo = u.kv_lo;
    m->kv_end = u.kv_end;
    m->pos0 = seq.ctx - seq.n;
    const int tok0 = u.row0 / seq.G;
    m->tok0 = tok0;
    m->rest = u.row0 - tok0 * seq.G;
}

// This CTA's share of the work, into *start (left 0, parts 0: none) and *share:
// the sequences' weights, scanned over the block.  red: 16 bytes a warp.
template <class Z, int MODE>
__device__ __forceinline__ void pp_start(const PpArgs& A, long long* red, PpCursor* start, long long* share, int* status) {
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
    const int each = (A.B + Z::kThreads - 1) / Z::kThreads;
    const int b0 = min(A.B, tid * each), b1 = min(A.B, b0 + each);
    PpSeq<Z, MODE> q;
    long long mine = 0;
    int items = 0;
    float most = 0.f;  // the largest item's work
    for (int b = b0; b < b1; ++b) {
        q.load(A, b, blockIdx.x == 0 ? status : nullptr);
        mine += (long long)A.Hkv * q.before(q.tiles);
        if (q.tiles) most = fmaxf(most, fmaxf((float)q.work(q.tiles - 1), (float)q.work(max(0, q.tiles - 2))));
        items += (int)min((int64_t)1 << 10, (int64_t)A.Hkv * q.tiles);  // exact where it counts: below the CTAs
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) red[warp] = incl;
    uint32_t* red2 = reinterpret_cast<uint32_t*>(red + Z::kWarps);
    const uint32_t wi = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)items);
    const uint32_t wm = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most));
    if (lane == 0) red2[2 * warp] = wi, red2[2 * warp + 1] = wm;
    __syncthreads();
    long long total = 0, before = 0;
    uint32_t all = 0, top = 0;
#pragma unroll
    for (int w = 0; w < Z::kWarps; ++w) {
        if (w < warp) before += red[w];
        total += red[w];
        all += red2[2 * w];
        top = max(top, red2[2 * w + 1]);
    }
    before += incl - mine;
    const float sum = (float)total, grid = (float)gridDim.x;
    // a little over total / grid: the last CTA's share may be smaller
    const long long per = (long long)(sum * (1.000001f / grid)) + 1;
    if (tid == 0) *share = per;
    // Shares along the line of all items cross from one item into the next, and
    // then pay for two items' rotations and outputs.  With few items a share is
    // a part of one item instead: an item gets (work / cut) + 1 shares, no more
    // than there are CTAs in all.  Taken where the largest of them is no more
    // than a share of the line: the drafts of 4 sequences over 400-2000
    // positions took 24.7 us along the line, 20.8 us so.
    float cut = 0.f;
    int each_cta = 1;  // items of a CTA, of which each is whole where they are more than one
    if (Z::kWhole && A.whole) {
        cut = 1e30f;  // one part each
        // (sequences of rows that others have too, as a cu_q that steps back gives)
        if (all > gridDim.x) each_cta = (all + gridDim.x - 1) / gridDim.x;
    } else if (each == 1 && all > 0 && all < gridDim.x) {
        const float over = (float)Z::kCostItem * Z::kN * (A.Hq / A.Hkv);
        const float c = fmaxf(1.f, __fdividef((sum - (float)all * over) * 1.000002f, grid - (float)all));
        if (fminf(c, __uint_as_float(top)) * grid <= sum) cut = c;
    }
    if (cut > 0.f) {
        auto parts = [&](int i) { return (int)__fdividef((float)q.work(i), cut) + 1; };
        int sums = 0;
        for (int i = 0; i < q.tiles; ++i) sums += A.Hkv * parts(i);
        int ins = sums;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, ins, o);
            if (lane >= o) ins += u;
        }
        __syncthreads();  // red2 is free
        if (lane == 31) red2[warp] = ins;
        __syncthreads();
        for (int w = 0; w < warp; ++w) ins += red2[w];
        int v = (int)blockIdx.x * each_cta - (ins - sums);
        if (v >= 0 && v < sums) {  // this thread's sequence holds this CTA's share
            int i = 0, n;
            for (;; ++i) {
                n = parts(i);
                if (v < A.Hkv * n) break;
                v -= A.Hkv * n;
            }
            start->b = b0;
            start->i = i;
            start->h = v / n;
            start->off = v % n;
            start->parts = n;
            start->n = q.n;
            start->ctx = q.ctx;
            start->q0 = q.q0;
            if (Z::kWhole && each_cta > 1) {  // along the line, from this item's start to the end of the last
                long long units = 0;
                int b = b0, h = v;
                for (int k = 0; k < each_cta; ++k, ++h) {
                    if (h >= A.Hkv) h = 0, ++i;
                    while (i >= q.tiles && ++b < A.B) q.load(A, b, nullptr), i = h = 0;
                    if (b >= A.B) break;
                    units += q.weight(i);
                }
                start->parts = 0;
                start->left = units;
            }
        }
        return;
    }
    const long long u0 = per * blockIdx.x, u1 = min(total, u0 + per);
    if (u0 < u1 && u0 >= before && u0 < before + mine) {  // this thread's sequences hold the start
        long long v = u0 - before;
        int b = b0;
        if (each > 1)
            for (;; ++b) {
                q.load(A, b, nullptr);
                const long long w = (long long)A.Hkv * q.before(q.tiles);
                if (v < w) break;
                v -= w;
            }
        int lo = 0, hi = q.tiles - 1;  // the last tile whose units start at or before v
        while (lo < hi) {
            const int m = (lo + hi + 1) / 2;
            if ((long long)A.Hkv * q.before(m) <= v) lo = m;
            else hi = m - 1;
        }
        v -= (long long)A.Hkv * q.before(lo);
        const long long w = q.weight(lo);
        start->b = b;
        start->i = lo;
        int h = (int)((float)v / (float)w);  // v / w, to within one
        h -= (long long)h * w > v;
        h += (long long)(h + 1) * w <= v;
        start->h = h;
        start->off = v - (long long)h * w;
        start->left = u1 - u0;
        start->n = q.n;
        start->ctx = q.ctx;
        start->q0 = q.q0;
    }
}

// Which parts this share left, and the item it owns: the one that starts in this
// share and ends in a later one.  One thread.
template <class Z, int MODE>
__device__ __forceinline__ void pp_report(const PpArgs& A, const PpCursor& start, long long share, const PpCursor& cur,
                                          const PpSeq<Z, MODE>& seq, bool ok, int has) {
    int last = blockIdx.x;
    bool owner;
    if (cur.parts > 0) {
        // (an item of one block is some share's whole)
        owner = ok && cur.off == 0 && cur.parts > 1 && pp_blocks(A, seq, cur.i) > 1;
        last += cur.parts - 1;
    } else {
        owner = ok && cur.off > 0 &&
                !(start.off > 0 && start.b == cur.b && start.i == cur.i && start.h == cur.h);
        if (owner) {
            const int64_t w = seq.weight(cur.i), per = share;
            const int nblk = pp_blocks(A, seq, cur.i);
            // no join where one share has all of the item's blocks
            owner = nblk > 0 && pp_cut(nblk, cur.off, w, seq.over) < nblk;
            for (int64_t x = cur.off; x < w && pp_cut(nblk, x, w, seq.over) == 0; x += per)
                if (pp_cut(nblk, min(w, x + per), w, seq.over) == nblk) owner = false;
            last += (int)((w - cur.off + per - 1) / per);
        }
    }
    const int row0 = cur.i * Z::kRows;
    int4* m = reinterpret_cast<int4*>(A.meta + (int64_t)blockIdx.x * kPpMeta);
    m[0] = make_int4(has, owner ? last : -1, owner ? seq.q0 : 0, cur.h);
    m[1] = make_int4(row0, owner ? min(Z::kRows, seq.rows - row0) : 0, 0, 0);
}

// The positions that a query row attends to, as bits of a block's columns.
template <int MODE>
struct PpVis {
    int c0, c1;           // kPpCausal, kPpSinks: columns [c0, c1)
    int cs;               // kPpSinks: and [0, cs)
    const uint32_t* row;  // kPpTree: the token's mask row, its words, the column of node 0, and the sequence's end
    int words, node0, end;
    // columns c .. c + 31
    __device__ __forceinline__ uint32_t word(int c) const {
        auto below = [](int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; };
        if constexpr (MODE == kPpTree) {
            const int rel = c - node0;  // the first column's node
            if (rel <= -32) return 0xFFFFFFFFu;
            const int k = rel < 0 ? -1 : rel >> 5, sh = rel & 31;
            const uint32_t w0 = k < 0 ? 0xFFFFFFFFu : k < words ? row[k] : 0u, w1 = k + 1 < words ? row[k + 1] : 0u;
            return __funnelshift_r(w0, w1, sh) & below(end - c);
        } else {
            uint32_t on = below(c1 - c) & ~below(c0 - c);
            if (MODE == kPpSinks) on |= below(cs - c);
            return on;
        }
    }
};

__device__ __forceinline__ float pp_pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

__device__ __forceinline__ float pp_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e;
}

// The value of lane 0: known to the compiler to be the same in the whole warp.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }
__device__ __forceinline__ uint64_t uniform(uint64_t v) {
    return ((uint64_t)uniform((uint32_t)(v >> 32)) << 32) | uniform((uint32_t)v);
}

// A try_wait that may suspend the warp for up to 100 us.
__device__ __forceinline__ bool pp_try_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(100000u)
        : "memory");
    return ok != 0;
}

// Bounded wait; gives up at once when the CTA's abort flag is set.
__device__ __forceinline__ bool pp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_f, int* status) {
    if (pp_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    while (!pp_try_wait(bar, parity)) {
        if (*abort_f) return false;
        if (global_ns() - t0 > kWaitLimitNs) {
            *abort_f = 1;
            report_timeout(status, kPpStatusWait);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// The largest of 32 columns as fp32, NaN left out: the load's own reduction.
__device__ __forceinline__ float tmem_max32(uint32_t taddr) {
    uint32_t r[32];
    float m;
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=f"(m)
        : "r"(taddr));
    // completes the load; naming its registers keeps them the load's until then
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+f"(m)::"memory");
    return m;
}

// Shared-memory descriptor of the V tile as an N-major B operand (N = dims):
// 128-byte swizzle, 64-dim columns `lbo` bytes apart (leading offset), groups
// of 8 positions 1024 bytes apart (stride offset).
__device__ __forceinline__ uint64_t umma_desc_sw128_mn(uint32_t addr, uint32_t lbo) {
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFF);
    d |= (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
constexpr uint32_t kIdescBTransposed = 1u << 16;

// Byte permute whose selector nibbles are below 8 already (__byte_perm masks
// them first).
__device__ __forceinline__ uint32_t pp_prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}
// Bits of b where m is set, of a elsewhere.
__device__ __forceinline__ uint32_t pp_select(uint32_t a, uint32_t b, uint32_t m) { return (a & ~m) | (b & m); }

// Four fp16 levels from four 4-bit selectors (nibbles of sel's low half) and
// the level bytes: two byte permutes pick the high and the low bytes, two
// interleave them.  4-bit indices: hi/lo hold the 8 positive levels; x has a 1
// in the nibble of every positive index, and the sign byte is permuted from
// it.  Narrower indices: hi/lo hold all levels with their signs.
template <int BITS>
__device__ __forceinline__ void pp_levels4(uint32_t sel, uint32_t x, const uint32_t* hi, const uint32_t* lo,
                                           uint32_t& p01, uint32_t& p23) {
    uint32_t h = pp_prmt(hi[0], hi[1], sel);
    const uint32_t l = pp_prmt(lo[0], lo[1], sel);
    if constexpr (BITS == 4) h ^= pp_prmt(0x00000080u, 0u, x);
    p01 = pp_prmt(l, h, 0x5140);
    p23 = pp_prmt(l, h, 0x7362);
}

// Which pair of 16-byte chunks a row's thread starts with (an xor on the pair
// number): a permutation per row under which a warp's reads of the staged
// words fall into different banks, and each eight lanes' writes to the
// swizzled tile too.
template <int BITS, int D>
__device__ __forceinline__ int pp_turn(int r) {
    if constexpr (BITS == 4)
        return D == 128 ? ((r >> 2) & 3) | ((r & 2) << 1)
                        : D == 256 ? ((r >> 2) & 3) | ((r & 3) << 2) : D == 64 ? (r >> 2) & 3 : (r >> 3) & 1;
    else if constexpr (BITS == 3)
        return D == 128 ? ((r >> 3) & 3) << 1
                        : D == 256 ? (((r >> 3) & 3) << 1) | ((r & 4) << 1) : D == 64 ? (r >> 4) & 1 : 0;
    else
        return D == 128 ? (r >> 2) & 7
                        : D == 256 ? ((r >> 2) & 7) | ((r & 2) << 2) : D == 64 ? (r >> 3) & 3 : (r >> 4) & 1;
}

__device__ __forceinline__ float pp_max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Sums of 2^(s - m) of two sets of positions put together (m -inf: an empty set,
// its sum 0 or NaN).
__device__ __forceinline__ void pp_join_sums(float& l, float& m, float l1, float m1) {
    const float mx = fmaxf(m, m1), mr = mx == -INFINITY ? 0.f : mx;
    l = l * pp_exp2(m - mr) + l1 * pp_exp2(m1 - mr);
    m = mx;
}

// Items have up to ROWS rows.  Block (share, y): rows 32 y .. + 31 of the item that the share owns, its
// parts summed in the order of the shares, AT parts' loads in flight, divided
// and rotated back.
template <int D, int AT, int ROWS>
__global__ void __launch_bounds__(256, D < 256 && AT == 2 ? 3 : 2)
k_prefill_paged_join(const __grid_constant__ PpArgs A, const __grid_constant__ PagedPrefillConsts P) {
    constexpr int C = D / 32;  // 16-byte columns per thread, and elements per lane of a row
    __shared__ float tile[32][D + 1];
    griddep_wait();
    const int sh = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int4* meta = reinterpret_cast<const int4*>(A.meta);
    const int4 m0 = __ldcg(meta + 2 * sh), m1 = __ldcg(meta + 2 * sh + 1);
    int near = 0;  // what the shares up to 31 further on left, looked up together with the item
    if (sh + lane < (int)gridDim.x) near = __ldcg(A.meta + (sh + lane) * kPpMeta + kMetaHas);
    const int last = m0.y, rows = m1.y;
    if (last < 0 || 32 * (int)blockIdx.y >= rows) return;
    const int G = A.Hq / A.Hkv;
    const int lrow = 32 * blockIdx.y + lane;  // every warp: the same 32 rows
    constexpr int64_t PF = (int64_t)(D + 3) * ROWS;
    const bool in = lrow < rows;
    float M = -INFINITY, l = 0.f, m = -INFINITY;
    float4 o[C];
#pragma unroll
    for (int k = 0; k < C; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = sh; c0 <= last; c0 += 32) {
        const int cl = c0 + lane;
        if (c0 > sh && cl <= last) near = __ldcg(A.meta + cl * kPpMeta + kMetaHas);
        unsigned has = __ballot_sync(0xFFFFFFFFu, cl <= last && (near & (cl == sh ? 2 : 1)));
        if (__any_sync(0xFFFFFFFFu, cl <= last && (near & kShareFailed))) return;  // every warp sees the same
        while (has && in) {
            // a few parts' loads in flight at once
            float4 v[AT][C];
            float Mc[AT], lc[AT], mc[AT];
            unsigned left = has;
#pragma unroll
            for (int t = 0; t < AT; ++t) {
                Mc[t] = -INFINITY, lc[t] = 0.f, mc[t] = -INFINITY;
                if (left) {
                    const int c = c0 + __ffs(left) - 1;
                    left &= left - 1;
                    const float* pt = A.part + ((int64_t)c * 2 + (c == sh)) * PF;
                    const float* x = pt + D * ROWS + lrow;
                    Mc[t] = __ldcg(x), lc[t] = __ldcg(x + ROWS), mc[t] = __ldcg(x + 2 * ROWS);
#pragma unroll
                    for (int k = 0; k < C; ++k)
                        v[t][k] = __ldcg(reinterpret_cast<const float4*>(pt) + lrow + (warp + 8 * k) * ROWS);
                }
            }
#pragma unroll
            for (int t = 0; t < AT; ++t) {
                if (!has) break;
                has &= has - 1;
                // both sides to the larger maximum; a side that attended to nothing
                // has -inf, no output and the sum 0 (or NaN)
                const float Mx = fmaxf(M, Mc[t]);
                const float a = M == -INFINITY ? 0.f : pp_exp2(M - Mx), a1 = Mc[t] == -INFINITY ? 0.f : pp_exp2(Mc[t] - Mx);
                pp_join_sums(l, m, lc[t], mc[t]);
                M = Mx;
#pragma unroll
                for (int k = 0; k < C; ++k) {
                    o[k].x = o[k].x * a + v[t][k].x * a1;
                    o[k].y = o[k].y * a + v[t][k].y * a1;
                    o[k].z = o[k].z * a + v[t][k].z * a1;
                    o[k].w = o[k].w * a + v[t][k].w * a1;
                }
            }
        }
    }
    const float inv = l == 0.f ? 0.f : pp_exp2(M - m) * P.out_mul * P.inv_sqrt_d / l;
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const float v[4] = {o[k].x, o[k].y, o[k].z, o[k].w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int j = 4 * (warp + 8 * k) + u;
            tile[lane][j] = __uint_as_float(__float_as_uint(v[u] * inv) ^ (P.two_sided ? sign_mask(P.sgn2b, j) : 0u));
        }
    }
    __syncthreads();
    // rows rotated back, one per warp at a time: elements lane + 32 k, the
    // transform's low five bits across lanes, the rest in registers
    for (int r = warp; r < 32; r += 8) {
        const int lr = 32 * blockIdx.y + r;
        if (lr >= rows) break;
        float e[C];
#pragma unroll
        for (int k = 0; k < C; ++k) e[k] = tile[r][lane + 32 * k];
#pragma unroll
        for (int m = 1; m < 32; m *= 2)
#pragma unroll
            for (int k = 0; k < C; ++k) {
                const float u = __shfl_xor_sync(0xFFFFFFFFu, e[k], m);
                e[k] = lane & m ? u - e[k] : e[k] + u;
            }
#pragma unroll
        for (int len = 1; len < C; len *= 2)
#pragma unroll
            for (int k = 0; k < C; ++k)
                if (!(k & len)) {
                    const float u = e[k], v = e[k + len];
                    e[k] = u + v;
                    e[k + len] = u - v;
                }
        const int grow = m1.x + lr, tok = grow / G, hd = grow - tok * G;
        const int64_t at = (((int64_t)m0.z + tok) * A.Hq + (int64_t)m0.w * G + hd) * D;
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const int j = lane + 32 * k;
            const float v = __uint_as_float(__float_as_uint(e[k]) ^ sign_mask(P.sgnb, j));
            if (A.out_bf16) static_cast<__nv_bfloat16*>(A.out)[at + j] = __float2bfloat16_rn(v);
            else static_cast<float*>(A.out)[at + j] = v;
        }
    }
}

// The kernels' arguments; part_floats: the floats of a part.
inline PpArgs pp_args(const PagedPrefillCall& c, int shares, size_t part_floats) {
    PpArgs A = {};
    A.q = static_cast<const __nv_bfloat16*>(c.q);
    A.out = c.out;
    A.cu = c.cu_q;
    A.ctx = c.ctx_lens;
    A.bt = c.block_table;
    A.c = c.cache;
    A.n_q = c.n_q;
    A.B = c.B;
    A.Hq = c.Hq;
    A.Hkv = c.Hkv;
    A.max_pages = c.max_pages;
    A.shift = c.page_shift;
    A.window = c.window;
    A.k_bits = c.k_bits;
    A.v_bits = c.v_bits;
    A.out_bf16 = c.out_bf16;
    A.sinks = c.sinks;
    A.mask = c.mask;
    A.words = c.mask_words;
    for (int i = 0; i < 4; ++i) {
        A.khi[i] = c.k_levels[i];
        A.klo[i] = c.k_levels[4 + i];
        A.vhi[i] = c.v_levels[i];
        A.vlo[i] = c.v_levels[4 + i];
    }
    A.part = static_cast<float*>(c.workspace);
    A.meta = reinterpret_cast<int32_t*>(A.part + (size_t)shares * 2 * part_floats);
    return A;
}

}  // namespace dev
}  // namespace tq
