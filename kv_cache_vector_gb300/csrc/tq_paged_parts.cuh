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

#include <climits>

#include "tq_async.cuh"
#include "tq_device.cuh"

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
    int sinks;             // kPpSinks (window > 0)
    const uint32_t* mask;  // kPpTree: [n_q][words]
    int words;
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
        if (MODE == kPpSinks) cap += (int64_t)A.sinks * G;
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

}  // namespace dev
}  // namespace tq
