// tq_prefill_paged.cu -- attention of several query tokens per sequence over
// the paged packed cache, ragged chunks, on the 5th-generation tensor cores.
//
// Sequence b has n_b query tokens (rows cu_q[b] .. cu_q[b + 1] - 1 of q), the
// last n_b of its ctx_b positions; token t sits at p = ctx_b - n_b + t and
// attends over positions max(0, p - window + 1) .. p (or, by MODE, over the
// sinks too, or as a node of a tree: tq_paged_parts.cuh):
//   out = R^-1 ( sum_j p_j n^v_j c[v_j] ),  p = softmax_j( scale n^k_j <R q, c[k_j]> )
// with R the codec's rotation, c the codebook's levels and n the rows' norms.
//
// The packed rows are expanded inside the kernel, straight from the pages
// into the shared-memory tiles that the tensor cores read: no expanded copy of
// the cache passes through memory.  A CTA's query tile is 256 rows (tokens
// times the query heads of one KV head; 128 at d = 256), so that one expansion
// serves two MMA row tiles.
//
//   warps 0-7    softmax, one thread per query row (4 warps at d = 256)
//   8 warps      expansion: bytes -> fp16 levels times the row's norm
//   1 warp       MMAs
//   1 warp       copies of packed rows and norms from the pages (bulk copies);
//                it also walks along the CTA's parts and hands them out
//   1 warp       the blocks' powers of two and the rows' factors
//
// The work is cut into equal shares, one per SM, along a line of all (query
// tile, KV head, block of positions) units: a share may end inside an item.
// (With few items a share is a part of one item.)  The two or more parts of
// such an item go to the workspace and k_prefill_paged_join adds them up in
// order.  All lengths are read on the device: the launch is the same for every
// batch.
//
// Two streams of steps keep the tensor cores and the softmax warps busy at
// once (d <= 128): with more than 128 query rows, stream g takes row tile g
// and both take every block; with at most 128 rows, the streams take the
// blocks in turn for the same rows and are merged at the end.  At d = 256 the
// output fills tensor memory: one stream, with two score buffers.
//
// Numbers.  fp16 operands, fp32 sums.  A block's K rows are scaled by a power
// of two 2^-Ek (its largest norm is below 2^(Ek + 14)), its V rows by 2^-Ev; Ek
// goes into the factor of the scores, Ev into the exponent of the probabilities,
//   P' = 2^(s + Ev - M),  M a running maximum of s + Ev, less 7,
// so that O = sum P' V' keeps its precision however the norms vary from block
// to block.  M moves only when it grows by more than 8, so P' < 2^15.  The
// denominator is held apart, l = sum 2^(s - m) with m the running maximum of the
// scores, from a block's sum of P' times 2^(M - Ev - m).
//   The norms that set a block's powers may belong to positions that a row does
// not attend to.  Its own K rows keep all their bits down to 2^-16 of the
// largest (fp16 has 28 powers of two below 2^14, the levels use 7 of them) and
// its V rows and probabilities to 2^-10.  A block whose norms are further apart (a
// K norm of 0 left out, and a block without any V norm), or whose Ev is 60 below an earlier one (the sum of P' could lose
// what l needs), is "wide": every position has its own Ek and Ev, and the softmax
// warps first put them into the scores (pp_wide).  Such steps are slower, and no
// size of norms that a row does not attend to changes its result.
// The query, P and the products of level and norm are rounded to fp16 once,
// 2^-11 relative, an eighth of the bf16 output's step (V's norms once more,
// before the product).  A non-finite norm makes the scores of its row NaN (only rows
// that attend to it see them) and its V row zero.
//
// What bounds it.  Two chunks of 4096 tokens over 12-16k positions (32 / 8
// heads, d = 128, K4/V3): 1.35 to 1.41 ms by GPU, 1.17 to 1.12 PFLOP/s of useful
// products, 61 to 58% of the measured burst rate; about 4300 cycles per block and
// 256 rows, of which the products need 2048.  A stream's step is a chain (scores 512 cycles and more,
// as both operands come from shared memory that the expansion writes at the
// same time; softmax about 2300; product with V 512; a barrier's wake-up of
// about 110 between each), and two streams do not fill all of it.  With one
// row tile the expansion's byte permutes set the pace, about 3800 cycles per
// block: 24 sequences of 1-4 tokens over 6-9k positions read 1.1 TB/s of
// packed rows.  Measured and not taken, against 1418 us of that step: score
// buffers of 64 columns, two per stream (1886 us); two softmax threads per row
// (1532 us); separate warps for the two kinds of products (1633 us); 4 or 16
// expansion warps (1486 and 1570 us).  Nor taken: the transform's stages across
// the 64-dim pieces first, straight from the queries' tile, and outputs staged
// there (d = 256: 120 us against 100; the same elements are read several times).
//
// Every wait on an mbarrier is bounded (2 s); one that gives up sets the
// device status word and a flag that ends the others.  The softmax warps go
// on through their (then failing) waits so that their barriers stay paired.  No
// output is written after the flag, and the join leaves out every item that a
// share with the flag may have had a part of.
#include <cfloat>
#include <climits>
#include <type_traits>

#include "tq_paged_parts.cuh"

#if !defined(TQ_UNIT_D) || !defined(TQ_UNIT_MODE)
#error "compile once per head dimension and mode with -DTQ_UNIT_D=<d> -DTQ_UNIT_MODE=<mode>"
#endif

namespace tq {
namespace dev {

// Sizes for head dimension D.
template <int D>
struct PpGeo {
    static constexpr int kD = D < 64 ? 64 : D;        // tile width: d = 32 is padded with zeros
    static constexpr int kN = D == 256 ? 64 : 128;    // positions per block
    static constexpr int kRows = PagedPrefillGeo<D>::kRows;
    static constexpr int kStreams = D == 256 ? 1 : 2;
    // The cost of a block for two row tiles and for one, and of an item's query
    // rotation and output, by which the line of work is cut into shares.  One row
    // tile costs nearly what two do (the expansion is the same).  32 sequences of
    // 1-496 tokens over 0.2-8k positions took 339 us with 2 : 1 and 2 blocks an
    // item, 223 us with these (238 and 229 us with 3 and 7 blocks an item); at
    // d = 256, 5 chunks with a window of 1024, 4 blocks 95 us and 5 blocks 98 us.
    static constexpr int kCostPair = kStreams == 2 ? 6 : 1, kCostSplit = kStreams == 2 ? 5 : 1;
    static constexpr int kCostItem = kStreams == 2 ? 5 * kCostPair : 4;
    static constexpr bool kWhole = false;  // (pp_start)
    static constexpr int kSoftWarps = 4 * kStreams;
    static constexpr int kDeqWarps = 8;
    static constexpr int kWarps = kSoftWarps + kDeqWarps + 3;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kStages = D <= 64 ? 4 : 2;   // staged packed blocks
    static constexpr uint32_t kTile = kN * kD * 2;    // an expanded K or V tile
    static constexpr uint32_t kQTile = 128 * kD * 2;
    static constexpr uint32_t kStage = kN * D + 8 * kN;  // 4-bit K and V rows, norms
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kRing = kQ + kStreams * kQTile;  // 4 tiles: K, V of two blocks
    static constexpr uint32_t kStg = kRing + 4 * kTile;
    static constexpr uint32_t kMeta = kStg + kStages * kStage;  // [8] float2: 2^Ek (0: wide), Ev
    static constexpr uint32_t kSegs = kMeta + 64;               // [kStages] segments staged
    static constexpr uint32_t kRed = kSegs + 16;                // scan scratch, then
    static constexpr uint32_t kCols = kRed;  // [kN] the wide block's Ek and Ev per position, a signed byte each
    static constexpr uint32_t kRedBytes = 2 * 8 * kWarps;
    static_assert(2 * kN <= kRedBytes && kRed % 16 == 0, "the positions' powers of two");
    static constexpr uint32_t kCur = (kRed + kRedBytes + 15) / 16 * 16;  // start cursor
    static constexpr uint32_t kJobs = kCur + 80;                // [2] jobs
    static constexpr uint32_t kBar = kJobs + 2 * 48;
    static constexpr int kBars = 2 * kStages + 4 + 4 + 8 + 2 + 2 + 2 + 2 + 2 + 1 + 1 + 1 + 1;
    static constexpr uint32_t kMisc = kBar + 8 * kBars;  // tensor-memory base, abort flag
    static constexpr uint32_t kSmem = (kMisc + 8 + 127) / 128 * 128;
    static constexpr uint32_t kTmemS = 0, kTmemO = 256;  // buffer b at kN b; output g at 128 g further
};

// Chunk c (8 dims, 16 bytes) of row r of a query tile.
__device__ __forceinline__ unsigned char* pp_place(unsigned char* tile, int r, int c) {
    return tile + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// ------------------------------------------------------------------ expansion

// 8 indices (fp16 pairs of their levels times the row's norm) to 16 bytes at
// dst.  The norm comes as fp16 high part r; with LOW also its rest rl, so that
// only the product is rounded (a rounded norm would shift a key's scores for
// every query alike).
template <int BITS, bool LOW>
__device__ __forceinline__ void pp_expand8(uint32_t f, __half2 r, __half2 rl, const uint32_t* hi, const uint32_t* lo,
                                           unsigned char* dst) {
    uint32_t sel, x = 0;
    if constexpr (BITS == 4) {
        // an index with its top bit set is positive level (index - 8), one
        // without is the negative of level 7 - index
        const uint32_t t = f & 0x88888888u;
        x = t >> 3;
        sel = (f ^ ~(t - x)) & 0x77777777u;
    } else if constexpr (BITS == 3) {
        // 3-bit fields spread to nibbles; the bits between them are cleared last
        sel = pp_select(f, f << 4, 0xFFFF0000u);
        sel = pp_select(sel, sel << 2, 0xFF00FF00u);
        sel = pp_select(sel, sel << 1, 0xF0F0F0F0u) & 0x77777777u;
    } else {
        sel = pp_select(f, f << 8, 0xFFFF0000u);
        sel = pp_select(sel, sel << 4, 0xFF00FF00u);
        sel = pp_select(sel, sel << 2, 0xF0F0F0F0u) & 0x33333333u;
    }
    uint32_t v[4];
    pp_levels4<BITS>(sel, x, hi, lo, v[0], v[1]);
    pp_levels4<BITS>(sel >> 16, x >> 16, hi, lo, v[2], v[3]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __half2 c = *reinterpret_cast<const __half2*>(&v[k]);
        const __half2 y = LOW ? __hfma2(c, r, __hmul2(c, rl)) : __hmul2(c, r);
        v[k] = *reinterpret_cast<const uint32_t*>(&y);
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
}

// This thread's share of one staged row, 16 indices per turn of a rolled loop.
// (All of the kernel's inner loops are rolled to stay within the instruction
// cache: unrolled, its warps waited for instructions most of the time.)
template <int BITS, int D, int TPR, bool LOW>
__device__ __forceinline__ void pp_expand_row(const unsigned char* rows, float rf, const uint32_t* hi,
                                              const uint32_t* lo, unsigned char* tile, uint32_t half_bytes, int row,
                                              int sub) {
    constexpr int EACH = D / 16 >= TPR ? D / 16 / TPR : 1;
    if (D / 16 < TPR && sub >= D / 16) return;
    const __half rh = __float2half_rn(rf);
    const __half2 r = __half2half2(rh), rl = __float2half2_rn(rf - __half2float(rh));
    const unsigned char* src = rows + row * (D * BITS / 8);
    unsigned char* dst = tile + (uint32_t)row * 128;
    const int turn = pp_turn<BITS, D>(row);
    const uint32_t sw = (row & 7) << 4;
#pragma unroll 1
    for (int e = sub * EACH; e < sub * EACH + EACH; ++e) {
        const int c = e ^ turn;
        uint32_t f0, f1;
        if constexpr (BITS == 4) {
            const uint2 u = reinterpret_cast<const uint2*>(src)[c];
            f0 = u.x;
            f1 = u.y;
        } else if constexpr (BITS == 3) {
            // 48 bits from a 32-bit boundary or 16 bits past one
            const uint32_t* w = reinterpret_cast<const uint32_t*>(src) + ((3 * c) >> 1);
            const uint32_t a = w[0], b = w[1];
            f0 = c & 1 ? __funnelshift_r(a, b, 16) : a;
            f1 = c & 1 ? b >> 8 : __funnelshift_r(a, b, 24);
        } else {
            f0 = reinterpret_cast<const uint32_t*>(src)[c];
            f1 = f0 >> 16;
        }
        unsigned char* d0 = dst + (uint32_t)(c >> 2) * half_bytes;
        const uint32_t at = ((uint32_t)(c & 3) << 5) ^ sw;
        pp_expand8<BITS, LOW>(f0, r, rl, hi, lo, d0 + at);
        pp_expand8<BITS, LOW>(f1, r, rl, hi, lo, d0 + (at ^ 16u));
    }
}

template <int D, int TPR, bool LOW>
__device__ __forceinline__ void pp_expand(int bits, const unsigned char* rows, float rf, const uint32_t* hi,
                                          const uint32_t* lo, unsigned char* tile, uint32_t half_bytes, int row,
                                          int sub) {
    if (bits == 4) pp_expand_row<4, D, TPR, LOW>(rows, rf, hi, lo, tile, half_bytes, row, sub);
    else if (bits == 3) pp_expand_row<3, D, TPR, LOW>(rows, rf, hi, lo, tile, half_bytes, row, sub);
    else pp_expand_row<2, D, TPR, LOW>(rows, rf, hi, lo, tile, half_bytes, row, sub);
}

// The largest of 32 values, NaN left out, in four chains.
__device__ __forceinline__ float pp_max32(const uint32_t (&s)[32]) {
    float m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = fmaxf(__uint_as_float(s[k]), __uint_as_float(s[4 + k]));
#pragma unroll
    for (int j = 8; j < 32; j += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = pp_max3(m[k], __uint_as_float(s[j + k]), __uint_as_float(s[j + 4 + k]));
    return fmaxf(pp_max3(m[0], m[1], m[2]), m[3]);
}

// Flip y[j] where bit j of the words is set.
template <int E>
__device__ __forceinline__ void pp_signs(float (&y)[E], const uint32_t* bits) {
#pragma unroll
    for (int w = 0; w < E / 32; ++w) {
        const uint32_t b = bits[w];
#pragma unroll
        for (int k = 0; k < 32; ++k)
            y[32 * w + k] = __uint_as_float(__float_as_uint(y[32 * w + k]) ^ ((b << (31 - k)) & 0x80000000u));
    }
}

// A piece of a row to and from this lane's tensor-memory columns.
template <int E>
__device__ __forceinline__ void pp_store_row(uint32_t t, const float (&y)[E]) {
#pragma unroll
    for (int c = 0; c < E / 32; ++c) {
        uint32_t o[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(y[32 * c + k]);
        tmem_st32(t + 32 * c, o);
    }
}
template <int E>
__device__ __forceinline__ void pp_load_row(uint32_t t, float (&y)[E]) {
    uint32_t o[E / 32][32];
#pragma unroll
    for (int c = 0; c < E / 32; ++c) tmem_ld32(t + 32 * c, o[c]);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < E; ++k) y[k] = __uint_as_float(o[k / 32][k % 32]);
}

// 16 columns of each of a row's pieces (64 columns apart), and the
// transform's stages across the pieces.
template <int PARTS>
__device__ __forceinline__ void pp_across(uint32_t t, uint32_t (&y)[PARTS][16]) {
#pragma unroll
    for (int h = 0; h < PARTS; ++h) tmem_ld16(t + 64 * h, y[h]);
    tmem_wait_ld();
#pragma unroll
    for (int len = 1; len < PARTS; len *= 2)
#pragma unroll
        for (int h = 0; h < PARTS; ++h)
            if (!(h & len)) {
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float u = __uint_as_float(y[h][k]), v = __uint_as_float(y[h + len][k]);
                    y[h][k] = __float_as_uint(u + v);
                    y[h + len][k] = __float_as_uint(u - v);
                }
            }
}

// Scores whose bit is not set become -inf.
template <int C>
__device__ __forceinline__ void pp_mask(uint32_t (&s)[C], uint32_t on) {
#pragma unroll
    for (int k = 0; k < C; ++k) s[k] = (on >> k) & 1u ? s[k] : 0xFF800000u;
}

// A wide block's scores, 16 columns from column c on, times their own factors;
// columns that are not the row's become -inf.
template <int MODE>
__device__ __forceinline__ void pp_wide16(uint32_t t_s, const unsigned char* cols, float cq, int c,
                                          const PpVis<MODE>& vis, float (&x)[16]) {
    const uint32_t on = vis.word(c);
    uint32_t s[16];
    tmem_ld16(t_s + c, s);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int e = *reinterpret_cast<const volatile int8_t*>(cols + 2 * (c + k));
        x[k] = (on >> k) & 1u ? __uint_as_float(s[k]) * (cq * pp_pow2(e)) : -INFINITY;
    }
}
// A wide block becomes one without powers of two: its scores times their factors
// plus the positions' V exponents, in the scores' place.  Returns the larger of m
// and the block's maximum score, and the row's sum of 2^(s - that).  (A call by
// itself, with values only: inlined in the step it took registers and instruction
// cache from all steps, 1.37 -> 1.63 ms for the long chunks.)
template <int N, int MODE>
__device__ __noinline__ float2 pp_wide(uint32_t t_s, const unsigned char* cols, float cq, PpVis<MODE> vis, float m) {
    float sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < N; c += 16) {
        float x[16];
        pp_wide16(t_s, cols, cq, c, vis, x);
#pragma unroll
        for (int k = 0; k < 16; ++k) m = fmaxf(m, x[k]);
    }
    const float mr = m == -INFINITY ? 0.f : m;
#pragma unroll 1
    for (int c = 0; c < N; c += 16) {
        float x[16];
        uint32_t w[16];
        pp_wide16(t_s, cols, cq, c, vis, x);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            sum += pp_exp2(x[k] - mr);
            w[k] = __float_as_uint(x[k] + (float)*reinterpret_cast<const volatile int8_t*>(cols + 2 * (c + k) + 1));
        }
        tmem_st16(t_s + c, w);
    }
    tmem_wait_st();
    return make_float2(m, sum);
}
// The finite norms' bits, 0 for the others; the power of two that goes with them:
// norms below 2^(e + 14), and a range that keeps every factor of the kernel a
// normal fp32.
__device__ __forceinline__ uint32_t pp_finite(float v) {
    const uint32_t x = __float_as_uint(v) & 0x7FFFFFFFu;
    return x < 0x7F800000u ? x : 0u;
}
__device__ __forceinline__ int pp_exponent(uint32_t m) { return min(100, max(-100, (int)(m >> 23) - 140)); }

// The factors of a wide block (norms kn and, behind them, vn), and its
// positions' powers of two.
template <int N>
__device__ __noinline__ void pp_wide_norms(float* kn, unsigned char* cols, uint32_t segs, int from, int snk,
                                           int lim, int seg_sh) {
#pragma unroll 1
    for (int r = threadIdx.x & 31; r < N; r += 32) {
        const bool in = (r >= from || r < snk) && r < lim && ((segs >> (4 * (r >> seg_sh))) & 1u);
        const float k = in ? kn[r] : 0.f, v = in ? kn[N + r] : 0.f;
        const int ek = pp_exponent(pp_finite(k)), ev = pp_exponent(pp_finite(v));
        kn[r] = fmaf(v, 0.f, k * pp_pow2(-ek));  // NaN if either norm is not finite
        kn[N + r] = fabsf(v) <= FLT_MAX ? v * pp_pow2(-ev) : 0.f;
        reinterpret_cast<uint16_t*>(cols)[r] = (uint16_t)((ek & 0xFF) | (ev & 0xFF) << 8);
    }
}

// ---------------------------------------------------------------- the kernel

template <int D, int MODE>
__global__ void __launch_bounds__(PpGeo<D>::kThreads, 1)
k_prefill_paged(const __grid_constant__ PpArgs A, const __grid_constant__ PagedPrefillConsts P, int* status) {
    using Z = PpGeo<D>;
    constexpr int N = Z::kN, W = Z::kD, SW = Z::kSoftWarps, DW = Z::kDeqWarps, NS = Z::kStages;
    constexpr int PARTS = D < 64 ? 1 : D / 64;  // register-sized pieces of a row
    constexpr int E = D < 64 ? D : 64;
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t sa = smem_addr(sm);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // known to be the same in a warp
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Z::kBar);
    uint64_t* stage_full = bars;              // [NS] the block's packed rows have landed
    uint64_t* stage_free = stage_full + NS;   // [NS] the expansion has read them
    uint64_t* kv_full = stage_free + NS;      // [4] a tile is expanded
    uint64_t* kv_free = kv_full + 4;          // [4] its products are done
    uint64_t* meta_full = kv_free + 4;        // [8] the block's row factors and powers of two are written
    uint64_t* s_full = meta_full + 8;         // [2] scores of the buffer's step are done
    uint64_t* p_full = s_full + 2;            // [2] the softmax warps wrote P over them
    uint64_t* pv_done = p_full + 2;           // [2] its PV product is done
    uint64_t* job_full = pv_done + 2;         // [2] a job is written
    uint64_t* job_free = job_full + 2;        // [2] every warp has read it
    uint64_t* q_full = job_free + 2;          // the item's queries are in shared memory
    uint64_t* meet = q_full + 1;              // all softmax warps are here
    uint64_t* drain = meet + 1;               // products in flight, on the abort path
    uint64_t* cols_free = drain + 1;          // the softmax warps have read a wide block's powers
    volatile int* abort_f = reinterpret_cast<volatile int*>(sm + Z::kMisc + 4);
    uint32_t* slot = reinterpret_cast<uint32_t*>(sm + Z::kMisc);
    PpCursor* start = reinterpret_cast<PpCursor*>(sm + Z::kCur);
    long long* share = reinterpret_cast<long long*>(sm + Z::kCur + 64);  // units of a share
    long long* red = reinterpret_cast<long long*>(sm + Z::kRed);

    if (sa & 1023u) {  // the tiles' swizzle needs it; the whole grid leaves, with nothing to join
        if (tid == 0) {
            report_timeout(status, kPpStatusAlign);
            griddep_wait();
            *reinterpret_cast<int4*>(A.meta + (int64_t)blockIdx.x * kPpMeta) = make_int4(kShareFailed, -1, 0, 0);
        }
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&stage_full[i], 1);
            mbar_init(&stage_free[i], DW);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&kv_full[i], DW);
            mbar_init(&kv_free[i], 1);
        }
        for (int i = 0; i < 8; ++i) mbar_init(&meta_full[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&pv_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&job_full[i], 1);
            mbar_init(&job_free[i], SW + DW + 2);
        }
        mbar_init(q_full, SW);
        mbar_init(meet, SW);
        mbar_init(drain, 1);
        mbar_init(cols_free, SW);
        *abort_f = 0;
        mbar_fence_init();
        start->left = 0;
        start->parts = 0;
    }
    if (warp == SW + DW) tmem_alloc<512>(slot);

    // From here on: what earlier kernels wrote.  No read-only loads (__ldg): they
    // may be taken ahead of the wait, as these values change within the grid's life.
    griddep_wait();
    pp_start<Z, MODE>(A, red, start, share, status);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*slot);
    PpJob p;
    int job = 0;
    // The next job; false at the end.
    auto next_job = [&]() {
        const bool ok = pp_wait(&job_full[job & 1], (job >> 1) & 1, abort_f, status);
        if (!__all_sync(0xFFFFFFFFu, ok)) return false;
        const volatile PpJob* m = reinterpret_cast<const volatile PpJob*>(sm + Z::kJobs) + (job & 1);
        p.nb = m->nb;
        p.flags = m->flags;
        p.q0 = m->q0;
        p.h = m->h;
        p.row0 = m->row0;
        p.rows = m->rows;
        p.blk = m->blk;
        p.kv_lo = m->kv_lo;
        p.kv_end = m->kv_end;
        p.pos0 = m->pos0;
        p.tok0 = m->tok0;
        p.rest = m->rest;
        __syncwarp();
        if (lane == 0) mbar_arrive(&job_free[job & 1]);
        ++job;
        return p.nb >= 0;
    };

    if (warp == SW + DW + 1) {
        // ---- copies: lane 4 s + a brings array a of segment s (min(page, N)
        // positions) of a block
        const int seg = min(1 << A.shift, N), nseg = N / seg;
        const int s = lane >> 2, a = lane & 3;
        const uint32_t row_bytes = a == 0 ? D * A.k_bits / 8 : a == 1 ? D * A.v_bits / 8 : 4u;
        const unsigned char* arr = reinterpret_cast<const unsigned char*>(
            a == 0 ? (const void*)A.c.k_packed : a == 1 ? (const void*)A.c.v_packed : a == 2 ? (const void*)A.c.k_norm
                                                                                             : (const void*)A.c.v_norm);
        const uint32_t at = a == 0 ? 0u : a == 1 ? N * D / 2 : a == 2 ? N * D : N * D + 4 * N;
        PpCursor cur = *start;
        PpSeq<Z, MODE> seq;
        if (cur.left > 0 || cur.parts > 0) seq.set(A, cur.n, cur.ctx, cur.q0);
        uint32_t tc = 0;
        int has = 0;  // parts left in the workspace
        bool ok = true;
        for (; ok; ++job) {
            PpPart u;
            const bool more = pp_next_part(A, cur, seq, u, job == 0);
            if (job >= 2) ok = pp_wait(&job_free[job & 1], ((job >> 1) - 1) & 1, abort_f, status);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            if (lane == 0) {
                pp_write_job(reinterpret_cast<volatile PpJob*>(sm + Z::kJobs) + (job & 1), more, u, seq);
                mbar_arrive(&job_full[job & 1]);
            }
            __syncwarp();
            if (!more) break;
            if (!u.whole) has |= u.head ? 2 : 1;
            // this lane's segment of block j: its page, or -1; looked up a block ahead
            auto block_at = [&](int j) { return pp_block_at<Z, MODE>(A, u.kv_lo, u.kv_end, u.lo_blk + j); };
            auto page_of = [&](int j) {
                const int pos = block_at(j) * N + s * seg;
                return s < nseg && j < u.blk1 && pos < u.kv_end &&
                               (pos + seg > u.kv_lo || (MODE == kPpSinks && pos < A.sinks))
                           ? A.bt[(int64_t)u.b * A.max_pages + (pos >> A.shift)]
                           : INT_MIN;
            };
            int next_page = page_of(u.blk0);
            for (int j = u.blk0; j < u.blk1; ++j, ++tc) {
                const int st = tc % NS;
                const int pos = block_at(j) * N + s * seg;
                const int page = next_page;
                next_page = page_of(j + 1);
                bool have = page != INT_MIN;
                if (have && (page < 0 || page >= A.c.n_pages)) {
                    report_timeout(status, kPpStatusPage);
                    have = false;
                }
                const int64_t src = (((int64_t)page * A.Hkv + u.h) << A.shift) + (pos & ((1 << A.shift) - 1));
                if (tc >= (uint32_t)NS) ok = pp_wait(&stage_free[st], (tc / NS - 1) & 1, abort_f, status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const uint32_t bytes = have ? row_bytes * seg : 0u;
                const uint32_t all = __reduce_add_sync(0xFFFFFFFFu, bytes);
                const uint32_t mask = __ballot_sync(0xFFFFFFFFu, have && a == 0);
                if (lane == 0) {
                    reinterpret_cast<volatile uint32_t*>(sm + Z::kSegs)[st] = mask;  // bit 4 s: segment s is there
                    mbar_arrive_expect_tx(&stage_full[st], all);
                }
                __syncwarp();
                if (have)
                    bulk_load(sa + Z::kStg + st * Z::kStage + at + s * seg * row_bytes, arr + src * row_bytes, bytes,
                              &stage_full[st]);
            }
        }
        if (lane == 0) pp_report<Z, MODE>(A, *start, *share, cur, seq, ok, has);
        // the copies issued have landed before the CTA leaves (bounded)
        if (lane == 0 && tc > 0)
            for (uint32_t t = tc > (uint32_t)NS ? tc - NS : 0; t < tc; ++t) mbar_wait(&stage_full[t % NS], (t / NS) & 1);
    } else if (warp == SW + DW) {
        // ---- MMAs.  The whole warp walks through the steps and one elected lane
        // issues: with a warp-uniform flow the descriptors are computed in
        // uniform registers and the products follow one another at the tensor
        // cores' rate (64 cycles for M = N = 128, K = 16, shared-memory or
        // tensor-memory A, either order of B); inside a one-thread branch each
        // took 150 to 250 cycles to issue.
        constexpr uint32_t idesc_s = umma_idesc_f16(128, N, false);
        constexpr uint32_t idesc_o = umma_idesc_f16(128, W, false) | kIdescBTransposed;
        const uint32_t elected = elect_one();
        const uint64_t dq = umma_desc_sw128(sa + Z::kQ), dk = umma_desc_sw128(sa + Z::kRing),
                       dv = umma_desc_sw128_mn(sa + Z::kRing, N * 128);
        uint32_t tc0 = 0, items = 0;
        uint32_t n0 = 0, n1 = 0;  // products of each buffer so far
        bool ok = true;
        // each lane for itself: the lanes agree once a step
        auto wait = [&](uint64_t* bar, uint32_t parity) { return pp_wait(bar, parity, abort_f, status); };
        while (ok && next_job()) {
            const int nb = (int)uniform((uint32_t)p.nb);
            const bool pair = uniform((uint32_t)p.flags) & kJobPair;
            if (nb == 0) continue;
            ok = __all_sync(0xFFFFFFFFu, wait(q_full, items & 1));
            ++items;
            const int T = pair ? 2 * nb : nb;
            for (int t = 0; t < T + 2; ++t) {
                const int g = t & 1;
                // a pair's second step reads the tiles that the first one waited
                // for, and frees them
                const bool first_use = !(pair && g), last_use = !pair || g;
                const uint32_t tk = tc0 + (pair ? t >> 1 : t), tv = tk - (pair ? 1 : 2);  // blocks of S and PV
                const uint32_t slk = (2 * tk) & 3, slv = (2 * tv + 1) & 3;
                // operands and barriers first: nothing is left between a wait and its products
                const uint64_t vt = dv + ((slv * Z::kTile) >> 4), kt = dk + ((slk * Z::kTile) >> 4);
                const uint64_t qt = dq + ((pair && g ? Z::kQTile : 0u) >> 4);
                const uint32_t o = tmem + Z::kTmemO + (Z::kStreams == 2 ? 128 * g : 0);
                const uint32_t d = tmem + Z::kTmemS + N * g;
                const uint32_t more = (Z::kStreams == 2 ? t < 4 : t == 2) ? 0u : 1u;  // 0: the output's first product
                uint64_t *bp = &p_full[g], *bpv = &pv_done[g], *bs = &s_full[g], *bvf = &kv_free[slv], *bkf = &kv_free[slk];
                if (t < T && first_use && t < 2) ok = wait(&kv_full[slk], (tk >> 1) & 1) && ok;
                if (t >= 2) {
                    const uint32_t n = g ? n1++ : n0++;
                    ok = wait(bp, n & 1) && ok;
                    tc_fence_after();
                    if (elected) {
#pragma unroll
                        for (int kk = 0; kk < N / 16; ++kk)
                            umma_f16_ts(o, d + 8 * kk, vt + ((kk * 2048) >> 4), idesc_o, kk > 0 ? 1u : more);
                        umma_commit(bpv);
                        if (last_use) umma_commit(bvf);
                    }
                    __syncwarp();
                    // under the products: the next step's V tile, this step's K tile;
                    // the buffer takes the next scores once P has been read
                    if (t < T) {
                        if (first_use) ok = wait(&kv_full[slk], (tk >> 1) & 1) && ok;
                        ok = wait(bpv, n & 1) && ok;
                    }
                }
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                if (t < T) {
                    tc_fence_after();
                    if (elected) {
#pragma unroll
                        for (int kk = 0; kk < W / 16; ++kk)
                            umma_f16(d, qt + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                                     kt + (((kk >> 2) * (N * 128) + (kk & 3) * 32) >> 4), idesc_s, kk > 0 ? 1u : 0u);
                        umma_commit(bs);
                        if (last_use) umma_commit(bkf);
                    }
                    __syncwarp();
                }
                // under the scores' product: the V tile of the next step's product
                if (t >= 1 && t + 1 < T + 2 && !(pair && !g)) {
                    const uint32_t tn = tc0 + (pair ? (t + 1) >> 1 : t + 1) - (pair ? 1 : 2);
                    ok = wait(&kv_full[(2 * tn + 1) & 3], (tn >> 1) & 1) && ok;
                }
            }
            tc0 += nb;
        }
        if (!ok) {  // products in flight finish before the tensor memory is freed (bounded)
            if (elected) umma_commit(drain);
            __syncwarp();
            mbar_wait(drain, 0);
        }
    } else if (warp == SW + DW + 2) {
        // ---- norms: a block's powers of two, and its rows' factors in the
        // norms' place
        uint32_t tc = 0, wides = 0;
        bool ok = true;
        while (ok && next_job()) {
            int emax = -1000;
            for (int j = 0; j < p.nb; ++j, ++tc) {
                const int st = tc % NS;
                float* knp = reinterpret_cast<float*>(sm + Z::kStg + st * Z::kStage + N * D);
                float* vnp = knp + N;
                ok = __all_sync(0xFFFFFFFFu, pp_wait(&stage_full[st], (tc / NS) & 1, abort_f, status));
                if (!ok) break;
                const uint32_t segs = reinterpret_cast<volatile uint32_t*>(sm + Z::kSegs)[st];
                const int t0 = pp_block_at<Z, MODE>(A, p.kv_lo, p.kv_end, p.blk + j) * N;
                const int from = p.kv_lo - t0, lim = p.kv_end - t0;  // the block's positions that count
                const int snk = MODE == kPpSinks ? A.sinks - t0 : 0;  // and the sinks among those in front
                const int seg_sh = min(A.shift, N == 64 ? 6 : 7);
                float kn[N / 32], vn[N / 32];
                bool in[N / 32];
                // the largest finite norms, as bits
                uint32_t mk = 0, mv = 0;
#pragma unroll
                for (int k = 0; k < N / 32; ++k) {
                    const int r = 32 * k + lane;
                    in[k] = (r >= from || r < snk) && r < lim && ((segs >> (4 * (r >> seg_sh))) & 1u);
                    kn[k] = in[k] ? knp[r] : 0.f;
                    vn[k] = in[k] ? vnp[r] : 0.f;
                    const uint32_t x = pp_finite(kn[k]), y = pp_finite(vn[k]);
                    mk = max(mk, x), mv = max(mv, y);
                }
                mk = __reduce_max_sync(0xFFFFFFFFu, mk);
                mv = __reduce_max_sync(0xFFFFFFFFu, mv);
                // (a block without a V norm must not raise the running maximum)
                const int ek = mk ? pp_exponent(mk) : 0, ev = pp_exponent(mv);
                emax = max(emax, ev);
                const float sk = pp_pow2(-ek), sv = pp_pow2(-ev);
                bool far = ev < emax - 60;
#pragma unroll
                for (int k = 0; k < N / 32; ++k) {
                    const float x = fabsf(kn[k] * sk), y = fabsf(vn[k] * sv);  // the largest: 2^13 to 2^14
                    // (a V norm of 0 beside others: a row that attends to it alone has no use for their exponent)
                    far = far || (x < 0.25f && x > 0.f) || (y < 8.f && in[k] && mv > 0u);
                }
                const bool wide = __any_sync(0xFFFFFFFFu, far);
                if (!wide) {
#pragma unroll
                    for (int k = 0; k < N / 32; ++k) {
                        const int r = 32 * k + lane;
                        knp[r] = fmaf(vn[k], 0.f, kn[k] * sk);  // NaN if either norm is not finite
                        vnp[r] = fabsf(vn[k]) <= FLT_MAX ? vn[k] * sv : 0.f;
                    }
                } else {
                    if (wides) ok = __all_sync(0xFFFFFFFFu, pp_wait(cols_free, (wides - 1) & 1, abort_f, status));
                    if (!ok) break;
                    ++wides;
                    pp_wide_norms<N>(knp, sm + Z::kCols, segs, from, snk, lim, seg_sh);
                }
                __syncwarp();
                if (lane == 0) {
                    reinterpret_cast<float2*>(sm + Z::kMeta)[tc & 7] = make_float2(wide ? 0.f : pp_pow2(ek), (float)ev);
                    mbar_arrive(&meta_full[tc & 7]);
                }
            }
        }
    } else if (warp >= SW) {
        // ---- expansion: thread = (row, sub) of the block
        constexpr int TPR = 32 * DW / N;  // threads per row
        const int dt = tid - 32 * SW;
        const int row = dt % N, sub = dt / N;
        if (D < 64) {  // the padded half of the tiles stays zero
            for (uint32_t i = dt; i < 4 * Z::kTile / 16; i += 32 * DW)
                reinterpret_cast<uint4*>(sm + Z::kRing)[i] = make_uint4(0, 0, 0, 0);
            asm volatile("bar.sync 2, %0;" ::"n"(32 * DW) : "memory");
        }
        uint32_t tc = 0;
        bool ok = true;
        while (ok && next_job()) {
            for (int j = 0; j < p.nb; ++j, ++tc) {
                const int st = tc % NS;
                const unsigned char* stg = sm + Z::kStg + st * Z::kStage;
                const float* fac = reinterpret_cast<const float*>(stg + N * D);
                const uint32_t slk = (2 * tc) & 3, slv = (2 * tc + 1) & 3;
                // (whoever wrote the factors has seen the rows land)
                ok = pp_wait(&meta_full[tc & 7], (tc >> 3) & 1, abort_f, status) &&
                     (tc < 2 || pp_wait(&kv_free[slk], ((tc >> 1) - 1) & 1, abort_f, status));
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                pp_expand<D, TPR, true>(A.k_bits, stg, fac[row], A.khi, A.klo, sm + Z::kRing + slk * Z::kTile, N * 128,
                                        row, sub);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&kv_full[slk]);
                if (tc >= 2) ok = pp_wait(&kv_free[slv], ((tc >> 1) - 1) & 1, abort_f, status);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                pp_expand<D, TPR, false>(A.v_bits, stg + N * D / 2, fac[N + row], A.vhi, A.vlo,
                                         sm + Z::kRing + slv * Z::kTile, N * 128, row, sub);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&kv_full[slv]);
                    mbar_arrive(&stage_free[st]);
                }
            }
        }
    } else {
        // ---- softmax: stream g, row r of its tile
        const int g = warp >> 2, r = 32 * (warp & 3) + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t t_out = t_lane + Z::kTmemO + 128 * g;
        const int G = A.Hq / A.Hkv;
        const uint32_t invG = (65536u + G - 1) / G;  // x / G = x invG >> 16 for x < 384, G <= 128
        const float q_sign = P.q_mul > 0.f ? 1.f : (P.q_mul < 0.f ? -1.f : 0.f);
        const float q_abs = P.q_mul == 0.f ? 1.f : fabsf(P.q_mul);
        uint32_t ns[2] = {0, 0}, npv[2] = {0, 0}, tc0 = 0, met = 0;
        // All softmax warps arrive and wait for one another (bounded).
        auto meet_all = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(meet);
            pp_wait(meet, met & 1, abort_f, status);
            ++met;
            __syncwarp();
            tc_fence_after();
        };
        // This warp's 32 rows of the next item's queries, into their places of the
        // tile (all products with the item's before are done): asynchronous copies
        // of 16 bytes a lane.
        auto fetch = [&]() {
            const bool ok = pp_wait(&job_full[job & 1], (job >> 1) & 1, abort_f, status);
            if (!__all_sync(0xFFFFFFFFu, ok)) return;
            const volatile PpJob* m = reinterpret_cast<const volatile PpJob*>(sm + Z::kJobs) + (job & 1);
            const bool pair = m->flags & kJobPair;
            if (m->nb <= 0 || (g && !pair)) return;
            const int lrow = r + (pair ? 128 * g : 0), left = m->rows - (pair ? 128 * g : 0) - 32 * (warp & 3);
            if (left <= 0) return;
            const int x = m->rest + lrow, tok = x * invG >> 16;  // from the item's first token on
            const int rel = tok * A.Hq + x - tok * G;
            const __nv_bfloat16* src = A.q + (((int64_t)m->q0 + m->tok0) * A.Hq + (int64_t)m->h * G) * D + 8 * (lane % (D / 8));
            unsigned char* qt = sm + Z::kQ + (pair ? g * Z::kQTile : 0) + 4096 * (warp & 3);
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
                const int rr = (32 * i + lane) / (D / 8);
                const int at = __shfl_sync(0xFFFFFFFFu, rel, rr);
                const bool in = rr < left;
                cp_async16(smem_addr(pp_place(qt, rr, lane % (D / 8))), src + (int64_t)(in ? at : 0) * D, in ? 16 : 0);
            }
            cp_async_commit();
        };
        for (;;) {
            fetch();
            if (!next_job()) break;
            const int nb = p.nb;
            const bool pair = p.flags & kJobPair, split = Z::kStreams == 2 && !pair;
            // the row of this thread: in split mode both streams have row r
            const int lrow = pair ? 128 * g + r : r;
            const bool rvalid = lrow < p.rows;
            const int x = rvalid ? p.rest + lrow : 0, dt = x * invG >> 16;
            const int tok = p.tok0 + dt, hd = x - dt * G;
            const int64_t qrow = ((int64_t)p.q0 + tok) * A.Hq + (int64_t)p.h * G + hd;
            const int pos = rvalid ? p.pos0 + tok : -1;
            // a warp without rows only keeps the barriers' count
            const bool rows_here = __any_sync(0xFFFFFFFFu, rvalid);
            const int lo = A.window > 0 ? max(0, pos - A.window + 1) : 0;
            const uint32_t* mask_row = MODE == kPpTree && rvalid ? A.mask + ((int64_t)p.q0 + tok) * A.words : nullptr;
            // ---- queries: each thread rotates its row in registers and tensor
            // memory (the output columns, free until the item's first product), 64
            // dims at a time, and rounds it to fp16 under a power of two.  A warp
            // without rows leaves its part of the tile as it is: those rows' scores
            // go nowhere.
            float cq = q_abs;
            if (nb > 0 && (pair || g == 0) && rows_here) {
                float amax = 0.f;
                unsigned char* qt = sm + Z::kQ + (pair ? g * Z::kQTile : 0) + 4096 * (warp & 3);
                cp_async_wait_all();
                __syncwarp();
#pragma unroll 1
                for (int h = 0; h < PARTS; ++h) {
                    float y[E];
                    {
                        uint32_t u[E / 2];
#pragma unroll
                        for (int k = 0; k < E / 8; ++k) {
                            const uint4 v = *reinterpret_cast<const uint4*>(pp_place(qt, lane, 8 * h + k));
                            u[4 * k] = v.x, u[4 * k + 1] = v.y, u[4 * k + 2] = v.z, u[4 * k + 3] = v.w;
                        }
#pragma unroll
                        for (int k = 0; k < E / 2; ++k) {
                            const uint32_t v = u[k] ^ P.sgnh[32 * h + k];
                            y[2 * k] = __uint_as_float(v << 16);
                            y[2 * k + 1] = __uint_as_float(v & 0xFFFF0000u);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < E; k += 2) amax = pp_max3(amax, fabsf(y[k]), fabsf(y[k + 1]));
                    fwht_reg2<E>(y);
                    pp_store_row<E>(t_out + 64 * h, y);
                }
                tmem_wait_st();
                // |rotated| <= D amax: below 2^14 after the scaling by 2^-e
                int e = 0;
                if (amax > 0.f && amax <= FLT_MAX) {
                    constexpr int LD = D == 32 ? 5 : D == 64 ? 6 : D == 128 ? 7 : 8;
                    e = min(100, max(-100, (int)(__float_as_uint(amax) >> 23) - 126 + LD - 14));
                }
                cq = q_abs * pp_pow2(e);
                const float inv = q_sign * pp_pow2(-e);
#pragma unroll 1
                for (int c = 0; c < E / 16; ++c) {
                    uint32_t y[PARTS][16];
                    pp_across<PARTS>(t_out + 16 * c, y);
#pragma unroll
                    for (int h = 0; h < PARTS; ++h) {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const __half2 hh = __floats2half2_rn(__uint_as_float(y[h][2 * k]) * inv,
                                                                 __uint_as_float(y[h][2 * k + 1]) * inv);
                            w[k] = *reinterpret_cast<const uint32_t*>(&hh);
                        }
                        if (P.two_sided) {  // signs of dims 2 k and 2 k + 1 onto bits 15 and 31
                            const uint32_t flip = (P.sgn2b[2 * h + (c >> 1)] >> (16 * (c & 1))) & 0xFFFFu;
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                w[k] ^= ((flip << (15 - 2 * k)) & 0x8000u) | ((flip << (30 - 2 * k)) & 0x80000000u);
                        }
                        *reinterpret_cast<uint4*>(pp_place(qt, lane, 8 * h + 2 * c)) = make_uint4(w[0], w[1], w[2], w[3]);
                        *reinterpret_cast<uint4*>(pp_place(qt, lane, 8 * h + 2 * c + 1)) = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                }
                if constexpr (D < 64) {
#pragma unroll
                    for (int k8 = D / 8; k8 < 8; ++k8)
                        *reinterpret_cast<uint4*>(pp_place(qt, lane, k8)) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            float* xs = reinterpret_cast<float*>(sm + Z::kQ + Z::kQTile);  // split mode: row tile 1 is free
            if (split && nb > 0) {
                // stream 1 has the same rows: it takes their factor from stream 0
                if (g == 0) xs[384 + r] = cq;
                meet_all();
                if (g == 1) cq = xs[384 + r];
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && nb > 0) mbar_arrive(q_full);

            // ---- the steps
            float M = -INFINITY, l = 0.f, m = -INFINITY;
            int lastb = -1;  // buffer of this stream's last step
            int j = split ? g : 0;
            // Twice in the code: the wide blocks apart (in one loop, with the call in it,
            // all steps were 4% slower)
            auto steps = [&](auto with) __attribute__((always_inline)) {
                constexpr bool kWide = decltype(with)::value;
                for (; j < nb; j += split ? 2 : 1) {
                    const int buf = Z::kStreams == 2 ? g : (j & 1);
                    const uint32_t tc = tc0 + j;
                    pp_wait(&meta_full[tc & 7], (tc >> 3) & 1, abort_f, status);
                    const volatile float* mp = reinterpret_cast<const volatile float*>(sm + Z::kMeta) + 2 * (tc & 7);
                    const float2 meta = make_float2(mp[0], mp[1]);
                    // a vote, so that the warp stays together also where a wait gave up and the lanes
                    // read the slot at different times
                    const bool wide = __any_sync(0xFFFFFFFFu, meta.x == 0.f);
                    if (kWide != wide) break;
                    // what the step sees, ahead of its scores (behind the wait it cost 260 to 530
                    // cycles of a step's 4400)
                    const int t0 = pp_block_at<Z, MODE>(A, p.kv_lo, p.kv_end, p.blk + j) * N;
                    PpVis<MODE> vis;  // the columns of the block that are this row's
                    bool all = true;
                    if constexpr (MODE == kPpTree) {
                        vis.row = mask_row;
                        vis.words = rvalid ? A.words : 0;
                        vis.node0 = p.pos0 - t0;
                        vis.end = rvalid ? p.kv_end - t0 : 0;
                        all = vis.node0 >= N;
                    } else {
                        vis.c1 = min(N, pos + 1 - t0), vis.c0 = max(0, lo - t0);
                        if constexpr (MODE == kPpSinks) {
                            vis.cs = min(vis.c1, A.sinks - t0);
                            if (vis.cs >= vis.c0) vis.c0 = 0;
                        }
                        all = vis.c1 == N && vis.c0 == 0;
                    }
                    const bool full = __all_sync(0xFFFFFFFFu, !rvalid || all);
                    pp_wait(&s_full[buf], ns[buf] & 1, abort_f, status);
                    ++ns[buf];
                    __syncwarp();
                    lastb = buf;
                    if (!rows_here) {
                        tc_fence_before();
                        __syncwarp();
                        if (kWide && lane <= (split ? 1 : 0)) mbar_arrive(cols_free);
                        if (lane == 0) mbar_arrive(&p_full[buf]);
                        ++npv[buf];
                        continue;
                    }
                    tc_fence_after();
                    const uint32_t t_s = t_lane + Z::kTmemS + N * buf;
                    // not 0, which a masked score of -inf would make NaN: tiny queries over tiny norms
                    float cs = fmaxf(cq * meta.x, FLT_MIN), ev = meta.y;
                    float2 w2;  // a wide block's
                    if (kWide) {
                        w2 = pp_wide<N>(t_s, sm + Z::kCols, cq, vis, m);
                        cs = 1.f, ev = 0.f;
                        __syncwarp();
                        if (lane <= (split ? 1 : 0)) mbar_arrive(cols_free);
                    }
                    float mx = -INFINITY;
                    if (full) {
#pragma unroll 1
                        for (int c = 0; c < N; c += 32) mx = fmaxf(mx, tmem_max32(t_s + c));
                    } else {
#pragma unroll 1
                        for (int c = 0; c < N; c += 32) {
                            uint32_t s[32];
                            tmem_ld32(t_s + c, s);
                            tmem_wait_ld();
                            pp_mask(s, vis.word(c));
                            mx = fmaxf(mx, pp_max32(s));
                        }
                    }
                    const float top = mx * cs, cand = top + ev;  // -inf where nothing is attended
                    const bool move = cand > M + 15.f || (M == -INFINITY && cand > -INFINITY);
                    const bool rescale = move && M != -INFINITY;
                    if (__any_sync(0xFFFFFFFFu, rescale)) {
                        const float alpha = rescale ? pp_exp2(M - (cand - 7.f)) : 1.f;
                        if (Z::kStreams == 1)  // the other buffer's product wrote the output last
                            pp_wait(&pv_done[buf ^ 1], (npv[buf ^ 1] - 1) & 1, abort_f, status);
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < W; c += 32) {
                            uint32_t o[32];
                            tmem_ld32(t_out + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                            tmem_st32(t_out + c, o);
                        }
                    }
                    if (move) M = cand - 7.f;
                    const float m1 = kWide ? w2.x : fmaxf(m, top), mr = m1 == -INFINITY ? 0.f : m1;
                    l *= pp_exp2(m - mr);  // (NaN stays)
                    m = m1;
                    const float off = M == -INFINITY ? 0.f : ev - M;
                    const F2 CS = f2(cs, cs), OFF = f2(off, off);
                    F2 sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
                    // Columns at a time.  d = 256, 5 chunks with a window: 32 97.7 us, 16 93.8 (four
                    // softmax warps beside eight of the expansion: the shorter loop leaves those
                    // more of the instruction cache); two streams, long chunks: 1356 and 1454 us.
                    constexpr int C = Z::kStreams == 1 ? 16 : 32;
#pragma unroll 1
                    for (int c = 0; c < N; c += C) {
                        uint32_t s[C];
                        if constexpr (C == 16) tmem_ld16(t_s + c, s);
                        else tmem_ld32(t_s + c, s);
                        tmem_wait_ld();
                        if (!full) pp_mask(s, vis.word(c));
                        uint32_t w[C / 2];
#pragma unroll
                        for (int k = 0; k < C / 2; ++k) {
                            float a0, a1;
                            f2_split(f2_fma(f2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), CS, OFF), a0, a1);
                            a0 = pp_exp2(a0);
                            a1 = pp_exp2(a1);
                            sum[k & 1] = f2_add(sum[k & 1], f2(a0, a1));
                            const __half2 hh = __floats2half2_rn(a0, a1);
                            w[k] = *reinterpret_cast<const uint32_t*>(&hh);
                        }
                        if constexpr (C == 16) tmem_st8(t_s + c / 2, w);
                        else tmem_st16(t_s + c / 2, w);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[buf]);
                    ++npv[buf];
                    float s0, s1;
                    f2_split(f2_add(sum[0], sum[1]), s0, s1);
                    l = kWide ? l + w2.y : fmaf(s0 + s1, pp_exp2(M - ev - mr), l);
                }
            };
            while (j < nb) {
                steps(std::false_type{});
                steps(std::true_type{});
            }
            if (lastb >= 0) {
                if (Z::kStreams == 1 && nb > 1) pp_wait(&pv_done[lastb ^ 1], (npv[lastb ^ 1] - 1) & 1, abort_f, status);
                pp_wait(&pv_done[lastb], (npv[lastb] - 1) & 1, abort_f, status);
            }
            __syncwarp();
            tc_fence_after();
            // ---- split mode: stream 0 adds stream 1's output and sums to its own
            if (split && nb > 0) {
                if (g == 1) {
                    xs[r] = M;
                    xs[128 + r] = l;
                    xs[256 + r] = m;
                }
                meet_all();
                if (g == 0 && nb > 1 && rows_here) {
                    const float M1 = xs[r], l1 = xs[128 + r], m1 = xs[256 + r];
                    const float Mx = fmaxf(M, M1);
                    const float a0 = M == -INFINITY ? 0.f : pp_exp2(M - Mx), a1 = M1 == -INFINITY ? 0.f : pp_exp2(M1 - Mx);
#pragma unroll 1
                    for (int c = 0; c < W; c += 16) {
                        uint32_t o[16], o1[16];
                        tmem_ld16(t_out + c, o);
                        tmem_ld16(t_out + 128 + c, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            o[k] = __float_as_uint(__uint_as_float(o[k]) * a0 + __uint_as_float(o1[k]) * a1);
                        tmem_st16(t_out + c, o);
                    }
                    tmem_wait_st();
                    pp_join_sums(l, m, l1, m1);
                    M = Mx;
                }
                meet_all();
            }
            // ---- the rows leave: finished, or as a part
            if ((pair || g == 0) && rows_here) {
                if (p.flags & kJobWhole) {
                    float inv = l == 0.f ? 0.f : pp_exp2(M - m) * P.out_mul * P.inv_sqrt_d / l;
                    // rotated back, s . H (s2 . o): 64 dims at a time, then across
#pragma unroll 1
                    for (int h = 0; h < PARTS; ++h) {
                        float y[E];
                        pp_load_row<E>(t_out + 64 * h, y);
                        if (nb == 0) {  // no position to attend to: the columns hold nothing of this item
#pragma unroll
                            for (int k = 0; k < E; ++k) y[k] = 0.f;
                        }
                        if (P.two_sided) pp_signs<E>(y, P.sgn2b + 2 * h);
                        fwht_reg2<E>(y);
                        pp_store_row<E>(t_out + 64 * h, y);
                    }
                    tmem_wait_st();
                    const bool write = rvalid && *abort_f == 0;
#pragma unroll 1
                    for (int c = 0; c < E / 16; ++c) {
                        uint32_t y[PARTS][16];
                        pp_across<PARTS>(t_out + 16 * c, y);
                        if (write) {
#pragma unroll
                            for (int h = 0; h < PARTS; ++h) {
                                const int64_t at = qrow * D + 64 * h + 16 * c;
                                if (A.out_bf16) {
                                    uint32_t w[8];
#pragma unroll
                                    for (int k = 0; k < 8; ++k) {
                                        const __nv_bfloat162 bb = __floats2bfloat162_rn(
                                            __uint_as_float(y[h][2 * k]) * inv, __uint_as_float(y[h][2 * k + 1]) * inv);
                                        w[k] = *reinterpret_cast<const uint32_t*>(&bb) ^ P.sgnh[32 * h + 8 * c + k];
                                    }
                                    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(A.out) + at);
                                    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                                    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                                } else {
                                    const uint32_t flip = P.sgnb[2 * h + (c >> 1)] >> (16 * (c & 1));
                                    uint32_t v[16];
#pragma unroll
                                    for (int k = 0; k < 16; ++k)
                                        v[k] = __float_as_uint(__uint_as_float(y[h][k]) * inv) ^
                                               ((flip << (31 - k)) & 0x80000000u);
                                    uint4* dst = reinterpret_cast<uint4*>(static_cast<float*>(A.out) + at);
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        dst[k] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                                }
                            }
                        }
                        __syncwarp();
                    }
                } else {
                    const int which = p.flags & kJobHead ? 1 : 0;
                    float* w = A.part + ((int64_t)blockIdx.x * 2 + which) * PagedPrefillGeo<D>::kPartFloats;
                    float4* o4 = reinterpret_cast<float4*>(w) + lrow;
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(t_out + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (rvalid)
                                o4[(c / 4 + k) * Z::kRows] =
                                    make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                                __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
                    }
                    float* x = w + D * Z::kRows;
                    x[lrow] = M;
                    x[Z::kRows + lrow] = l;
                    x[2 * Z::kRows + lrow] = m;
                }
                tc_fence_before();
            }
            tc0 += nb;
        }
        cp_async_wait_all();
    }
    griddep_launch();
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_f)  // over what the copy warp wrote
        *reinterpret_cast<int4*>(A.meta + (int64_t)blockIdx.x * kPpMeta) = make_int4(kShareFailed, -1, 0, 0);
    if (warp == SW + DW) {
        tc_fence_after();
        tmem_dealloc<512>(tmem);
    }
}

}  // namespace dev

template <int D, int MODE>
cudaError_t launch_prefill_paged(const PagedPrefillCall& c, cudaStream_t s) {
    const PagedPrefillConsts& P = c.consts;
    using namespace dev;
    using Z = PpGeo<D>;
    static_assert(Z::kSmem <= 232448, "shared memory per CTA");
    const int shares = num_sms();
    const PpArgs A = pp_args(c, shares, PagedPrefillGeo<D>::kPartFloats);
    static int attr_done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !attr_done[dev]) {
        e = cudaFuncSetAttribute(k_prefill_paged<D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Z::kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_done[dev] = 1;
    }
    e = launch_pdl(k_prefill_paged<D, MODE>, dim3(shares), dim3(Z::kThreads), Z::kSmem, s, A, P, status_word());
    if (e != cudaSuccess) return e;
    // groups of 32 rows that an item can have
    const int64_t rows = c.n_q * (c.Hq / c.Hkv);
    const unsigned groups = (unsigned)((rows < Z::kRows ? rows : Z::kRows) + 31) / 32;
    // Few rows: few items in many parts, four parts' loads in flight.  More: mostly
    // two parts an item, and three CTAs per SM count for more (two in flight: drafts
    // 21.1 -> 21.5 us, but 32 mixed sequences 222 -> 220, 2048 tokens after 4000 238
    // -> 235).
    if (D < 256 && rows < Z::kRows)
        return launch_pdl(k_prefill_paged_join<D, D < 256 ? 4 : 2, Z::kRows>, dim3(shares, groups), dim3(256), 0, s, A, P);
    return launch_pdl(k_prefill_paged_join<D, 2, Z::kRows>, dim3(shares, groups), dim3(256), 0, s, A, P);
}

template cudaError_t launch_prefill_paged<TQ_UNIT_D, TQ_UNIT_MODE>(const PagedPrefillCall&, cudaStream_t);

}  // namespace tq
