// tq_attn_few.cu -- attention of few query rows per (sequence, KV head) over the
// paged packed cache: single tokens over a window with sinks, small trees.
//
// With few rows the packed rows are what there is to read, and expanding them is
// the work: tiles in shared memory for the 5th-generation tensor cores take
// 512 bytes of writes and as many of operand reads per position (d = 128).  Here the products are mma.sync m16n8k16 with
// positions (scores) and dims (output) as rows and query rows as the 8 columns,
// and the packed rows go from shared memory straight into their A fragments: a
// pair of indices is one lookup in a table of fp16 pairs, replicated for the 32
// lanes (as in the decode attention, tq_attn.cu).
//
//   S^T[position, row] = K[position, :] . Q[row, :]
//   O^T[dim, row]     += V[:, dim]^T . P^T[position, row]
//
// Four warps at a time take a block of 128 positions of the CTA's part, 32 each,
// from a ring of two blocks of their own (one bulk copy per array and page:
// issuing one costs a warp some 100 cycles).  Every warp keeps a running maximum
// and output; the warps are merged at the part's end.  Work is cut into shares, parts of items
// are joined and lengths are read as in tq_prefill_paged.cu (tq_paged_parts.cuh).
//
// Numbers.  s = log2 score, in fp32 from the fp16 products.  Per row a running
// maximum m of s (p = 2^(s - m), l = sum p), moved only when s exceeds it by 8,
// and one M of s + log2 |V norm|:
//   P = p |V norm| 2^(m - M) <= 2^15, in fp16,
// so neither the size of a norm nor its spread takes bits from a row, whatever
// positions it does not attend to hold.  The query, the levels and P are rounded
// to fp16 (2^-11 relative each).  A non-finite norm makes the scores of its
// position NaN, for the rows that attend to it, and its V row zero.
//
// What bounds it.  32 sequences of 6000 positions, 32 / 8 heads, one query token
// (4 rows), d = 128, K4/V3: 76 us, 2.43 TB/s of packed rows; 16 rows 109 us; d = 64
// 61 us; d = 256, K4/V4 127 us, 3.2 TB/s.  About 960 instructions a chunk and warp,
// half of them byte permutes and shifts: the ALU is 45% busy, the lookups' pipe 44%,
// an issue slot in two is used, and 12 warps of 168 registers leave 0.8 of 3 ready.
// Measured and not kept: 16 warps of 128 registers (87 us, spills), chunks of 64
// positions in 8 warps (88), V by byte permutes instead of lookups (87), a warp that
// copies for the others (82: a bulk copy costs it some 100 cycles), rings of 3 blocks
// with 10 warps (96).  Tiles of 32 rows take 5800 cycles a block of positions, where
// the multi-token kernel takes 3500 for up to 128.  The same products transposed on
// tcgen05 (positions on the lanes) took 236 us at 24 rows: a row's factors come to
// every lane by shared-memory reads, and those and the tiles' own fill that pipe.
//
// Every wait is bounded; one that gives up sets the device status word and a
// flag, and the warps go on without computing, so that the block's barriers stay
// paired.
#include "tq_paged_parts.cuh"

#if !defined(TQ_UNIT_D) || !defined(TQ_UNIT_MODE)
#error "compile once per head dimension and mode with -DTQ_UNIT_D=<d> -DTQ_UNIT_MODE=<mode>"
#endif

namespace tq {
namespace dev {

constexpr int kFwStatusLayout = 76;  // dynamic shared memory starts above kFwLow

// Shared memory by absolute shared-window address (the dynamic block starts at
// or below kFwLow): the pair table 64 KiB aligned, so that a lookup's address is
// one byte permute: row e (256 bytes) holds pair e, keys in bytes 0..127 and
// values in 128..255, 4 bytes a lane.  The rings' blocks lie below it and, where
// they do not all fit, above.
constexpr uint32_t kFwLow = 2048, kFwTop = 232448;

struct FwJob {
    int b, h, nb, flags, q0, row0, rows, blk, kv_lo, kv_end, pos0, tok0, rest;
};
constexpr int kFwJobs = 24;  // parts known at a time

template <int D, int NT>
struct FwGeo {
    static constexpr int kN = 128;       // positions per block
    static constexpr int kRows = 8 * NT;  // query rows of an item
    static constexpr int kStreams = 1;
    static constexpr int kCostPair = 1, kCostSplit = 1, kCostItem = 4;  // of a block and an item (pp_start)
    static constexpr bool kWhole = true;  // shares may be items
    // registers: the output takes D / 4 NT, the queries D / 8 NT
        static constexpr int kWarps = D * NT >= 256 ? 8 : 12;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kQuads = kWarps / 4;
    static constexpr int kStages = 2;
    static constexpr uint32_t kStage = kN * (D + 8);  // 4-bit K and V rows, K and V norms
    static constexpr uint32_t kTable = D == 256 ? 131072 : 65536, kHigh = kTable + 65536;
    static constexpr int kAll = kQuads * kStages, kFitLow = (int)((kTable - kFwLow) / kStage);
    static constexpr int kLow = kFitLow < kAll ? kFitLow : kAll;  // blocks below the table
    static constexpr uint32_t kLowEnd = kFwLow + kLow * kStage;
    static constexpr uint32_t kHighEnd = kHigh + (kAll - kLow) * kStage;
    // queries in the order of the B fragments, row factors, parts, barriers, ...
    static constexpr uint32_t kQBytes = kRows * D * 2;
    static constexpr uint32_t kMiscBytes =
        kQBytes + 4 * kRows + kFwJobs * sizeof(FwJob) + 16 + (16 + 16) * kQuads * kStages + 16 * kWarps + 16 + 96 + 16;
    static constexpr bool kMiscLow = kLowEnd + kMiscBytes <= kTable;
    static constexpr uint32_t kQ = kMiscLow ? kLowEnd : kHighEnd;
    static constexpr uint32_t kFac = kQ + kQBytes;
    static constexpr uint32_t kJobs = kFac + 4 * kRows;
    static constexpr uint32_t kBar = (kJobs + kFwJobs * sizeof(FwJob) + 15) / 16 * 16;
    static constexpr uint32_t kRec = kBar + 16 * kQuads * kStages;  // [quads][stages] int4: position, part, segments
    static constexpr uint32_t kRed = kRec + 16 * kQuads * kStages;
    static constexpr uint32_t kCur = (kRed + 16 * kWarps + 15) / 16 * 16;
    static constexpr uint32_t kMisc = kCur + 96;  // parts at hand, abort flag
    static constexpr uint32_t kMiscEnd = kMisc + 16;
    // merge buffer, where more is left: [warps][rows at a time] of D floats and m, M, l
    static constexpr bool kMergeLow = kMiscLow && kTable - kMiscEnd > kFwTop - kHighEnd;
    static constexpr uint32_t kMerge = kMiscLow && !kMergeLow ? kHighEnd : kMiscEnd, kMergeTop = kMergeLow ? kTable : kFwTop;
    static constexpr uint32_t kMergeRow = 4 * (D + 4);
    static constexpr int kFit = (int)((kMergeTop - kMerge) / (kWarps * kMergeRow));
    static constexpr int kMergeRows = kFit < kRows ? kFit : kRows;
    static constexpr uint32_t kMergeEnd = kMerge + kWarps * kMergeRows * kMergeRow;
    static constexpr uint32_t kEnd = kMergeEnd > kHighEnd ? kMergeEnd : kHighEnd;
    static_assert(kMergeRows >= 1 && kMergeEnd <= kMergeTop && kEnd <= kFwTop && kHighEnd <= kFwTop && (!kMiscLow || kMiscEnd <= kTable) && kMerge % 16 == 0 && kQ % 16 == 0 &&
                      kStage % 16 == 0,
                  "shared-memory plan");
};

__device__ __forceinline__ void fw_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transposes an 8 x 8 matrix of 16-bit elements, two of a row per lane.
__device__ __forceinline__ uint32_t fw_transpose(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// The table is written once; the ring is read after a wait (volatile).
__device__ __forceinline__ uint32_t fw_lookup(uint32_t addr) {
    uint32_t v;
    asm("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t fw_word(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
// N consecutive words, by the widest loads that their number allows (aligned so).
template <int N>
__device__ __forceinline__ void fw_words(uint32_t addr, uint32_t (&w)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                         : "r"(addr + 4 * i));
    } else if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[i]), "=r"(w[i + 1]) : "r"(addr + 4 * i));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = fw_word(addr + 4 * i);
    }
}
// Field number `at` of BITS bits each of the row at `row`, as bits 0.. of w.
template <int BITS>
__device__ __forceinline__ void fw_field(uint32_t row, int at, uint32_t (&w)[(BITS + 31) / 32]) {
    constexpr int N = (BITS + 31) / 32;
    if constexpr (BITS % 32 == 0) {
        fw_words<N>(row + at * (BITS / 8), w);
    } else {
        const uint32_t off = (uint32_t)at * BITS, sh = off & 31, a = row + (off >> 5) * 4;
        // a field starts at a multiple of the power of two in BITS: the words that it touches
        constexpr int STEP = BITS & -BITS, M = (BITS + 32 - STEP + 31) / 32;
        uint32_t r[M];
#pragma unroll
        for (int i = 0; i < M; ++i) r[i] = fw_word(a + 4 * i);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = i + 1 < M ? __funnelshift_r(r[i], r[i + 1 < M ? i + 1 : i], sh) : r[i] >> sh;
    }
}
// Pair q of a field: the byte that holds the pair's first bit (of the field, or
// of it shifted by the pair's place in a byte) becomes the table's row.
template <int BITS, int N>
__device__ __forceinline__ uint32_t fw_pair(const uint32_t (&w)[N], int q, uint32_t slot) {
    const int o = q * 2 * BITS, sh = o & 7, wi = o >> 5, bi = (o >> 3) & 3;
    uint32_t x;
    if (sh == 0) x = w[wi];
    else if (wi + 1 < N) x = __funnelshift_r(w[wi], w[wi + 1], sh);
    else x = w[wi] >> sh;
    return fw_lookup(__byte_perm(x, slot, 0x7604u | ((uint32_t)bi << 4)));
}

// Which position of its 16 a row of the scores' tile is: lanes t of the value
// rows 2 t then read words of different banks.
__device__ __forceinline__ int fw_at(int r) { return r ^ ((r >> 1) & 1); }

// Scores of 32 positions: acc[u][nt], u the 16 positions.
template <int D, int NT, int BITS, bool QREG>
__device__ __forceinline__ void fw_scores(uint32_t rows, uint32_t slot, const uint32_t (&qf)[QREG ? NT : 1][QREG ? D / 16 : 1][2],
                                          uint32_t qs, int g, int t, float (&acc)[2][NT][4]) {
    constexpr int FB = D / 4 * BITS, ROW = D * BITS / 8, KK = D / 16;
    // D = 256: the fields in two parts, for the registers
    constexpr int PARTS = D == 256 ? 2 : 1;
    constexpr int NW = (FB / PARTS + 31) / 32;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[u][nt][0] = acc[u][nt][1] = acc[u][nt][2] = acc[u][nt][3] = 0.f;
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
        uint32_t w[2][2][NW];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                fw_field<FB / PARTS>(rows + (16 * u + 8 * h + fw_at(g)) * ROW, PARTS * t + part, w[u][h]);
#pragma unroll
        for (int k = 0; k < KK / PARTS; ++k) {
            const int kk = part * (KK / PARTS) + k;
            uint32_t b[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if constexpr (QREG) {
                    b[nt][0] = qf[nt][kk][0], b[nt][1] = qf[nt][kk][1];
                } else {
                    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                        : "=r"(b[nt][0]), "=r"(b[nt][1])
                        : "r"(qs + (uint32_t)(nt * KK + kk) * 256));
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t a0 = fw_pair<BITS>(w[u][0], 2 * k, slot), a1 = fw_pair<BITS>(w[u][1], 2 * k, slot);
                const uint32_t a2 = fw_pair<BITS>(w[u][0], 2 * k + 1, slot), a3 = fw_pair<BITS>(w[u][1], 2 * k + 1, slot);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) fw_mma(acc[u][nt], a0, a1, a2, a3, b[nt][0], b[nt][1]);
            }
        }
    }
}

// The output of 32 positions: pb[u][nt] the B fragments of P.
template <int D, int NT, int BITS>
__device__ __forceinline__ void fw_output(uint32_t rows, uint32_t slot, const uint32_t (&pb)[2][NT][2], int g, int t,
                                          float (&O)[NT][D / 16][4]) {
    constexpr int FB = D / 8 * BITS, ROW = D * BITS / 8;
    constexpr int NW = (FB + 31) / 32;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        uint32_t f[4][NW];
#pragma unroll
        for (int i = 0; i < 4; ++i) fw_field<FB>(rows + (16 * u + fw_at(2 * t + (i & 1) + 8 * (i >> 1))) * ROW, g, f[i]);
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
            const uint32_t A = fw_pair<BITS>(f[0], mt, slot), B = fw_pair<BITS>(f[1], mt, slot);
            const uint32_t C = fw_pair<BITS>(f[2], mt, slot), E = fw_pair<BITS>(f[3], mt, slot);
            const uint32_t a0 = __byte_perm(A, B, 0x5410), a1 = __byte_perm(A, B, 0x7632);
            const uint32_t a2 = __byte_perm(C, E, 0x5410), a3 = __byte_perm(C, E, 0x7632);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) fw_mma(O[nt][mt], a0, a1, a2, a3, pb[u][nt][0], pb[u][nt][1]);
        }
    }
}

struct FwLevels {
    uint16_t k[16], v[16];  // fp16 c * s of the plan's levels
};

template <int D, int NT, int MODE>
__global__ void __launch_bounds__(FwGeo<D, NT>::kThreads, 1)
k_attn_few(const __grid_constant__ PpArgs A, const __grid_constant__ PagedPrefillConsts P, const __grid_constant__ FwLevels L,
           int* status) {
    using Z = FwGeo<D, NT>;
    constexpr int W = Z::kWarps, S = Z::kStages, KK = D / 16;
    constexpr bool QREG = NT == 2 || D == 256;  // queries in registers, where they cost no warps
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    extern __shared__ __align__(16) unsigned char fw_smem[];
    const uint32_t base = smem_addr(fw_smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto at = [&](uint32_t abs) { return fw_smem + (abs - base); };
    if (base > kFwLow) {  // the whole grid leaves, with nothing to join
        if (tid == 0) {
            report_timeout(status, kFwStatusLayout);
            griddep_wait();
            *reinterpret_cast<int4*>(A.meta + (int64_t)blockIdx.x * kPpMeta) = make_int4(kShareFailed, -1, 0, 0);
        }
        return;
    }
    PpCursor* start = reinterpret_cast<PpCursor*>(at(Z::kCur));
    long long* share = reinterpret_cast<long long*>(at(Z::kCur + 80));
    volatile int* n_jobs = reinterpret_cast<volatile int*>(at(Z::kMisc));
    volatile int* abort_f = n_jobs + 1;
    FwJob* jobs = reinterpret_cast<FwJob*>(at(Z::kJobs));
    float* fac = reinterpret_cast<float*>(at(Z::kFac));
    const int quad = warp >> 2, sub = warp & 3;
    uint64_t* full = reinterpret_cast<uint64_t*>(at(Z::kBar)) + quad * S;  // [S] a block has landed
    uint64_t* free_ = full + Z::kQuads * S;                                // [S] its four warps have read it
    volatile int4* recs = reinterpret_cast<volatile int4*>(at(Z::kRec)) + quad * S;

    // ---- pair tables: row e holds the pair e mod 2^(2 bits)
    {
        const int mk = (1 << A.k_bits) - 1, mv = (1 << A.v_bits) - 1;
        for (int e = warp; e < 256; e += W) {
            const uint32_t k = L.k[e & mk] | (uint32_t)L.k[(e >> A.k_bits) & mk] << 16;
            const uint32_t v = L.v[e & mv] | (uint32_t)L.v[(e >> A.v_bits) & mv] << 16;
            *reinterpret_cast<uint32_t*>(at(Z::kTable + 256u * e + 4u * lane)) = k;
            *reinterpret_cast<uint32_t*>(at(Z::kTable + 256u * e + 128u + 4u * lane)) = v;
        }
    }
    if (tid == 0) {
        for (int i = 0; i < Z::kQuads * S; ++i) mbar_init(full + i, 1), mbar_init(free_ + i, 4);
        mbar_fence_init();
        start->left = 0;
        start->parts = 0;
        *abort_f = 0;
    }
    // From here on: what earlier kernels wrote (no read-only loads).
    griddep_wait();
    pp_start<Z, MODE>(A, reinterpret_cast<long long*>(at(Z::kRed)), start, share, status);
    __syncthreads();

    const int g = lane >> 2, t = lane & 3;
    const int G = A.Hq / A.Hkv;
    const uint32_t kslot = Z::kTable + 4u * lane, vslot = kslot + 128u;
    auto stage_at = [&](uint32_t st) {
        const int i = quad * S + (int)st;
        return i < Z::kLow ? kFwLow + i * Z::kStage : Z::kHigh + (i - Z::kLow) * Z::kStage;
    };
    const uint32_t k_row = D * A.k_bits / 8, v_row = D * A.v_bits / 8;
    // lane 4 s + a copies array a of segment s (min(page, 128) positions) of a block
    const int seg = min(1 << A.shift, Z::kN), seg_at = (lane >> 2) * seg;
    const unsigned char* my_src = reinterpret_cast<const unsigned char*>(
        (lane & 3) == 0 ? (const void*)A.c.k_packed : (lane & 3) == 1 ? (const void*)A.c.v_packed
                                                  : (lane & 3) == 2 ? (const void*)A.c.k_norm : (const void*)A.c.v_norm);
    const uint32_t my_row = (lane & 3) == 0 ? k_row : (lane & 3) == 1 ? v_row : 4u;
    const uint32_t my_dst = ((lane & 3) == 0 ? 0 : (lane & 3) == 1 ? 64 * D : (lane & 3) == 2 ? 128 * D : 128 * D + 512) + seg_at * my_row;  // in the block
    const float q_sign = P.q_mul > 0.f ? 1.f : (P.q_mul < 0.f ? -1.f : 0.f);
    const float q_abs = P.q_mul == 0.f ? 1.f : fabsf(P.q_mul);
    bool bad = false;              // a wait gave up: nothing is computed from then on
    uint32_t put = 0, taken = 0;   // blocks of the ring so far: copied (or on their way), and read by this warp

    PpCursor cur;  // of thread 0
    PpSeq<Z, MODE> seq;
    int has = 0;
    bool more = true, first_part = true;
    if (tid == 0) {
        cur = *start;
        if (cur.left > 0 || cur.parts > 0) seq.set(A, cur.n, cur.ctx, cur.q0);
    }
    for (;;) {
        // ---- the next parts of the share
        if (tid == 0) {
            int n = 0;
            while (n < kFwJobs && more) {
                PpPart u;
                more = pp_next_part(A, cur, seq, u, first_part);
                first_part = false;
                if (!more) break;
                if (!u.whole) has |= u.head ? 2 : 1;
                FwJob& x = jobs[n++];
                x.b = u.b, x.h = u.h, x.nb = u.blk1 - u.blk0;
                x.flags = (u.whole ? kJobWhole : 0) | (u.head ? kJobHead : 0);
                x.q0 = seq.q0, x.row0 = u.row0, x.rows = u.rows, x.blk = u.lo_blk + u.blk0;
                x.kv_lo = u.kv_lo, x.kv_end = u.kv_end, x.pos0 = seq.ctx - seq.n;
                x.tok0 = u.row0 / seq.G, x.rest = u.row0 - x.tok0 * seq.G;
            }
            *n_jobs = n;
        }
        __syncthreads();
        const int nj = *n_jobs;
        if (nj == 0) break;

        // The quad's blocks: numbers quad, quad + kQuads, ... of every part's, and then
        // a record without one.  Its warps bring them in turn, each the fourth after its
        // last, whose page ids it looks up that long before.
        const int blocks = (int)__reduce_add_sync(
            kAll, lane < nj ? (unsigned)max(0, (jobs[lane].nb - quad + Z::kQuads - 1) / Z::kQuads) : 0u);
        const uint32_t put0 = put;
        int mj = -1, mc = 0, mn = 0, m_t0 = 0, m_page = INT_MIN;  // this warp's next: part, block, the part's blocks; position, page
        auto look = [&](int steps) {
            for (; steps > 0 && mj < nj; --steps) {
                mc += Z::kQuads;
                while (mc >= mn && ++mj < nj) mc = quad, mn = jobs[mj].nb;
            }
            m_page = INT_MIN;
            if (mj >= nj) return;
            const FwJob& x = jobs[mj];
            m_t0 = pp_block_at<Z, MODE>(A, x.kv_lo, x.kv_end, x.blk + mc) * Z::kN;
            const int pos = m_t0 + seg_at;
            if (seg_at < Z::kN && pos < x.kv_end && (pos + seg > x.kv_lo || (MODE == kPpSinks && pos < A.sinks)))
                m_page = A.bt[(int64_t)x.b * A.max_pages + (pos >> A.shift)];
        };
        look(1 + (int)((sub - put0) & 3));
        auto bring = [&]() {
            if (bad || (int)(put - put0) > blocks) return;
            const uint32_t st = put % S;
            if ((put & 3) == (uint32_t)sub) {
                const bool have = m_page >= 0 && m_page < A.c.n_pages;
                if (m_page != INT_MIN && !have) report_timeout(status, kPpStatusPage);
                const uint32_t mask = __ballot_sync(kAll, have && (lane & 3) == 0);
                // (a wait that gives up is noticed at the block's own)
                if (put >= (uint32_t)S) pp_wait(free_ + st, (put / S - 1) & 1, abort_f, status);
                __syncwarp();
                if (lane == 0) {
                    recs[st].x = m_t0;
                    recs[st].y = mj;
                    recs[st].z = (int)mask;
                    mbar_arrive_expect_tx(full + st, __popc(mask) * seg * (k_row + v_row + 8));
                }
                __syncwarp();
                if (have && *abort_f == 0) {
                    const int pos = m_t0 + seg_at;
                    const int64_t row = (((int64_t)m_page * A.Hkv + jobs[mj].h) << A.shift) + (pos & ((1 << A.shift) - 1));
                    fence_async_smem();  // earlier reads of this stage come first
                    bulk_load(stage_at(st) + my_dst, my_src + row * my_row, seg * my_row, full + st);
                }
                look(4);
            }
            ++put;
        };
        for (int i = 0; i < S; ++i) bring();

        // this warp's rows of a part's queries, looked up a part ahead
        constexpr int E = D / 32, RW = (Z::kRows + W - 1) / W;
        uint32_t raw[RW][E < 2 ? 1 : E / 2];
        auto fetch = [&](int j) {
            if (j >= nj) return;
            const FwJob& x = jobs[j];
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                const int r = warp + W * i;
                if (r >= x.rows) break;
                const int at_row = x.rest + r, tok = at_row / G;
                const __nv_bfloat16* src =
                    A.q + (((int64_t)x.q0 + x.tok0 + tok) * A.Hq + (int64_t)x.h * G + (at_row - tok * G)) * D + E * lane;
                if constexpr (E == 1) raw[i][0] = *reinterpret_cast<const uint16_t*>(src);
                else if constexpr (E == 2) raw[i][0] = *reinterpret_cast<const uint32_t*>(src);
                else if constexpr (E == 4) {
                    const uint2 v = *reinterpret_cast<const uint2*>(src);
                    raw[i][0] = v.x, raw[i][1] = v.y;
                } else {
                    const uint4 v = *reinterpret_cast<const uint4*>(src);
                    raw[i][0] = v.x, raw[i][1] = v.y, raw[i][2] = v.z, raw[i][3] = v.w;
                }
            }
        };
        fetch(0);

        for (int j = 0; j < nj; ++j) {
            const FwJob& x = jobs[j];  // (not copied: registers)
            // ---- queries: a warp rotates a row, rounds it to fp16 under a power of
            // two and stores it in the order of the B fragments
            if (x.nb > 0) {
#pragma unroll
                for (int i = 0; i < RW; ++i) {
                    const int r = warp + W * i;
                    if (r >= Z::kRows) break;
                    float y[E];
                    if (r < x.rows) {
#pragma unroll
                        for (int k = 0; k < E; ++k) {
                            const uint32_t bits = E == 1 ? raw[i][0] << 16 : k & 1 ? raw[i][k / 2] & 0xFFFF0000u : raw[i][k / 2] << 16;
                            y[k] = __uint_as_float(bits ^ sign_mask(P.sgnb, E * lane + k));
                        }
#pragma unroll
                        for (int len = 1; len < E; len *= 2)
#pragma unroll
                            for (int k = 0; k < E; ++k)
                                if (!(k & len)) {
                                    const float a = y[k], c = y[k + len];
                                    y[k] = a + c;
                                    y[k + len] = a - c;
                                }
#pragma unroll
                        for (int m = 1; m < 32; m *= 2)
#pragma unroll
                            for (int k = 0; k < E; ++k) {
                                const float o = __shfl_xor_sync(kAll, y[k], m);
                                y[k] = lane & m ? o - y[k] : y[k] + o;
                            }
                    } else {
#pragma unroll
                        for (int k = 0; k < E; ++k) y[k] = 0.f;
                    }
                    float amax = 0.f;
#pragma unroll
                    for (int k = 0; k < E; ++k) amax = fmaxf(amax, fabsf(y[k]));
                    amax = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(amax)));
                    int e = 0;  // below 2^14 after the scaling
                    if (amax > 0.f && amax <= FLT_MAX) e = min(100, max(-100, (int)(__float_as_uint(amax) >> 23) - 126 - 14));
                    const float inv = q_sign * pp_pow2(-e);
#pragma unroll
                    for (int k = 0; k < E; ++k) {
                        const int dim = E * lane + k, tt = dim / (D / 4), rem = dim % (D / 4);
                        const __half v = __float2half_rn(
                            __uint_as_float(__float_as_uint(y[k] * inv) ^ (P.two_sided ? sign_mask(P.sgn2b, dim) : 0u)));
                        *reinterpret_cast<__half*>(at(Z::kQ + (((r >> 3) * KK + rem / 4) * 32 + 4 * (r & 7) + tt) * 8 + 2 * (rem & 3))) = v;
                    }
                    if (lane == 0) fac[r] = r < x.rows ? q_abs * pp_pow2(e) : 0.f;
                }
            }
            __syncthreads();
            fetch(j + 1);
            uint32_t qf[QREG ? NT : 1][QREG ? KK : 1][2];
            const uint32_t qs = Z::kQ + 8u * lane;
            if constexpr (QREG) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk)
                        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                                     : "=r"(qf[nt][kk][0]), "=r"(qf[nt][kk][1])
                                     : "r"(qs + (uint32_t)(nt * KK + kk) * 256));
            }
            // this lane's columns: rows 8 nt + 2 t and the next.  nm = -m, +inf for a row
            // that has attended to nothing; a row past the item's has factor 0 and -inf
            float O[NT][KK][4], cq[NT][2], nm[NT][2], M[NT][2], l[NT][2], cc[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int mt = 0; mt < KK; ++mt) O[nt][mt][0] = O[nt][mt][1] = O[nt][mt][2] = O[nt][mt][3] = 0.f;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = 8 * nt + 2 * t + c;
                    cq[nt][c] = fac[r];
                    nm[nt][c] = r < x.rows ? INFINITY : -INFINITY;
                    M[nt][c] = -INFINITY;
                    l[nt][c] = cc[nt][c] = 0.f;
                }
            }

            // a row of the lane's has attended to V norms of 0 alone (its factor is 0), or leads them
            // so far that its factor has left fp32 (times a V norm of 0 it would be NaN)
            bool lost = false;
            const int first_p = x.pos0 + x.tok0, last_p = x.pos0 + (x.row0 + x.rows - 1) / G;  // the rows' positions
            for (;;) {
                const uint32_t st = taken % S;
                if (bad) break;
                if (!__all_sync(kAll, pp_wait(full + st, (taken / S) & 1, abort_f, status))) {
                    bad = true;
                    break;
                }
                const int pos = recs[st].x + 32 * sub;
                if (recs[st].y != j) break;  // of a later part, or the end: it stays
                const uint32_t segs = (uint32_t)recs[st].z;
                const uint32_t sb = stage_at(st), s_k = sb + sub * 32 * k_row, s_v = sb + 64 * D + sub * 32 * v_row,
                               s_n = sb + 128 * D + sub * 128;
                if (pos < x.kv_end && (pos + 32 > x.kv_lo || (MODE == kPpSinks && pos < A.sinks))) {
                float acc[2][NT][4];
                if (A.k_bits == 4) fw_scores<D, NT, 4, QREG>(s_k, kslot, qf, qs, g, t, acc);
                else if (A.k_bits == 3) fw_scores<D, NT, 3, QREG>(s_k, kslot, qf, qs, g, t, acc);
                else fw_scores<D, NT, 2, QREG>(s_k, kslot, qf, qs, g, t, acc);
                // this lane's positions: 16 u + 8 h + fw_at(g)
                float kn[2][2], vn[2][2];
                {
                    const uint32_t sn = s_n + 4 * fw_at(g);
                    const bool none = !((segs >> (4 * (32 * sub / seg))) & 1u);  // the page is out of range: rows of norm 0
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        kn[i >> 1][i & 1] = none ? 0.f : __uint_as_float(fw_word(sn + 32 * i));
                        vn[i >> 1][i & 1] = none ? 0.f : __uint_as_float(fw_word(sn + 512 + 32 * i));
                    }
                }
                bool all;  // every row attends to every position
                if (MODE == kPpTree) all = pos + 32 <= x.pos0;
                else all = pos + 31 <= first_p && (A.window == 0 || pos > last_p - A.window || (MODE == kPpSinks && pos + 32 <= A.sinks));
                uint32_t on[2][2];  // of the position: bit 2 nt + k, the lane's columns
                if (!all) {
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        const int p = pos + 8 * i + fw_at(g);
                        int r0 = 0, r1 = 0;  // rows [r0, r1) attend to the position
                        if constexpr (MODE == kPpTree) {
                            if (p < x.pos0) r1 = Z::kRows;
                        } else {
                            const int first = p - first_p;
                            r0 = max(0, min(first, Z::kRows + 1)) * G - x.rest;
                            r1 = Z::kRows;
                            if (A.window > 0 && !(MODE == kPpSinks && p < A.sinks))
                                r1 = max(0, min(min(first, Z::kRows + 1) + A.window, Z::kRows + 1)) * G - x.rest;
                        }
                        uint32_t w = 0;
                        const int node = p - x.pos0;
#pragma unroll
                        for (int c = 0; c < 2 * NT; ++c) {
                            const int r = 8 * (c >> 1) + 2 * t + (c & 1);
                            bool is = r >= r0 && r < r1;
                            if (MODE == kPpTree && node >= 0 && p < x.kv_end && r < x.rows)
                                is = (A.mask[((int64_t)x.q0 + x.tok0 + (x.rest + r) / G) * A.words + (node >> 5)] >> (node & 31)) & 1u;
                            w |= is ? 1u << c : 0u;
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (i == k) on[k >> 1][k & 1] = w;
                    }
                }
                // ---- probabilities, as B fragments.  Turn 0 takes the maxima as they are; if a
                // score is 8 above m, a P above 2^15, or a norm not finite, they move and
                // turn 1 follows, and where the factor of P is above 2^100 (a p that is lost
                // could count) or is lost itself turn 2, by exponents
                float p[2][NT][4], lv[2][2];
                uint32_t pb[2][NT][2];
#pragma unroll 1
                for (int turn = 0;; ++turn) {
                    float top = -INFINITY, ymax = 0.f, odd = 0.f;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            odd = fmaf(kn[u][h], 0.f, fmaf(vn[u][h], 0.f, odd));
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float x[2], y[2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    x[k] = fmaf(acc[u][nt][2 * h + k] * kn[u][h], cq[nt][k], nm[nt][k]);
                                    if (!all) x[k] = (on[u][h] >> (2 * nt + k)) & 1u ? x[k] : -INFINITY;
                                }
                                top = pp_max3(top, x[0], x[1]);
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const float e = pp_exp2(x[k]), w = vn[u][h] * cc[nt][k];
                                    p[u][nt][2 * h + k] = e;
                                    y[k] = e * w;
                                    ymax = pp_max3(ymax, fabsf(y[k]), fabsf(w) * 0x1p-85f);
                                    if (turn == 2) {  // (no M: no V norm but 0)
                                        const float d = M[nt][k] == -INFINITY ? 0.f : -nm[nt][k] - M[nt][k];
                                        y[k] = copysignf(pp_exp2(x[k] + (lv[u][h] + d)), vn[u][h]);
                                    }
                                }
                                const __half2 hh = __floats2half2_rn(y[0], y[1]);
                                pb[u][nt][h] = *reinterpret_cast<const uint32_t*>(&hh);
                            }
                        }
                    if (turn == 2 || !__any_sync(kAll, top > 8.f || ymax > 32768.f || odd != 0.f || lost)) break;
                    if (turn == 1) continue;
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!(fabsf(kn[u][h]) <= FLT_MAX && fabsf(vn[u][h]) <= FLT_MAX))
                                kn[u][h] = __uint_as_float(0x7FFFFFFFu), vn[u][h] = 0.f;
                            lv[u][h] = __log2f(fabsf(vn[u][h]));
                        }
                    lost = false;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float a = -INFINITY, b = -INFINITY;  // the most score, and with the V norm (NaN left out)
#pragma unroll
                            for (int u = 0; u < 2; ++u)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    float v = acc[u][nt][2 * h + k] * kn[u][h] * cq[nt][k];
                                    if (!all) v = (on[u][h] >> (2 * nt + k)) & 1u ? v : -INFINITY;
                                    a = fmaxf(a, v);
                                    b = fmaxf(b, v + lv[u][h]);
                                }
#pragma unroll
                            for (int o = 4; o < 32; o *= 2) {
                                a = fmaxf(a, __shfl_xor_sync(kAll, a, o));
                                b = fmaxf(b, __shfl_xor_sync(kAll, b, o));
                            }
                            if (nm[nt][k] == -INFINITY) continue;  // past the item's rows
                            const float m0 = -nm[nt][k], M0 = M[nt][k], m1 = fmaxf(m0, a);
                            const float M1 = b > M0 + 15.f || (M0 == -INFINITY && b > -INFINITY) ? b - 7.f : M0;
                            const float fl = m0 == m1 ? 1.f : pp_exp2(m0 - m1), fo = M0 == M1 ? 1.f : pp_exp2(M0 - M1);
                            nm[nt][k] = -m1;
                            M[nt][k] = M1;
                            l[nt][k] *= fl;
#pragma unroll
                            for (int mt = 0; mt < KK; ++mt) {
                                O[nt][mt][k] *= fo;
                                O[nt][mt][2 + k] *= fo;
                            }
                            cc[nt][k] = m1 == -INFINITY || M1 == -INFINITY ? 0.f : pp_exp2(m1 - M1);
                            lost = lost || (m1 > -INFINITY && (M1 == -INFINITY || cc[nt][k] > FLT_MAX));
                        }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            l[nt][0] += p[u][nt][2 * h];
                            l[nt][1] += p[u][nt][2 * h + 1];
                            pb[u][nt][h] = fw_transpose(pb[u][nt][h]);
                        }
                // the next block but one: by now the other warps have read the last
                if (put - taken < (uint32_t)S) bring();
                if (A.v_bits == 4) fw_output<D, NT, 4>(s_v, vslot, pb, g, t, O);
                else if (A.v_bits == 3) fw_output<D, NT, 3>(s_v, vslot, pb, g, t, O);
                else fw_output<D, NT, 2>(s_v, vslot, pb, g, t, O);
                }
                if (put - taken < (uint32_t)S) bring();  // (this block's sub-chunk was not worked on)
                __syncwarp();
                if (lane == 0) mbar_arrive(free_ + st);
                ++taken;
            }

            // ---- the warps' rows put together
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int o = 4; o < 32; o *= 2) l[nt][k] += __shfl_xor_sync(kAll, l[nt][k], o);
            const bool whole = x.flags & kJobWhole;
            float* part = A.part + ((int64_t)blockIdx.x * 2 + (x.flags & kJobHead ? 1 : 0)) * ((D + 3) * Z::kRows);
            float* merge = reinterpret_cast<float*>(at(Z::kMerge));
            constexpr int MR = Z::kMergeRows, MS = Z::kMergeRow / 4;
            for (int r0 = 0; r0 < x.rows; r0 += MR) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int r = 8 * nt + 2 * t + k - r0;
                        if (r < 0 || r >= MR || r + r0 >= x.rows) continue;
                        float* o = merge + (warp * MR + r) * MS;
#pragma unroll
                        for (int mt = 0; mt < KK; ++mt)
                            *reinterpret_cast<float2*>(o + (D / 8) * g + 2 * mt) = make_float2(O[nt][mt][k], O[nt][mt][2 + k]);
                        if (g == 0) o[D] = -nm[nt][k], o[D + 1] = M[nt][k], o[D + 2] = l[nt][k];
                    }
                __syncthreads();
                const bool write = *abort_f == 0;
                for (int r = warp; r < MR && r0 + r < x.rows; r += W) {
                    constexpr int C = D / 32;
                    float mm = -INFINITY, MM = -INFINITY, ll = 0.f, e[C];
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const float* o = merge + (w * MR + r) * MS + D;
                        mm = fmaxf(mm, o[0]);
                        MM = fmaxf(MM, o[1]);
                    }
#pragma unroll
                    for (int k = 0; k < C; ++k) e[k] = 0.f;
                    const float mr = mm == -INFINITY ? 0.f : mm, Mr = MM == -INFINITY ? 0.f : MM;
#pragma unroll 4
                    for (int w = 0; w < W; ++w) {
                        const float* o = merge + (w * MR + r) * MS;
                        ll = fmaf(o[D + 2], pp_exp2(o[D] - mr), ll);
                        const float f = pp_exp2(o[D + 1] - Mr);
#pragma unroll
                        for (int k = 0; k < C; ++k) e[k] = fmaf(o[lane + 32 * k], f, e[k]);
                    }
                    const int row = r0 + r;
                    if (!whole) {
                        float* st = part + D * Z::kRows;
                        if (lane == 0) st[row] = MM, st[Z::kRows + row] = ll, st[2 * Z::kRows + row] = mm;
#pragma unroll
                        for (int k = 0; k < C; ++k) {
                            const int i = lane + 32 * k;
                            part[((i >> 2) * Z::kRows + row) * 4 + (i & 3)] = e[k];
                        }
                        continue;
                    }
                    // rotated back, s . H (s2 . o)
                    const float inv = ll == 0.f ? 0.f : pp_exp2(MM - mr) * P.out_mul * P.inv_sqrt_d / ll;
#pragma unroll
                    for (int k = 0; k < C; ++k)
                        e[k] = __uint_as_float(__float_as_uint(e[k] * inv) ^ (P.two_sided ? sign_mask(P.sgn2b, lane + 32 * k) : 0u));
#pragma unroll
                    for (int b = 1; b < 32; b *= 2)
#pragma unroll
                        for (int k = 0; k < C; ++k) {
                            const float o = __shfl_xor_sync(kAll, e[k], b);
                            e[k] = lane & b ? o - e[k] : e[k] + o;
                        }
#pragma unroll
                    for (int len = 1; len < C; len *= 2)
#pragma unroll
                        for (int k = 0; k < C; ++k)
                            if (!(k & len)) {
                                const float a = e[k], c = e[k + len];
                                e[k] = a + c;
                                e[k + len] = a - c;
                            }
                    const int i = x.rest + row, tok = i / G;
                    const int64_t o = (((int64_t)x.q0 + x.tok0 + tok) * A.Hq + (int64_t)x.h * G + (i - tok * G)) * D;
#pragma unroll
                    for (int k = 0; k < C; ++k) {
                        const int d = lane + 32 * k;
                        const float v = __uint_as_float(__float_as_uint(e[k]) ^ sign_mask(P.sgnb, d));
                        if (!write) continue;
                        if (A.out_bf16) static_cast<__nv_bfloat16*>(A.out)[o + d] = __float2bfloat16_rn(v);
                        else static_cast<float*>(A.out)[o + d] = v;
                    }
                }
                __syncthreads();
            }
        }
        if (!bad) {  // the record at the end
            if (__all_sync(kAll, pp_wait(full + taken % S, (taken / S) & 1, abort_f, status))) {
                if (lane == 0) mbar_arrive(free_ + taken % S);
                ++taken;
            } else {
                bad = true;
            }
        }
        __syncthreads();  // the jobs have been read
    }
    if (tid == 0) pp_report<Z, MODE>(A, *start, *share, cur, seq, true, has);
    // after a wait that gave up: the copies in flight land before the CTA leaves (bounded)
    if (bad)
        for (uint32_t i = put > (uint32_t)S ? put - S : 0; i < put; ++i) mbar_wait(full + i % S, (i / S) & 1);
    griddep_launch();
    __syncthreads();
    if (tid == 0 && *abort_f) *reinterpret_cast<int4*>(A.meta + (int64_t)blockIdx.x * kPpMeta) = make_int4(kShareFailed, -1, 0, 0);
}

template <int D, int NT, int MODE>
static cudaError_t launch_few(const PagedPrefillCall& c, cudaStream_t s) {
    using Z = FwGeo<D, NT>;
    static_assert(Z::kRows <= PagedPrefillGeo<D>::kRows, "the workspace holds the parts");
    const int shares = num_sms(), G = c.Hq / c.Hkv;
    PpArgs A = pp_args(c, shares, (size_t)(D + 3) * Z::kRows);
    // Few items of few blocks (a short window, a small table): one CTA takes all of an
    // item, and no join follows.  By the most items and blocks that there can be, as the
    // lengths are on the device.  4 sequences, 8 KV heads, windows of 256 (5 blocks), 512
    // (7) and 768 (9), us in parts and whole: d = 128, 4 rows 13.8 12.2, 13.7 12.8 and 13.9
    // 14.3, 16 rows 16.4 15.2, 16.7 17.0 and 17.0 19.3; d = 64, 4 rows 13.1 11.1, 13.0 11.5
    // and 13.2 12.5; d = 256, 4 rows 16.0 15.1, 16.5 17.4 and 16.9 19.8.  The host saves a
    // launch.  (A cu_q that steps back can give more items than CTAs: pp_start gives each a
    // few.)
    const int64_t items = (c.n_q * G / Z::kRows + c.B) * c.Hkv;
    int64_t blocks = ((int64_t)c.max_pages << c.page_shift) / Z::kN + 1;
    if (MODE == kPpSinks && c.window > 0) {
        const int64_t reach = ((int64_t)c.window + Z::kRows / G) / Z::kN + 2 + (c.sinks + Z::kN - 1) / Z::kN;
        if (reach < blocks) blocks = reach;
    }
    A.whole = items <= shares && blocks <= (NT == 1 && D <= 128 ? 7 : 5);
    FwLevels L;
    for (int i = 0; i < 16; ++i) L.k[i] = c.k_cen[i], L.v[i] = c.v_cen[i];
    static int attr_done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !attr_done[dev]) {
        e = cudaFuncSetAttribute(k_attn_few<D, NT, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Z::kEnd);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_done[dev] = 1;
    }
    e = launch_pdl(k_attn_few<D, NT, MODE>, dim3(A.whole ? (unsigned)items : shares), dim3(Z::kThreads), Z::kEnd, s, A, c.consts, L, status_word());
    if (e != cudaSuccess) return e;
    if (A.whole) return e;  // no parts to join
    const int64_t rows = c.n_q * G;
    const unsigned groups = (unsigned)((rows < Z::kRows ? rows : Z::kRows) + 31) / 32;
    return launch_pdl(k_prefill_paged_join<D, D < 256 ? 4 : 2, Z::kRows>, dim3(shares, groups), dim3(256), 0, s, A,
                      c.consts);
}

}  // namespace dev

template <int D, int MODE>
cudaError_t launch_attn_few(const PagedPrefillCall& c, cudaStream_t s) {
    // One tile of 8 rows, or two for more than 8 rows (of a sequence and KV head, as an
    // average), which read the positions once: 32 sequences of 6000 positions, 8 rows 79
    // us, 12 rows 109 us.  At d = 256 two tiles leave no registers (the output alone takes
    // 128).
    const int64_t rows = c.n_q * (c.Hq / c.Hkv);
    if (D == 256 || rows <= (int64_t)8 * c.B) return dev::launch_few<D, 1, MODE>(c, s);
    return dev::launch_few<D, D == 256 ? 1 : 2, MODE>(c, s);
}

template cudaError_t launch_attn_few<TQ_UNIT_D, TQ_UNIT_MODE>(const PagedPrefillCall&, cudaStream_t);

}  // namespace tq
