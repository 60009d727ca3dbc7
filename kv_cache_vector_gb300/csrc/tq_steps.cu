// tq_steps.cu -- a serving step's tokens: where the new ones go (tq_pages_slots),
// their append (tq_append_slots), and the drafted ones that are kept
// (tq_pages_keep).
#include <climits>

#include "tq_async.cuh"
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace dev {

constexpr int kStepStatusCounts = 63;  // counts or lengths outside their ranges, or more tokens than the outputs hold
constexpr int kStepStatusPage = 64;    // a page id outside [0, n_pages)
constexpr int kStepStatusParent = 65;  // a parent outside [-1, its child)
constexpr int kStepStatusKeep = 66;    // a row's kept tokens outside their ranges, or in pages that it shares

// ------------------------------------------------------------------ slot map
//
// cu_q is the running sum of the rows' counts; token t belongs to the last row
// whose sum is not above t.  Every CTA sums all counts for itself (a chain of
// two reads, no second launch and no workspace), then looks its tokens up by a
// binary search over the threads' sums in shared memory.  A tree's node walks up
// its parents: they come in descending order, so each word of its mask is
// written once, complete.
//
// Bound by latency: 64 rows of one token take 2.4 to 2.9 us in a graph, the trees of 256
// rows (9500 nodes) 7.2 us.  A walk takes a dependent read a level, about 170 ns: 1024
// nodes in one chain 174 us, with parents at random behind them 12 us.  The sums of all
// rows in each CTA: 4096 rows 6 us, 2^16 154 us, 2^18 872 us.
constexpr int kSlThreads = 512;

struct SlotsArgs {
    const int32_t* bt;
    const int32_t* lens;
    const int32_t* counts;
    const int32_t* parents;  // or nullptr
    int32_t* cu_q;
    int32_t* positions;
    int64_t* slots;
    uint32_t* mask;  // with parents
    int64_t n_tokens, n_pages;
    int n_seqs, max_pages, shift, words;
};

__global__ void __launch_bounds__(kSlThreads) k_pages_slots(const SlotsArgs A, int* status) {
    __shared__ int before[kSlThreads];  // tokens of the rows of the threads before this one
    __shared__ int2 last[kSlThreads];   // count and length of the thread's last row
    __shared__ long long sums[kSlThreads / 32];
    __shared__ int flags[kSlThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_wait();
    griddep_launch();
    const int each = (A.n_seqs + kSlThreads - 1) / kSlThreads;
    const int b0 = min(A.n_seqs, tid * each), b1 = min(A.n_seqs, b0 + each);
    const int64_t cap = (int64_t)A.max_pages << A.shift;
    long long mine = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        const int n = A.counts[b], len = A.lens[b];
        bad = bad || n < 0 || len < n || len > cap || (A.parents && n > 32 * A.words);
        mine += max(n, 0);
        last[tid] = make_int2(n, len);
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) sums[warp] = incl;
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (lane == 0) flags[warp] = bad;
    __syncthreads();
    long long total = 0, first = incl - mine;
    bad = false;
#pragma unroll
    for (int w = 0; w < kSlThreads / 32; ++w) {
        if (w < warp) first += sums[w];
        total += sums[w];
        bad = bad || flags[w];
    }
    if (bad || total > A.n_tokens) {  // no token at all
        if (tid == 0 && blockIdx.x == 0) report_timeout(status, kStepStatusCounts);
        total = first = 0;
        bad = true;
    }
    before[tid] = (int)first;
    if (blockIdx.x == 0) {
        int at = (int)first;
        for (int b = b0; b < b1; ++b) {
            A.cu_q[b] = at;
            if (!bad) at += A.counts[b];
        }
        if (tid == 0) A.cu_q[A.n_seqs] = (int)total;
    }
    __syncthreads();
    for (int64_t t = (int64_t)blockIdx.x * kSlThreads + tid; t < A.n_tokens; t += (int64_t)gridDim.x * kSlThreads) {
        uint32_t* mask = A.parents ? A.mask + t * A.words : nullptr;
        if (t >= total) {
            A.slots[t] = -1;
            A.positions[t] = 0;
            if (mask)
                for (int w = 0; w < A.words; ++w) mask[w] = 0u;
            continue;
        }
        int lo = 0, hi = kSlThreads;  // before[lo] <= t
        while (hi - lo > 1) {
            const int m = (lo + hi) / 2;
            if (before[m] <= t) lo = m;
            else hi = m;
        }
        int b = lo * each, i = (int)t - before[lo], n = last[lo].x, base = last[lo].y - n;
        if (each > 1) {
            n = A.counts[b];
            while (i >= n) {  // (ends: the threads' rows hold the token)
                i -= n;
                n = A.counts[++b];
            }
            base = A.lens[b] - n;
        }
        const int at = base + i;
        const int page = A.bt[(int64_t)b * A.max_pages + (at >> A.shift)];
        const bool ok = page >= 0 && page < A.n_pages;
        if (!ok) report_timeout(status, kStepStatusPage);
        A.slots[t] = ok ? ((int64_t)page << A.shift) + (at & ((1 << A.shift) - 1)) : -1;
        int depth = i;
        if (mask) {
            const int32_t* up = A.parents + (t - i);
            int w = A.words - 1, x = i;
            uint32_t bits = 0;
            for (depth = -1; x >= 0; ++depth) {
                for (; w > x >> 5; --w) {
                    mask[w] = bits;
                    bits = 0;
                }
                bits |= 1u << (x & 31);
                const int p = up[x];
                if (p >= x || p < -1) {  // a root
                    report_timeout(status, kStepStatusParent);
                    break;
                }
                x = p;
            }
            if (x >= 0) ++depth;
            for (; w >= 0; --w) {
                mask[w] = bits;
                bits = 0;
            }
        }
        A.positions[t] = base + depth;
    }
}

// -------------------------------------------------------------------- append
//
// A step's tokens at the slots that tq_pages_slots gives them: row
// (t, h) goes to offset slots[t] % page_size of page slots[t] / page_size; a
// negative slot has no token.  One warp per row, as the append of one token per
// sequence: made for a step's tokens.  Bound by a warp's chain of encoding steps and
// their shuffles, K4/V3, 8 KV heads, d = 128, bf16 or fp32: 64 tokens 3.1 us, 1024
// tokens 13.9 us, 4096 tokens 46.6 us (bf16: 445 GB/s, 3.1 us of bytes).
constexpr int kAsWarps = 4;
constexpr int kAsStatusRange = 42;  // a slot past the pool's end (as the other appends)

template <int D, typename T>
__global__ void __launch_bounds__(32 * kAsWarps) k_append_slots(const SlotRows A, tq_cache_view cache, int k_bits,
                                                                 int v_bits, const __grid_constant__ RowParams PK,
                                                                 const __grid_constant__ RowParams PV, int* status) {
    __shared__ uint32_t sg[D], sg2[D];
    __shared__ uint8_t idxbuf[kAsWarps][D];
    const bool is_v = blockIdx.y == 1;
    const RowParams& P = is_v ? PV : PK;
    for (int i = threadIdx.x; i < D; i += blockDim.x) {
        sg[i] = sign_mask(P.sgnb, i);
        sg2[i] = sign_mask(P.sgn2b, i);
    }
    __syncthreads();
    griddep_wait();    // the new rows and slots, and readers of the cache, of the previous kernel
    griddep_launch();  // the next kernel may set itself up; it waits for this grid
    const int bits = is_v ? v_bits : k_bits;
    const T* src = static_cast<const T*>(is_v ? A.v_new : A.k_new);
    const int64_t stride = is_v ? A.v_stride : A.k_stride;
    uint8_t* pk = is_v ? cache.v_packed : cache.k_packed;
    float* nrm = is_v ? cache.v_norm : cache.k_norm;
    const int rb = D * bits / 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* ib = idxbuf[warp];
    const int64_t rows = A.n_tokens * A.Hkv;
    for (int64_t r = (int64_t)blockIdx.x * kAsWarps + warp; r < rows; r += (int64_t)gridDim.x * kAsWarps) {
        const int64_t t = r / A.Hkv;
        const int h = (int)(r - t * A.Hkv);
        const int64_t slot = A.slots[t];
        if (slot < 0) continue;
        const int64_t page = slot >> A.page_shift;
        if (page >= A.n_pages) {
            if (lane == 0) report_timeout(status, kAsStatusRange);
            continue;
        }
        const float n = warp_encode_indices<D, T>(src + t * stride + (int64_t)h * D, lane, sg, P.two_sided ? sg2 : nullptr,
                                                  P, (1 << bits) - 1, ib);
        const int64_t drow = ((page * A.Hkv + h) << A.page_shift) + (slot & ((int64_t(1) << A.page_shift) - 1));
        warp_pack_row<D>(ib, lane, bits, pk + drow * rb);
        if (lane == 0) nrm[drow] = n;
        __syncwarp();
    }
}

// ---------------------------------------------------------------- kept tokens
//
// Of row b's counts[b] last tokens those in keep[b] stay: token keep[b][i] moves
// to the place of token i.  The list ascends, so keep[b][i] >= i, and a place
// that a token moves to is the source of no later one: a warp moves a (row,
// layer, KV head)'s tokens a few at a time, each time reading all of them before
// it writes.  A CTA works out one row's places once, for kKpEach (layer, KV
// head) pairs a warp; every CTA of a row checks its list alike.
//
// Bound by latency (lists, pages, then the rows): 64 rows of which 122 tokens
// move in 32 layers, 7.5 MB in all, 12.3 us in a graph (15.8 with a list for
// every warp); 4 rows in 2 layers 4.0 us.
constexpr int kKpWarps = 8;
constexpr int kKpThreads = 32 * kKpWarps;
// (layer, KV head) pairs of a warp, us with 1 / 2 / 4 / 8: 4 rows in 2 layers 3.0 3.9 4.0 4.0,
// 64 rows in 4 layers 3.5 4.4 6.2 6.2 and in 32 layers 16.9 12.7 12.4 11.1, 128 rows in 64
// layers 56 40 32 31: the places are worked out once for them, and they follow one another
constexpr int kKpEach = 4;
constexpr int kKpList = 128;   // tokens whose places are known at a time
constexpr int kKpBatch = 8;    // tokens that a warp moves at a time
constexpr int kKpLayers = 64;  // most layers per launch

struct KeepLayers {
    void* at[kKpLayers][4];  // packed K, K norms, packed V, V norms
};

struct KeepArgs {
    const int32_t* bt;
    const int32_t* lens;
    const int32_t* refs;
    const int32_t* counts;
    const int32_t* keep;
    const int32_t* n_keep;
    int32_t* new_lens;  // nullptr: another launch writes them
    int64_t n_pages;
    int n_seqs, max_pages, max_keep, shift, Hkv, k_bytes, v_bytes, slices;  // bytes of a packed row
};

// n rows of `units` T each, from the places src to the places dst (rows of KV
// head 0; `up` further on): the loads, and the stores.
template <typename T, int U>
struct KeepRows {
    T v[U];
    __device__ __forceinline__ void load(const void* base, int units, int n, const long long* src, int64_t up, int lane) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int w = 32 * k + lane, r = w / units;
            if (w < n * units) v[k] = static_cast<const T*>(base)[(src[r] + up) * units + (w - r * units)];
        }
    }
    __device__ __forceinline__ void store(void* base, int units, int n, const long long* dst, int64_t up, int lane) const {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int w = 32 * k + lane, r = w / units;
            if (w < n * units) static_cast<T*>(base)[(dst[r] + up) * units + (w - r * units)] = v[k];
        }
    }
};

// A batch of tokens, packed rows in units of TK and TV (at most 128 bytes a row).
template <typename TK, typename TV>
__device__ __forceinline__ void keep_batch(void* const (&at)[4], int k_bytes, int v_bytes, int n, const long long* src,
                                           const long long* dst, int64_t up, int lane) {
    KeepRows<TK, sizeof(TK) == 16 ? 2 : 1> k;
    KeepRows<TV, sizeof(TV) == 16 ? 2 : 1> v;
    KeepRows<uint32_t, 1> kn, vn;
    k.load(at[0], k_bytes / (int)sizeof(TK), n, src, up, lane);
    v.load(at[2], v_bytes / (int)sizeof(TV), n, src, up, lane);
    kn.load(at[1], 1, n, src, up, lane);
    vn.load(at[3], 1, n, src, up, lane);
    __syncwarp();
    k.store(at[0], k_bytes / (int)sizeof(TK), n, dst, up, lane);
    v.store(at[2], v_bytes / (int)sizeof(TV), n, dst, up, lane);
    kn.store(at[1], 1, n, dst, up, lane);
    vn.store(at[3], 1, n, dst, up, lane);
}
template <typename TK>
__device__ __forceinline__ void keep_batch(void* const (&at)[4], int k_bytes, int v_bytes, int n, const long long* src,
                                           const long long* dst, int64_t up, int lane) {
    if (v_bytes % 16 == 0) keep_batch<TK, uint4>(at, k_bytes, v_bytes, n, src, dst, up, lane);
    else if (v_bytes % 8 == 0) keep_batch<TK, uint2>(at, k_bytes, v_bytes, n, src, dst, up, lane);
    else keep_batch<TK, uint32_t>(at, k_bytes, v_bytes, n, src, dst, up, lane);
}

__global__ void __launch_bounds__(kKpThreads) k_pages_keep(const __grid_constant__ KeepLayers P, int L, const KeepArgs A,
                                                           int* status) {
    __shared__ long long s_src[kKpList], s_dst[kKpList];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / A.slices, slice = blockIdx.x - b * A.slices;
    griddep_wait();
    griddep_launch();
    const int n = A.counts[b], len = A.lens[b], k = A.n_keep[b];
    const int32_t* keep = A.keep + (int64_t)b * A.max_keep;
    const int32_t* row = A.bt + (int64_t)b * A.max_pages;
    bool ok = n >= 0 && len >= n && len <= ((int64_t)A.max_pages << A.shift) && k >= 0 && k <= n && k <= A.max_keep;
    const int base = len - n;
    // token i of the list: where it is and where it goes, as rows of KV head 0
    auto find = [&](int i, bool& moves) {
        moves = false;
        if (i >= k) return true;
        const int x = keep[i];
        if (x < i || x >= n || (i > 0 && x <= keep[i - 1])) return false;
        if (x == i) return true;
        moves = true;
        const int a = base + x, z = base + i, m = (1 << A.shift) - 1;
        const int pa = row[a >> A.shift], pz = row[z >> A.shift];
        if (pa < 0 || pa >= A.n_pages || pz < 0 || pz >= A.n_pages || A.refs[pa] > 1 || A.refs[pz] > 1) return false;
        s_src[i % kKpList] = (((int64_t)pa * A.Hkv) << A.shift) + (a & m);
        s_dst[i % kKpList] = (((int64_t)pz * A.Hkv) << A.shift) + (z & m);
        return true;
    };
    int moving = 0;
    if (ok) {
        for (int i0 = 0; i0 < k; i0 += kKpList) {
            bool moves = false, fine = true;
            if (tid < kKpList) fine = find(i0 + tid, moves);
            moving += __syncthreads_count(moves);
            ok = __syncthreads_and(fine) && ok;
        }
    }
    if (slice == 0 && tid == 0 && A.new_lens) {
        A.new_lens[b] = ok ? base + k : len;
        if (!ok) report_timeout(status, kStepStatusKeep);
    }
    if (!ok || moving == 0) return;
    const int first = k - moving;  // all behind the first that moves do
    const int LH = L * A.Hkv;
    for (int i0 = k <= kKpList ? first : first / kKpList * kKpList; i0 < k; i0 += kKpList) {
        int end = k;
        if (k > kKpList) {  // the list in pieces: their places once more
            __syncthreads();
            bool moves;
            if (tid < kKpList) find(i0 + tid, moves);
            end = min(k, i0 + kKpList);
            __syncthreads();
        }
        for (int e = 0; e < kKpEach; ++e) {
            const int lh = (slice * kKpEach + e) * kKpWarps + warp;
            if (lh >= LH) break;
            const int l = lh / A.Hkv, h = lh - l * A.Hkv;
            const int64_t up = (int64_t)h << A.shift;
            for (int i = max(i0, first); i < end; i += kKpBatch) {
                const int m = min(kKpBatch, end - i);
                const long long *src = s_src + i % kKpList, *dst = s_dst + i % kKpList;
                if (A.k_bytes % 16 == 0) keep_batch<uint4>(P.at[l], A.k_bytes, A.v_bytes, m, src, dst, up, lane);
                else if (A.k_bytes % 8 == 0) keep_batch<uint2>(P.at[l], A.k_bytes, A.v_bytes, m, src, dst, up, lane);
                else keep_batch<uint32_t>(P.at[l], A.k_bytes, A.v_bytes, m, src, dst, up, lane);
            }
        }
        if (k <= kKpList) break;
    }
}

static cudaError_t launch_keep(const StepKeepCall& c, int l0, int L, KeepArgs A, cudaStream_t s) {
    KeepLayers P;
    for (int l = 0; l < L; ++l) {
        const tq_paged_cache& x = c.layers[l0 + l];
        P.at[l][0] = x.k_packed;
        P.at[l][1] = x.k_norm;
        P.at[l][2] = x.v_packed;
        P.at[l][3] = x.v_norm;
    }
    A.slices = (L * A.Hkv + kKpWarps * kKpEach - 1) / (kKpWarps * kKpEach);
    return launch_pdl(k_pages_keep, dim3((unsigned)A.n_seqs * A.slices), dim3(kKpThreads), 0, s, P, L, A, status_word());
}

}  // namespace dev

template <int D>
cudaError_t launch_append_slots_d(int k_bits, int v_bits, tq_dtype dt, const SlotRows& r, const tq_cache_view& pages,
                                  const RowParams& PK, const RowParams& PV, cudaStream_t s) {
    auto launch = [&](auto tag) {
        auto fn = dev::k_append_slots<D, decltype(tag)>;
        int64_t g = (r.n_tokens * r.Hkv + dev::kAsWarps - 1) / dev::kAsWarps;
        const int64_t cap = (int64_t)num_sms() * blocks_per_sm((const void*)fn, 32 * dev::kAsWarps, 0);
        if (g > cap) g = cap;
        return dev::launch_pdl(fn, dim3((unsigned)g, 2), dim3(32 * dev::kAsWarps), 0, s, r, pages, k_bits, v_bits,
                               PK, PV, status_word());
    };
    return dt == TQ_BF16 ? launch(__nv_bfloat16{}) : launch(float{});
}
template cudaError_t launch_append_slots_d<32>(int, int, tq_dtype, const SlotRows&, const tq_cache_view&, const RowParams&,
                                               const RowParams&, cudaStream_t);
template cudaError_t launch_append_slots_d<64>(int, int, tq_dtype, const SlotRows&, const tq_cache_view&, const RowParams&,
                                               const RowParams&, cudaStream_t);
template cudaError_t launch_append_slots_d<128>(int, int, tq_dtype, const SlotRows&, const tq_cache_view&,
                                                const RowParams&, const RowParams&, cudaStream_t);
template cudaError_t launch_append_slots_d<256>(int, int, tq_dtype, const SlotRows&, const tq_cache_view&,
                                                const RowParams&, const RowParams&, cudaStream_t);

cudaError_t launch_slots(const StepSlotsCall& c, cudaStream_t s) {
    using namespace dev;
    SlotsArgs A = {};
    A.bt = c.table.block_table;
    A.lens = c.table.lens;
    A.counts = c.counts;
    A.parents = c.parents;
    A.cu_q = c.cu_q;
    A.positions = c.positions;
    A.slots = c.slots;
    A.mask = c.mask;
    A.n_tokens = c.n_tokens;
    A.n_pages = c.n_pages;
    A.n_seqs = c.n_seqs;
    A.max_pages = c.max_pages;
    A.shift = c.page_shift;
    A.words = c.words;
    const int64_t want = (c.n_tokens + kSlThreads - 1) / kSlThreads, most = 2 * num_sms();
    const int64_t grid = want < 1 ? 1 : want < most ? want : most;
    return launch_pdl(k_pages_slots, dim3((unsigned)grid), dim3(kSlThreads), 0, s, A, status_word());
}

cudaError_t launch_keep(const StepKeepCall& c, cudaStream_t s) {
    using namespace dev;
    KeepArgs A = {};
    A.bt = c.table.block_table;
    A.lens = c.table.lens;
    A.refs = c.table.refs;
    A.counts = c.counts;
    A.keep = c.keep;
    A.n_keep = c.n_keep;
    A.n_pages = c.layers[0].n_pages;
    A.n_seqs = c.n_seqs;
    A.max_pages = c.max_pages;
    A.max_keep = c.max_keep;
    A.shift = c.page_shift;
    A.Hkv = c.Hkv;
    A.k_bytes = c.d * c.k_bits / 8;
    A.v_bytes = c.d * c.v_bits / 8;
    for (int l0 = 0; l0 < c.n_layers; l0 += kKpLayers) {
        const int L = c.n_layers - l0 < kKpLayers ? c.n_layers - l0 : kKpLayers;
        A.new_lens = l0 == 0 ? c.new_lens : nullptr;
        const cudaError_t e = launch_keep(c, l0, L, A, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace tq
