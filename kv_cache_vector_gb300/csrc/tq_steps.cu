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
// Bound by latency: 64 rows of one token take three dependent reads.
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
    __shared__ int before[kSlThreads + 1];  // tokens of the rows of the threads before this one
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
        int b = lo * each, i = (int)t - before[lo], n = A.counts[b];
        while (i >= n) {  // (ends: the threads' rows hold the token)
            i -= n;
            n = A.counts[++b];
        }
        const int base = A.lens[b] - n, at = base + i;
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
// sequence.
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
// it writes.  Lists of the same row are checked by every warp alike.
constexpr int kKpWarps = 8;
constexpr int kKpLayers = 64;  // most layers per launch

template <int MAX>
struct KeepLayers {
    void* at[MAX][4];  // packed K, K norms, packed V, V norms
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
    int n_seqs, max_pages, max_keep, shift, Hkv, k_bytes, v_bytes;  // bytes of a packed row
};

// Rows of `units` T each: lanes of the batch's rows [0, n), whose places are
// src and dst of lane r.  All loads first.
template <typename T, int U>
__device__ __forceinline__ void keep_rows(void* base, int units, int n, int64_t src, int64_t dst, int lane) {
    T v[U];
    T* p = static_cast<T*>(base);
    const int all = n * units;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int w = 32 * k + lane, r = w < all ? w / units : 0;
        const int64_t s = __shfl_sync(0xFFFFFFFFu, src, r);
        if (w < all) v[k] = p[s * units + (w - r * units)];
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int w = 32 * k + lane, r = w < all ? w / units : 0;
        const int64_t t = __shfl_sync(0xFFFFFFFFu, dst, r);
        if (w < all) p[t * units + (w - r * units)] = v[k];
    }
}
// A batch of up to 8 packed rows of at most 128 bytes.
__device__ __forceinline__ void keep_packed(void* base, int bytes, int n, int64_t src, int64_t dst, int lane) {
    if (bytes % 16 == 0) keep_rows<uint4, 2>(base, bytes / 16, n, src, dst, lane);
    else if (bytes % 8 == 0) keep_rows<uint2, 1>(base, bytes / 8, n, src, dst, lane);
    else keep_rows<uint32_t, 1>(base, bytes / 4, n, src, dst, lane);
}
constexpr int kKpBatch = 8;

template <int MAX>
__global__ void __launch_bounds__(32 * kKpWarps) k_pages_keep(const __grid_constant__ KeepLayers<MAX> P, int L,
                                                              const KeepArgs A, int* status) {
    const int lane = threadIdx.x & 31;
    griddep_wait();
    griddep_launch();
    const int LH = L * A.Hkv;
    const int64_t items = (int64_t)A.n_seqs * LH;
    for (int64_t it = (int64_t)blockIdx.x * kKpWarps + (threadIdx.x >> 5); it < items;
         it += (int64_t)gridDim.x * kKpWarps) {
        const int b = (int)(it / LH), lh = (int)(it - (int64_t)b * LH), l = lh / A.Hkv, h = lh - l * A.Hkv;
        const int n = A.counts[b], len = A.lens[b], k = A.n_keep[b];
        const int32_t* keep = A.keep + (int64_t)b * A.max_keep;
        const int32_t* row = A.bt + (int64_t)b * A.max_pages;
        bool ok = n >= 0 && len >= n && len <= ((int64_t)A.max_pages << A.shift) && k >= 0 && k <= n && k <= A.max_keep;
        const int base = len - n;
        // lane r's token of the list from i on: where it is and where it goes, as rows of head 0
        auto find = [&](int i, int64_t& src, int64_t& dst, bool& moves) {
            const int x = i < k ? keep[i] : n + i;
            const int below = i > 0 && i < k ? keep[i - 1] : -1;
            moves = false;
            if (i >= k) return true;
            if (x < i || x >= n || x <= below) return false;
            moves = x != i;
            if (!moves) return true;
            const int a = base + x, z = base + i;
            const int pa = row[a >> A.shift], pz = row[z >> A.shift];
            if (pa < 0 || pa >= A.n_pages || pz < 0 || pz >= A.n_pages || A.refs[pa] > 1 || A.refs[pz] > 1) return false;
            const int m = (1 << A.shift) - 1;
            src = (((int64_t)pa * A.Hkv + h) << A.shift) + (a & m);
            dst = (((int64_t)pz * A.Hkv + h) << A.shift) + (z & m);
            return true;
        };
        int64_t src = 0, dst = 0;
        bool moves = false, any = false;
        int first = k;  // the first token that moves: all behind it do
        if (ok)
            for (int i0 = 0; i0 < k; i0 += 32) {
                const bool fine = find(i0 + lane, src, dst, moves);
                ok = __all_sync(0xFFFFFFFFu, fine) && ok;
                const unsigned who = __ballot_sync(0xFFFFFFFFu, moves);
                if (who && !any) first = i0 + __ffs(who) - 1;
                any = any || who;
            }
        if (lh == 0 && A.new_lens && lane == 0) {
            A.new_lens[b] = ok ? base + k : len;
            if (!ok) report_timeout(status, kStepStatusKeep);
        }
        if (!ok || !any) continue;
        for (int i = first; i < k; i += kKpBatch) {
            const int m = min(kKpBatch, k - i);
            find(lane < m ? i + lane : k, src, dst, moves);
            keep_packed(P.at[l][0], A.k_bytes, m, src, dst, lane);
            keep_packed(P.at[l][2], A.v_bytes, m, src, dst, lane);
            keep_rows<uint32_t, 1>(P.at[l][1], 1, m, src, dst, lane);
            keep_rows<uint32_t, 1>(P.at[l][3], 1, m, src, dst, lane);
        }
    }
}

template <int MAX>
static cudaError_t launch_keep(const StepKeepCall& c, int l0, int L, const KeepArgs& A, cudaStream_t s) {
    KeepLayers<MAX> P;
    for (int l = 0; l < L; ++l) {
        const tq_paged_cache& x = c.layers[l0 + l];
        P.at[l][0] = x.k_packed;
        P.at[l][1] = x.k_norm;
        P.at[l][2] = x.v_packed;
        P.at[l][3] = x.v_norm;
    }
    const int64_t items = (int64_t)A.n_seqs * L * A.Hkv, want = (items + kKpWarps - 1) / kKpWarps;
    const int64_t most = (int64_t)num_sms() * 64;
    return launch_pdl(k_pages_keep<MAX>, dim3((unsigned)(want < most ? want : most)), dim3(32 * kKpWarps), 0, s, P, L, A,
                      status_word());
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
        const cudaError_t e = L <= 4 ? launch_keep<4>(c, l0, L, A, s) : launch_keep<kKpLayers>(c, l0, L, A, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace tq
