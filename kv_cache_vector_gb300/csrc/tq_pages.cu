// tq_pages.cu -- the upkeep of a paged cache's pages: copy, fork, resize
// (grow, cut, free) and compaction.
//
// A page table holds, per sequence row, its page ids and its length, and per
// page the number of rows that hold it (0: free).  Every operator is two
// launches (a copy of few pairs one, k_pages_copy_few):
//   k_pages_plan   one thread-block cluster (1 or 8 CTAs of 1024 threads)
//     works out the new table and the list of (source, destination) page
//     pairs to copy.  All of its decisions follow row order and take the
//     lowest free page ids first, so the result does not depend on timing;
//     the only atomics are integer sums, minima and maxima.  Nothing is written to
//     the output table before the call is known to succeed (valid input,
//     enough free pages): a call that fails returns the table as it was.
//     The steps exchange data through the workspace with a cluster barrier
//     between them (hardware barriers: nothing spins).
//   k_pages_copy   copies the pairs' pages, in every layer, 32 KB per CTA and
//     step.  Bound by memory: a copied page is read once and written once.
//     473 pages of 2 MB (32 layers): 293 to 297 us, 6.35 TB/s; with 4, 8 and 16 KB
//     steps 413, 322 and 304 us (too few bytes in flight).
// Both are launched with programmatic stream serialization, so that their CTAs
// are there when the kernel before ends.  Small calls are bound by the launches
// and the plan's chain of dependent reads (steps of 1 to 2 us each): 4 us for a
// copy of 5 pages, 9 to 16 us for a fork, resize or compaction with few pages
// to copy (8 to 512 rows, 100 to 6500 pages), in a graph.
#include <climits>

#include <cooperative_groups.h>

#include "tq_async.cuh"
#include "tq_internal.h"

namespace cg = cooperative_groups;

namespace tq {
namespace dev {

constexpr int kPgThreads = 1024;
constexpr int kPgWarps = kPgThreads / 32;
constexpr int kPgClusterMax = 8;
constexpr int kPgStatusInput = 61;     // a page id, length, row number outside its range
constexpr int kPgStatusConflict = 62;  // copy: a destination given twice, or also a source
// words of the workspace head
enum { kHeadBad = 0, kHeadTakes = 1, kHeadPairs = 2, kHeadWords = 16 };

struct PagesWs {
    int32_t* head;   // [kHeadWords]
    int32_t* delta;  // [n_pages] change of the holders (copy: first pair per destination; compact: holders of movers)
    int32_t* cow;    // [n_pages] fork, resize: holders lost to private copies (copy: page is a source)
    int32_t* fresh;  // [n_pages] free pages, ascending (compact: holes)
    int32_t* src;    // [n_pages] pairs: source page, or -1 for none (resize, first: rows that write into the page)
    int32_t* dst;    // [n_pages] pairs: destination page (resize, first: the last such row)
    int32_t* first;  // [n_seqs] fork: first child of a row; resize: the tail page the row writes into, or -1
    int32_t* start;  // [n_seqs] the row's place in the list of fresh pages
    int32_t* pair;   // [n_seqs] the row's place in the list of pairs; bit 31: it has one
};

__host__ __device__ inline PagesWs pages_ws(void* w, int64_t n_pages, int n_seqs) {
    int32_t* p = static_cast<int32_t*>(w);
    PagesWs r;
    r.head = p;
    p += kHeadWords;
    r.delta = p;
    p += n_pages;
    r.cow = p;
    p += n_pages;
    r.fresh = p;
    p += n_pages;
    r.src = p;
    p += n_pages;
    r.dst = p;
    p += n_pages;
    r.first = p;
    p += n_seqs;
    r.start = p;
    p += n_seqs;
    r.pair = p;
    return r;
}

// Inclusive scan of v over the block; *total receives the block's sum.
// `s` holds kPgWarps values.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* s, T* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();  // s is free
    if (lane == 31) s[warp] = v;
    __syncthreads();
    if (warp == 0) {
        T w = s[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T u = __shfl_up_sync(0xFFFFFFFFu, w, o);
            if (lane >= o) w += u;
        }
        s[lane] = w;
    }
    __syncthreads();
    if (warp > 0) v += s[warp - 1];
    *total = s[kPgWarps - 1];
    return v;
}

enum PagesOp { kOpCopy, kOpFork, kOpResize, kOpCompact };

struct PagesPlan {
    const int32_t* table;  // [n_seqs][max_pages]
    const int32_t* lens;
    const int32_t* refs;
    int32_t* table_out;
    int32_t* lens_out;
    int32_t* refs_out;
    const int32_t* arg;   // parents (fork), new lengths (resize), source ids (copy)
    const int32_t* arg2;  // destination ids (copy)
    int32_t* moved;       // compact: [n_pages]
    int32_t* info;        // [2]
    void* ws;
    int64_t n;  // pairs (copy)
    int n_seqs, max_pages, n_pages, n_src, shift;
    int same;  // copy: source and destination are one pool
};

// Counts of this CTA's segment, summed over the lower CTAs of the cluster and
// over all of them.  Contains a cluster barrier, which also makes the global
// writes before it visible to the cluster.
__device__ __forceinline__ void cluster_sums(cg::cluster_group& cl, int* slot, int mine, int* before, int* all) {
    if (threadIdx.x == 0) *slot = mine;
    cl.sync();
    int b = 0, a = 0;
    for (unsigned r = 0; r < cl.num_blocks(); ++r) {
        const int v = *cl.map_shared_rank(slot, r);
        if (r < cl.block_rank()) b += v;
        a += v;
    }
    *before = b;
    *all = a;
}

template <int OP>
__global__ void __launch_bounds__(kPgThreads, 1) k_pages_plan(const PagesPlan A, int* status) {
    cg::cluster_group cl = cg::this_cluster();
    __shared__ int s_scan[kPgWarps];
    __shared__ long long s_scan64[kPgWarps];
    __shared__ int s_cnt[2];
    __shared__ int s_warp[2][kPgWarps];  // per-warp counts, then their exclusive sums
    griddep_wait();
    griddep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nb = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int gt = rank * kPgThreads + tid, GT = nb * kPgThreads;  // thread of the cluster
    const int gw = rank * kPgWarps + warp, GW = nb * kPgWarps;    // warp of the cluster
    const PagesWs W = pages_ws(A.ws, A.n_pages, A.n_seqs);
    const int N = A.n_pages;
    const int ps = 1 << A.shift;
    const int64_t cap = (int64_t)A.max_pages << A.shift;
    // pages of this warp: a contiguous segment, multiples of 32
    const int64_t seg = ((int64_t)N + (int64_t)GW * 32 - 1) / ((int64_t)GW * 32) * 32;
    const int lo = (int)((int64_t)gw * seg < N ? (int64_t)gw * seg : N);
    const int hi = (int)((int64_t)lo + seg < N ? (int64_t)lo + seg : N);
    volatile int32_t* head = W.head;
    auto bad = [&](int code) {
        head[kHeadBad] = 1;
        report_timeout(status, code);
    };
    auto clamp_len = [&](int l) { return l < 0 ? 0 : ((int64_t)l > cap ? (int)cap : l); };
    auto pages_of = [&](int l) { return (int)(((int64_t)l + ps - 1) >> A.shift); };
    auto in_range = [&](int p) { return p >= 0 && p < N; };

    // ---- start: the workspace's sums
    if (gt < kHeadWords) W.head[gt] = 0;
    if constexpr (OP != kOpCompact)
        for (int p = gt; p < N; p += GT) {
            W.delta[p] = OP == kOpCopy ? INT_MAX : 0;
            W.cow[p] = 0;
            if constexpr (OP == kOpResize) {
                W.src[p] = 0;
                W.dst[p] = -1;
            }
        }
    if constexpr (OP == kOpFork)
        for (int i = gt; i < A.n_seqs; i += GT) W.first[i] = INT_MAX;
    cl.sync();

    if constexpr (OP == kOpCopy) {
        // the first pair per destination, and the pages that are sources
        for (int64_t i = gt; i < A.n; i += GT) {
            const int s = A.arg[i], t = A.arg2[i];
            if (s < 0 || t < 0) continue;
            if (s >= A.n_src || t >= N) {
                report_timeout(status, kPgStatusInput);
                continue;
            }
            atomicMin(&W.delta[t], (int)i);
            if (A.same && s < N) W.cow[s] = 1;
        }
        cl.sync();
        for (int64_t i = gt; i < A.n; i += GT) {
            int s = A.arg[i];
            const int t = A.arg2[i];
            if (s < 0 || t < 0 || s >= A.n_src || t >= N) {
                s = -1;
            } else if (W.delta[t] != (int)i || W.cow[t]) {
                report_timeout(status, kPgStatusConflict);
                s = -1;
            }
            W.src[i] = s;
            W.dst[i] = t;
        }
        if (gt == 0) W.head[kHeadPairs] = (int)A.n;
        return;
    }

    if constexpr (OP == kOpFork || OP == kOpResize) {
        // ---- holders lost and gained, and what each row takes
        if constexpr (OP == kOpFork) {
            for (int i = gt; i < A.n_seqs; i += GT) {
                const int p = A.arg[i], l = A.lens[i];
                if (p < -1 || p >= A.n_seqs || l != clamp_len(l)) bad(kPgStatusInput);
                if (p >= 0 && p < A.n_seqs) atomicMin(&W.first[p], p == i ? 0 : i + 1);
            }
            cl.sync();
        }
        for (int i = gw; i < A.n_seqs; i += GW) {
            const int32_t* row = A.table + (int64_t)i * A.max_pages;
            const int old = clamp_len(A.lens[i]);
            const int had = pages_of(old);
            if constexpr (OP == kOpFork) {
                int p = A.arg[i];
                if (p < 0 || p >= A.n_seqs) p = -1;
                for (int j = lane; j < had; j += 32) {
                    const int e = row[j];
                    if (!in_range(e)) bad(kPgStatusInput);
                    else if (p != i) atomicSub(&W.delta[e], 1);
                }
                int own = 0;  // the row needs a last page of its own
                if (p >= 0 && p != i) {
                    const int32_t* prow = A.table + (int64_t)p * A.max_pages;
                    const int len = clamp_len(A.lens[p]);
                    const int used = pages_of(len);
                    own = (len & (ps - 1)) != 0 && W.first[p] != i + 1;
                    for (int j = lane; j < used - own; j += 32) {
                        const int e = prow[j];
                        if (in_range(e)) atomicAdd(&W.delta[e], 1);
                    }
                }
                if (lane == 0) {
                    W.start[i] = own;
                    W.pair[i] = own;
                }
            } else {
                const int to = A.arg[i] < 0 ? old : A.arg[i];
                const int len = clamp_len(to);
                const int used = pages_of(len);
                if (lane == 0 && (A.lens[i] != old || to != len)) bad(kPgStatusInput);
                for (int j = lane; j < had; j += 32) {
                    const int e = row[j];
                    if (!in_range(e)) bad(kPgStatusInput);
                    else if (j >= used) atomicSub(&W.delta[e], 1);
                }
                // the row goes on inside its last page
                if (lane == 0) {
                    const bool writes = len > old && (old & (ps - 1)) != 0;
                    const int tail = writes ? row[had - 1] : -1;
                    W.first[i] = in_range(tail) ? tail : -1;
                    if (in_range(tail)) {
                        atomicAdd(&W.src[tail], 1);
                        atomicMax(&W.dst[tail], i);
                    }
                }
            }
        }
        cl.sync();
        if constexpr (OP == kOpResize) {
            // in row order, a row whose last page has other holders takes a
            // private copy of it: of k such rows on a page with r >= k holders,
            // all but the last if k = r, else all
            for (int i = gt; i < A.n_seqs; i += GT) {
                const int old = clamp_len(A.lens[i]);
                const int len = A.arg[i] < 0 ? old : clamp_len(A.arg[i]);
                const int more = pages_of(len) - pages_of(old);
                const int tail = W.first[i];
                int own = 0;
                if (tail >= 0) {
                    const int r = A.refs[tail] + W.delta[tail];
                    own = r > 1 && (W.src[tail] < r || W.dst[tail] != i);
                    if (own) atomicAdd(&W.cow[tail], 1);
                }
                W.start[i] = own + (more > 0 ? more : 0);
                W.pair[i] = own;
            }
            cl.sync();
        }
        // ---- free pages of this CTA's segments, and (last CTA) the rows' places
        int cnt = 0;
        for (int p = lo + lane; p - lane < hi; p += 32)
            cnt += __popc(__ballot_sync(0xFFFFFFFFu, p < hi && A.refs[p] + W.delta[p] <= 0));
        if (lane == 0) s_warp[0][warp] = cnt;
        __syncthreads();
        if (warp == 0) {  // the warps' counts to their exclusive sums
            const int own = s_warp[0][lane];
            int incl = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (lane >= o) incl += u;
            }
            s_warp[0][lane] = incl - own;
            cnt = __shfl_sync(0xFFFFFFFFu, incl, 31);  // thread 0 passes it on
        }
        if (rank == nb - 1) {
            long long base = 0;  // takes in the low 32 bits' place, pairs above
            for (int i0 = 0; i0 < A.n_seqs; i0 += kPgThreads) {
                const int i = i0 + tid;
                const long long v =
                    i < A.n_seqs ? ((long long)W.pair[i] << 40) + W.start[i] : 0;
                long long total;
                const long long ex = base + block_scan(v, s_scan64, &total) - v;
                if (i < A.n_seqs) {
                    const long long t = ex & ((1ll << 40) - 1);
                    W.start[i] = t > INT_MAX ? INT_MAX : (int)t;
                    W.pair[i] = (int)(ex >> 40) | (W.pair[i] ? INT_MIN : 0);
                }
                base += total;
            }
            if (tid == 0) {
                const long long t = base & ((1ll << 40) - 1);
                W.head[kHeadTakes] = t > INT_MAX ? INT_MAX : (int)t;
                W.head[kHeadPairs] = (int)(base >> 40);
            }
        }
        int before, all;
        __syncthreads();
        cluster_sums(cl, &s_cnt[0], cnt, &before, &all);
        const int takes = head[kHeadTakes];
        const bool invalid = head[kHeadBad] != 0;
        const bool fail = invalid || takes > all;
        // ---- the free pages in order, and the holders
        int r = before + s_warp[0][warp];
        for (int p = lo + lane; p - lane < hi; p += 32) {
            int ref = 0, d = 0;
            if (p < hi) {
                ref = A.refs[p];
                d = W.delta[p];
            }
            const unsigned m = __ballot_sync(0xFFFFFFFFu, p < hi && ref + d <= 0);
            const int k = r + __popc(m & ((1u << lane) - 1));
            r += __popc(m);
            if (p >= hi) continue;
            const bool is_free = (m >> lane) & 1;
            if (is_free && k < takes) W.fresh[k] = p;
            A.refs_out[p] = fail ? ref : (is_free ? (k < takes ? 1 : 0) : ref + d - W.cow[p]);
        }
        cl.sync();  // also: no CTA leaves while another reads its s_cnt
        // ---- the rows
        for (int i = gw; i < A.n_seqs; i += GW) {
            const int32_t* row = A.table + (int64_t)i * A.max_pages;
            int32_t* out = A.table_out + (int64_t)i * A.max_pages;
            if (fail) {
                if (out != row)
                    for (int j = lane; j < A.max_pages; j += 32) out[j] = row[j];
                if (lane == 0) A.lens_out[i] = A.lens[i];
                continue;
            }
            const int st = W.start[i], pr = W.pair[i];
            const int own = pr < 0;
            if constexpr (OP == kOpFork) {
                const int p = A.arg[i];
                const int len = p < 0 ? 0 : A.lens[p];
                const int used = pages_of(len);
                const int32_t* prow = A.table + (int64_t)(p < 0 ? 0 : p) * A.max_pages;
                for (int j = lane; j < A.max_pages; j += 32)
                    out[j] = j < used - own ? prow[j] : (j < used ? W.fresh[st] : -1);
                if (lane == 0) {
                    A.lens_out[i] = len;
                    if (own) {
                        W.src[pr & INT_MAX] = prow[used - 1];
                        W.dst[pr & INT_MAX] = W.fresh[st];
                    }
                }
            } else {
                const int old = A.lens[i];
                const int len = A.arg[i] < 0 ? old : A.arg[i];
                const int had = pages_of(old), used = pages_of(len);
                if (lane == 0 && own) {
                    W.src[pr & INT_MAX] = row[had - 1];
                    W.dst[pr & INT_MAX] = W.fresh[st];
                }
                __syncwarp();  // the row may be its own output
                for (int j = lane; j < A.max_pages; j += 32) {
                    const int e = row[j];
                    out[j] = j >= used ? -1 : (j >= had ? W.fresh[st + own + j - had] : (own && j == had - 1 ? W.fresh[st] : e));
                }
                if (lane == 0) A.lens_out[i] = len;
            }
        }
        if (gt == 0) {
            if (fail) W.head[kHeadPairs] = 0;
            A.info[0] = fail ? 0 : takes;
            A.info[1] = invalid ? -1 : (fail ? takes - all : 0);
        }
        return;
    }

    if constexpr (OP == kOpCompact) {
        // ---- live pages, and the rows' entries
        for (int i = gw; i < A.n_seqs; i += GW) {
            const int32_t* row = A.table + (int64_t)i * A.max_pages;
            const int l = A.lens[i], used = pages_of(clamp_len(l));
            if (lane == 0 && l != clamp_len(l)) bad(kPgStatusInput);
            for (int j = lane; j < used; j += 32) {
                const int e = row[j];
                if (!in_range(e) || A.refs[e] <= 0) bad(kPgStatusInput);
            }
        }
        int cnt = 0;
        for (int p = lo + lane; p - lane < hi; p += 32)
            cnt += __popc(__ballot_sync(0xFFFFFFFFu, p < hi && A.refs[p] > 0));
        int total;
        block_scan(lane == 0 ? cnt : 0, s_scan, &total);
        int before, live;
        __syncthreads();
        cluster_sums(cl, &s_cnt[0], total, &before, &live);
        const bool fail = head[kHeadBad] != 0;
        // ---- movers (live pages past the live count) and holes below it
        int movers = 0, holes = 0;
        for (int p = lo + lane; p - lane < hi; p += 32) {
            const bool on = p < hi && A.refs[p] > 0;
            movers += __popc(__ballot_sync(0xFFFFFFFFu, on && p >= live));
            holes += __popc(__ballot_sync(0xFFFFFFFFu, p < hi && !on && p < live));
        }
        if (lane == 0) {
            s_warp[0][warp] = movers;
            s_warp[1][warp] = holes;
        }
        __syncthreads();
        int tm, th;
        const int im = block_scan(tid < kPgWarps ? s_warp[0][tid] : 0, s_scan, &tm);
        const int ih = block_scan(tid < kPgWarps ? s_warp[1][tid] : 0, s_scan, &th);
        __syncthreads();
        if (tid < kPgWarps) {
            s_warp[0][tid] = im - s_warp[0][tid];
            s_warp[1][tid] = ih - s_warp[1][tid];
        }
        __syncthreads();
        cl.sync();  // s_cnt has been read
        int bm, am, bh, ah;
        if (tid == 0) s_cnt[1] = th;
        cluster_sums(cl, &s_cnt[0], tm, &bm, &am);
        bh = ah = 0;
        for (int c = 0; c < nb; ++c) {
            const int v = *cl.map_shared_rank(&s_cnt[1], c);
            if (c < rank) bh += v;
            ah += v;
        }
        (void)ah;
        int km = bm + s_warp[0][warp], kh = bh + s_warp[1][warp];
        for (int p = lo + lane; p - lane < hi; p += 32) {
            const int ref = p < hi ? A.refs[p] : 0;
            const bool on = p < hi && ref > 0;
            const unsigned mm = __ballot_sync(0xFFFFFFFFu, on && p >= live);
            const unsigned mh = __ballot_sync(0xFFFFFFFFu, p < hi && !on && p < live);
            const unsigned below = (1u << lane) - 1;
            if ((mm >> lane) & 1) {
                const int k = km + __popc(mm & below);
                W.src[k] = p;
                W.delta[k] = ref;  // the table's holders may be overwritten in place
            }
            if ((mh >> lane) & 1) W.dst[kh + __popc(mh & below)] = p;
            km += __popc(mm);
            kh += __popc(mh);
        }
        cl.sync();
        // ---- the new ids and holders (as many movers as holes)
        km = bm + s_warp[0][warp];
        kh = bh + s_warp[1][warp];
        for (int p = lo + lane; p - lane < hi; p += 32) {
            const int ref = p < hi ? A.refs[p] : 0;
            const bool on = p < hi && ref > 0;
            const unsigned mm = __ballot_sync(0xFFFFFFFFu, on && p >= live);
            const unsigned mh = __ballot_sync(0xFFFFFFFFu, p < hi && !on && p < live);
            const unsigned below = (1u << lane) - 1;
            if (p < hi) {
                int to = on ? p : -1, ref_out = ref;
                if (!fail) {
                    if ((mm >> lane) & 1) to = W.dst[km + __popc(mm & below)];
                    if (p >= live) ref_out = 0;
                    else if ((mh >> lane) & 1) ref_out = W.delta[kh + __popc(mh & below)];
                }
                A.moved[p] = to;
                A.refs_out[p] = ref_out;
            }
            km += __popc(mm);
            kh += __popc(mh);
        }
        cl.sync();
        for (int i = gw; i < A.n_seqs; i += GW) {
            const int32_t* row = A.table + (int64_t)i * A.max_pages;
            int32_t* out = A.table_out + (int64_t)i * A.max_pages;
            const int l = A.lens[i];
            const int used = pages_of(clamp_len(l));
            for (int j = lane; j < A.max_pages; j += 32) {
                const int e = row[j];
                out[j] = fail ? e : (j < used ? A.moved[e] : -1);
            }
            if (lane == 0) A.lens_out[i] = l;
        }
        if (gt == 0) {
            W.head[kHeadPairs] = fail ? 0 : am;
            A.info[0] = fail ? 0 : live;
            A.info[1] = fail ? -1 : am;
        }
    }
}

// ------------------------------------------------------------------- copying

constexpr int kPcThreads = 256;
constexpr int kPcUnroll = 8;
constexpr int kPcPerSm = 3;
constexpr int kPcChunk = kPcThreads * kPcUnroll;  // 16-byte words per step
constexpr int kPcLayers = 64;                     // most layers per launch (4 KB of parameters)

// A launch with few layers has few parameters: they are copied at every call.
template <int MAX>
struct CopyLayers {
    const uint4* src[MAX][4];
    uint4* dst[MAX][4];
};

// 16-byte words of a page's four arrays: n[0] packed K, n[1] K norms, ...
struct CopySizes {
    uint32_t n[4];
};

// A run of 32 KB of a page pair in one layer: the page's four arrays taken as
// one run of words, from word w0 on (each thread's first).
template <int MAX>
__device__ __forceinline__ void copy_step(const CopyLayers<MAX>& P, const CopySizes& Z, int l, int64_t s, int64_t t,
                                          uint32_t w0, uint32_t words) {
    uint4 v[kPcUnroll];
    uint4* to[kPcUnroll];
#pragma unroll
    for (int k = 0; k < kPcUnroll; ++k) {
        uint32_t w = w0 + k * kPcThreads;
        to[k] = nullptr;
        if (w >= words) continue;
        int a = 0;
        if (w >= Z.n[0]) {
            w -= Z.n[0];
            a = 1;
            if (w >= Z.n[1]) {
                w -= Z.n[1];
                a = 2;
                if (w >= Z.n[2]) {
                    w -= Z.n[2];
                    a = 3;
                }
            }
        }
        to[k] = P.dst[l][a] + t * Z.n[a] + w;
        v[k] = __ldcg(P.src[l][a] + s * Z.n[a] + w);
    }
#pragma unroll
    for (int k = 0; k < kPcUnroll; ++k)
        if (to[k]) __stcg(to[k], v[k]);
}

// Step u of the copy: words [u % steps * kPcChunk, ..) of page pair u / steps
// / L in layer u / steps % L, the page's four arrays taken as one run of
// words.
template <int MAX>
__global__ void __launch_bounds__(kPcThreads, kPcPerSm)
k_pages_copy(const __grid_constant__ CopyLayers<MAX> P, const CopySizes Z, int L, const int32_t* head,
             const int32_t* src, const int32_t* dst) {
    griddep_wait();
    // read at the L2, where the plan's writes are: this kernel's CTAs were
    // resident while it wrote
    const int64_t pairs = __ldcg(head + kHeadPairs);
    const uint32_t words = Z.n[0] + Z.n[1] + Z.n[2] + Z.n[3];
    const uint32_t steps = (words + kPcChunk - 1) / kPcChunk;
    const int64_t units = pairs * L * steps;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t pl = u / steps;
        const uint32_t w0 = (uint32_t)(u - pl * steps) * kPcChunk + threadIdx.x;
        const int64_t pair = pl / L;
        const int l = (int)(pl - pair * L);
        const int64_t s = __ldcg(src + pair), t = __ldcg(dst + pair);
        if (s < 0) continue;
        copy_step(P, Z, l, s, t, w0, words);
    }
}

// tq_pages_copy with few pairs: every CTA looks all of them over for itself, so
// that there is no plan to wait for.  In a graph, with the plan and so: 5 pages
// of 2 layers 6.5 and 3.6 us; 128 pages of 768 bytes 4.9 and 3.2 us; 128 of
// 0.25 MB in 2 layers 23.8 and 21.3 us.
constexpr int kPcFew = TQ_PAGES_COPY_FEW;

template <int MAX>
__global__ void __launch_bounds__(kPcThreads, kPcPerSm)
k_pages_copy_few(const __grid_constant__ CopyLayers<MAX> P, const CopySizes Z, int L, const int32_t* src,
                 const int32_t* dst, int n, int n_src, int n_dst, int same, int* status) {
    static_assert(2 * kPcFew == kPcThreads, "two threads a pair");
    __shared__ __align__(16) int s_src[kPcFew], s_dst[kPcFew];  // -1: no pair
    __shared__ int s_skip[kPcFew];
    griddep_wait();
    const int tid = threadIdx.x;
    if (tid < kPcFew) {
        int s = -1, t = -1;
        if (tid < n) {
            s = __ldcg(src + tid), t = __ldcg(dst + tid);
            if (s < 0 || t < 0) s = t = -1;
            if (s >= n_src || t >= n_dst) {
                if (blockIdx.x == 0) report_timeout(status, kPgStatusInput);
                s = t = -1;
            }
        }
        s_src[tid] = s;
        s_dst[tid] = t;
        s_skip[tid] = s < 0;
    }
    __syncthreads();
    // pair i is skipped if an earlier pair has its destination, or within one
    // pool any pair has it as a source: each of two threads looks at half of them
    {
        const int i = tid & (kPcFew - 1), t = s_dst[i], j0 = (tid / kPcFew) * (kPcFew / 2);
        bool skip = false;
        for (int j = j0; j < min(n, j0 + kPcFew / 2); j += 4) {
            const int4 d = *reinterpret_cast<const int4*>(s_dst + j), c = *reinterpret_cast<const int4*>(s_src + j);
            skip |= (d.x == t && j < i) || (d.y == t && j + 1 < i) || (d.z == t && j + 2 < i) || (d.w == t && j + 3 < i);
            skip |= same && (c.x == t || c.y == t || c.z == t || c.w == t);
        }
        if (skip && t >= 0) s_skip[i] = 2;
    }
    __syncthreads();
    if (blockIdx.x == 0 && tid < n && s_skip[tid] == 2) report_timeout(status, kPgStatusConflict);
    const uint32_t words = Z.n[0] + Z.n[1] + Z.n[2] + Z.n[3];
    const uint32_t steps = (words + kPcChunk - 1) / kPcChunk;
    const int64_t units = (int64_t)n * L * steps;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t pl = u / steps;
        const uint32_t w0 = (uint32_t)(u - pl * steps) * kPcChunk + tid;
        const int pair = (int)(pl / L), l = (int)(pl - (int64_t)pair * L);
        if (!s_skip[pair]) copy_step(P, Z, l, s_src[pair], s_dst[pair], w0, words);
    }
}

template <int MAX>
static cudaError_t launch_copy(const PagesCall& c, int l0, int L, const CopySizes& Z, const PagesWs& W, int64_t grid,
                               bool few, cudaStream_t s) {
    CopyLayers<MAX> P;
    for (int l = 0; l < L; ++l) {
        const tq_paged_cache &f = c.src[l0 + l], &t = c.dst[l0 + l];
        P.src[l][0] = reinterpret_cast<const uint4*>(f.k_packed);
        P.src[l][1] = reinterpret_cast<const uint4*>(f.k_norm);
        P.src[l][2] = reinterpret_cast<const uint4*>(f.v_packed);
        P.src[l][3] = reinterpret_cast<const uint4*>(f.v_norm);
        P.dst[l][0] = reinterpret_cast<uint4*>(t.k_packed);
        P.dst[l][1] = reinterpret_cast<uint4*>(t.k_norm);
        P.dst[l][2] = reinterpret_cast<uint4*>(t.v_packed);
        P.dst[l][3] = reinterpret_cast<uint4*>(t.v_norm);
    }
    if (few)
        return launch_pdl(k_pages_copy_few<MAX>, dim3((unsigned)grid), dim3(kPcThreads), 0, s, P, Z, L, c.arg, c.arg2,
                          (int)c.n, (int)c.src[0].n_pages, (int)c.dst[0].n_pages, c.same, status_word());
    return launch_pdl(k_pages_copy<MAX>, dim3((unsigned)grid), dim3(kPcThreads), 0, s, P, Z, L,
                      (const int32_t*)W.head, (const int32_t*)W.src, (const int32_t*)W.dst);
}

// One CTA, or a cluster of 8 once the books are long enough for the barriers
// between CTAs to cost less than they save.  A resize, fork and compaction of
// 4048 words of books took 9.1, 10.1 and 10.8 us with one CTA and 10.5, 11.6 and
// 13.4 with 8; of 8096 words 13.1, 12.8 and 14.3 against 11.0, 11.5 and 14.7; of
// 16,000 words 19.0, 18.0 and 21.0 against 11.4, 12.2 and 17.3.
static int plan_ctas(const PagesPlan& A) {
    const int64_t words = (int64_t)A.n_pages + (int64_t)A.n_seqs * A.max_pages + A.n;
    return words > 6144 ? kPgClusterMax : 1;
}

template <int OP>
static cudaError_t launch_plan(const PagesPlan& A, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    const int nb = plan_ctas(A);
    cfg.gridDim = dim3(nb);
    cfg.blockDim = dim3(kPgThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = nb;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = nb > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_pages_plan<OP>, A, status_word());
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace dev

size_t pages_workspace_bytes(int n_seqs, int64_t n_pages) {
    return (4 * (size_t)(dev::kHeadWords + 5 * n_pages + 3 * (int64_t)n_seqs) + 255) / 256 * 256;
}

cudaError_t launch_pages(int op, const PagesCall& c, cudaStream_t s) {
    using namespace dev;
    PagesPlan A = {};
    A.table = c.in.block_table;
    A.lens = c.in.lens;
    A.refs = c.in.refs;
    A.table_out = c.out.block_table;
    A.lens_out = c.out.lens;
    A.refs_out = c.out.refs;
    A.arg = c.arg;
    A.arg2 = c.arg2;
    A.moved = c.moved;
    A.info = c.info;
    A.ws = c.ws;
    A.n = c.n;
    A.n_seqs = c.n_seqs;
    A.max_pages = c.max_pages;
    A.n_pages = (int)c.dst[0].n_pages;
    A.n_src = (int)c.src[0].n_pages;
    A.shift = c.page_shift;
    A.same = c.same;
    cudaError_t e = cudaSuccess;
    const bool few = op == kPagesCopy && c.n <= kPcFew;
    switch (op) {
        case kPagesCopy:
            if (!few) e = launch_plan<kOpCopy>(A, s);
            break;
        case kPagesFork: e = launch_plan<kOpFork>(A, s); break;
        case kPagesResize: e = launch_plan<kOpResize>(A, s); break;
        default: e = launch_plan<kOpCompact>(A, s); break;
    }
    if (e != cudaSuccess) return e;
    CopySizes Z;
    const uint32_t rows = (uint32_t)c.Hkv << c.page_shift;
    Z.n[0] = rows * (uint32_t)(c.d * c.k_bits / 8) / 16;
    Z.n[1] = Z.n[3] = rows / 4;
    Z.n[2] = rows * (uint32_t)(c.d * c.v_bits / 8) / 16;
    const PagesWs W = few ? PagesWs{} : pages_ws(c.ws, A.n_pages, A.n_seqs);
    // the most pairs that the plan can ask for: a small call gets a small grid
    const int64_t most = op == kPagesCopy ? c.n : (op == kPagesCompact ? (int64_t)A.n_pages / 2 : (int64_t)c.n_seqs);
    const uint32_t words = Z.n[0] + Z.n[1] + Z.n[2] + Z.n[3];
    const int64_t steps = (words + kPcChunk - 1) / kPcChunk;
    for (int l0 = 0; l0 < c.n_layers; l0 += kPcLayers) {
        const int L = c.n_layers - l0 < kPcLayers ? c.n_layers - l0 : kPcLayers;
        const int64_t cap = (int64_t)num_sms() * kPcPerSm;
        int64_t grid = most * L * steps;
        grid = grid < 1 ? 1 : (grid > cap ? cap : grid);
        e = L <= 4 ? launch_copy<4>(c, l0, L, Z, W, grid, few, s) : launch_copy<kPcLayers>(c, l0, L, Z, W, grid, few, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace tq
