// Eviction from the paged cache by accumulated attention weight.
//
// Per (sequence, key-value head): of the tokens between the protected first
// `sink` and last `recent`, the T = budget - sink - recent heaviest stay.
//
// evict_select finds the T-th largest weight by radix selection on 32-bit keys
// whose unsigned order is the floats' order: three digits of 11, 11 and 10
// bits, each a histogram of the digit among the keys that share the prefix
// found so far and a scan of it from the top.  It then lists the kept tokens
// in their order.  A cluster of up to 16 blocks shares one (sequence,
// head); each holds its slice of the keys in shared memory, so the weights are
// read once, and sums the others' histograms over distributed shared memory.
//
// Carrying the rows is a copy bound by HBM: evict_copy for another cache, and
// evict_shift in place, where a row may overwrite one that is still to be read.

#include <cooperative_groups.h>

#include "paged.cuh"

namespace cg = cooperative_groups;

namespace gdn2 {

constexpr int kBins = 2048;
constexpr int kDigits = 3;
constexpr int kMostRanks = 16;     // blocks of a cluster
constexpr int kMaxKeys = 40960;    // keys of a block's slice in shared memory
constexpr int kMoveThreads = 256;

__device__ __forceinline__ int ld_acquire(const int *p) {
    int x;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
    return x;
}
__device__ __forceinline__ void st_release(int *p, int x) {
    asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(x) : "memory");
}

struct EvictPlan {
    int first, count;  // rows [first, count) move; count < 0: nothing, the length included
};

// larger float <=> larger key; -0 as +0, NaN below everything
__device__ __forceinline__ unsigned weight_key(float x) {
    if (x != x) return 0u;
    const unsigned u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ unsigned key_at(const PagedView &c, int n, int h, int j, unsigned int *status) {
    int entry, slot;
    page_slot(c, j, entry, slot);
    const int page = page_of(c, n, entry);
    if (page < 0) {
        record_status(status, GDN2_ERR_INVALID_ARG);
        return 0u;
    }
    return weight_key(c.w[weight_off(c, page, slot, h)]);
}

// inclusive scan over the block's NT threads
template <int NT>
__device__ __forceinline__ int block_scan(int x, int *warp_tot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) warp_tot[warp] = x;
    __syncthreads();
    int t = lane < NT / 32 ? warp_tot[lane] : 0;
#pragma unroll
    for (int off = 1; off < NT / 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, t, off);
        if (lane >= off) t += y;
    }
    const int before = __shfl_sync(0xffffffffu, t, warp == 0 ? 0 : warp - 1);
    __syncthreads();
    return x + (warp == 0 ? 0 : before);
}

// Block (n h, rank) of a cluster.  slots: the keys that dynamic shared memory
// holds; stride: entries of a list; flags: evict_shift's, one a chunk of each
// list and the ticket behind them, or nullptr; ticket: the first to be drawn.
template <int NT>
__global__ void __launch_bounds__(NT)
evict_select_kernel(const PagedView c, const PagedView to, int in_place, int budget, int sink, int recent,
                    int slots, int stride, int *list_all, EvictPlan *plan, int *flags, int chunks, int ticket, unsigned int *status) {
    constexpr int kWarps = NT / 32, kOwn = kBins / NT;  // digits of a thread
    extern __shared__ unsigned s_key[];
    __shared__ __align__(16) int hist[kDigits][kBins];
    __shared__ int warp_tot[32], s_digit, s_above;
    __shared__ int2 s_warp[kWarps];  // kept for certain, equal to the threshold: a warp's
    __shared__ int2 s_block;            // the block's
    __shared__ int s_first;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nh = blockIdx.x / ranks, n = nh / c.Hkv, h = nh - n * c.Hkv;
    int *list = list_all + (size_t)nh * stride;
    follow_previous();
    if (flags) {  // for evict_shift: no chunk read
        for (int j = rank * NT + tid; j < chunks; j += ranks * NT) flags[(size_t)nh * chunks + j] = 0;
        if (blockIdx.x == 0 && tid == 0) flags[(size_t)c.N * c.Hkv * chunks] = ticket;
    }
    const int raw = c.lens[n];
    int len = checked_len(c, n, status);
    if (min(len, budget) > to.cap) {
        record_status(status, GDN2_ERR_INVALID_ARG);
        len = 0;
    }
    if (len <= budget) {
        for (int j = rank * NT + tid; j < stride; j += ranks * NT) list[j] = j < len ? j : -1;
        if (rank == 0 && tid == 0) plan[nh] = EvictPlan{in_place ? len : 0, in_place && raw != len ? -1 : len};
        return;
    }
    const int lo = sink, hi = len - recent, T = budget - sink - recent;  // T < hi - lo
    for (int j = rank * NT + tid; j < sink; j += ranks * NT) list[j] = j;
    for (int j = rank * NT + tid; j < recent; j += ranks * NT) list[budget - recent + j] = hi + j;
    if (T == 0) {
        if (rank == 0 && tid == 0) plan[nh] = EvictPlan{in_place ? sink : 0, budget};
        return;
    }
    const int per = (hi - lo + ranks - 1) / ranks, a = min(hi, lo + rank * per), b = min(hi, a + per);
    const bool held = per <= slots;
    auto key = [&](int j) { return held ? s_key[j - a] : key_at(c, n, h, j, status); };
    for (int x = tid; x < kDigits * kBins; x += NT) (&hist[0][0])[x] = 0;
    if (tid == 0) s_first = len;
    if (held) {  // eight at a time, each load before any is used
        constexpr int kAhead = 8;
        for (int j0 = a + tid; j0 < b; j0 += kAhead * NT) {
            int page[kAhead], slot[kAhead];
            float w[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int j = min(j0 + u * NT, b - 1);
                int entry;
                page_slot(c, j, entry, slot[u]);
                page[u] = page_of(c, n, entry);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) w[u] = page[u] < 0 ? __uint_as_float(0x7fc00000u) : c.w[weight_off(c, page[u], slot[u], h)];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (page[u] < 0) record_status(status, GDN2_ERR_INVALID_ARG);
                if (j0 + u * NT < b) s_key[j0 + u * NT - a] = weight_key(w[u]);
            }
        }
    }
    __syncthreads();
    unsigned prefix = 0, mask = 0;
    int need = T;
#pragma unroll
    for (int d = 0; d < kDigits; ++d) {
        const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, width = d == 2 ? 10 : 11;
        for (int j = a + tid; j < b; j += NT) {
            const unsigned k = key(j);
            if ((k & mask) == prefix) atomicAdd(&hist[d][(k >> shift) & ((1u << width) - 1)], 1);
        }
        cluster.sync();
        // Each block sums its share of the bins over the cluster, in place (the
        // others read only their own shares of it), and then reads the sums:
        // two short trips over the cluster's network instead of every block
        // reading all of every histogram.
        const int share = kBins / ranks;
        if (ranks > 1) {
            for (int i = tid; i < share; i += NT) {
                int sum = 0;
#pragma unroll
                for (int r = 0; r < kMostRanks; ++r)
                    if (r < ranks) sum += *cluster.map_shared_rank(&hist[d][rank * share + i], r);
                hist[d][rank * share + i] = sum;
            }
            cluster.sync();
        }
        // thread t: the t-th kOwn digits from the top
        const int top = kBins - 1 - kOwn * tid;
        int own[kOwn];
        const int *summed = cluster.map_shared_rank(&hist[d][top - kOwn + 1], (top - kOwn + 1) / share);
#pragma unroll
        for (int i = 0; i < kOwn; i += 2) {
            const int2 y = *reinterpret_cast<const int2 *>(summed + i);
            own[i] = y.x;
            own[i + 1] = y.y;
        }
        int sum = 0;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) sum += own[i];
        const int inc = block_scan<NT>(sum, warp_tot);
        int above = inc - sum;
        if (above < need && need <= inc) {  // one thread: its digit with the need-th largest
            int i = kOwn - 1;
            for (; i > 0 && above + own[i] < need; --i) above += own[i];
            s_digit = top - kOwn + 1 + i;
            s_above = above;
        }
        __syncthreads();
        prefix |= (unsigned)s_digit << shift;
        mask |= ((1u << width) - 1) << shift;
        need -= s_above;
        __syncthreads();  // both have been read
    }
    // all keys above `prefix` stay, and the first `need` of those equal to it.
    // Each warp takes a contiguous piece of the slice: first it counts.
    const int piece = ((b - a + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int wa = min(b, a + warp * piece), wb = min(b, wa + piece);
    int2 cnt = make_int2(0, 0);
    for (int j0 = wa; j0 < wb; j0 += 32) {
        const int j = j0 + lane;
        const unsigned k = j < wb ? key(j) : 0u;
        cnt.x += __popc(__ballot_sync(0xffffffffu, j < wb && k > prefix));
        cnt.y += __popc(__ballot_sync(0xffffffffu, j < wb && k == prefix));
    }
    if (lane == 0) s_warp[warp] = cnt;
    __syncthreads();
    int2 before = make_int2(0, 0);
    for (int w = 0; w < kWarps; ++w) {
        const int2 x = s_warp[w];
        if (w == warp) cnt = before;
        before.x += x.x;
        before.y += x.y;
    }
    if (tid == 0) s_block = before;
    cluster.sync();
    int2 other = lane < rank ? *cluster.map_shared_rank(&s_block, lane) : make_int2(0, 0);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        other.x += __shfl_xor_sync(0xffffffffu, other.x, off);
        other.y += __shfl_xor_sync(0xffffffffu, other.y, off);
    }
    cnt.x += other.x;
    cnt.y += other.y;
    int first = len;  // the first token that goes: up to there no row moves
    const unsigned below = (1u << lane) - 1;
    for (int j0 = wa; j0 < wb; j0 += 32) {
        const int j = j0 + lane;
        const unsigned k = j < wb ? key(j) : 0u;
        const unsigned gt = __ballot_sync(0xffffffffu, j < wb && k > prefix);
        const unsigned eq = __ballot_sync(0xffffffffu, j < wb && k == prefix);
        if (j < wb) {
            const int e = cnt.y + __popc(eq & below);
            if (k > prefix || (k == prefix && e < need)) {
                const int at = sink + cnt.x + __popc(gt & below) + min(e, need);
                if (at < sink + T) list[at] = j;  // always, unless the weights change under the call
            } else first = min(first, j);
        }
        cnt.x += __popc(gt);
        cnt.y += __popc(eq);
    }
    if (first < len) atomicMin(&s_first, first);
    cluster.sync();
    if (rank == 0 && warp == 0) {
        first = lane < ranks ? *cluster.map_shared_rank(&s_first, lane) : len;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) first = min(first, __shfl_xor_sync(0xffffffffu, first, off));
        if (lane == 0) plan[nh] = EvictPlan{in_place ? first : 0, budget};
    }
    cluster.sync();  // no block ends while another reads its memory
}

// Into another cache: the kept rows in any order.  An item is a chunk of rows
// of one (sequence, head), a thread carrying the same 16-byte piece of kDeep
// rows of k and of v; the next item's places are looked up (list, then tables)
// while this one's rows are on their way.  The weights are items of their own.
constexpr int kDeep = 2;  // 16 sequences to 2K tokens of 16 heads: 114 us a call; with 4 rows a thread 146, with 8 262
constexpr int kCopyBlocksPerSm = 4;

// The most rows that any of the lists moves, for every thread of the block:
// a budget may be far beyond what the sequences hold.
__device__ __forceinline__ int most_rows(const EvictPlan *plan, int nhs) {
    __shared__ int s_most[kMoveThreads / 32];
    int most = 0;
    for (int i = threadIdx.x; i < nhs; i += kMoveThreads) most = max(most, plan[i].count - plan[i].first);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
    if ((threadIdx.x & 31) == 0) s_most[threadIdx.x >> 5] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kMoveThreads / 32; ++w) most = max(most, s_most[w]);
    return most;
}
// the new lengths, shared out over the grid
__device__ __forceinline__ void write_lens(const PagedView &to, const EvictPlan *plan) {
    for (int n = blockIdx.x * kMoveThreads + threadIdx.x; n < to.N; n += gridDim.x * kMoveThreads) {
        const int count = plan[(size_t)n * to.Hkv].count;
        if (count >= 0) to.lens[n] = count;
    }
}
__global__ void __launch_bounds__(kMoveThreads, kCopyBlocksPerSm)
evict_copy_kernel(const PagedView c, const PagedView to, int stride, const int *list_all,
                  const EvictPlan *plan, unsigned int *status) {
    const int pieces = c.d * c.es / 16, at_once = kMoveThreads / pieces;
    const int piece = threadIdx.x % pieces, r = threadIdx.x / pieces;
    long long from[kDeep], dst[kDeep];
    follow_previous();
    write_lens(to, plan);
    const int most = most_rows(plan, c.N * c.Hkv);
    if (most == 0) return;
    const int chunks = (most + at_once * kDeep - 1) / (at_once * kDeep);
    const int wchunks = (most + kMoveThreads * kDeep - 1) / (kMoveThreads * kDeep);
    const long long rows = (long long)c.N * c.Hkv * chunks, total = rows + (long long)c.N * c.Hkv * wchunks;
    // the places of row i0 + u step, u < kDeep, of (sequence, head) nh; -1: not written
    auto places = [&](int nh, long long i0, int step, auto place) {
        const int n = nh / c.Hkv, h = nh - n * c.Hkv, count = plan[nh].count;
        const int *list = list_all + (size_t)nh * stride;
        int src[kDeep], page[kDeep], page2[kDeep], slot[kDeep], slot2[kDeep];
#pragma unroll
        for (int u = 0; u < kDeep; ++u) src[u] = i0 + u * step < count ? list[i0 + u * step] : -1;
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            page[u] = page2[u] = -1;
            if (src[u] < 0) continue;
            int entry, entry2;
            page_slot(c, src[u], entry, slot[u]);
            page_slot(to, (int)(i0 + u * step), entry2, slot2[u]);
            page[u] = page_of(c, n, entry);
            page2[u] = page_of(to, n, entry2);
        }
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            const bool ok = page[u] >= 0 && page2[u] >= 0;
            if (src[u] >= 0 && !ok) record_status(status, GDN2_ERR_INVALID_ARG);
            from[u] = dst[u] = -1;
            if (ok) place(u, page[u], slot[u], page2[u], slot2[u], h);
        }
    };
    auto row_places = [&](long long x) {
        // heads first: blocks at work at once then read and write the same pages
        const long long y = x / c.Hkv;
        const int n = (int)(y / chunks), chunk = (int)(y - (long long)n * chunks), nh = n * c.Hkv + (int)(x - y * c.Hkv);
        places(nh, (long long)chunk * at_once * kDeep + r, at_once, [&](int u, int pg, int sl, int pg2, int sl2, int h) {
            from[u] = row_off(c, pg, sl, h) + piece * 16;
            dst[u] = row_off(to, pg2, sl2, h) + piece * 16;
        });
    };
    long long x = blockIdx.x;
    if (x < rows) row_places(x);
    for (; x < rows; x += gridDim.x) {
        uint4 k[kDeep], v[kDeep];
        long long at[kDeep];
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            at[u] = dst[u];
            if (at[u] < 0) continue;
            k[u] = *reinterpret_cast<const uint4 *>(c.k + from[u]);
            v[u] = *reinterpret_cast<const uint4 *>(c.v + from[u]);
        }
        if (x + gridDim.x < rows) row_places(x + gridDim.x);
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            if (at[u] < 0) continue;
            *reinterpret_cast<uint4 *>(to.k + at[u]) = k[u];
            *reinterpret_cast<uint4 *>(to.v + at[u]) = v[u];
        }
    }
    for (; x < total; x += gridDim.x) {
        const int nh = (int)((x - rows) / wchunks), chunk = (int)(x - rows - (long long)nh * wchunks);
        places(nh, (long long)chunk * kMoveThreads * kDeep + threadIdx.x, kMoveThreads,
               [&](int u, int pg, int sl, int pg2, int sl2, int h) {
                   from[u] = (long long)weight_off(c, pg, sl, h);
                   dst[u] = (long long)weight_off(to, pg2, sl2, h);
               });
        float w[kDeep];
#pragma unroll
        for (int u = 0; u < kDeep; ++u)
            if (dst[u] >= 0) w[u] = c.w[from[u]];
#pragma unroll
        for (int u = 0; u < kDeep; ++u)
            if (dst[u] >= 0) to.w[dst[u]] = w[u];
    }
}

constexpr int kShiftDeep = 8;
constexpr int kShiftBlocksPerSm = 2;
// In place, where a row may overwrite one that is still to be read.  Chunks of
// rows are taken in the order of a ticket: chunk by chunk, in each the
// (sequence, head)s.  A block reads its chunk, says so in the chunk's flag, and
// writes it once every earlier chunk of that (sequence, head) has been read:
// row i comes from list[i] >= i, so the rows that chunk x overwrites belong to
// chunks up to x.  Every wait ends, whichever blocks the GPU runs: a block
// waits, with its own chunk read, for chunks of earlier tickets only, so the
// block that holds the earliest ticket not yet read is either reading it or
// (the next ticket is drawn early) waits for nothing that is not read.  It
// gives up all the same after `limit` clocks (GDN2_ERR_TIMEOUT), and leaves its
// chunk's rows where they were, under lengths that are new already.  Chunks of 128 rows (bf16, d = 128)
// make the agreement cheap: 16 sequences of up to 8K tokens and 16 heads to 2K
// take 141 us, with 32 rows and twice the blocks 153; the copy above, 114.  One
// of 131K tokens, halved: 80, 117 and 47.
__global__ void __launch_bounds__(kMoveThreads, kShiftBlocksPerSm)
evict_shift_kernel(const PagedView c, int stride, int chunks, const int *list_all, const EvictPlan *plan, int *flags,
                   int *ticket, long long limit, unsigned int *status) {
    __shared__ int s_ticket;
    const int pieces = c.d * c.es / 16, at_once = kMoveThreads / pieces, nhs = c.N * c.Hkv;
    const int piece = threadIdx.x % pieces, r = threadIdx.x / pieces;
    follow_previous();
    write_lens(c, plan);
    const long long total = (long long)nhs * ((most_rows(plan, nhs) + at_once * kShiftDeep - 1) / (at_once * kShiftDeep));
    if (total == 0) return;
    int next = threadIdx.x == 0 ? atomicAdd(ticket, 1) : 0;
    for (;;) {
        __syncthreads();  // the last ticket has been read
        if (threadIdx.x == 0) s_ticket = next;
        __syncthreads();
        const long long x = (unsigned)s_ticket;
        if (threadIdx.x == 0 && x < total) next = atomicAdd(ticket, 1);  // under this chunk's reads
        if (x >= total) return;
        const int chunk = (int)(x / nhs), nh = (int)(x - (long long)chunk * nhs), n = nh / c.Hkv, h = nh - n * c.Hkv;
        const EvictPlan p = plan[nh];
        const long long i0 = p.first + (long long)chunk * at_once * kShiftDeep;
        if (i0 >= p.count) continue;
        const int *list = list_all + (size_t)nh * stride;
        int *flag = flags + (size_t)nh * chunks;
        uint4 k[kShiftDeep], v[kShiftDeep];
        float w[kShiftDeep];
        int src[kShiftDeep], page[kShiftDeep], slot[kShiftDeep];
#pragma unroll
        for (int u = 0; u < kShiftDeep; ++u) {
            const long long i = i0 + r + u * at_once;
            src[u] = i < p.count ? list[i] : -1;
        }
#pragma unroll
        for (int u = 0; u < kShiftDeep; ++u) {
            page[u] = -1;
            if (src[u] < 0) continue;
            int entry;
            page_slot(c, src[u], entry, slot[u]);
            page[u] = page_of(c, n, entry);
            if (page[u] < 0) record_status(status, GDN2_ERR_INVALID_ARG);
        }
#pragma unroll
        for (int u = 0; u < kShiftDeep; ++u) {
            if (page[u] < 0) continue;
            const long long at = row_off(c, page[u], slot[u], h) + piece * 16;
            k[u] = *reinterpret_cast<const uint4 *>(c.k + at);
            v[u] = *reinterpret_cast<const uint4 *>(c.v + at);
            if (piece == 0) w[u] = c.w[weight_off(c, page[u], slot[u], h)];
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            __threadfence();
            st_release(flag + chunk, 1);
        }
        bool ready = true;
        for (int j = threadIdx.x; j < chunk && ready; j += kMoveThreads) {
            if (ld_acquire(flag + j)) continue;
            const long long t0 = clock64();
            while (!ld_acquire(flag + j) && ready) ready = clock64() - t0 < limit;
        }
        if (!__syncthreads_and(ready)) {
            if (threadIdx.x == 0) record_status(status, GDN2_ERR_TIMEOUT);
            continue;
        }
#pragma unroll
        for (int u = 0; u < kShiftDeep; ++u) {
            if (page[u] < 0) continue;
            int entry, to_slot;
            page_slot(c, (int)(i0 + r + u * at_once), entry, to_slot);
            const int to_page = page_of(c, n, entry);
            if (to_page < 0) {
                record_status(status, GDN2_ERR_INVALID_ARG);
                continue;
            }
            const long long at = row_off(c, to_page, to_slot, h) + piece * 16;
            *reinterpret_cast<uint4 *>(c.k + at) = k[u];
            *reinterpret_cast<uint4 *>(c.v + at) = v[u];
            if (piece == 0) c.w[weight_off(c, to_page, to_slot, h)] = w[u];
        }
    }
}

// entries of a list in the workspace
static int list_stride(const PagedView &c, int budget) { return budget < c.cap ? budget : c.cap; }

// items of a list when a thread carries `deep` rows, and evict_shift's
static int item_count(const PagedView &c, int stride, int deep) {
    const int rows = kMoveThreads / (c.d * c.es / 16) * deep;
    return (stride + rows - 1) / rows;
}
static int chunk_count(const PagedView &c, int stride) { return item_count(c, stride, kShiftDeep); }

// chunks that the tickets may have to count
bool evict_countable(const PagedView &c, int budget) {
    return (long long)c.N * c.Hkv * chunk_count(c, list_stride(c, budget)) < 1LL << 30;
}

size_t evict_ws_bytes(const PagedView &c, int budget) {
    const size_t nh = (size_t)c.N * c.Hkv;
    const int stride = list_stride(c, budget);
    return align256(nh * sizeof(EvictPlan)) + align256(nh * stride * sizeof(int)) +
           align256((nh * chunk_count(c, stride) + 1) * sizeof(int));
}

template <int NT>
static cudaError_t select_launch(const PagedView &src, const PagedView &dst, bool in_place, int budget, int sink, int recent,
                                 int ranks, int slots, int stride, int *list, EvictPlan *plan, int *flags, int chunks,
                                 int ticket, unsigned int *status, cudaStream_t s) {
    const auto kernel = evict_select_kernel<NT>;
    cudaError_t e = cudaSuccess;
    if (slots * 4 > 16 << 10)  // with the static arrays above what any kernel may have
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxKeys * 4);
    if (e == cudaSuccess && ranks > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    return launch_clusters(K_EVICT_SELECT, kernel, ranks, src.N * src.Hkv * ranks, NT, slots * 4, s, src, dst, (int)in_place,
                           budget, sink, recent, slots, stride, list, plan, flags, chunks, ticket, status);
}

cudaError_t evict_launch(const PagedView &src, const PagedView &dst, bool in_place, int budget, int sink,
                         int recent, int *kept, void *ws, unsigned int *status, cudaStream_t s, long long wait_clocks,
                         int ticket) {
    const int nh = src.N * src.Hkv;
    EvictPlan *plan = static_cast<EvictPlan *>(ws);
    const int stride = kept ? budget : list_stride(src, budget);  // entries of a list
    const int own = list_stride(src, budget), chunks = chunk_count(src, own);
    int *const own_list = at<int>(ws, align256((size_t)nh * sizeof(EvictPlan)));
    int *list = kept ? kept : own_list;
    int *flags = at<int>(own_list, align256((size_t)nh * own * sizeof(int)));
    // blocks of a cluster: until a slice is 4096 tokens or the GPU is full
    int ranks = 1;
    while (ranks < kMostRanks && src.cap / ranks > 4096 && (long long)nh * ranks < sm_count()) ranks *= 2;
    const int slice = (int)(((long long)src.cap + ranks - 1) / ranks), slots = slice < kMaxKeys ? slice : kMaxKeys;
    // one block an SM has 1024 threads; several hide each other's waits with 512
    cudaError_t e = (long long)nh * ranks <= sm_count()
                        ? select_launch<1024>(src, dst, in_place, budget, sink, recent, ranks, slots, stride, list, plan, in_place ? flags : nullptr, chunks, ticket, status, s)
                        : select_launch<512>(src, dst, in_place, budget, sink, recent, ranks, slots, stride, list, plan, in_place ? flags : nullptr, chunks, ticket, status, s);
    if (e != cudaSuccess) return e;
    if (in_place) {
        const long long items = (long long)nh * chunks;
        const long long blocks = (long long)kShiftBlocksPerSm * sm_count();
        return launch_behind(K_EVICT_MOVE, evict_shift_kernel, (int)(items < blocks ? items : blocks), kMoveThreads, 0, s,
                             src, stride, chunks, list, plan, flags, flags + (size_t)nh * chunks, wait_clocks, status);
    }
    const long long items = (long long)nh * (item_count(src, stride, kDeep) + 1);
    const long long blocks = (long long)kCopyBlocksPerSm * sm_count();
    return launch_behind(K_EVICT_MOVE, evict_copy_kernel, (int)(items < blocks ? items : blocks), kMoveThreads, 0, s, src,
                         dst, stride, list, plan, status);
}

}  // namespace gdn2
