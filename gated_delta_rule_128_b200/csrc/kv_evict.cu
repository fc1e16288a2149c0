// Eviction from the paged cache by accumulated attention weight.
//
// Per (sequence, key-value head): of the tokens between the protected first
// `sink` and last `recent`, the T = budget - sink - recent heaviest stay.
//
// evict_select finds the T-th largest weight by radix selection on 32-bit keys
// whose unsigned order is the floats' order: three digits of 11, 11 and 10
// bits, each a histogram of the digit among the keys that share the prefix
// found so far and a scan of it from the top.  It then lists the kept tokens
// in their order.  A cluster of up to 8 blocks shares one (sequence, head);
// each holds its slice of the keys in shared memory, so the weights are read
// once, and sums the others' histograms over distributed shared memory.
//
// Carrying the rows is a copy bound by HBM: evict_copy for another cache, and
// evict_shift in place, where a row may overwrite one that is still to be read.

#include <cooperative_groups.h>

#include "paged.cuh"

namespace cg = cooperative_groups;

namespace gdn2 {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kDigits = 3;
constexpr int kMaxKeys = 40960;    // keys of a block's slice in shared memory
constexpr int kMoveThreads = 256;

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

// inclusive scan over the block's threads
__device__ __forceinline__ int block_scan(int x, int *warp_tot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) warp_tot[warp] = x;
    __syncthreads();
    int t = warp_tot[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, t, off);
        if (lane >= off) t += y;
    }
    const int before = __shfl_sync(0xffffffffu, t, warp == 0 ? 0 : warp - 1);
    __syncthreads();
    return x + (warp == 0 ? 0 : before);
}

// Block (n h, rank) of a cluster.  slots: the keys that dynamic shared memory
// holds; stride: entries of a list.
__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const PagedView c, const PagedView to, int in_place, int budget, int sink, int recent,
                    int slots, int stride, int *list_all, EvictPlan *plan, unsigned int *status) {
    extern __shared__ unsigned s_key[];
    __shared__ int hist[kDigits][kBins], warp_tot[32], s_digit, s_above;
    __shared__ int2 s_warp[kSelWarps];  // kept for certain, equal to the threshold: a warp's
    __shared__ int2 s_block;            // the block's
    __shared__ int s_first;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nh = blockIdx.x / ranks, n = nh / c.Hkv, h = nh - n * c.Hkv;
    int *list = list_all + (size_t)nh * stride;
    allow_next_launch();
    const int raw = c.lens[n];
    int len = checked_len(c, n, status);
    if (min(len, budget) > to.cap) {
        record_status(status, GDN2_ERR_INVALID_ARG);
        len = 0;
    }
    if (len <= budget) {
        for (int j = rank * kSelThreads + tid; j < stride; j += ranks * kSelThreads) list[j] = j < len ? j : -1;
        if (rank == 0 && tid == 0) plan[nh] = EvictPlan{in_place ? len : 0, in_place && raw != len ? -1 : len};
        return;
    }
    const int lo = sink, hi = len - recent, T = budget - sink - recent;  // T < hi - lo
    for (int j = rank * kSelThreads + tid; j < sink; j += ranks * kSelThreads) list[j] = j;
    for (int j = rank * kSelThreads + tid; j < recent; j += ranks * kSelThreads) list[budget - recent + j] = hi + j;
    if (T == 0) {
        if (rank == 0 && tid == 0) plan[nh] = EvictPlan{in_place ? sink : 0, budget};
        return;
    }
    const int per = (hi - lo + ranks - 1) / ranks, a = min(hi, lo + rank * per), b = min(hi, a + per);
    const bool held = per <= slots;
    auto key = [&](int j) { return held ? s_key[j - a] : key_at(c, n, h, j, status); };
    for (int x = tid; x < kDigits * kBins; x += kSelThreads) (&hist[0][0])[x] = 0;
    if (tid == 0) s_first = len;
    if (held) {
#pragma unroll 8
        for (int j = a + tid; j < b; j += kSelThreads) s_key[j - a] = key_at(c, n, h, j, status);
    }
    __syncthreads();
    unsigned prefix = 0, mask = 0;
    int need = T;
#pragma unroll
    for (int d = 0; d < kDigits; ++d) {
        const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, width = d == 2 ? 10 : 11;
        for (int j = a + tid; j < b; j += kSelThreads) {
            const unsigned k = key(j);
            if ((k & mask) == prefix) atomicAdd(&hist[d][(k >> shift) & ((1u << width) - 1)], 1);
        }
        cluster.sync();
        // thread t: the t-th pair of digits from the top
        const int top = kBins - 1 - 2 * tid;
        int c1 = 0, c0 = 0;
        for (int r = 0; r < ranks; ++r) {
            const int2 x = *reinterpret_cast<const int2 *>(cluster.map_shared_rank(&hist[d][top - 1], r));
            c0 += x.x;
            c1 += x.y;
        }
        const int inc = block_scan(c0 + c1, warp_tot), above = inc - c0 - c1;
        if (above < need && need <= inc) {
            s_digit = above + c1 >= need ? top : top - 1;
            s_above = above + c1 >= need ? above : above + c1;
        }
        __syncthreads();
        prefix |= (unsigned)s_digit << shift;
        mask |= ((1u << width) - 1) << shift;
        need -= s_above;
        __syncthreads();  // both have been read
    }
    // all keys above `prefix` stay, and the first `need` of those equal to it.
    // Each warp takes a contiguous piece of the slice: first it counts.
    const int piece = ((b - a + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
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
    for (int w = 0; w < kSelWarps; ++w) {
        const int2 x = s_warp[w];
        if (w == warp) cnt = before;
        before.x += x.x;
        before.y += x.y;
    }
    if (tid == 0) s_block = before;
    cluster.sync();
    for (int r = 0; r < rank; ++r) {
        const int2 x = *cluster.map_shared_rank(&s_block, r);
        cnt.x += x.x;
        cnt.y += x.y;
    }
    int first = len;  // the first token that goes: up to there no row moves
    const unsigned below = (1u << lane) - 1;
    for (int j0 = wa; j0 < wb; j0 += 32) {
        const int j = j0 + lane;
        const unsigned k = j < wb ? key(j) : 0u;
        const unsigned gt = __ballot_sync(0xffffffffu, j < wb && k > prefix);
        const unsigned eq = __ballot_sync(0xffffffffu, j < wb && k == prefix);
        if (j < wb) {
            const int e = cnt.y + __popc(eq & below);
            if (k > prefix || (k == prefix && e < need)) list[sink + cnt.x + __popc(gt & below) + min(e, need)] = j;
            else first = min(first, j);
        }
        cnt.x += __popc(gt);
        cnt.y += __popc(eq);
    }
    if (first < len) atomicMin(&s_first, first);
    cluster.sync();
    if (rank == 0 && tid == 0) {
        for (int r = 0; r < ranks; ++r) first = min(first, *cluster.map_shared_rank(&s_first, r));
        plan[nh] = EvictPlan{in_place ? first : 0, budget};
    }
    cluster.sync();  // no block ends while another reads its memory
}

// Into another cache: the kept rows in any order.  A block carries kRows rows
// of one (sequence, head) at a time, k and v, a thread the same 16-byte piece
// of kDeep rows of each.
constexpr int kDeep = 4;
__global__ void __launch_bounds__(kMoveThreads)
evict_copy_kernel(const PagedView c, const PagedView to, int stride, int chunks, const int *list_all,
                  const EvictPlan *plan, unsigned int *status) {
    const int pieces = c.d * c.es / 16, at_once = kMoveThreads / pieces;
    const int piece = threadIdx.x % pieces, r = threadIdx.x / pieces;
    const long long total = (long long)c.N * c.Hkv * chunks;
    wait_for_previous();
    for (long long x = blockIdx.x; x < total; x += gridDim.x) {
        const int nh = (int)(x / chunks), chunk = (int)(x - (long long)nh * chunks);
        const int n = nh / c.Hkv, h = nh - n * c.Hkv, count = plan[nh].count;
        const int *list = list_all + (size_t)nh * stride;
        const long long i0 = (long long)chunk * at_once * kDeep + r;
        uint4 k[kDeep], v[kDeep];
        float w[kDeep];
        long long dst[kDeep];
        size_t wd[kDeep];
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            const long long i = i0 + u * at_once;
            dst[u] = -1;
            if (i >= count) continue;
            int entry, slot, entry2, slot2;
            page_slot(c, list[i], entry, slot);
            page_slot(to, (int)i, entry2, slot2);
            const int page = page_of(c, n, entry), page2 = page_of(to, n, entry2);
            if (page < 0 || page2 < 0) {
                record_status(status, GDN2_ERR_INVALID_ARG);
                continue;
            }
            const long long from = row_off(c, page, slot, h) + piece * 16;
            k[u] = *reinterpret_cast<const uint4 *>(c.k + from);
            v[u] = *reinterpret_cast<const uint4 *>(c.v + from);
            if (piece == 0) w[u] = c.w[weight_off(c, page, slot, h)];
            dst[u] = row_off(to, page2, slot2, h) + piece * 16;
            wd[u] = weight_off(to, page2, slot2, h);
        }
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            if (dst[u] < 0) continue;
            *reinterpret_cast<uint4 *>(to.k + dst[u]) = k[u];
            *reinterpret_cast<uint4 *>(to.v + dst[u]) = v[u];
            if (piece == 0) to.w[wd[u]] = w[u];
        }
        if (h == 0 && chunk == 0 && threadIdx.x == 0) to.lens[n] = count;
    }
}

// In place.  Block (n h, column): 16 LANES bytes of every row of k or of v, the
// kept tokens in order, a batch ahead in registers.  Row i is read from
// list[i] >= i, so a batch overwrites only rows that it or earlier batches
// have read, and columns need no agreement between blocks.  The fewer
// (sequence, head) pairs there are, the narrower the columns, to have blocks.
constexpr int kBatch = 8;
template <int LANES>
__global__ void __launch_bounds__(kMoveThreads)
evict_shift_kernel(const PagedView c, int stride, const int *list_all, const EvictPlan *plan, unsigned int *status) {
    constexpr int kStep = kMoveThreads / LANES;
    const int columns = c.d * c.es / (16 * LANES);
    const int nh = blockIdx.x / (2 * columns), col = blockIdx.x % (2 * columns);
    const int n = nh / c.Hkv, h = nh - n * c.Hkv;
    wait_for_previous();
    const EvictPlan p = plan[nh];
    const int *list = list_all + (size_t)nh * stride;
    const int lane = threadIdx.x % LANES, r = threadIdx.x / LANES;
    char *pool = (col < columns ? c.k : c.v) + (size_t)(col % columns) * (16 * LANES) + lane * 16;
    const bool weights = col == 0 && lane == 0;
    uint4 x[kBatch], x2[kBatch];
    float w[kBatch], w2[kBatch];
    unsigned ok = 0, ok2 = 0;
    auto load = [&](int i0, uint4 *y, float *wy, unsigned &have) {
        have = 0;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = i0 + u * kStep + r;
            if (i >= p.count) continue;
            int entry, slot;
            page_slot(c, list[i], entry, slot);
            const int page = page_of(c, n, entry);
            if (page < 0) {
                record_status(status, GDN2_ERR_INVALID_ARG);
                continue;
            }
            y[u] = *reinterpret_cast<const uint4 *>(pool + row_off(c, page, slot, h));
            if (weights) wy[u] = c.w[weight_off(c, page, slot, h)];
            have |= 1u << u;
        }
    };
    load(p.first, x, w, ok);
    for (int i0 = p.first; i0 < p.count; i0 += kStep * kBatch) {
        if (i0 + kStep * kBatch < p.count) load(i0 + kStep * kBatch, x2, w2, ok2);
        else ok2 = 0;
        __syncthreads();  // the block has read this batch and the next before it writes
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (!(ok >> u & 1u)) continue;
            int entry, slot;
            page_slot(c, i0 + u * kStep + r, entry, slot);
            const int page = page_of(c, n, entry);
            if (page < 0) {
                record_status(status, GDN2_ERR_INVALID_ARG);
                continue;
            }
            *reinterpret_cast<uint4 *>(pool + row_off(c, page, slot, h)) = x[u];
            if (weights) c.w[weight_off(c, page, slot, h)] = w[u];
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            x[u] = x2[u];
            w[u] = w2[u];
        }
        ok = ok2;
    }
    if (h == 0 && col == 0 && threadIdx.x == 0 && p.count >= 0) c.lens[n] = p.count;
}

// entries of a list in the workspace
static int list_stride(const PagedView &c, int budget) { return budget < c.cap ? budget : c.cap; }

size_t evict_ws_bytes(const PagedView &c, int budget) {
    const size_t nh = (size_t)c.N * c.Hkv;
    return align256(nh * sizeof(EvictPlan)) + align256(nh * list_stride(c, budget) * sizeof(int));
}

template <int LANES>
static cudaError_t shift_launch(const PagedView &c, int stride, const int *list, const EvictPlan *plan,
                                unsigned int *status, cudaStream_t s) {
    return launch_behind(K_EVICT_MOVE, evict_shift_kernel<LANES>, c.N * c.Hkv * 2 * (c.d * c.es / (16 * LANES)),
                         kMoveThreads, 0, s, c, stride, list, plan, status);
}

cudaError_t evict_launch(const PagedView &src, const PagedView &dst, bool in_place, int budget, int sink,
                         int recent, int *kept, void *ws, unsigned int *status, cudaStream_t s) {
    const int nh = src.N * src.Hkv;
    EvictPlan *plan = static_cast<EvictPlan *>(ws);
    const int stride = kept ? budget : list_stride(src, budget);
    int *list = kept ? kept : at<int>(ws, align256((size_t)nh * sizeof(EvictPlan)));
    // blocks of a cluster: until a slice is 4096 tokens or the GPU is full
    int ranks = 1;
    while (ranks < 8 && src.cap / ranks > 4096 && (long long)nh * ranks < sm_count()) ranks *= 2;
    const int slots = (int)(((long long)src.cap + ranks - 1) / ranks < kMaxKeys ? (src.cap + ranks - 1) / ranks : kMaxKeys);
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxKeys * 4);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(nh * ranks);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = slots * 4;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    launch_begin(K_EVICT_SELECT, s);
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel, src, dst, (int)in_place, budget, sink, recent, slots, stride, list, plan, status);
    launch_end(K_EVICT_SELECT, s);
    if (e != cudaSuccess) return e;
    if (in_place) {
        const long long narrow = (long long)nh * 2 * (src.d * src.es / 16);  // blocks of 16-byte columns
        if (narrow >= 16LL * sm_count()) return shift_launch<4>(src, stride, list, plan, status, s);
        if (narrow >= 4LL * sm_count()) return shift_launch<2>(src, stride, list, plan, status, s);
        return shift_launch<1>(src, stride, list, plan, status, s);
    }
    const int rows = kMoveThreads / (src.d * src.es / 16) * kDeep, chunks = (stride + rows - 1) / rows;
    const long long blocks = (long long)nh * chunks, most = 64LL * sm_count();
    return launch_behind(K_EVICT_MOVE, evict_copy_kernel, (int)(blocks < most ? blocks : most), kMoveThreads, 0, s, src,
                         dst, stride, chunks, list, plan, status);
}

}  // namespace gdn2
