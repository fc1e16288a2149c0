// Eviction from the paged cache by accumulated attention weight.
//
// Per (sequence, key-value head): of the tokens between the protected first
// `sink` and last `recent`, the T = budget - sink - recent heaviest stay.
// evict_select finds the T-th largest weight by radix selection on 32-bit
// keys whose unsigned order is the floats' order (four passes of 8 bits: a
// histogram of the digit among the keys that share the prefix found so far),
// then lists the kept tokens in their order.  evict_move carries the rows.

#include "paged.cuh"

namespace gdn2 {

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 8;       // rows a thread holds at once
constexpr int kMovePiece = 64;     // bytes of a row that one block carries

struct EvictPlan {
    int first, count;  // rows [first, count) are written
};

// larger float <=> larger key; -0 as +0, NaN below everything
__device__ __forceinline__ unsigned weight_key(float x) {
    if (x != x) return 0u;
    const unsigned u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float weight_at(const PagedView &c, int n, int h, int j, unsigned int *status) {
    int entry, slot;
    page_slot(c, j, entry, slot);
    const int page = page_of(c, n, entry);
    if (page < 0) {
        record_status(status, GDN2_ERR_INVALID_ARG);
        return __uint_as_float(0x7fc00000u);
    }
    return c.w[weight_off(c, page, slot, h)];
}

// inclusive scan over the block; `total` for every thread
__device__ __forceinline__ int block_scan(int x, int *warp_tot, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) warp_tot[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int t = warp_tot[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, t, off);
            if (lane >= off) t += y;
        }
        warp_tot[lane] = t;
    }
    __syncthreads();
    const int before = warp ? warp_tot[warp - 1] : 0;
    total = warp_tot[31];
    __syncthreads();
    return x + before;
}

__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(const PagedView c, const PagedView to, int in_place, int budget, int sink, int recent,
                    int *list_all, EvictPlan *plan, unsigned int *status) {
    __shared__ int hist[256], warp_tot[32], s_digit, s_above, s_first;
    const int tid = threadIdx.x, n = blockIdx.x / c.Hkv, h = blockIdx.x % c.Hkv;
    int *list = list_all + (size_t)blockIdx.x * budget;
    const int raw = c.lens[n];
    int len = checked_len(c, n, status);
    const bool fits = min(len, budget) <= to.cap;
    if (!fits) {
        record_status(status, GDN2_ERR_INVALID_ARG);
        len = 0;
    }
    if (len <= budget) {
        for (int j = tid; j < budget; j += kSelThreads) list[j] = j < len ? j : -1;
        // -1: the length stays as it is too
        if (tid == 0) plan[blockIdx.x] = EvictPlan{in_place ? len : 0, in_place && raw != len ? -1 : len};
        return;
    }
    const int lo = sink, hi = len - recent;
    int need = budget - sink - recent;  // < hi - lo
    unsigned prefix = 0, mask = 0;
    if (tid == 0) s_first = budget;
    if (need > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int j = lo + tid; j < hi; j += kSelThreads) {
                const unsigned key = weight_key(weight_at(c, n, h, j, status));
                if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
            }
            __syncthreads();
            if (tid == 0) {  // the digit in which the need-th largest lies
                int above = 0, b = 255;
                while (b > 0 && above + hist[b] < need) above += hist[b--];
                s_digit = b;
                s_above = above;
            }
            __syncthreads();
            prefix |= (unsigned)s_digit << shift;
            mask |= 255u << shift;
            need -= s_above;
            __syncthreads();
        }
    }
    // `need` of the keys equal to `prefix` stay, the earliest; all above it do
    const int ties = need;
    const bool none = budget - sink - recent == 0;
    for (int j = tid; j < sink; j += kSelThreads) list[j] = j;
    for (int j = tid; j < recent; j += kSelThreads) list[budget - recent + j] = hi + j;
    int above = 0, equal = 0, first = budget;
    for (int j0 = lo; j0 < hi && !none; j0 += kSelThreads) {
        const int j = j0 + tid;
        int gt = 0, eq = 0;
        if (j < hi) {
            const unsigned key = weight_key(weight_at(c, n, h, j, status));
            gt = key > prefix;
            eq = key == prefix;
        }
        int total;
        const int inc = block_scan(gt | eq << 16, warp_tot, total);
        const int g = above + (inc & 0xffff) - gt, e = equal + (inc >> 16) - eq;
        if (gt || (eq && e < ties)) {
            const int at = sink + g + min(e, ties);
            list[at] = j;
            if (at != j) first = min(first, at);
        }
        above += total & 0xffff;
        equal += total >> 16;
    }
    if (recent > 0) first = min(first, budget - recent);
    __syncthreads();
    atomicMin(&s_first, first);
    __syncthreads();
    if (tid == 0) plan[blockIdx.x] = EvictPlan{in_place ? s_first : 0, budget};
}

// Block (piece, n h): one 64-byte piece of the rows of k or of v, for all kept
// tokens of a (sequence, head), in order.  In place this is safe without any
// agreement between blocks: row i is read from list[i] >= i, so a batch of
// rows only overwrites what its own and earlier batches read.
__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(const PagedView c, const PagedView to, int budget, const int *list_all, const EvictPlan *plan,
                  unsigned int *status) {
    const int nh = blockIdx.x, n = nh / c.Hkv, h = nh % c.Hkv, pieces = c.d * c.es / kMovePiece;
    const int which = blockIdx.y / pieces, piece = blockIdx.y % pieces;
    const EvictPlan p = plan[nh];
    const int *list = list_all + (size_t)nh * budget;
    const int lane = threadIdx.x & 3, r = threadIdx.x >> 2;
    const char *src = which ? c.v : c.k;
    char *dst = which ? to.v : to.k;
    const bool weights = blockIdx.y == 0 && lane == 0;
    constexpr int kStep = kMoveThreads / 4;
    for (int i0 = p.first; i0 < p.count; i0 += kStep * kMoveRows) {
        uint4 x[kMoveRows];
        float w[kMoveRows];
        bool ok[kMoveRows];
#pragma unroll
        for (int u = 0; u < kMoveRows; ++u) {
            const int i = i0 + u * kStep + r;
            ok[u] = false;
            if (i < p.count) {
                int entry, slot;
                page_slot(c, list[i], entry, slot);
                const int page = page_of(c, n, entry);
                ok[u] = page >= 0;
                if (ok[u]) {
                    x[u] = *reinterpret_cast<const uint4 *>(src + row_off(c, page, slot, h) + piece * kMovePiece + lane * 16);
                    if (weights) w[u] = c.w[weight_off(c, page, slot, h)];
                } else record_status(status, GDN2_ERR_INVALID_ARG);
            }
        }
        __syncthreads();  // the batch is read before any of it is written
#pragma unroll
        for (int u = 0; u < kMoveRows; ++u) {
            if (!ok[u]) continue;
            int entry, slot;
            page_slot(to, i0 + u * kStep + r, entry, slot);
            const int page = page_of(to, n, entry);
            if (page < 0) {
                record_status(status, GDN2_ERR_INVALID_ARG);
                continue;
            }
            *reinterpret_cast<uint4 *>(dst + row_off(to, page, slot, h) + piece * kMovePiece + lane * 16) = x[u];
            if (weights) to.w[weight_off(to, page, slot, h)] = w[u];
        }
    }
    if (h == 0 && blockIdx.y == 0 && threadIdx.x == 0 && p.count >= 0) to.lens[n] = p.count;
}

size_t evict_ws_bytes(const PagedView &c, int budget) {
    const size_t nh = (size_t)c.N * c.Hkv;
    return align256(nh * sizeof(EvictPlan)) + align256(nh * budget * sizeof(int));
}

cudaError_t evict_launch(const PagedView &src, const PagedView &dst, bool in_place, int budget, int sink,
                         int recent, int *kept, void *ws, unsigned int *status, cudaStream_t s) {
    const int nh = src.N * src.Hkv;
    EvictPlan *plan = static_cast<EvictPlan *>(ws);
    int *list = kept ? kept : at<int>(ws, align256((size_t)nh * sizeof(EvictPlan)));
    launch_begin(K_EVICT_SELECT, s);
    evict_select_kernel<<<nh, kSelThreads, 0, s>>>(src, dst, in_place, budget, sink, recent, list, plan, status);
    launch_end(K_EVICT_SELECT, s);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    launch_begin(K_EVICT_MOVE, s);
    evict_move_kernel<<<dim3(nh, 2 * src.d * src.es / kMovePiece), kMoveThreads, 0, s>>>(src, dst, budget, list, plan,
                                                                                       status);
    launch_end(K_EVICT_MOVE, s);
    return cudaGetLastError();
}

}  // namespace gdn2
