// Appending tokens to the paged key-value cache.
//
// Token i of sequence n's new ones goes to position len_n + i: a copy of
// H_kv d elements of k and of v, contiguous in the source, to one row per head
// in the token's page.  Nothing is computed, so the call is bound by the copy
// (2 T H_kv d elements read and written) or, for one token a sequence, by the
// launch.

#include "paged.cuh"

namespace gdn2 {

constexpr int kAppThreads = 256;
constexpr int kAppTokens = 64;  // most tokens of one block
// Bytes of k and v for one block: 17.5K prompt tokens of 16 KB take 48.6 us with
// 32 KB a block, 47.5 with 16 KB, 49 with 48 KB, 58 with 112 KB, 51 with 256 KB.
constexpr int kAppBytes = 32 << 10;

// cu[0 .. N] rises from 0 to T; every thread of the block gets the answer
__device__ __forceinline__ bool table_ok(const int *cu, int N, int T) {
    int bad = 0;
    for (int n = threadIdx.x; n < N; n += blockDim.x) bad |= cu[n + 1] < cu[n];
    if (threadIdx.x == 0) bad |= cu[0] != 0 || cu[N] != T;
    return !__syncthreads_or(bad);
}

// the lengths with the new tokens (`ok`: cu is as it should be)
__device__ __forceinline__ void write_lens(const PagedView &c, const int *cu, bool ok, int *lens_out, unsigned int *status) {
    for (int n = threadIdx.x; n < c.N; n += blockDim.x) {
        const int len = c.lens[n], count = ok ? cu[n + 1] - cu[n] : 0;
        const bool fits = len >= 0 && len <= c.cap - count;
        if (!fits) record_status(status, GDN2_ERR_INVALID_ARG);
        lens_out[n] = fits ? len + count : len;
    }
}

// Block b copies tokens [b per, b per + per).  Its first threads find each
// token's place (packed: a binary search in cu); then all threads copy 16-byte
// pieces, consecutive threads consecutive pieces of one token.
__global__ void __launch_bounds__(kAppThreads)
kv_append_kernel(const PagedView c, const uint4 *k, const uint4 *v, const int *cu, int T, int per,
                 int *lens_out, unsigned int *status) {
    __shared__ long long s_off[kAppTokens];  // byte offset of head 0's row, -1: not written
    __shared__ size_t s_w[kAppTokens];
    const int t0 = blockIdx.x * per, nt = min(per, T - t0), tid = threadIdx.x;
    follow_previous();
    if (cu && !table_ok(cu, c.N, T)) {
        if (tid == 0) record_status(status, GDN2_ERR_INVALID_ARG);
        if (lens_out != c.lens && blockIdx.x == 0) write_lens(c, cu, false, lens_out, status);
        return;
    }
    if (tid < nt) {
        const int t = t0 + tid;
        int n = t, i = 0, count = 1;
        if (cu) {  // the last sequence that starts at or before t and is not empty
            int lo = 0, hi = c.N;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= t) lo = mid;
                else hi = mid;
            }
            n = lo;
            i = t - cu[n];
            count = cu[n + 1] - cu[n];
        }
        const int len = c.lens[n];
        const bool fits = len >= 0 && len <= c.cap - count;
        int entry, slot, page = -1;
        if (fits) {
            page_slot(c, len + i, entry, slot);
            page = page_of(c, n, entry);
        }
        if (page < 0) record_status(status, GDN2_ERR_INVALID_ARG);
        s_off[tid] = page < 0 ? -1 : row_off(c, page, slot, 0);
        s_w[tid] = page < 0 ? 0 : weight_off(c, page, slot, 0);
        // one token a sequence: no other block reads this length
        if (!cu) lens_out[n] = fits ? len + 1 : len;
    }
    // packed, and the new lengths go to a place of their own: block 0 writes them
    if (cu && lens_out != c.lens && blockIdx.x == 0) write_lens(c, cu, true, lens_out, status);
    __syncthreads();
    const int rv = c.d * c.es / 16, tv = c.Hkv * rv;  // 16-byte pieces of a row, of a token
#pragma unroll 4
    for (int x = tid; x < nt * tv; x += kAppThreads) {
        const int t = x / tv, y = x - t * tv, h = y / rv, piece = y - h * rv;
        if (s_off[t] < 0) continue;
        const long long at = s_off[t] + h * c.sh + piece * 16;
        const size_t from = (size_t)(t0 + t) * tv + y;
        const uint4 a = k[from], b = v[from];
        *reinterpret_cast<uint4 *>(c.k + at) = a;
        *reinterpret_cast<uint4 *>(c.v + at) = b;
    }
    if (c.w)
        for (int x = tid; x < nt * c.Hkv; x += kAppThreads) {
            const int t = x / c.Hkv, h = x - t * c.Hkv;
            if (s_off[t] >= 0) c.w[s_w[t] + (size_t)h * c.page] = 0.f;
        }
}

// In place, the lengths after a packed append wait until its rows are written:
// the copy still reads the old ones.  (And without new tokens there is no copy.)
__global__ void __launch_bounds__(1024)
kv_lens_kernel(const PagedView c, const int *cu, int T, int *lens_out, unsigned int *status) {
    follow_previous();
    const bool ok = table_ok(cu, c.N, T);
    if (!ok && threadIdx.x == 0) record_status(status, GDN2_ERR_INVALID_ARG);
    write_lens(c, cu, ok, lens_out, status);
}

cudaError_t kv_append_launch(const PagedView &c, const void *k, const void *v, const int *cu, int T,
                             int *lens_out, unsigned int *status, cudaStream_t s) {
    if (T > 0) {
        const long long token = 2LL * c.Hkv * c.d * c.es, fill = T / (4 * sm_count());  // fewer tokens fill the GPU
        long long want = kAppBytes / token;
        want = want < fill ? want : fill;
        const int per = want < 1 ? 1 : (want > kAppTokens ? kAppTokens : (int)want);
        const cudaError_t e = launch_behind(K_KV_APPEND, kv_append_kernel, (T + per - 1) / per, kAppThreads, 0, s, c,
                                            static_cast<const uint4 *>(k), static_cast<const uint4 *>(v), cu, T, per,
                                            lens_out, status);
        if (e != cudaSuccess) return e;
    }
    return cu && (T == 0 || lens_out == c.lens)
               ? launch_behind(K_KV_LENS, kv_lens_kernel, 1, 1024, 0, s, c, cu, T, lens_out, status)
               : cudaSuccess;
}

}  // namespace gdn2
