// Softmax attention of one new token a sequence over the paged cache.
//
//   s_j = scale <q, k_j>,  o = sum_j e^(s_j - lse) v_j,  lse = log sum_j e^(s_j)
//
// One block per (sequence, key-value head) walks the cached tokens in tiles of
// 128 with a running maximum m and sum l: a tile's scores raise m, and what
// was summed before is scaled by e^(m_old - m_new).

#include "paged.cuh"

namespace gdn2 {

constexpr int kAttnThreads = 128;

template <typename E>
__global__ void __launch_bounds__(kAttnThreads)
attn_kernel(const PagedView c, const E *q, E *o, float *lse, int H, float scale, int window, int add_weights,
            unsigned int *status) {
    __shared__ float sq[kMaxD], sp[kAttnThreads], red[kAttnThreads / 32];
    __shared__ long long soff[kAttnThreads];
    const int tid = threadIdx.x, n = blockIdx.x / c.Hkv, kvh = blockIdx.x % c.Hkv, G = H / c.Hkv;
    const int len = checked_len(c, n, status), first = window > 0 && len > window ? len - window : 0;
    for (int g = 0; g < G; ++g) {
        const size_t row = ((size_t)n * H + kvh * G + g) * c.d;
        __syncthreads();
        if (tid < c.d) sq[tid] = ldx(q, row + tid);
        __syncthreads();
        float m = -INFINITY, l = 0.f, acc = 0.f, L = 0.f;
        for (int pass = 0; pass <= add_weights; ++pass) {
            for (int j0 = first; j0 < len; j0 += kAttnThreads) {
                const int j = j0 + tid;
                float x = -INFINITY;
                long long off = -1;
                size_t wo = 0;
                if (j < len) {
                    int entry, slot;
                    page_slot(c, j, entry, slot);
                    const int page = page_of(c, n, entry);
                    if (page < 0) record_status(status, GDN2_ERR_INVALID_ARG);
                    else {
                        off = row_off(c, page, slot, kvh);
                        wo = weight_off(c, page, slot, kvh);
                        const E *kr = reinterpret_cast<const E *>(c.k + off);
                        x = 0.f;
                        for (int i = 0; i < c.d; ++i) x += sq[i] * ldx(kr, i);
                        x *= scale;
                    }
                }
                if (pass == 1) {
                    if (off >= 0) atomicAdd(c.w + wo, expf(x - L));
                    continue;
                }
                float mx = x;
                for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
                if ((tid & 31) == 0) red[tid >> 5] = mx;
                __syncthreads();
                mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
                const float mn = fmaxf(m, mx), base = mn == -INFINITY ? 0.f : mn;
                sp[tid] = expf(x - base);
                soff[tid] = off;
                __syncthreads();
                const float f = expf(m - base);
                l *= f;
                acc *= f;
                const int cnt = min(kAttnThreads, len - j0);
                for (int i = 0; i < cnt; ++i) {
                    l += sp[i];
                    if (tid < c.d && soff[i] >= 0) acc += sp[i] * ldx(reinterpret_cast<const E *>(c.v + soff[i]), tid);
                }
                m = mn;
                __syncthreads();
            }
            if (pass == 0) L = l > 0.f ? m + logf(l) : (l == 0.f ? -INFINITY : l);
            if (l == 0.f) break;
        }
        if (tid < c.d) stx(o, row + tid, l == 0.f ? 0.f : acc / l);
        if (lse && tid == 0) lse[(size_t)n * H + kvh * G + g] = L;
    }
}

size_t attn_ws_bytes(const PagedView &, int, int) { return 256; }

cudaError_t attn_launch(const PagedView &c, const void *q, void *o, float *lse, int H, float scale, int window,
                        int add_weights, void *, unsigned int *status, cudaStream_t s) {
    launch_begin(K_ATTN_SPLIT, s);
    if (c.es == 2)
        attn_kernel<<<c.N * c.Hkv, kAttnThreads, 0, s>>>(c, static_cast<const __nv_bfloat16 *>(q),
                                                         static_cast<__nv_bfloat16 *>(o), lse, H, scale, window,
                                                         add_weights, status);
    else
        attn_kernel<<<c.N * c.Hkv, kAttnThreads, 0, s>>>(c, static_cast<const float *>(q), static_cast<float *>(o),
                                                         lse, H, scale, window, add_weights, status);
    launch_end(K_ATTN_SPLIT, s);
    return cudaGetLastError();
}

}  // namespace gdn2
