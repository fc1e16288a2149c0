// Host side of the paged-cache calls in include/gdn2.h: argument checks,
// workspace sizes and launches.  No allocation, no synchronisation.

#include <math.h>
#include <stdint.h>

#include "paged.cuh"

using namespace gdn2;

namespace {

bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Checks what the descriptor says and fills the kernels' view of it.  A stride
// along an axis of extent 1 is not read (frameworks leave anything there).
gdn2_status make_view(PagedView &c, const gdn2_paged_kv *kv) {
    if (!kv) return GDN2_ERR_INVALID_ARG;
    if (kv->io != GDN2_IO_F32 && kv->io != GDN2_IO_BF16) return GDN2_ERR_INVALID_ARG;
    if (kv->num_pages < 1 || kv->page_size < 1 || kv->max_pages < 1 || kv->N < 1 || kv->H_kv < 1)
        return GDN2_ERR_INVALID_ARG;
    if (kv->d != 32 && kv->d != 64 && kv->d != 128) return GDN2_ERR_UNSUPPORTED;
    if ((long long)kv->max_pages * kv->page_size > 1LL << 30) return GDN2_ERR_UNSUPPORTED;  // token numbers are ints
    // one block per (sequence, head) in the calls that split no further
    if ((long long)kv->N * kv->H_kv > 0x7fffffffLL / 64) return GDN2_ERR_UNSUPPORTED;
    const int es = kv->io == GDN2_IO_BF16 ? 2 : 4;
    struct Axis { long long stride; int extent; } ax[3] = {{kv->stride_page, kv->num_pages},
                                                          {kv->stride_slot, kv->page_size},
                                                          {kv->stride_head, kv->H_kv}};
    for (Axis &a : ax) {
        if (a.extent == 1) a.stride = 0;
        else if (a.stride < kv->d || a.stride > (1LL << 40) || (a.stride * es) % 16 != 0) return GDN2_ERR_INVALID_ARG;
    }
    c.sp = ax[0].stride * es;
    c.ss = ax[1].stride * es;
    c.sh = ax[2].stride * es;
    // rows must not overlap: by rising stride, each axis steps over the ones before
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j + 1 < 3 - i; ++j)
            if (ax[j].stride > ax[j + 1].stride) { const Axis t = ax[j]; ax[j] = ax[j + 1]; ax[j + 1] = t; }
    long long reach = kv->d;  // elements that the axes so far span
    for (const Axis &a : ax) {
        if (a.extent == 1) continue;
        if (a.stride < reach) return GDN2_ERR_INVALID_ARG;
        if (a.stride > (1LL << 60) / a.extent) return GDN2_ERR_UNSUPPORTED;
        reach += a.stride * (a.extent - 1);
    }
    if (!kv->k || !kv->v || !aligned(kv->k, 16) || !aligned(kv->v, 16)) return GDN2_ERR_INVALID_ARG;
    if (!kv->block_table || !kv->seq_lens || !aligned(kv->block_table, 4) || !aligned(kv->seq_lens, 4) ||
        !aligned(kv->weight, 4))
        return GDN2_ERR_INVALID_ARG;
    c.k = static_cast<char *>(kv->k);
    c.v = static_cast<char *>(kv->v);
    c.w = kv->weight;
    c.table = kv->block_table;
    c.lens = kv->seq_lens;
    c.num_pages = kv->num_pages;
    c.page = kv->page_size;
    c.page_shift = -1;
    for (int b = 0; b < 31; ++b)
        if (kv->page_size == 1 << b) c.page_shift = b;
    c.max_pages = kv->max_pages;
    c.N = kv->N;
    c.Hkv = kv->H_kv;
    c.d = kv->d;
    c.cap = kv->max_pages * kv->page_size;
    c.es = es;
    return GDN2_OK;
}

gdn2_status check_heads(const PagedView &c, int H) {
    if (H < 1 || H % c.Hkv != 0) return GDN2_ERR_INVALID_ARG;
    return H / c.Hkv > kMaxHeadGroup || (long long)c.N * H > 0x7fffffffLL / 64 || !attn_countable(c, H) ? GDN2_ERR_UNSUPPORTED : GDN2_OK;
}

gdn2_status launched(cudaError_t e) {
    if (e == cudaSuccess) return GDN2_OK;
    cudaGetLastError();  // the caller has the status; a later call does not find the error again
    return GDN2_ERR_CUDA;
}

}  // namespace

extern "C" {

gdn2_status gdn2_kv_append(const gdn2_paged_kv *kv, const void *k, const void *v, const int *cu_seqlens,
                           int T, int *lens_out, gdn2_stream_t stream) {
    PagedView c;
    gdn2_status st = make_view(c, kv);
    if (st != GDN2_OK) return st;
    if (T < 0 || (!cu_seqlens && T != c.N)) return GDN2_ERR_INVALID_ARG;
    if (T > 0 && (!k || !v || !aligned(k, 16) || !aligned(v, 16))) return GDN2_ERR_INVALID_ARG;
    if (!lens_out || !aligned(lens_out, 4) || !aligned(cu_seqlens, 4)) return GDN2_ERR_INVALID_ARG;
    unsigned int *status = status_word();
    if (!status) return GDN2_ERR_CUDA;
    return launched(kv_append_launch(c, k, v, cu_seqlens, T, lens_out, status, (cudaStream_t)stream));
}

size_t gdn2_attn_decode_workspace_bytes(const gdn2_paged_kv *kv, int H, int add_weights) {
    PagedView c;
    if (make_view(c, kv) != GDN2_OK || check_heads(c, H) != GDN2_OK) return 0;
    return attn_ws_bytes(c, H, add_weights != 0);
}

gdn2_status gdn2_attn_decode_step(const gdn2_paged_kv *kv, const void *q, void *o, float *lse, int H,
                                  float scale, int window, int add_weights, void *ws, size_t ws_bytes,
                                  gdn2_stream_t stream) {
    PagedView c;
    gdn2_status st = make_view(c, kv);
    if (st != GDN2_OK) return st;
    if ((st = check_heads(c, H)) != GDN2_OK) return st;
    if (!q || !o || !aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4)) return GDN2_ERR_INVALID_ARG;
    // o in q's place is written after q has been read, unless the weights need q again
    const size_t bytes = (size_t)c.N * H * c.d * c.es;
    const uintptr_t qa = (uintptr_t)q, oa = (uintptr_t)o;
    if (qa < oa + bytes && oa < qa + bytes && (qa != oa || add_weights)) return GDN2_ERR_INVALID_ARG;
    if (window < 0 || !isfinite(scale * 1.5f)  /* with log2 e in it too */ || (add_weights && !c.w)) return GDN2_ERR_INVALID_ARG;
    if (!ws || !aligned(ws, 16) || ws_bytes < attn_ws_bytes(c, H, add_weights != 0)) return GDN2_ERR_WORKSPACE;
    unsigned int *status = status_word();
    if (!status) return GDN2_ERR_CUDA;
    return launched(attn_launch(c, q, o, lse, H, scale, window, add_weights != 0, ws, status, (cudaStream_t)stream));
}

size_t gdn2_kv_evict_workspace_bytes(const gdn2_paged_kv *kv, int budget) {
    PagedView c;
    if (make_view(c, kv) != GDN2_OK || budget < 1 || !evict_countable(c, budget)) return 0;
    return evict_ws_bytes(c, budget);
}

gdn2_status gdn2_kv_evict(const gdn2_paged_kv *kv, const gdn2_paged_kv *dst, int budget, int sink, int recent,
                          int *kept, void *ws, size_t ws_bytes, gdn2_stream_t stream) {
    PagedView c, to;
    gdn2_status st = make_view(c, kv);
    if (st != GDN2_OK) return st;
    to = c;
    if (dst) {
        if ((st = make_view(to, dst)) != GDN2_OK) return st;
        if (to.N != c.N || to.Hkv != c.Hkv || to.d != c.d || to.es != c.es || to.lens == c.lens || !to.w)
            return GDN2_ERR_INVALID_ARG;
    }
    if (!c.w || budget < 1 || sink < 0 || recent < 0 || (long long)sink + recent > budget || !aligned(kept, 4))
        return GDN2_ERR_INVALID_ARG;
    if (!evict_countable(c, budget)) return GDN2_ERR_UNSUPPORTED;
    // a kept list has `budget` entries, whatever the table reaches; the kernels count them in ints
    if (kept && budget > 1 << 30) return GDN2_ERR_UNSUPPORTED;
    if (!ws || !aligned(ws, 16) || ws_bytes < evict_ws_bytes(c, budget)) return GDN2_ERR_WORKSPACE;
    unsigned int *status = status_word();
    if (!status) return GDN2_ERR_CUDA;
    return launched(evict_launch(c, to, dst == nullptr, budget, sink, recent, kept, ws, status, (cudaStream_t)stream));
}

gdn2_status gdn2_selftest_evict_timeout(const gdn2_paged_kv *kv, int budget, void *ws, size_t ws_bytes,
                                        long long limit_cycles, gdn2_stream_t stream) {
    PagedView c;
    gdn2_status st = make_view(c, kv);
    if (st != GDN2_OK) return st;
    if (!c.w || budget < 1) return GDN2_ERR_INVALID_ARG;
    if (!evict_countable(c, budget)) return GDN2_ERR_UNSUPPORTED;
    if (!ws || !aligned(ws, 16) || ws_bytes < evict_ws_bytes(c, budget)) return GDN2_ERR_WORKSPACE;
    unsigned int *status = status_word();
    if (!status) return GDN2_ERR_CUDA;
    const long long limit = limit_cycles < 1000 ? 1000 : (limit_cycles > 4000000LL ? 4000000LL : limit_cycles);
    return launched(evict_launch(c, c, true, budget, 0, 0, nullptr, ws, status, (cudaStream_t)stream, limit, c.N * c.Hkv));
}

}  // extern "C"
