// The paged key-value cache as its kernels see it, and the launchers of the
// calls on it (gdn2_kv_append, gdn2_attn_decode_step, gdn2_kv_evict).
#pragma once

#include "common.cuh"

namespace gdn2 {

// kernel kinds of these calls, behind common.cuh's
enum PagedKernelKind {
    K_KV_APPEND = K_KINDS, K_KV_LENS, K_ATTN_SPLIT, K_ATTN_FINISH, K_EVICT_SELECT, K_EVICT_MOVE, K_ALL_KINDS
};
// device address of the status word in the current context (nullptr on failure)
unsigned int *status_word();

constexpr int kMaxHeadGroup = 256;  // most query heads of a key-value head

struct PagedView {
    char *k, *v;
    float *w;          // [num_pages, Hkv, page] or nullptr
    const int *table;  // [N, max_pages]
    int *lens;         // [N]
    long long sp, ss, sh;  // strides in bytes; 0 along an axis of extent 1
    int num_pages, page, page_shift;  // page_shift: log2(page), or -1
    int max_pages, N, Hkv, d, cap;    // cap = max_pages * page
    int es;                           // bytes of an element
};

// token j -> (entry of the sequence's table row, slot in the page)
__device__ __forceinline__ void page_slot(const PagedView &c, int j, int &entry, int &slot) {
    if (c.page_shift >= 0) {
        entry = j >> c.page_shift;
        slot = j & (c.page - 1);
    } else {
        entry = j / c.page;
        slot = j - entry * c.page;
    }
}
// the page of table entry (n, entry), or -1 where the table names none
__device__ __forceinline__ int page_of(const PagedView &c, int n, int entry) {
    const int p = c.table[(size_t)n * c.max_pages + entry];
    return (unsigned)p < (unsigned)c.num_pages ? p : -1;
}
__device__ __forceinline__ long long row_off(const PagedView &c, int page, int slot, int h) {
    return page * c.sp + slot * c.ss + h * c.sh;
}
__device__ __forceinline__ size_t weight_off(const PagedView &c, int page, int slot, int h) {
    return ((size_t)page * c.Hkv + h) * c.page + slot;
}
// a sequence's length; 0, with the status recorded, where it is out of range
__device__ __forceinline__ int checked_len(const PagedView &c, int n, unsigned int *status) {
    const int len = c.lens[n];
    if (len >= 0 && len <= c.cap) return len;
    record_status(status, GDN2_ERR_INVALID_ARG);
    return 0;
}

// The kernels here follow each other on the stream without the launch between
// them: every kernel first waits until the one before it has finished and its
// writes are visible, whatever kernel that is, and then lets the next one's
// blocks come up, which wait in their turn.  Called by every thread, before
// any access to global memory.
__device__ __forceinline__ void follow_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
}
// launches a kernel whose blocks come up while the one before it still runs
// (they wait for it themselves), in clusters of `ranks` blocks
template <typename... P, typename... A>
static cudaError_t launch_clusters(int kind, void (*kernel)(P...), int ranks, int grid, int threads, int smem,
                                   cudaStream_t s, A... args) {
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = ranks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = ranks > 1 ? 2 : 1;
    launch_begin(kind, s);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
    launch_end(kind, s);
    return e;
}
template <typename... P, typename... A>
static cudaError_t launch_behind(int kind, void (*kernel)(P...), int grid, int threads, int smem, cudaStream_t s, A... args) {
    return launch_clusters(kind, kernel, 1, grid, threads, smem, s, args...);
}

cudaError_t kv_append_launch(const PagedView &c, const void *k, const void *v, const int *cu, int T,
                             int *lens_out, unsigned int *status, cudaStream_t s);
bool attn_countable(const PagedView &c, int H);
size_t attn_ws_bytes(const PagedView &c, int H, int add_weights);
cudaError_t attn_launch(const PagedView &c, const void *q, void *o, float *lse, int H, float scale,
                        int window, int add_weights, void *ws, unsigned int *status, cudaStream_t s);
bool evict_countable(const PagedView &c, int budget);
size_t evict_ws_bytes(const PagedView &c, int budget);
constexpr long long kEvictWaitClocks = 4000000000LL;  // about two seconds
// wait_clocks, ticket: the in-place form's longest wait, and the first ticket
// that it draws (the self-test leaves the chunks of earlier ones unread)
cudaError_t evict_launch(const PagedView &src, const PagedView &dst, bool in_place, int budget, int sink,
                         int recent, int *kept, void *ws, unsigned int *status, cudaStream_t s,
                         long long wait_clocks = kEvictWaitClocks, int ticket = 0);

}  // namespace gdn2
