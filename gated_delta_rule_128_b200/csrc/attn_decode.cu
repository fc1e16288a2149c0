// Softmax attention of one new token a sequence over the paged cache.
//
//   s_j = scale <q, k_j>,  o = sum_j e^(s_j - lse) v_j,  lse = log sum_j e^(s_j)
//
// The call reads each cached k and v once (4 d bytes a token and head in bf16)
// for 4 d G flops, G query heads sharing them: at most a few flops a byte, so
// HBM bounds it and everything else has to stay out of the way.
//
// Work is cut into units of 64 tokens of one (sequence, key-value head, block
// of at most 16 query heads), numbered in that order; every block takes an
// equal run of consecutive units, whatever the sequences' lengths (the lengths
// are on the device, so each block finds its own run with a scan over them).
// Before each (sequence, head)'s units stand kLead empty ones, for the time
// that starting and merging it takes: without them a block that gets 28 short
// sequences needs twice as long as one with 28 units of a long one (48
// sequences of 1 to 1000 tokens, 16 heads: 60 us without them, 41 with them; 64
// of 1 to 4000: 195 and 180).  Times in this file are a call's on the GPU, in a
// captured graph; d = 128, bf16, inputs from HBM, where nothing else is said.
// A block walks the part of its run that lies in one (sequence, head) as a
// segment with a running maximum m, sum l and accumulator of e^(s - m) v.  A
// segment that covers the whole (sequence, head) leaves the result, one that
// does not leaves (m, l, acc) in the workspace; at most the first and the last
// of a block's segments are such parts.  attn_finish combines them:
//   m = max m_i,  o = sum e^(m_i - m) acc_i / sum e^(m_i - m) l_i.
// Exponents are in base 2 throughout (scale carries log2 e).  A running maximum
// stays within +-FLT_MAX, so that no difference of two of them, or of a score
// and one, is infinity less itself: scores of -inf sum to 0, and one of +inf to
// +inf, which the log-sum-exp keeps.
//
// Within a block each warp owns 16-token (float32, d = 128: 8-token) slices of
// its own: it copies their k and v rows into its ring of stages in shared
// memory with 16-byte asynchronous copies and works on them without a
// block-wide barrier; the four warps' (m, l, acc) meet once a segment.  The
// copies run ahead across segments, so a merge does not empty the ring.

#include <float.h>

#include "paged.cuh"
#include "tc.cuh"

namespace gdn2 {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kUnit = 64;        // tokens of a unit
constexpr int kLead = 2;         // empty units before a (sequence, head)'s own
constexpr int kMinUnits = 1;     // fewest units of a block: one sequence of 1000 tokens, 16 heads, takes 9.4 us with 1, 9.8 with 2
constexpr int kHeadBlock = 16;   // most query heads of one pass
constexpr int kMostBlocksPerSm = 4;
// Sequences that cannot hold more than kSoloTokens (or kSoloTokensMany where
// there are kSoloRuns (sequence, head)s for each block that the GPU holds, so
// that blocks with short ones make room for others) go to blocks one
// (sequence, head) each: no search for a run, no join, and one launch, which
// counts where the host takes longer than the GPU (10 us a call from Python).
// One sequence, 16 heads: 100 tokens 4.8 us, split 8.0; 300 8.0 and 8.3; 400 9.7
// and 8.6; 500 10.6 and 8.8 (8.2 and 8.3 out of L2); 1000 17 and 9.4.  1024
// (sequence, head)s of up to 2000 tokens: 91 us, split 95; of up to 1000 48, 53.
constexpr int kSoloTokens = 512;
constexpr int kSoloTokensMany = 2048;
constexpr int kSoloRuns = 3;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnArgs {
    PagedView c;
    const void *q;
    void *o;
    float *lse;
    int H, G, HB, hpb;  // query heads, per kv head, blocks of them, heads of a block
    float scale2;       // scale log2 e
    int window;
    // workspace
    float2 *ml;         // [2 grid][kHeadBlock] m, l of a part
    float *part;        // [2 grid][kHeadBlock][d]
    int2 *parts;        // [N Hkv HB] first and last block with a part, or -1
    float *lse2;        // [N H] log-sum-exp in base 2 (for the weights), or nullptr
    float *scores;      // [score_units][hpb][kUnit] scores in base 2, or nullptr
    int score_units;    // units whose scores are kept
    unsigned int *status;
};

__device__ __forceinline__ int first_token(int len, int window) { return window > 0 && len > window ? len - window : 0; }
__device__ __forceinline__ int units_of(const PagedView &c, int n, int window, unsigned int *status) {
    const int len = checked_len(c, n, status);
    return len == 0 ? 0 : kLead + (len - first_token(len, window) + kUnit - 1) / kUnit;
}

// The run of units of block `block` out of `blocks`, `per` (= Hkv times
// head blocks) runs of units a sequence, at least `least` units a block:
// [u, end) and the sequence n, whose units start at `base`, that u lies in.
// (The host refuses calls of 2^30 units or more.)
struct Run {
    int u, end, share, base, n;
};
template <int NT>
__device__ __forceinline__ Run find_run(const PagedView &c, int window, int per, int least, unsigned int *status, int block,
                                        int blocks) {
    __shared__ int s_warp[NT / 32], s_n, s_base;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // A warp's lanes cover the sequences: each warp for itself, without barriers
    // (one sequence of 1000 tokens, 16 heads over 2: 8.4 us with them, 8.0 without).
    if (c.N <= 32) {
        const int own = lane < c.N ? units_of(c, lane, window, status) : 0;
        int sum = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += y;
        }
        const int all = __shfl_sync(0xffffffffu, sum, 31) * per, lo = (sum - own) * per;
        Run r;
        r.share = max(least, (all + blocks - 1) / blocks);
        r.u = r.share * block;
        r.end = min(r.u + r.share, all);
        const int at = __ffs(__ballot_sync(0xffffffffu, lo <= r.u && r.u < lo + own * per)) - 1;
        r.n = max(at, 0);
        r.base = __shfl_sync(0xffffffffu, lo, r.n);
        return r;
    }
    int x = 0, mine = 0;
    for (int n = tid; n < c.N; n += NT) x += mine = units_of(c, n, window, status);
    int inc = x;  // inclusive scan over the threads
    auto scan = [&]() {
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += y;
        }
        if (lane == 31) s_warp[warp] = inc;
        __syncthreads();
        int t = lane < NT / 32 ? s_warp[lane] : 0;
        int before = lane < warp ? t : 0;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            t += __shfl_xor_sync(0xffffffffu, t, off);
            before += __shfl_xor_sync(0xffffffffu, before, off);
        }
        inc += before;
        return t;  // the sum
    };
    int all = scan();
    const int total = all * per;
    Run r;
    r.share = max(least, (total + blocks - 1) / blocks);
    r.u = r.share * block;
    r.end = min(r.u + r.share, total);
    r.base = 0;
    r.n = 0;
    if (r.u >= total) return r;  // u >= end: nothing to do
    for (int n0 = 0, before = 0;;) {  // chunks of NT sequences; the only one's scan is the one above
        if (c.N > NT) {
            inc = mine = n0 + tid < c.N ? units_of(c, n0 + tid, window, status) : 0;
            __syncthreads();  // s_warp has been read
            all = scan();
        }
        const int lo = (before + inc - mine) * per;
        if (lo <= r.u && r.u < lo + mine * per) {
            s_n = n0 + tid;
            s_base = lo;
        }
        before += all;
        n0 += NT;
        if (before * per > r.u || n0 >= c.N) break;
    }
    __syncthreads();
    r.n = s_n;
    r.base = s_base;
    return r;
}

__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16_full(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// the two values of a packed pair of bf16
__device__ __forceinline__ float bf16_low(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_high(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
// a pair of bf16 with infinities, and what is no number, brought to the largest finite value
__device__ __forceinline__ uint32_t bf16_finite(uint32_t x) {
    uint32_t y;
    asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0x7f7f7f7fu));
    return y;
}
// an 8 x 8 block of 16-bit values (thread 4 r + c holds row r, columns 2c, 2c + 1), transposed
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// d += a b: a 16 x 16 (row), b 16 x 8 (column), bf16, float32 sums
__device__ __forceinline__ void mma16816(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A segment: tokens [begin, end) of sequence n, key-value head h, and query
// heads [head, head + rows).
struct Segment {
    int n, h, head, rows, begin, end;
    int run;             // (h, head block) in the sequence
    bool starts, whole;  // it starts at the run's first unit, and covers it
    int unit;            // the number of its first unit
    int run_end;         // one past the run's last unit
};
// the next segment of a run of units (false: there is none)
template <bool SOLO>
__device__ __forceinline__ bool next_segment(const AttnArgs &a, Run &run, Segment &sg) {
    const PagedView &c = a.c;
    const int per = c.Hkv * a.HB;
    while (run.u < run.end) {
        const int n = run.n, len = checked_len(c, n, a.status), first = first_token(len, a.window);
        const int T = (len - first + kUnit - 1) / kUnit;
        int t0 = 0, cnt = T;
        if constexpr (SOLO) {
            sg.run = blockIdx.x - run.n * per;
            sg.unit = blockIdx.x * ((c.cap + kUnit - 1) / kUnit);
            run.u = run.end;
        } else {
            if (T == 0) {
                ++run.n;
                continue;
            }
            const int U = T + kLead, in = run.u - run.base;
            sg.run = in / U;
            const int u0 = in - sg.run * U, n_units = min(U - u0, run.end - run.u);
            t0 = max(u0 - kLead, 0);
            cnt = u0 + n_units - kLead - t0;  // without a leading unit's share: nothing to do if <= 0
            sg.unit = run.u - u0 + kLead + t0;
            sg.run_end = run.base + (sg.run + 1) * U;
            run.u += n_units;
            if (run.u == run.base + per * U) {
                run.base = run.u;
                ++run.n;
            }
            if (cnt <= 0) continue;
        }
        sg.n = n;
        sg.h = sg.run / a.HB;
        const int hb = sg.run - sg.h * a.HB;
        sg.head = sg.h * a.G + hb * a.hpb;
        sg.rows = min(a.hpb, a.G - hb * a.hpb);
        sg.begin = first + t0 * kUnit;
        sg.end = min(len, sg.begin + cnt * kUnit);
        sg.starts = t0 == 0;
        sg.whole = t0 == 0 && cnt == T;
        return true;
    }
    return false;
}

// A warp's ring of stages and its copies.  Step i of a segment covers tokens
// begin + (i kAttnWarps + warp) KW + 0 .. KW-1; steps are taken segment by
// segment over the block's whole run.  A stage holds KW rows of k, then KW of
// v, rows of RB bytes with their 16-byte pieces permuted by the row (piece p
// of row r at p ^ key(r)), so that eight rows' equal pieces lie in different
// banks.  Rows without a token are zeros: their v must not be whatever the
// memory held, since 0 times NaN is NaN.
template <int KW, int RB, int STAGES, bool SOLO>
struct Ring {
    static constexpr int kStages = STAGES;
    static constexpr int kPieces = RB / 16;
    static constexpr int kHalf = KW * RB, kStage = 2 * kHalf;
    static constexpr int kBytes = kStages * kStage;
    static constexpr int kStep = kAttnWarps * KW;
    static constexpr uint32_t kAllRows = (1u << KW) - 1;
    const AttnArgs &a;
    uint32_t base;  // this warp's stages
    int warp, lane;
    Run run;        // what is left to copy behind the present segment
    int n, h, at_tok, end;  // the present segment: the warp's next token, the segment's end
    int steps;              // the segment's steps left
    bool more;              // there is a step to look up
    // the step that is issued next: whether there is one, whether row lane % KW
    // of it holds a token, and that row's page (as the table has it, not used
    // before the issue, so that the load does not hold anything up), slot, head
    bool ready, token;
    int page, slot, head;
    uint32_t live[kStages - 1];  // rows that hold a token, of the steps in flight, oldest first

    __device__ __forceinline__ static int key(int r) { return kPieces >= 8 ? r & 7 : (r >> 1) & (kPieces - 1); }
    __device__ __forceinline__ static uint32_t at(int r, int piece) { return (uint32_t)(r * RB + ((piece ^ key(r)) << 4)); }

    __device__ __forceinline__ void open() {
        Segment sg;
        steps = 0;
        more = false;
        while (steps == 0 && next_segment<SOLO>(a, run, sg)) {
            n = sg.n;
            h = sg.h;
            at_tok = sg.begin + warp * KW;
            end = sg.end;
            steps = (sg.end - sg.begin + kStep - 1) / kStep;
            more = steps > 0;
        }
    }
    // finds the rows of the next step
    __device__ __forceinline__ void lookup() {
        ready = more;
        token = false;
        if (!more) return;
        const int j = at_tok + lane % KW;
        if (j < end) {
            int entry;
            page_slot(a.c, j, entry, slot);
            page = a.c.table[(size_t)n * a.c.max_pages + entry];
            head = h;
            token = true;
        }
        at_tok += kStep;
        if (--steps == 0) open();
    }
    // the copies of a step to stage s, from lane r % KW's row r at `off`;
    // FULL: every row holds a token, otherwise those that do not become zeros
    template <bool FULL> __device__ __forceinline__ void copy(uint32_t s, long long off) const {
        constexpr int kRowsAtOnce = 32 / kPieces;  // rows of one instruction
        static_assert(kPieces <= 32 && KW * kPieces % 32 == 0, "whole warps of pieces");
        const int piece = lane % kPieces, mine = lane / kPieces;
        const char *k = a.c.k + piece * 16, *v = a.c.v + piece * 16;
        long long rows[KW * kPieces / 32];  // all fetched before the first is used
#pragma unroll
        for (int x = 0; x < KW * kPieces / 32; ++x) rows[x] = __shfl_sync(0xffffffffu, off, x * kRowsAtOnce + mine);
#pragma unroll
        for (int x = 0; x < KW * kPieces / 32; ++x) {
            const int r = x * kRowsAtOnce + mine;
            const long long ro = rows[x];
            const uint32_t to = s + at(r, piece);
            if (FULL) {
                cp_async16_full(to, k + ro);
                cp_async16_full(to + kHalf, v + ro);
            } else {
                cp_async16_zfill(to, ro < 0 ? k : k + ro, ro >= 0);
                cp_async16_zfill(to + kHalf, ro < 0 ? v : v + ro, ro >= 0);
            }
        }
    }
    // starts the copies of the step that was looked up (a group of its own,
    // empty past the last), and looks the one behind it up
    __device__ __forceinline__ uint32_t issue(int stage) {
        long long off = -1;
        if (token) {
            if ((unsigned)page < (unsigned)a.c.num_pages) off = row_off(a.c, page, slot, head);
            else record_status(a.status, GDN2_ERR_INVALID_ARG);
        }
        const uint32_t ok = __ballot_sync(0xffffffffu, off >= 0);
        if (ready) {
            const uint32_t s = base + stage * kStage;
            if ((ok & kAllRows) == kAllRows) copy<true>(s, off);
            else copy<false>(s, off);
        }
        tc::cp_async_commit();
        lookup();
        return ok;
    }
};

// where channel ch of row `row` lies in a warp's merge area [rows][D]: banks
// differ between the rows that a warp writes at once
template <int D> __device__ __forceinline__ int merge_at(int row, int ch) { return row * D + (ch ^ ((row >> 1 & 3) << 3)); }

// ---- bf16: products on the tensor cores, tokens (scores) and channels
// (values) as the 16 rows and the query heads as NT times 8 columns:
//   S^T [16 tokens x heads] = K Q^T,  acc^T [channels x heads] += V^T P^T.
// A mask, a maximum and a scale factor then belong to a column, which four
// registers of a thread share, and P^T turns from a result into an operand by
// transposing 8 x 8 blocks between registers.
template <int D, int NT>
struct EngineBf16 {
    using E = __nv_bfloat16;
    static constexpr int KW = 16, RB = 2 * D, kRows = 8 * NT, kBlocksPerSm = D == 128 ? 2 : 4, kStages = 3;
    static constexpr int kSoloBlocksPerSm = D == 128 ? (NT == 1 ? 3 : 2) : D == 64 ? (NT == 1 ? 5 : 4) : 6, kSoloStages = 2;
    uint32_t qf[NT][D / 16][2];
    float acc[NT][D / 16][4];
    float m[NT][2], l[NT][2];

    __device__ __forceinline__ void begin(const AttnArgs &a, const Segment &sg, int lane, float *) {
        const E *q = static_cast<const E *>(a.q) + ((size_t)sg.n * a.H + sg.head) * D;
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int row = 8 * i + g;
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    qf[i][x][y] = row < sg.rows ? *reinterpret_cast<const uint32_t *>(q + row * D + x * 16 + y * 8 + 2 * t) : 0u;
                acc[i][x][0] = acc[i][x][1] = acc[i][x][2] = acc[i][x][3] = 0.f;
            }
            m[i][0] = m[i][1] = -FLT_MAX;
            l[i][0] = l[i][1] = 0.f;
        }
    }
    // one step of 16 tokens; `scores`: this step's place in rows of kUnit scores, or nullptr
    template <class R>
    __device__ __forceinline__ void step(const AttnArgs &a, const Segment &sg, uint32_t ks, uint32_t vs, uint32_t live,
                                         int lane, float *scores, float *) {
        float s[NT][4];
        const int mi = lane >> 3, lr = lane & 7, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < NT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
            uint32_t k[4];
            ldmatrix4(ks + R::at((mi & 1) * 8 + lr, 2 * x + (mi >> 1)), k);
#pragma unroll
            for (int i = 0; i < NT; ++i) mma16816(s[i], k, qf[i][x][0], qf[i][x][1]);
        }
        const bool on[2] = {(live >> g & 1u) != 0, (live >> (g + 8) & 1u) != 0};
        float mn[NT][2];
        bool raised = false;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
#pragma unroll
                for (int x = 0; x < 2; ++x) s[i][2 * x + y] = on[x] ? s[i][2 * x + y] * a.scale2 : -INFINITY;
                float mx = fmaxf(s[i][y], s[i][2 + y]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                mn[i][y] = fmaxf(m[i][y], mx);
                raised |= mn[i][y] > m[i][y];
            }
        if (scores) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    if (8 * i + 2 * t + y < sg.rows) {
                        scores[(8 * i + 2 * t + y) * kUnit + g] = s[i][y];
                        scores[(8 * i + 2 * t + y) * kUnit + g + 8] = s[i][2 + y];
                    }
        }
        if (__any_sync(0xffffffffu, raised)) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float to = fminf(mn[i][y], FLT_MAX), f = exp2f(m[i][y] - to);
                    m[i][y] = to;
                    l[i][y] *= f;
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        acc[i][x][y] *= f;
                        acc[i][x][2 + y] *= f;
                    }
                }
        }
        uint32_t p[NT][2], rest[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                s[i][y] = exp2f(s[i][y] - m[i][y]);
                s[i][2 + y] = exp2f(s[i][2 + y] - m[i][y]);
                l[i][y] += s[i][y] + s[i][2 + y];
            }
            // The weights meet v as the sum of two bf16 numbers: rounded once,
            // to 2^-8, they would add as much error to o as its own rounding
            // (2.2e-3 against 1.7e-3 in all); in two parts it is 2^-16.  The
            // second product costs nothing up to 8 heads, where the copies set
            // the pace, and 3 us of 66 with 16 (64 sequences of up to 4000
            // tokens, 4 kv heads).
            const uint32_t h0 = tc::pack_bf16(s[i][0], s[i][1]), h1 = tc::pack_bf16(s[i][2], s[i][3]);
            p[i][0] = transpose8x8(h0);
            p[i][1] = transpose8x8(h1);
            rest[i][0] = transpose8x8(tc::pack_bf16(s[i][0] - bf16_low(h0), s[i][1] - bf16_high(h0)));
            rest[i][1] = transpose8x8(tc::pack_bf16(s[i][2] - bf16_low(h1), s[i][3] - bf16_high(h1)));
        }
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
            uint32_t v[4];
            ldmatrix4_trans(vs + R::at((mi >> 1) * 8 + lr, 2 * x + (mi & 1)), v);
#pragma unroll
            for (int i = 0; i < NT; ++i) mma16816(acc[i][x], v, p[i][0], p[i][1]);
            // An infinite value is in the sum already.  The rest, which may be 0
            // or negative, meets the largest finite one in its place (1 us of
            // those 66, nothing up to 8 heads).
#pragma unroll
            for (int y = 0; y < 4; ++y) v[y] = bf16_finite(v[y]);
#pragma unroll
            for (int i = 0; i < NT; ++i) mma16816(acc[i][x], v, rest[i][0], rest[i][1]);
        }
    }
    // this warp's m, l [kRows] and acc [kRows][D] to shared memory
    __device__ __forceinline__ void finish(float2 *ml, float *out, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int row = 8 * i + 2 * t + y;
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[i][y] += __shfl_xor_sync(0xffffffffu, l[i][y], d);
                if (g == 0) ml[row] = make_float2(m[i][y], l[i][y]);
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    out[merge_at<D>(row, 16 * x + g)] = acc[i][x][y];
                    out[merge_at<D>(row, 16 * x + g + 8)] = acc[i][x][2 + y];
                }
            }
    }
};

// ---- float32: products on the CUDA cores (the tensor cores' tf32 would lose
// what a float32 cache is kept for).  Scores: lane (part, token) = (lane / 8,
// lane % 8) sums a quarter of the channels of KT tokens, so that a piece of q
// is read from shared memory once for KT of them; values: a lane owns four
// channels of every (128 / D)-th token, and reads that token's weights for four
// heads at once.  GP: query heads, padded to a power of two.
template <int D, int GP>
struct EngineF32 {
    using E = float;
    static constexpr int KT = D == 128 || GP == 16 ? 1 : 2;
    static constexpr int KW = 8 * KT, RB = 4 * D, kRows = GP, kStages = 3;
    static constexpr int kBlocksPerSm = D == 32 && GP <= 4 ? 4 : 2;
    static constexpr int kSoloBlocksPerSm = GP == 16 ? 2 : GP == 8 || D == 128 ? 3 : 4, kSoloStages = 2;
    static constexpr int kLanes = D / 4;         // lanes of one token's channels
    static constexpr int kGroups = 32 / kLanes;  // tokens at once
    static constexpr int kVec = GP < 4 ? GP : 4;  // heads whose weights lie together, and that
                                                  // the parts share out: part p's are p, p + 4, ..
    static constexpr int kOwn = GP / kVec;
    float acc[GP][4];
    float m[GP], l[kOwn * (GP < 4 ? GP : 1)];

    // sq: [GP][D] of the block's
    __device__ __forceinline__ void begin(const AttnArgs &a, const Segment &sg, int, float *sq) {
        const float *q = static_cast<const float *>(a.q) + ((size_t)sg.n * a.H + sg.head) * D;
        __syncthreads();
        for (int i = threadIdx.x; i < GP * D; i += kAttnThreads) sq[i] = i < sg.rows * D ? q[i] : 0.f;
        __syncthreads();
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            acc[g][0] = acc[g][1] = acc[g][2] = acc[g][3] = 0.f;
            m[g] = -FLT_MAX;
        }
#pragma unroll
        for (float &x : l) x = 0.f;
    }
    // of four heads' values the one of this lane's part
    __device__ __forceinline__ static float of_part(const float *x, int part) {
        const float lo = part & 1 ? x[1] : x[0], hi = part & 1 ? x[3] : x[2];
        return part & 2 ? hi : lo;
    }
    // sp: [kAttnWarps][KW][GP] behind sq
    template <class R>
    __device__ __forceinline__ void step(const AttnArgs &a, const Segment &sg, uint32_t ks, uint32_t vs, uint32_t live,
                                         int lane, float *scores, float *sq) {
        float *sp = sq + GP * D + (threadIdx.x >> 5) * GP * KW;
        const int tok = lane & 7, part = lane >> 3;
        float s[KT][GP];
#pragma unroll
        for (int y = 0; y < KT; ++y)
#pragma unroll
            for (int g = 0; g < GP; ++g) s[y][g] = 0.f;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
            const int piece = 4 * x + part;
            float4 k[KT];
#pragma unroll
            for (int y = 0; y < KT; ++y) k[y] = ld4(ks + R::at(tok + 8 * y, piece));
#pragma unroll
            for (int g = 0; g < GP; ++g) {
                const float4 q = *reinterpret_cast<const float4 *>(sq + g * D + piece * 4);
#pragma unroll
                for (int y = 0; y < KT; ++y)
                    s[y][g] = fmaf(k[y].x, q.x, fmaf(k[y].y, q.y, fmaf(k[y].z, q.z, fmaf(k[y].w, q.w, s[y][g]))));
            }
        }
        bool raised = false;
        float mn[GP];
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            mn[g] = -INFINITY;
#pragma unroll
            for (int y = 0; y < KT; ++y) {
                s[y][g] += __shfl_xor_sync(0xffffffffu, s[y][g], 8);
                s[y][g] += __shfl_xor_sync(0xffffffffu, s[y][g], 16);
                s[y][g] = live >> (tok + 8 * y) & 1u ? s[y][g] * a.scale2 : -INFINITY;
                mn[g] = fmaxf(mn[g], s[y][g]);
            }
#pragma unroll
            for (int off = 1; off < 8; off <<= 1) mn[g] = fmaxf(mn[g], __shfl_xor_sync(0xffffffffu, mn[g], off));
            mn[g] = fmaxf(m[g], mn[g]);
            raised |= mn[g] > m[g];
        }
        if (scores && part == 0)
#pragma unroll
            for (int g = 0; g < GP; ++g)
                if (g < sg.rows)
#pragma unroll
                    for (int y = 0; y < KT; ++y) scores[g * kUnit + tok + 8 * y] = s[y][g];
        if (raised) {  // the same on every lane: m and mn are
            float f[GP];
#pragma unroll
            for (int g = 0; g < GP; ++g) {
                mn[g] = fminf(mn[g], FLT_MAX);
                f[g] = exp2f(m[g] - mn[g]);
                m[g] = mn[g];
                acc[g][0] *= f[g]; acc[g][1] *= f[g]; acc[g][2] *= f[g]; acc[g][3] *= f[g];
            }
            if constexpr (GP >= 4) {
#pragma unroll
                for (int i = 0; i < kOwn; ++i) l[i] *= of_part(f + 4 * i, part);
            } else {
#pragma unroll
                for (int g = 0; g < GP; ++g) l[g] *= f[g];
            }
        }
        __syncwarp();  // the last step's sp has been read
#pragma unroll
        for (int y = 0; y < KT; ++y) {
            if constexpr (GP >= 4) {
#pragma unroll
                for (int i = 0; i < kOwn; ++i) {
                    const float e = exp2f(of_part(&s[y][4 * i], part) - of_part(m + 4 * i, part));
                    l[i] += e;
                    sp[(tok + 8 * y) * GP + 4 * i + part] = e;
                }
            } else {
#pragma unroll
                for (int g = 0; g < GP; ++g) {
                    const float e = exp2f(s[y][g] - m[g]);
                    l[g] += e;
                    if (part == 0) sp[(tok + 8 * y) * GP + g] = e;
                }
            }
        }
        __syncwarp();
        const int grp = lane / kLanes, ch = lane % kLanes;
#pragma unroll
        for (int x = 0; x < KW / kGroups; ++x) {
            const int r = x * kGroups + grp;
            const float4 v = ld4(vs + R::at(r, ch));
#pragma unroll
            for (int g0 = 0; g0 < GP; g0 += kVec) {
                float e[kVec];
                if constexpr (kVec == 4) {
                    const float4 t = *reinterpret_cast<const float4 *>(sp + r * GP + g0);
                    e[0] = t.x; e[1] = t.y; e[2] = t.z; e[3] = t.w;
                } else {
#pragma unroll
                    for (int i = 0; i < kVec; ++i) e[i] = sp[r * GP + i];
                }
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    acc[g0 + i][0] = fmaf(e[i], v.x, acc[g0 + i][0]);
                    acc[g0 + i][1] = fmaf(e[i], v.y, acc[g0 + i][1]);
                    acc[g0 + i][2] = fmaf(e[i], v.z, acc[g0 + i][2]);
                    acc[g0 + i][3] = fmaf(e[i], v.w, acc[g0 + i][3]);
                }
            }
        }
    }
    __device__ __forceinline__ void finish(float2 *ml, float *out, int lane) {
        const int part = lane >> 3, ch = lane % kLanes;
#pragma unroll
        for (int g = 0; g < GP; ++g) {
            // a row's sum lies with one part's lanes (or, the same, with all four)
            float x = GP >= 4 ? ((g & 3) == part ? l[g / 4] : 0.f) : (part == 0 ? l[g % kVec] : 0.f);
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
            if (lane == 0) ml[g] = make_float2(m[g], x);
#pragma unroll
            for (int off = kLanes; off < 32; off <<= 1)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[g][i] += __shfl_xor_sync(0xffffffffu, acc[g][i], off);
            if (lane < kLanes)
                *reinterpret_cast<float4 *>(out + merge_at<D>(g, ch * 4)) =
                    make_float4(acc[g][0], acc[g][1], acc[g][2], acc[g][3]);
        }
    }
    __device__ __forceinline__ static float4 ld4(uint32_t addr) {
        float4 v;
        asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
        return v;
    }
};

__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(tc::pack_bf16(v.x, v.y), tc::pack_bf16(v.z, v.w));
}

// what a part with maximum and sum (m, l) = y counts for at the joint maximum m
// (0 for a part of nothing; not-a-numbers in its sums stay what they are)
__device__ __forceinline__ float part_factor(float2 y, float m) { return exp2f(y.x - m); }
// the row of ml and part where block b's part of a run, in blocks pr.x .. pr.y,
// has head `row`: the block where the run begins has it second, the others first
__device__ __forceinline__ size_t part_row(int2 pr, int b, int row) { return (size_t)(2 * b + (b == pr.x)) * kHeadBlock + row; }
// four channels of o, and (first: once a head) the log-sum-exp
template <typename E>
__device__ __forceinline__ void write_result(const AttnArgs &a, E *o, size_t hd, bool first, float m, float l, float4 x) {
    const bool none = l == 0.f;
    const float inv = none ? 0.f : 1.f / l;
    store4(o, none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
    if (!first) return;
    if (a.lse) a.lse[hd] = none ? -INFINITY : m * kLn2 + logf(l);
    if (a.lse2) a.lse2[hd] = none ? -INFINITY : m + log2f(l);
}

// shared memory of a block: the warps' rings, then what the engine keeps
template <class En, int D, bool SOLO> constexpr int attn_smem() {
    return kAttnWarps * Ring<En::KW, En::RB, SOLO ? En::kSoloStages : En::kStages, SOLO>::kBytes +
           (sizeof(typename En::E) == 4 ? En::kRows * (D + kAttnWarps * En::KW) * 4 : 0);
}

// SOLO: block b takes run b whole (no parts, no join).
template <class En, int D, bool SOLO>
__global__ void __launch_bounds__(kAttnThreads, SOLO ? En::kSoloBlocksPerSm : En::kBlocksPerSm)
attn_split_kernel(const AttnArgs a) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float2 s_ml[kAttnWarps][En::kRows];
    constexpr int kStages = SOLO ? En::kSoloStages : En::kStages;
    using R = Ring<En::KW, En::RB, kStages, SOLO>;
    using E = typename En::E;
    static_assert(R::kStage >= En::kRows * D * 4, "a stage holds a warp's accumulator");
    float *own = reinterpret_cast<float *>(smem + kAttnWarps * R::kBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const PagedView &c = a.c;
    const int per = c.Hkv * a.HB;
    follow_previous();
    Run run;
    if constexpr (SOLO) {
        run.n = blockIdx.x / per;
        run.u = 0;
        run.end = 1;
    } else run = find_run<kAttnThreads>(c, a.window, per, kMinUnits, a.status, blockIdx.x, gridDim.x);

    R ring{a, tc::smem_addr(smem) + warp * R::kBytes, warp, lane, run};
    ring.open();
    ring.lookup();
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) ring.live[s] = ring.issue(s);
    int stage = 0;  // the oldest step in flight
    En en;
    Segment sg;
    while (next_segment<SOLO>(a, run, sg)) {
        en.begin(a, sg, lane, own);
        const int steps = (sg.end - sg.begin + R::kStep - 1) / R::kStep;
        for (int i = 0; i < steps; ++i) {
            const uint32_t live = ring.live[0];
#pragma unroll
            for (int s = 0; s + 1 < kStages - 1; ++s) ring.live[s] = ring.live[s + 1];
            __syncwarp();  // the stage that the next copies go to has been read
            ring.live[kStages - 2] = ring.issue(stage == 0 ? kStages - 1 : stage - 1);
            cp_async_wait<kStages - 1>();
            __syncwarp();
            const int tok = (i * kAttnWarps + warp) * En::KW;  // in the segment
            float *sc = a.scores && sg.unit + tok / kUnit < a.score_units ? a.scores + (size_t)(sg.unit + tok / kUnit) * a.hpb * kUnit + tok % kUnit : nullptr;
            const uint32_t st = ring.base + stage * R::kStage;
            if (live) en.template step<R>(a, sg, st, st + R::kHalf, live, lane, sc, own);
            stage = stage == kStages - 1 ? 0 : stage + 1;
        }
        // the stage before the oldest in flight is free: the accumulators go there
        float *area = reinterpret_cast<float *>(smem + (stage == 0 ? kStages - 1 : stage - 1) * R::kStage);
        __syncwarp();
        en.finish(s_ml[warp], area + warp * (R::kBytes / 4), lane);
        __syncthreads();
        const int slot = 2 * blockIdx.x + sg.starts;
        for (int x = tid; x < sg.rows * (D / 4); x += kAttnThreads) {
            const int row = x / (D / 4), ch = (x - row * (D / 4)) * 4;
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) m = fmaxf(m, s_ml[w][row].x);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float2 y = s_ml[w][row];
                const float f = part_factor(y, m);
                const float4 v = *reinterpret_cast<const float4 *>(area + w * (R::kBytes / 4) + merge_at<D>(row, ch));
                l += f * y.y;
                o.x += f * v.x; o.y += f * v.y; o.z += f * v.z; o.w += f * v.w;
            }
            if (sg.whole) {
                const size_t hd = (size_t)sg.n * a.H + sg.head + row;
                write_result(a, static_cast<E *>(a.o) + hd * D + ch, hd, ch == 0, m, l, o);
            } else {
                store4(a.part + ((size_t)slot * kHeadBlock + row) * D + ch, o);
                if (ch == 0) a.ml[(size_t)slot * kHeadBlock + row] = make_float2(m, l);
            }
        }
        if constexpr (!SOLO) {
            if (tid == 0 && sg.starts)
                a.parts[(size_t)sg.n * per + sg.run] =
                    sg.whole ? make_int2(-1, -1) : make_int2((int)blockIdx.x, (sg.run_end - 1) / run.share);
        }
        __syncthreads();  // the area is a stage again
    }
    cp_async_wait<0>();
}

// After the split.  The first N H blocks: one a (sequence, query head) that
// joins its parts, or writes the empty sequence's result, or (no parts: it is
// written already) ends.  Each of a block's groups of D / 4 lanes takes every
// kGroups-th part, four loads ahead.  One sequence alone leaves a part in
// every block of the GPU, and then the blocks here are few and have 1024
// threads (NT); otherwise 128.
template <typename E, int D, int NT>
__device__ __forceinline__ void join_head(const AttnArgs &a) {
    constexpr int kLanes = D / 4, kGroups = NT / kLanes, kAhead = 4;
    __shared__ float s_m[NT / 32];
    __shared__ float s_l[kGroups];
    __shared__ float4 s_o[kGroups][kLanes];
    const int tid = threadIdx.x, n = blockIdx.x / a.H, h = blockIdx.x - n * a.H, kvh = h / a.G, g = h - kvh * a.G;
    const int hb = g / a.hpb, row = g - hb * a.hpb;
    const size_t hd = blockIdx.x;
    E *o = static_cast<E *>(a.o) + hd * D;
    const int2 pr = a.parts[((size_t)n * a.c.Hkv + kvh) * a.HB + hb];  // means nothing for an empty sequence
    if (checked_len(a.c, n, a.status) == 0) {
        if (tid < kLanes) write_result(a, o + tid * 4, hd, tid == 0, -INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f));
        return;
    }
    if (pr.x < 0) return;
    const int grp = tid / kLanes, ch = tid - grp * kLanes;
    float4 v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {  // the first parts come while the maximum is found
        const int b = pr.x + grp + i * kGroups;
        if (b <= pr.y) v[i] = *reinterpret_cast<const float4 *>(a.part + part_row(pr, b, row) * D + ch * 4);
    }
    float m = -INFINITY;
    for (int b = pr.x + tid; b <= pr.y; b += NT) m = fmaxf(m, a.ml[part_row(pr, b, row)].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if ((tid & 31) == 0) s_m[tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) m = fmaxf(m, s_m[w]);
    float l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b0 = pr.x + grp; b0 <= pr.y; b0 += kAhead * kGroups) {
        float2 y[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int b = b0 + i * kGroups;
            y[i] = b <= pr.y ? a.ml[part_row(pr, b, row)] : make_float2(-INFINITY, 0.f);
            if (b0 != pr.x + grp && b <= pr.y) v[i] = *reinterpret_cast<const float4 *>(a.part + part_row(pr, b, row) * D + ch * 4);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (b0 + i * kGroups > pr.y) break;
            const float f = part_factor(y[i], m);
            l += f * y[i].y;
            x.x += f * v[i].x; x.y += f * v[i].y; x.z += f * v[i].z; x.w += f * v[i].w;
        }
    }
    if (ch == 0) s_l[grp] = l;
    s_o[grp][ch] = x;
    // the groups' sums: 8 (kSome) groups take what the others have, then one
    constexpr int kSome = kGroups < 8 ? kGroups : 8;
    for (int left = kGroups, to = kSome; left > 1; left = to, to = 1) {
        __syncthreads();
        if (grp < to) {
            for (int i = grp + to; i < left; i += to) {
                const float4 w = s_o[i][ch];
                l += s_l[i];
                x.x += w.x; x.y += w.y; x.z += w.z; x.w += w.w;
            }
        }
        __syncthreads();
        if (grp < to) {
            if (ch == 0) s_l[grp] = l;
            s_o[grp][ch] = x;
        }
        if (to == 1) break;
    }
    if (tid >= kLanes) return;
    write_result(a, o + tid * 4, hd, tid == 0, m, l, x);
}

// sum over `rows` query heads of 2^(s - lse) for one cached row
template <typename E, int D>
__device__ __noinline__ float weight_of_row(const AttnArgs &a, const E *q, const E *k, const float *L, int rows) {
    float sum = 0.f;
    for (int r = 0; r < rows; ++r) {
        float s = 0.f;
#pragma unroll 8
        for (int i = 0; i < D; ++i) s = fmaf(ldx(q, r * D + i), ldx(k, i), s);
        sum += L[r] == -INFINITY ? 0.f : exp2f(s * a.scale2 - L[r]);
    }
    return sum;
}

// The blocks behind those (first = N H; none unless weights are wanted):
//   weight_j += sum over the group's heads of 2^(s_j - lse),
// from the scores that the split kernel kept, 64 threads a unit, a token each.
// A head's lse is the one written, or comes from its parts once more.  One
// addition a token and call, so that no order matters unless sequences share
// the page.
template <typename E, int D, int NT, bool SOLO>
__device__ __forceinline__ void add_weights(const AttnArgs &a, int first_block) {
    __shared__ float s_L[kMaxHeadGroup];
    const PagedView &c = a.c;
    Run run = find_run<NT>(c, a.window, c.Hkv, 1, a.status, blockIdx.x - first_block, gridDim.x - first_block);
    const int tid = threadIdx.x, lane = tid & 31, sub = tid / kUnit, tok = tid % kUnit;
    while (run.u < run.end) {
        const int len = checked_len(c, run.n, a.status), first = first_token(len, a.window);
        const int T = (len - first + kUnit - 1) / kUnit;
        if (T == 0) {
            ++run.n;
            continue;
        }
        const int U = T + kLead, h = (run.u - run.base) / U, u0 = run.u - run.base - h * U;
        const int n_units = min(U - u0, run.end - run.u), n = run.n, base = run.base;
        const int t0 = max(u0 - kLead, 0), cnt = u0 + n_units - kLead - t0;
        run.u += n_units;
        if (run.u == run.base + c.Hkv * U) {
            run.base = run.u;
            ++run.n;
        }
        if (cnt <= 0) continue;
        __syncthreads();  // the last segment's s_L has been read
        for (int g = tid >> 5; g < a.G; g += NT / 32) {
            const int hb = g / a.hpb, row = g - hb * a.hpb;
            const int2 pr = SOLO ? make_int2(-1, -1) : a.parts[((size_t)n * c.Hkv + h) * a.HB + hb];
            float L;
            if (pr.x < 0) L = a.lse2[(size_t)n * a.H + h * a.G + g];
            else {
                float m = -INFINITY, l = 0.f;
                for (int b = pr.x + lane; b <= pr.y; b += 32) m = fmaxf(m, a.ml[part_row(pr, b, row)].x);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                for (int b = pr.x + lane; b <= pr.y; b += 32) {
                    const float2 y = a.ml[part_row(pr, b, row)];
                    l += part_factor(y, m) * y.y;
                }
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
                L = l == 0.f ? -INFINITY : m + log2f(l);
            }
            if (lane == 0) s_L[g] = L;
        }
        __syncthreads();
        constexpr int kStep = NT / kUnit, kAhead = 2;  // units at once, and a thread's whose loads go out together
        for (int t = t0 + sub; t < t0 + cnt; t += kAhead * kStep) {
            int page[kAhead], slot[kAhead], at[kAhead];
            float sum[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int j = first + (t + u * kStep) * kUnit + tok;
                page[u] = -1;
                sum[u] = 0.f;
                at[u] = 0;  // what is not wanted reads unit t's, without a branch
                if (t + u * kStep >= t0 + cnt || j >= len) continue;
                at[u] = u * kStep * a.hpb * kUnit;
                int entry;
                page_slot(c, j, entry, slot[u]);
                page[u] = page_of(c, n, entry);
            }
            for (int hb = 0; hb < a.HB; ++hb) {
                // the split kernel's number of this unit: it has Hkv HB runs a sequence
                const int run_of = h * a.HB + hb;
                const int unit = SOLO ? (n * c.Hkv * a.HB + run_of) * ((c.cap + kUnit - 1) / kUnit) + t
                                      : base * a.HB + run_of * U + kLead + t;
                const float *s = a.scores + (size_t)unit * a.hpb * kUnit + tok;
                const int rows = min(a.hpb, a.G - hb * a.hpb);
                if (unit - t + min(t + (kAhead - 1) * kStep, t0 + cnt - 1) >= a.score_units) {
                    // past what was kept (sequences that share pages can hold more
                    // tokens together than the pool): the scores once more
#pragma unroll 1
                    for (int u = 0; u < kAhead; ++u)
                        if (page[u] >= 0)
                            sum[u] += weight_of_row<E, D>(a, static_cast<const E *>(a.q) + ((size_t)n * a.H + h * a.G + hb * a.hpb) * D,
                                                          reinterpret_cast<const E *>(c.k + row_off(c, page[u], slot[u], h)),
                                                          s_L + hb * a.hpb, rows);
                    continue;
                }
#pragma unroll 4
                for (int r = 0; r < rows; ++r) {
                    const float L = s_L[hb * a.hpb + r];
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        const float e = exp2f(s[at[u] + r * kUnit] - L);
                        sum[u] += L == -INFINITY ? 0.f : e;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (page[u] >= 0) atomicAdd(c.w + weight_off(c, page[u], slot[u], h), sum[u]);
        }
    }
}

template <typename E, int D, int NT, bool SOLO>
__global__ void __launch_bounds__(NT)
attn_finish_kernel(const AttnArgs a) {
    follow_previous();
    const int heads = SOLO ? 0 : a.c.N * a.H;
    if (!SOLO && blockIdx.x < heads) join_head<E, D, NT>(a);
    else add_weights<E, D, NT, SOLO>(a, heads);
}

// ---- host side
static void head_blocks(const PagedView &c, int H, AttnArgs &a) {
    a.c = c;
    a.H = H;
    a.G = H / c.Hkv;
    a.HB = (a.G + kHeadBlock - 1) / kHeadBlock;
    a.hpb = (a.G + a.HB - 1) / a.HB;
}

// The kept scores of a solo call are laid out by what the table reaches, so the
// window counts only without them (the workspace query does not know it).
static bool solo(const AttnArgs &a, bool weights, int window) {
    const PagedView &c = a.c;
    const int reach = window > 0 && !weights ? min(window, c.cap) : c.cap;
    return reach <= kSoloTokens || (reach <= kSoloTokensMany && (long long)c.N * c.Hkv * a.HB >= kSoloRuns * 2LL * sm_count());
}
static bool solo(const AttnArgs &a) { return solo(a, a.scores != nullptr, a.window); }

// places the workspace's regions (ws may be null: sizes only); returns its bytes
static size_t attn_ws(AttnArgs &a, int add_weights, void *ws) {
    const PagedView &c = a.c;
    a.ml = nullptr;
    a.part = a.lse2 = a.scores = nullptr;
    a.score_units = 0;
    a.parts = nullptr;
    if (!add_weights && solo(a, false, 0)) return 256;  // not touched
    const size_t slots = 2 * (size_t)kMostBlocksPerSm * sm_count(), runs = (size_t)c.N * c.Hkv * a.HB;
    size_t o = 0;
    auto take = [&](size_t bytes) { const size_t at = o; o = align256(o + bytes); return static_cast<char *>(ws) + at; };
    a.ml = reinterpret_cast<float2 *>(take(slots * kHeadBlock * sizeof(float2)));
    a.part = reinterpret_cast<float *>(take(slots * kHeadBlock * c.d * sizeof(float)));
    a.parts = reinterpret_cast<int2 *>(take(runs * sizeof(int2)));
    if (add_weights) {
        a.lse2 = reinterpret_cast<float *>(take((size_t)c.N * a.H * sizeof(float)));
        // every unit there can be, or if that is less, as many as the pool has
        // tokens for; a table much wider than the sequences costs nothing
        const long long all = (long long)runs * ((c.cap + kUnit - 1) / kUnit + kLead);
        const long long pool = ((long long)c.num_pages * c.page / kUnit + (1 + kLead) * (long long)c.N) * c.Hkv * a.HB;
        a.score_units = (int)(solo(a, true, 0) || all < pool ? all : pool);
        a.scores = reinterpret_cast<float *>(take((size_t)a.score_units * a.hpb * kUnit * sizeof(float)));
    }
    return o;
}

// units of 64 tokens that the call may have to count
bool attn_countable(const PagedView &c, int H) {
    AttnArgs a;
    head_blocks(c, H, a);
    return (double)c.N * c.Hkv * a.HB * ((c.cap + kUnit - 1) / kUnit + kLead) < (double)(1 << 30);
}

size_t attn_ws_bytes(const PagedView &c, int H, int add_weights) {
    AttnArgs a;
    head_blocks(c, H, a);
    return attn_ws(a, add_weights, nullptr);
}

template <class En, int D, bool SOLO>
static cudaError_t attn_run_as(const AttnArgs &a, cudaStream_t s) {
    static_assert(En::kBlocksPerSm <= kMostBlocksPerSm, "the workspace has parts for so many");
    constexpr int bytes = attn_smem<En, D, SOLO>();
    using E = typename En::E;
    const int heads = a.c.N * a.H;
    cudaError_t e = cudaFuncSetAttribute(attn_split_kernel<En, D, SOLO>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    e = launch_behind(K_ATTN_SPLIT, attn_split_kernel<En, D, SOLO>,
                      SOLO ? a.c.N * a.c.Hkv * a.HB : En::kBlocksPerSm * sm_count(), kAttnThreads, bytes, s, a);
    if (e != cudaSuccess) return e;
    if (SOLO && !a.scores) return cudaSuccess;
    if (heads <= sm_count())
        return launch_behind(K_ATTN_FINISH, attn_finish_kernel<E, D, 1024, SOLO>, (SOLO ? 0 : heads) + (a.scores ? 2 * sm_count() : 0),
                             1024, 0, s, a);
    return launch_behind(K_ATTN_FINISH, attn_finish_kernel<E, D, 128, SOLO>, (SOLO ? 0 : heads) + (a.scores ? 8 * sm_count() : 0),
                         128, 0, s, a);
}
template <class En, int D>
static cudaError_t attn_run(const AttnArgs &a, cudaStream_t s) {
    return solo(a) ? attn_run_as<En, D, true>(a, s) : attn_run_as<En, D, false>(a, s);
}

template <int D>
static cudaError_t attn_for_d(const AttnArgs &a, cudaStream_t s) {
    if (a.c.es == 2) return a.hpb <= 8 ? attn_run<EngineBf16<D, 1>, D>(a, s) : attn_run<EngineBf16<D, 2>, D>(a, s);
    if (a.hpb == 1) return attn_run<EngineF32<D, 1>, D>(a, s);
    if (a.hpb == 2) return attn_run<EngineF32<D, 2>, D>(a, s);
    if (a.hpb <= 4) return attn_run<EngineF32<D, 4>, D>(a, s);
    if (a.hpb <= 8) return attn_run<EngineF32<D, 8>, D>(a, s);
    return attn_run<EngineF32<D, 16>, D>(a, s);
}

cudaError_t attn_launch(const PagedView &c, const void *q, void *o, float *lse, int H, float scale, int window,
                        int add_weights, void *ws, unsigned int *status, cudaStream_t s) {
    AttnArgs a;
    a.q = q;
    a.o = o;
    a.lse = lse;
    head_blocks(c, H, a);
    a.scale2 = scale * kLog2e;
    a.window = window;
    a.status = status;
    attn_ws(a, add_weights, ws);
    if (c.d == 32) return attn_for_d<32>(a, s);
    if (c.d == 64) return attn_for_d<64>(a, s);
    return attn_for_d<128>(a, s);
}

}  // namespace gdn2
