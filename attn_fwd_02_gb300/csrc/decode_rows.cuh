// decode_rows.cuh -- paged decode with the query heads as the columns of the products: the kernel of the
// decode with modified scores and of a batch's own pages behind shared ones, and the merge of partials, which
// the splits of a row do themselves where they fit a cluster (cluster_splits).
//
// One query per sequence attends over its pages.  A CTA takes a range of pages of one (sequence,
// key/value head) for up to 8 NT of the query heads that share the head; its four warps take every
// fourth page each, through private rings of page blocks that TMA fills.  Per page of 16 tokens a warp
// computes, with mma.sync m16n8k16,
//     S^T = K Q^T        16 tokens x 8 heads: K is the A operand (ldmatrix), Q the B operand in registers,
//     O^T += V^T P^T     16 dims x 8 heads per product: V^T by transposing ldmatrix, P^T by two movmatrix
//                        of the packed scores (their tokens move from the rows to the pairs).
// With the tokens as the M rows, the 16-row products are full and the heads pad to 8 instead of 16: for
// up to 8 query heads that halves the products, exponentials and accumulators of the form with the heads
// as the rows.  The softmax keeps a reference max per head that moves only when some score exceeds it by
// 2^8 (one vote per page; the maxima are reduced over the lanes only then), and each lane keeps its own
// tokens' part of the normaliser until the end.
//
// e4m3 pages are widened in registers to f16 (exact) and both products run in f16; ldmatrix hands a lane
// four codes of a token, so a k-step's 16 dims are taken in the order 4t, 4t + 1, 4t + 2, 4t + 3 per lane
// t, for K and Q alike, and the rows of O^T stand for the even and odd dims of a chunk.
#pragma once

#include "launch.h"
#include "mma_sync.cuh"
#include "scoremod.cuh"
#include "sm103_ptx.cuh"

namespace attn {

// Arguments of the rows kernel and the merge (device-side; filled by the launchers).
struct RowsParams {
    const void *q;
    const int32_t *page_table, *ctx_lens;
    void *o;
    float *lse;  // may be null
    float *ws;   // [B, H, ws_splits, d + 4] partials: O, m (log2), l
    int *status;
    int B, H, Hkv, group, rgroups, max_pages, num_pages;
    int n_splits, ws_splits, ws_first;  // this kernel writes partials ws_first .. ws_first + n_splits - 1
    float c;                            // scale * log2(e) (times the key scale of an e4m3 cache)
    float v_scale;
    int q_low;                          // of the queries' powers of two (query_shift)
    // groups of S sequences: the first shared_pages[b / S] pages are those of the group's first row of the
    // table; own_only: they are not read here
    const int32_t *shared_pages;
    int S, own_only;
    // modified scores: cap_in (0: none) = scale * key scale / cap, cap_out = cap * log2(e)
    float cap_in, cap_out;
    const float *slopes;       // [H], may be null
    const int32_t *key_begin;  // [B], may be null
    int chunk_pages;           // pages per split (0: even shares of the pages)
    int cluster;               // splits of a row that are the CTAs of one cluster, which merges them itself (0: none)
};

namespace {

constexpr int kRowWarps = 4;
constexpr int kRowPS = 16;
constexpr float kRowLog2e = 1.4426950408889634f;
constexpr float kRowLn2 = 0.6931471805599453f;
// Ring slots (page blocks of K and V in flight) per warp.
template <bool FP8> constexpr int kRowSlots = 2;
constexpr int kRowCluster = 16;  // most splits of a row that one cluster merges
template <int D, bool FP8> constexpr int kRowBoxes = FP8 ? 1 : (D + 63) / 64;  // 128-byte-row boxes per block
template <int D, bool FP8> constexpr int kRowBlock = kRowBoxes<D, FP8> * kRowPS * 128;

// What a CTA's warps leave for the merge.
template <int D, int NT>
struct RowsRed {
    float o[kRowWarps][8 * NT][D];
    float m[kRowWarps][8 * NT];
    float l[kRowWarps][8 * NT];
    float2 ml[8 * NT];  // of the CTA (whose O is then in o[0])
};

template <int D, bool FP8, int NT>
struct RowsSmem {
    // the merge starts after every warp has consumed its last page: it shares the ring's bytes
    union {
        alignas(1024) uint8_t kv[kRowWarps][kRowSlots<FP8>][2][kRowBlock<D, FP8>];
        RowsRed<D, NT> red;
    } u;
    uint64_t full[kRowWarps][kRowSlots<FP8>];
    int abort_flag;
};

// Transposes an 8 x 8 matrix of 16-bit elements held as one register per lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Barrier over the cluster's threads, ordering their shared-memory accesses.
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
// The same shared-memory address in CTA `rank` of the cluster, and a load from there.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, int rank) {
    uint32_t d;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(addr), "r"(rank));
    return d;
}
__device__ __forceinline__ float2 cluster_load2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// Pages [p0, p1) of this split, and the tokens lo <= t < hi among them that the query sees.
struct PageRange {
    int p0, p1, lo, hi;
};
__device__ __forceinline__ int shared_pages_of(const RowsParams &a, int b) {
    return min(max(a.shared_pages[b / a.S], 0), a.max_pages);
}
template <bool MOD>
__device__ __forceinline__ PageRange rows_range(const RowsParams &a, int b, int split) {
    PageRange r;
    r.hi = min(max(a.ctx_lens[b], 0), a.max_pages * kRowPS);
    const int pages = (r.hi + kRowPS - 1) / kRowPS;
    if constexpr (MOD) {
        r.lo = a.key_begin ? min(max(a.key_begin[b], 0), r.hi) : 0;
        if (a.chunk_pages == 0) {
            const int base = r.lo / kRowPS;
            const long long n = max(pages - base, 0);
            r.p0 = base + (int)(n * split / a.n_splits);
            r.p1 = r.lo < r.hi ? base + (int)(n * (split + 1) / a.n_splits) : 0;
        } else {
            r.p0 = max(split * a.chunk_pages, r.lo / kRowPS);
            r.p1 = r.lo < r.hi ? min((split + 1) * a.chunk_pages, pages) : 0;
        }
    } else {
        r.lo = 0;
        const int base = a.own_only ? shared_pages_of(a, b) : 0;
        const long long n = max(pages - base, 0);
        r.p0 = base + (int)(n * split / a.n_splits);
        r.p1 = base + (int)(n * (split + 1) / a.n_splits);
    }
    return r;
}

// O / L of values with a scale.  Of a scale near the smallest and a large sum the quotient would leave fp32's normal numbers where
// the result does not, so for scales below 1 it is taken 2^64 times as large (an exact power: nothing else changes).
struct OverSum {
    float f, back;
    __device__ __forceinline__ OverSum(float scale, float L, bool any) {
        const bool small = scale < 1.f;
        f = any ? (small ? scale * 0x1p64f : scale) / L : 0.f;
        back = small ? 0x1p-64f : 1.f;
    }
    __device__ __forceinline__ float operator()(float O) const { return O * f * back; }
};

// The end of a CTA's splits: its warps' states are merged in shared memory, over the ring once every warp is done with its
// pages, and the CTA's goes to the workspace or, through distributed shared memory, into the cluster's result.  CODES: rows
// g, g + 8 of a tile of O^T are the even and odd dims of its 16, not its halves, and the values have a scale.
template <int D, int NT, bool CODES, bool MOD>
__device__ __forceinline__ void rows_finish(RowsRed<D, NT> &red, volatile int *abort_flag, const RowsParams &a,
                                            const float (&o)[NT][D / 16][4], const float (&m_ref)[NT][2],
                                            const float (&l)[NT][2], int rows, int h0, int b, int split, float *ws,
                                            size_t ws_row) {
    constexpr int KS = D / 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 8 * nt + 2 * t + j;
            float ls = l[nt][j];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, off);
            if (g == 0) {
                // (a sum of NaN counts as seen, so that a query with NaN gives NaN)
                red.m[warp][r] = ls == ls ? m_ref[nt][j] : 0.f;
                red.l[warp][r] = ls;
            }
#pragma unroll
            for (int nd = 0; nd < KS; ++nd) {
                const int d0 = CODES ? 16 * nd + 2 * g : 16 * nd + g;
                red.o[warp][r][d0] = o[nt][nd][j];
                red.o[warp][r][d0 + (CODES ? 1 : 8)] = o[nt][nd][j + 2];
            }
        }
    __syncthreads();
    if (a.cluster) {
        // the CTA's state, over the first warp's
        for (int e = threadIdx.x; e < rows * D; e += kRowWarps * 32) {
            const int r = e / D, dd = e % D;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, red.m[w][r]);
            float L = 0.f, O = 0.f;
            if (M != -INFINITY) {
#pragma unroll
                for (int w = 0; w < kRowWarps; ++w) {
                    const float wgt = ex2_approx(red.m[w][r] - M);
                    L += red.l[w][r] * wgt;
                    O += red.o[w][r][dd] * wgt;
                }
            }
            red.o[0][r][dd] = O;
            if (dd == 0) red.ml[r] = make_float2(M, L);
        }
        cluster_sync_all();
        // the cluster's: the rows' pairs of columns are shared out over its threads
        const uint32_t ml0 = smem_u32(red.ml), o0 = smem_u32(red.o[0]);
        __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(a.o) + ((size_t)b * a.H + h0) * D;
        for (int e = split * kRowWarps * 32 + threadIdx.x; e < rows * (D / 2); e += a.n_splits * kRowWarps * 32) {
            const int r = e / (D / 2), pair = e % (D / 2);
            float2 ml[kRowCluster], ov[kRowCluster];
#pragma unroll
            for (int c0 = 0; c0 < kRowCluster; ++c0) {
                ml[c0] = make_float2(-INFINITY, 0.f), ov[c0] = make_float2(0.f, 0.f);
                if (c0 < a.n_splits) {
                    ml[c0] = cluster_load2(cluster_map(ml0 + r * 8, c0));
                    ov[c0] = cluster_load2(cluster_map(o0 + (r * D + 2 * pair) * 4, c0));
                }
            }
            float M = -INFINITY;
#pragma unroll
            for (int c0 = 0; c0 < kRowCluster; ++c0) M = fmaxf(M, ml[c0].x);
            float L = 0.f;
            float2 O = make_float2(0.f, 0.f);
            if (M != -INFINITY) {
#pragma unroll
                for (int c0 = 0; c0 < kRowCluster; ++c0) {
                    const float wgt = ex2_approx(ml[c0].x - M);  // 0 for an empty one, whose O is 0
                    L = fmaf(ml[c0].y, wgt, L);
                    O.x = fmaf(ov[c0].x, wgt, O.x);
                    O.y = fmaf(ov[c0].y, wgt, O.y);
                }
            }
            const bool any = L != 0.f;
            const OverSum over(CODES ? a.v_scale : 1.f, L, any);
            *reinterpret_cast<uint32_t *>(out + (size_t)r * D + 2 * pair) = pack_bf16x2(over(O.x), over(O.y));
            if (pair == 0 && a.lse) a.lse[(size_t)b * a.H + h0 + r] = any ? kRowLn2 * (M + __log2f(L)) : -INFINITY;
        }
        cluster_sync_all();  // no CTA leaves while another reads its state
        return;
    }
    if (!*abort_flag) {
        for (int e = threadIdx.x; e < rows * D; e += kRowWarps * 32) {
            const int r = e / D, dd = e % D;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, red.m[w][r]);
            float L = 0.f, O = 0.f;
            if (M != -INFINITY) {
#pragma unroll
                for (int w = 0; w < kRowWarps; ++w) {
                    const float wgt = ex2_approx(red.m[w][r] - M);
                    L += red.l[w][r] * wgt;
                    O += red.o[w][r][dd] * wgt;
                }
            }
            ws[r * ws_row + dd] = CODES ? O * a.v_scale : O;
            if (dd == 0) {
                ws[r * ws_row + D] = M;
                ws[r * ws_row + D + 1] = L;
            }
        }
    }
    // own pages: this grid may have started while the shared pages' grid was still running; its
    // completion, which the merge relies on, is to include that grid's
    if (!MOD) griddep_wait();
    griddep_launch_dependents();
}

template <int D, bool FP8, int NT, bool MOD>
__global__ void __launch_bounds__(kRowWarps * 32, 4)
    decode_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const RowsParams a) {
    constexpr int kSl = kRowSlots<FP8>;
    constexpr int kBx = kRowBoxes<D, FP8>;
    constexpr uint32_t kBlockBytes = kRowBlock<D, FP8>;
    constexpr int KS = D / 16;  // k-steps of S^T, and 16-dim tiles of O^T
    constexpr float kThresh = 8.0f;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    using Smem = RowsSmem<D, FP8, NT>;
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

    const int split = blockIdx.x, b = blockIdx.z;
    const int kvh = (int)blockIdx.y / a.rgroups;
    const int row0 = ((int)blockIdx.y % a.rgroups) * 8 * NT;
    const int rows = min(8 * NT, a.group - row0);
    const int h0 = kvh * a.group + row0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const PageRange pr = rows_range<MOD>(a, b, split);
    float *ws = a.ws + (((size_t)b * a.H + h0) * a.ws_splits + a.ws_first + split) * (D + 4);
    const size_t ws_row = (size_t)a.ws_splits * (D + 4);
    if (pr.p0 >= pr.p1 && !a.cluster) {  // nothing here (uniform over the CTA)
        if (!MOD) {
            if ((int)threadIdx.x < rows) {
                ws[threadIdx.x * ws_row + D] = -INFINITY;
                ws[threadIdx.x * ws_row + D + 1] = 0.f;
            }
            griddep_wait();
            griddep_launch_dependents();
        }
        return;
    }
    const int npages = pr.p1 - pr.p0;
    const int nk = npages > warp ? (npages - warp + kRowWarps - 1) / kRowWarps : 0;

    if (threadIdx.x == 0) {
        for (int w = 0; w < kRowWarps; ++w)
            for (int s = 0; s < kSl; ++s) mbar_init(&sm.full[w][s], 1);
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    WaitCtx wc{&sm.abort_flag, a.status};
    if (lane == 0) {
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }

    // Page ids, 32 of this warp's pages at a time (lane l: page k0 + l); bit k % 32 of mapped: page k's id
    // lies in the pool (an unmapped page holds no token)
    const int32_t *table = a.page_table + (size_t)b * a.max_pages + pr.p0 + warp;
    // shared pages (not own_only): the entries of the group's first row, `back` before this row's
    const int shared = !MOD && !a.own_only ? shared_pages_of(a, b) - pr.p0 - warp : 0;
    const size_t back = !MOD ? (size_t)(b % a.S) * a.max_pages : 0;
    int my_pid = -1;
    uint32_t mapped = 0;
    auto issue = [&](int k) {
        if ((k & 31) == 0) {
            const int at = kRowWarps * (k + lane);
            my_pid = k + lane < nk ? (!MOD && at < shared ? table - back : table)[at] : -1;
        }
        const int pid = __shfl_sync(0xffffffffu, my_pid, k & 31);
        const bool ok = pid >= 0 && pid < a.num_pages;
        mapped = (mapped & ~(1u << (k & 31))) | ((ok ? 1u : 0u) << (k & 31));
        if (lane == 0) {
            uint64_t *bar = &sm.full[warp][k % kSl];
            if (ok) {
                const int row = pid * a.Hkv + kvh;
                mbar_arrive_expect_tx(bar, 2 * kBlockBytes);
#pragma unroll
                for (int i = 0; i < kBx; ++i) {
                    tma_load_3d(sm.u.kv[warp][k % kSl][0] + i * (16 * 128), &tmK, bar, i * 64, 0, row);
                    tma_load_3d(sm.u.kv[warp][k % kSl][1] + i * (16 * 128), &tmV, bar, i * 64, 0, row);
                }
            } else {
                mbar_arrive(bar);
            }
        }
    };
    const int first = nk < kSl ? nk : kSl;
    for (int k = 0; k < first; ++k) issue(k);

    // Q as B fragments: column n = g of n-tile nt is query head h0 + 8 nt + g (zero past the group)
    uint32_t qb[NT][KS][2];
    // per score column (heads 2t, 2t + 1 of an n-tile): the factor of its products, to the cap's argument or, without
    // a cap, to the log2 domain
    const float c = MOD && a.cap_in > 0.f ? a.cap_in : a.c;
    float cc[NT][2];
    {
        const __nv_bfloat16 *q = reinterpret_cast<const __nv_bfloat16 *>(a.q) + ((size_t)b * a.H + h0) * D;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float amax = 0.f;
            const uint32_t *qr = reinterpret_cast<const uint32_t *>(q + (size_t)(8 * nt + g) * D);
            const bool have = 8 * nt + g < rows;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                if constexpr (FP8) {  // dims 16 ks + 4 t + {0, 1} and + {2, 3}: the order of the K codes
                    const uint2 u = have ? *reinterpret_cast<const uint2 *>(qr + ks * 8 + 2 * t) : make_uint2(0u, 0u);
                    qb[nt][ks][0] = u.x;
                    qb[nt][ks][1] = u.y;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(qb[nt][ks][i] << 16)),
                                                 fabsf(__uint_as_float(qb[nt][ks][i] & 0xffff0000u))));
                } else {
                    qb[nt][ks][0] = have ? qr[ks * 8 + t] : 0u;
                    qb[nt][ks][1] = have ? qr[ks * 8 + 4 + t] : 0u;
                }
            }
            cc[nt][0] = cc[nt][1] = c;
            if constexpr (FP8) {
                // each head is rounded to f16 after a 2^-sh of its own (query_shift); its four lanes hold its dims
#pragma unroll
                for (int off = 1; off <= 2; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
                const int sh = query_shift(amax, a.q_low);
                const float f = __uint_as_float((uint32_t)(127 - sh) << 23), back = __uint_as_float((uint32_t)(127 + sh) << 23);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        qb[nt][ks][i] = pack_f16x2(__uint_as_float(qb[nt][ks][i] << 16) * f,
                                                   __uint_as_float(qb[nt][ks][i] & 0xffff0000u) * f);
#pragma unroll
                for (int j = 0; j < 2; ++j) cc[nt][j] *= __shfl_sync(0xffffffffu, back, 4 * (2 * t + j));
            }
        }
    }
    // modified scores: the slopes of this lane's heads (columns 2t, 2t + 1)
    [[maybe_unused]] float slope2[NT][2];
    if constexpr (MOD) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = 8 * nt + 2 * t + j;
                slope2[nt][j] = a.slopes && r < rows ? bias_slope(a.slopes[h0 + r]) : 0.f;
            }
    }

    float o[NT][KS][4];
    float m_ref[NT][2], l[NT][2];  // of heads 2t, 2t + 1; l: this lane's tokens only
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int nd = 0; nd < KS; ++nd) o[nt][nd][0] = o[nt][nd][1] = o[nt][nd][2] = o[nt][nd][3] = 0.f;
        m_ref[nt][0] = m_ref[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
    }

    // ldmatrix: lane l gives row l & 7 of 8x8 matrix l >> 3.  K (A operand): tokens 0-7, 8-15, then the
    // next 8 columns; V (transposed): dims in the low bit, tokens in the high one.  e4m3 boxes: matrices
    // {tokens 0-7, tokens 8-15} x {chunk c, chunk c + 1} of 16 codes.
    const int mi = lane >> 3, mr = lane & 7;
    const int k_row = (mi & 1) * 8 + mr, k_col = (mi >> 1) * 8;
    const int v_row = (mi >> 1) * 8 + mr, v_col = (mi & 1) * 8;
    const int f_row = (mi & 1) * 8 + mr, f_chunk = mi >> 1;
    auto f_off = [](int r, int chunk) { return (uint32_t)(r * 128 + ((chunk ^ (r & 7)) << 4)); };

    int issued = first;
    bool failed = false;
    for (int k = 0; k < nk; ++k) {
        const int slot = k % kSl;
        if (!mbar_wait(&sm.full[warp][slot], (uint32_t)((k / kSl) & 1), wc, 140 + warp)) {
            failed = true;
            break;
        }
        if ((mapped >> (k & 31)) & 1u) {
            const int tok0 = (pr.p0 + warp + kRowWarps * k) * kRowPS;
            const int lo = pr.lo - tok0, hi = pr.hi - tok0;  // slots lo <= i < hi are seen
            const uint32_t Ks = smem_u32(sm.u.kv[warp][slot][0]);
            const uint32_t Vs = smem_u32(sm.u.kv[warp][slot][1]);
            const bool ragged = hi < kRowPS || (MOD && lo > 0);
            if (ragged) {
                // slots outside may hold anything: their V rows become zero so that P = 0 meets finite values
                for (int i = lane; i < kRowPS * 8 * kBx; i += 32) {
                    const int r = (i >> 3) & 15;
                    if (r >= hi || r < lo)
                        *reinterpret_cast<uint4 *>(sm.u.kv[warp][slot][1] + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                __syncwarp();
            }
            float sc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
            float sc2[NT][4];  // odd k-steps: two shorter chains
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) sc2[nt][0] = sc2[nt][1] = sc2[nt][2] = sc2[nt][3] = 0.f;
            if constexpr (FP8) {
#pragma unroll
                for (int ks = 0; ks < KS; ks += 2) {
                    uint32_t w[4];
                    ldsm_x4(Ks + f_off(f_row, ks + f_chunk), w);
                    uint32_t ka[4];
                    e4m3x4_to_f16x2x2(w[0], ka[0], ka[2]);
                    e4m3x4_to_f16x2x2(w[1], ka[1], ka[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_16816_f16(sc[nt], ka, qb[nt][ks][0], qb[nt][ks][1]);
                    if (ks + 1 < KS) {
                        e4m3x4_to_f16x2x2(w[2], ka[0], ka[2]);
                        e4m3x4_to_f16x2x2(w[3], ka[1], ka[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_16816_f16(sc2[nt], ka, qb[nt][ks + 1][0], qb[nt][ks + 1][1]);
                    }
                }
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t ka[4];
                    ldsm_x4(Ks + swz_off(k_row, ks * 16 + k_col), ka);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_16816((ks & 1) ? sc2[nt] : sc[nt], ka, qb[nt][ks][0], qb[nt][ks][1]);
                }
            }
            // log2-domain scores: rows (tokens) g, g + 8, columns (heads) 2t, 2t + 1
            uint32_t pb[NT][2];
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[nt][i] += sc2[nt][i];
                if constexpr (MOD) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[nt][i] *= cc[nt][i & 1];
                    if (a.cap_in > 0.f) {
                        const float big = fmaxf(fmaxf(fabsf(sc[nt][0]), fabsf(sc[nt][1])),
                                                fmaxf(fabsf(sc[nt][2]), fabsf(sc[nt][3])));
                        const uint64_t u01 = f32x2_pack(sc[nt][0], sc[nt][1]), u23 = f32x2_pack(sc[nt][2], sc[nt][3]);
                        if (__any_sync(0xffffffffu, big > 1.f)) {
                            f32x2_unpack(TanhCap::eval_u<2>(u01, a.cap_out), sc[nt][0], sc[nt][1]);
                            f32x2_unpack(TanhCap::eval_u<2>(u23, a.cap_out), sc[nt][2], sc[nt][3]);
                        } else {
                            f32x2_unpack(TanhCap::eval_u<1>(u01, a.cap_out), sc[nt][0], sc[nt][1]);
                            f32x2_unpack(TanhCap::eval_u<1>(u23, a.cap_out), sc[nt][2], sc[nt][3]);
                        }
                    }
                    const float far0 = (float)(pr.hi - 1 - tok0 - g);  // distance of token g (token g + 8: 8 less)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sc[nt][i] = fmaf(-slope2[nt][i & 1], i < 2 ? far0 : far0 - 8.f, sc[nt][i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[nt][i] *= cc[nt][i & 1];
                }
                if (ragged) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = g + (i < 2 ? 0 : 8);
                        if (r >= hi || r < lo) sc[nt][i] = -INFINITY;
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) grow = grow || fmaxf(sc[nt][j], sc[nt][j + 2]) > m_ref[nt][j] + kThresh;
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float al[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float mx = fmaxf(sc[nt][j], sc[nt][j + 2]);
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                        al[j] = 1.f;
                        if (mx > m_ref[nt][j] + kThresh) {
                            al[j] = ex2_approx(m_ref[nt][j] - mx);  // 0 when the reference was -inf
                            m_ref[nt][j] = mx;
                            l[nt][j] *= al[j];
                        }
                    }
#pragma unroll
                    for (int nd = 0; nd < KS; ++nd) {
                        o[nt][nd][0] *= al[0];
                        o[nt][nd][1] *= al[1];
                        o[nt][nd][2] *= al[0];
                        o[nt][nd][3] *= al[1];
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float m = m_ref[nt][i & 1] == -INFINITY ? 0.f : m_ref[nt][i & 1];
                    p[i] = ex2_approx(sc[nt][i] - m);
                    l[nt][i & 1] += p[i];
                }
                // tokens from the rows into the pairs of the B operand
                pb[nt][0] = movmatrix_trans(FP8 ? pack_f16x2(p[0], p[1]) : pack_bf16x2(p[0], p[1]));
                pb[nt][1] = movmatrix_trans(FP8 ? pack_f16x2(p[2], p[3]) : pack_bf16x2(p[2], p[3]));
            }
            if constexpr (FP8) {
#pragma unroll
                for (int ch = 0; ch < KS; ch += 2) {
                    uint32_t w[4];  // tokens 2t, 2t + 1 (then + 8) x dims 2g, 2g + 1 of chunks ch, ch + 1
                    ldsm_x4_trans(Vs + f_off(f_row, ch + f_chunk), w);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (ch + j < KS) {
                            uint32_t va[4];  // rows g: the chunk's even dims, rows g + 8: its odd dims
                            e4m3x4_to_f16x2x2(prmt(w[2 * j], 0u, 0x3120u), va[0], va[1]);
                            e4m3x4_to_f16x2x2(prmt(w[2 * j + 1], 0u, 0x3120u), va[2], va[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma_16816_f16(o[nt][ch + j], va, pb[nt][0], pb[nt][1]);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int nd = 0; nd < KS; ++nd) {
                    uint32_t va[4];
                    ldsm_x4_trans(Vs + swz_off(v_row, nd * 16 + v_col), va);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_16816(o[nt][nd], va, pb[nt][0], pb[nt][1]);
                }
            }
        }
        // the slot is free: order this warp's reads and writes before the next TMA write
        fence_proxy_async_smem();
        __syncwarp();
        if (k + kSl < nk) {
            issue(k + kSl);
            ++issued;
        }
    }
    if (failed) {  // drain this warp's copies in flight (bounded) before the CTA exits
        WaitCtx drain{nullptr, a.status};
        for (int k = 0; k < issued; ++k)
            if (lane == 0 && k + kSl >= issued)
                (void)mbar_wait(&sm.full[warp][k % kSl], (uint32_t)((k / kSl) & 1), drain, 197);
        __syncwarp();
    }

    rows_finish<D, NT, FP8, MOD>(sm.u.red, &sm.abort_flag, a, o, m_ref, l, rows, h0, b, split, ws, ws_row);
}

// Merge of the partials of one (sequence, query head) per warp: lanes hold 4 columns each, the weights
// of up to 32 partials at a time sit one per lane.  Partials 0 .. n_first - 1 (shared pages) and those of
// the rows kernel; an empty one (m = -inf) may hold anything in O and is skipped.
template <int D, bool MOD>
__global__ void __launch_bounds__(128) decode_rows_merge_kernel(const RowsParams a) {
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (long long)a.B * a.H) return;
    const int b = (int)(row / a.H);
    int s0 = 0, s1 = a.ws_first + a.n_splits;
    if constexpr (MOD) {  // only the splits with a visible page were written
        const PageRange r = rows_range<true>(a, b, 0);
        s0 = r.lo / (a.chunk_pages * kRowPS);
        s1 = r.lo < r.hi ? (r.hi + a.chunk_pages * kRowPS - 1) / (a.chunk_pages * kRowPS) : 0;
    }
    const float *ws = a.ws + (size_t)row * a.ws_splits * (D + 4);
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int base = s0; base < s1; base += 32) {
        float2 ml = make_float2(-INFINITY, 0.f);
        if (base + lane < s1) ml = *reinterpret_cast<const float2 *>(ws + (size_t)(base + lane) * (D + 4) + D);
        float mx = ml.x;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        if (mx == -INFINITY) continue;
        const float m_new = fmaxf(M, mx), al = ex2_approx(M - m_new);
        M = m_new;
        const float w = ex2_approx(ml.x - M);  // 0 for an empty one
        float ls = ml.y * w;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, off);
        L = L * al + ls;
        acc.x *= al, acc.y *= al, acc.z *= al, acc.w *= al;
        const int n = min(32, s1 - base);
        const uint32_t some = __ballot_sync(0xffffffffu, ml.x != -INFINITY);
        for (int s = 0; s < n; s += 8) {  // eight partials' columns in flight
            float4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = 4 * lane < D && ((some >> (s + i)) & 1u)
                           ? *reinterpret_cast<const float4 *>(ws + (size_t)(base + s + i) * (D + 4) + 4 * lane)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float wt = __shfl_sync(0xffffffffu, w, s + i);
                acc.x = fmaf(v[i].x, wt, acc.x);
                acc.y = fmaf(v[i].y, wt, acc.y);
                acc.z = fmaf(v[i].z, wt, acc.z);
                acc.w = fmaf(v[i].w, wt, acc.w);
            }
        }
    }
    const bool any = L != 0.f;
    const float inv = any ? 1.f / L : 0.f;
    if (4 * lane < D)
        *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(a.o) + (size_t)row * D + 4 * lane) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0 && a.lse) a.lse[row] = any ? kRowLn2 * (M + __log2f(L)) : -INFINITY;
}

// Splits of a row (a sequence's heads that one CTA takes) for the form whose splits are one cluster: it merges
// them through distributed shared memory, without the workspace and the second launch.  0: splits through the
// workspace.  The clusters are to be resident all at once (clusters of more than 4 leave some slots unused); a
// row that outruns its share is cut finer through the workspace, and so is a long context of so few rows that
// the clusters leave SMs empty.  Both ways, us (32 query heads, d 128 unless said; cluster / workspace):
//   1 sequence, 8 key/value heads    8 pages 4.8 / 6.4, 97 6.8 / 7.1, 262 8.8 / 9.6, 1000 16.3 / 24.1
//   the same, 2 key/value heads      51 pages 7.5 / 9.0, 262 11.4 / 11.4, 1000 22.5 / 19.8
//   8 sequences, 8 heads (6 splits)  22 pages 6.4 / 7.3, 250 15.6 / 20.8, 497 34.4 / 36.7; all in flight or not:
//                                    62 pages 8.2 with 6 splits, 12.9 with 8
//   32 sequences, 8 heads, e4m3 (2)  63 pages 13.2 / 17.1, 250 38.4 / 44.7, 497 70.6 / 71.2
//   the same in bf16 (1 split)       63 pages 17.0 / 19.1, 123 37.1 / 36.6, 497 125.9 / 118.2
//   128 sequences, 12 heads, d 64    7 pages 14.1 / 12.2 (not resident at once)
inline int cluster_splits(int B, int H, int Hkv, int d, int max_pages, bool fp8) {
    const int group = H / Hkv;
    const long long rows = (long long)B * Hkv * (group <= 8 ? 1 : (group + 15) / 16);
    const long long slots = 152 * (d > 64 && !fp8 ? 3 : 4);  // by shared memory, and by registers
    long long n = slots * 95 / 100 / rows;
    if (n > 4) n = slots * 85 / 100 / rows > 4 ? slots * 85 / 100 / rows : 4;
    if (n > kRowCluster) n = kRowCluster;
    if (n > (max_pages + kRowWarps - 1) / kRowWarps) n = (max_pages + kRowWarps - 1) / kRowWarps;
    if (max_pages > 32 * kRowWarps * n || (max_pages > 256 && rows * n < 128)) return 0;
    return (int)n;
}

// Page boxes of the rows kernel over a pool of `pool` page blocks.
template <int D>
bool encode_rows_maps(bool fp8, const void *k_pages, const void *v_pages, int pool, CUtensorMap &tk, CUtensorMap &tv) {
    return fp8 ? (encode_page_map_u8(&tk, k_pages, pool, kRowPS, D) && encode_page_map_u8(&tv, v_pages, pool, kRowPS, D))
               : (encode_qkv_map(&tk, k_pages, pool, kRowPS, D, kRowPS) &&
                  encode_qkv_map(&tv, v_pages, pool, kRowPS, D, kRowPS));
}

// Launches a kernel with the CTAs of each blockIdx.y, blockIdx.z as one cluster.
template <class K, class... A>
cudaError_t launch_cluster(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = grid.x;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The rows kernel (dependent: it may overlap the grid before it) and the merge, or one kernel whose
// clusters merge, where the device can place them.
template <int D, bool FP8, int NT, bool MOD>
cudaError_t launch_rows_n(RowsParams p, const CUtensorMap &tk, const CUtensorMap &tv, bool dependent,
                          cudaStream_t stream) {
    const size_t smem = sizeof(RowsSmem<D, FP8, NT>) + 1024;
    auto kernel = decode_rows_kernel<D, FP8, NT, MOD>;
    cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void *>(kernel), (int)smem);
    if (e != cudaSuccess) return e;
    const dim3 grid(p.n_splits, p.Hkv * p.rgroups, p.B);
    if (p.cluster) {
        if (p.cluster > 8) e = ensure_large_clusters(reinterpret_cast<const void *>(kernel));
        if (e == cudaSuccess && cluster_fits(reinterpret_cast<const void *>(kernel), p.cluster, kRowWarps * 32, smem)) {
            RowsParams c = p;
            c.n_splits = p.cluster;
            c.chunk_pages = 0;
            return launch_cluster(kernel, dim3(p.cluster, grid.y, grid.z), kRowWarps * 32, smem, stream, tk, tv, c);
        }
        (void)cudaGetLastError();
        p.cluster = 0;  // no room for the cluster (a part of a GPU): the splits go through the workspace
    }
    if (dependent) {
        e = launch_dependent(kernel, grid, kRowWarps * 32, smem, stream, tk, tv, p);
    } else {
        kernel<<<grid, kRowWarps * 32, smem, stream>>>(tk, tv, p);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
    const unsigned blocks = (unsigned)(((long long)p.B * p.H + 3) / 4);
    return launch_dependent(decode_rows_merge_kernel<D, MOD>, dim3(blocks), 128, 0, stream, p);
}

// Up to 8 query heads per key/value head take one n-tile of 8; larger groups take 16 heads per CTA.
template <int D, bool MOD>
cudaError_t launch_rows_d(RowsParams p, const CUtensorMap &tk, const CUtensorMap &tv, bool fp8, bool dependent,
                          cudaStream_t stream) {
    p.rgroups = p.group <= 8 ? 1 : (p.group + 15) / 16;
    if (fp8)
        return p.group <= 8 ? launch_rows_n<D, true, 1, MOD>(p, tk, tv, dependent, stream)
                            : launch_rows_n<D, true, 2, MOD>(p, tk, tv, dependent, stream);
    return p.group <= 8 ? launch_rows_n<D, false, 1, MOD>(p, tk, tv, dependent, stream)
                        : launch_rows_n<D, false, 2, MOD>(p, tk, tv, dependent, stream);
}

}  // namespace
}  // namespace attn
