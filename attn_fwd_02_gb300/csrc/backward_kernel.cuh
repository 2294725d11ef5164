// backward_kernel.cuh -- attention backward on the sm_103a tensor cores; instantiated by backward.cu and,
// for modified scores, by backward_scoremod.cu.
//
// The method (gpu-inference blog, section 02 "FlashAttention-2 in Triton"): the backward keeps
// no probability matrix; it recomputes the probabilities tile by tile from the log-sum-exp the
// forward saved, and it is split into three kernels: a pass that computes the row term
// D_i = dO_i . O_i, a dK/dV kernel and a dQ kernel.  With P = exp(s - LSE) on the valid keys
// (s = scale q.k), dP = dO V^T and dS = P * (dP - D):
//     dV = P^T dO,   dK = scale dS^T Q,   dQ = scale dS K.
//
// GB300 mapping of the two tile kernels (d in {32, 64, 80, 96, 128}):
//   * One CTA owns a 128-row tile of what it accumulates (dK and dV of 128 keys, or dQ of 128
//     queries) in TMEM, and streams the other side's 128-row tiles through a 2-slot TMA ring
//     (128-byte swizzled boxes of 128 rows x 64 columns).
//   * 10 warps.  Warps 0-7 are two compute warpgroups: thread r of warpgroup w owns TMEM lane r
//     (row r of the CTA's own tile) and columns 64w .. 64w+63 of each 128 x 128 score tile.
//     Warp 8 loads; warp 9 owns the TMEM and one of its threads issues every MMA.  (Capped scores: four
//     warpgroups of 32 columns, then those two warps.)
//   * dK/dV: S^T = K Q^T and dP^T = V dO^T land in TMEM with lane = key.  The warpgroups write
//     P^T and dS^T (bf16 pairs) back over the columns they read, where dV += P^T dO and
//     dK += dS^T Q take them as the A operand straight from TMEM.  Each Q or dO tile is the
//     K-major B operand of a score product and the MN-major B operand of an accumulation.
//     TMEM: S^T 128 | dP^T 128 | dV d | dK d columns.
//   * dQ: S = Q K^T and dP = dO V^T with lane = query; dS (bf16) over dP feeds dQ += dS K.
//     TMEM: S 128 | dP 128 | dQ d columns.
//   * Modified scores (forms F >= 0: an interval of keys per query and, bit 0, the cap, bit 1, the distance
//     bias of s = cap tanh(scale q.k / cap) - slope |distance|): P = exp(s - LSE) as before, and dS, the
//     gradient of the modified score, times 1 - tanh^2 is that of scale q.k.  P times that factor takes the place of P in registers once P itself is
//     packed, so the cap holds no further registers.  Key tiles visit the query tiles from the first to
//     the last whose intervals meet them (the row-term kernel also writes each query tile's interval).
//   * Issue order per step j.  dK/dV: dV(j), S^T(j+1), then dK(j), dP^T(j+1).  dQ: S(j+1),
//     then dQ(j), dP(j+1).  The tensor core computes the next scores while the warpgroups turn
//     dP(j) into dS(j), and the next dP while they turn S(j+1) into P(j+1).  The MMAs of one
//     thread run in issue order, so a product that overwrites a TMEM buffer never overtakes the
//     earlier product that reads the same columns as its operand.
#pragma once

#include <cmath>

#include "launch.h"
#include "scoremod.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kT = 128;  // rows of every tile (queries or keys)
// Forms: plain scores, or modified ones (kMod .. kMod + 3).
constexpr int kPlain = -1, kMod = 0;
template <int F> constexpr bool kIsMod = (F >= kMod);
template <int F> constexpr bool kHasCap = (F > 0 && (F & 1) != 0);
template <int F> constexpr bool kHasBias = (F > 0 && (F & 2) != 0);
// Compute warpgroups, and the columns of a score tile that each takes.  The capped forms do the most per score and
// take four of 32 columns, whose warps hide one another's latency; the others two of 64.  Measured (causal, 16
// heads x 8192, the whole backward, four / two): d 128 cap 1049 / 1080 us, cap and bias 1151 / 1217, no cap 964 /
// 930, bias 1057 / 1018; d 64 cap 889 / 949, both 984 / 1123, no cap 775 / 722, bias 902 / 854.  (With the distances
// multiplied as they are, the forms kept take 1021 for the bias and 1143 for both; at d 64 843 and 966.)
template <int F> constexpr int kGroups = kHasCap<F> ? 4 : 2;
template <int F> constexpr int kCols = kT / kGroups<F>;
// Two groups of a modified form hold more per thread than the plain form's: a third warpgroup is launched whose
// idle warps give it their registers (setmaxnreg: 128 x (2 x 216 + 64) of the 384 x 168 at launch; with 320 threads
// the dK/dV kernel spilled 528 bytes).
template <int F> constexpr bool kSplitRegs = kIsMod<F> && kGroups<F> == 2;
template <int F> constexpr int kThreadsOf = 128 * kGroups<F> + (kSplitRegs<F> ? 128 : 64);
constexpr uint32_t kRegsCompute = 216, kRegsOther = 64;
template <int F> constexpr int kProducerWarp = 4 * kGroups<F>;
template <int F> constexpr int kMmaWarp = kProducerWarp<F> + 1;
constexpr int kStages = 2;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kBoxBytes = 128 * 64 * 2;  // one 128-row x 64-column bf16 box
constexpr float kLog2e = 1.4426950408889634f;
constexpr unsigned kFull = 0xffffffffu;
// Tiles are padded to 64 (d <= 64) or 128 columns of 64-column TMA boxes, which read zeros past d:
// the score products run over d/16 k-steps and the accumulations over N = d columns, so the padding
// costs shared memory only.  Accumulators in TMEM sit at padded column offsets.
template <int D> constexpr int kBPad = D <= 64 ? 64 : 128;
template <int D> constexpr int kBBoxes = kBPad<D> / 64;
// dQ columns of the first warpgroup (the second takes the rest): halves in multiples of 16
template <int D> constexpr int kDqSplit = ((D / 16 + 1) / 2) * 16;

struct BwdParams {
    const float *lse, *dterm;
    __nv_bfloat16 *dq, *dk, *dv;
    const int32_t *kv_lens;
    int *status;
    int B, Hq, Hkv, group, Nq, Nkv, causal;
    int units_per_head;   // query tiles (dQ kernel) or key tiles (dK/dV kernel) of one head
    int heads_per_chunk;  // heads whose streamed operands share L2 at a time
    float scale, scale_log2;
};
// With modified scores (see the forward's parameters); spans [B, query tiles] holds the union {lo, hi} of
// the intervals of a query tile's rows.  A type of its own: the plain kernels' registers depend on the
// size of their parameters (spilled bytes of the dK/dV kernel 20 / 12 without these fields, 56 / 76 with).
struct BwdModParams : BwdParams {
    const int32_t *key_begin, *key_end;
    const float *slopes;
    float cap_in, cap_out;
    int2 *spans;
    int kv_target;    // dK/dV kernel: steps of a key tile that a CTA is to take (0: all of them); see tile_splits
    float *kv_parts;  // the sums of key tiles with several CTAs: [CTA][dV, dK][B, Hkv, Nkv, d]
};
template <bool MOD> struct ParamsOf { using type = BwdParams; };
template <> struct ParamsOf<true> { using type = BwdModParams; };
template <int F> using Params = typename ParamsOf<kIsMod<F>>::type;

// CTAs of key tile t in the dK/dV kernel: equal shares of its steps (query tiles x query heads of the group, as the
// causal mask leaves them; the intervals, which may leave fewer, are on the device), of at most `target` steps where
// kMaxSplits shares allow it, else kMaxSplits longer ones.
constexpr int kMaxSplits = 16;
__host__ __device__ inline int tile_splits(int t, int target, int group, int Nq, int Nkv, bool causal) {
    if (target <= 0) return 1;
    const int n_qt = (Nq + kT - 1) / kT, first = causal ? (t * kT - (Nkv - Nq)) / kT : 0;
    const int steps = group * (n_qt - (first > 0 ? first : 0)), n = (steps + target - 1) / target;
    return n < 1 ? 1 : (n > kMaxSplits ? kMaxSplits : n);
}

// Keys lo <= j < hi that query `row` of sequence b sees (none past the last query).
__device__ __forceinline__ int2 bwd_row_span(const BwdModParams &p, int b, int row, int kv_end) {
    if (row >= p.Nq) return make_int2(0, 0);
    const size_t at = (size_t)b * p.Nq + row;
    int2 s;
    s.x = p.key_begin ? max(p.key_begin[at], 0) : 0;
    s.y = p.key_end ? min(p.key_end[at], kv_end) : kv_end;
    if (p.causal) s.y = min(s.y, row + p.Nkv - p.Nq + 1);
    return s.x < s.y ? s : make_int2(0, 0);  // (the bounds given may be any int)
}

// CTA order (as in the forward): heads in chunks small enough that the chunk's streamed tiles
// stay in L2; inside a chunk, unit levels in order (level 0 = the heaviest unit of a head
// under the causal mask) across the chunk's heads.
__device__ __forceinline__ void unit_of(const BwdParams &p, int n_heads, unsigned unit, int &head, int &level) {
    const int per_chunk = p.heads_per_chunk * p.units_per_head;
    const int chunk = (int)(unit / per_chunk);
    const int h0 = chunk * p.heads_per_chunk;
    const int heads = min(p.heads_per_chunk, n_heads - h0);
    const int in_chunk = (int)(unit % per_chunk);
    level = in_chunk / heads;
    head = h0 + in_chunk % heads;
}

__device__ __forceinline__ int kv_end_for(const BwdParams &p, int b) {
    return p.kv_lens ? min(max(p.kv_lens[b], 0), p.Nkv) : p.Nkv;
}

// 128 x 128 score tile: D[tmem] = A B^T over the head dimension (both operands K-major tiles).
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t d_tmem, const __nv_bfloat16 *a, const __nv_bfloat16 *b) {
    constexpr uint32_t id = idesc_bf16_f32(kT, kT, false, false);
    const uint64_t da = sdesc_sw128(smem_u32(a), 16, 1024), db = sdesc_sw128(smem_u32(b), 16, 1024);
    static_assert(kBoxBytes == 16384, "k-step layout of the grouped issue");
    tc_mma_ss_ksteps<D / 16>(d_tmem, da, db, id, 0u);
}

// tc_mma_ts_k8_halves for A in four groups of two k-steps, 32 columns apart.
#define ATTN_TS_QUARTER(COLS, STEP)                                                                   \
    "add.u32 ta, %1, " #COLS ";\n\tadd.s64 rb, %2, " #STEP                                            \
    ";\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [ta], rb, %3, q;\n\t"
__device__ __forceinline__ void tc_mma_ts_k8_quarters(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                                      uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 ta;\n\t.reg .b64 rb;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, %4, %4;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        ATTN_TS_QUARTER(8, 128) ATTN_TS_QUARTER(32, 256) ATTN_TS_QUARTER(40, 384) ATTN_TS_QUARTER(64, 512)
        ATTN_TS_QUARTER(72, 640) ATTN_TS_QUARTER(96, 768) ATTN_TS_QUARTER(104, 896) "}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
#undef ATTN_TS_QUARTER

// 128 x d accumulation: D[tmem] (+)= A[tmem] B, A = 128 x 128 bf16 written by the warpgroups (each its
// columns' pairs at the first of them: k-indices 0-63 and 64-127 in columns 0-31 and 64-95 of a_tmem, or
// 0-31 in columns 0-15 and so on), B = a 128-row tile read MN-major (k-index = tile row).
template <int D, int F>
__device__ __forceinline__ void mma_accum(uint32_t d_tmem, uint32_t a_tmem, const __nv_bfloat16 *b, bool first) {
    constexpr uint32_t id = idesc_bf16_f32(kT, D, false, true);
    const uint64_t db = sdesc_sw128(smem_u32(b), kBoxBytes, 1024);
    static_assert(kT / 16 == 8, "one group of eight k-steps");
    if constexpr (kGroups<F> == 2) tc_mma_ts_k8_halves(d_tmem, a_tmem, db, id, first ? 0u : 1u);
    else tc_mma_ts_k8_quarters(d_tmem, a_tmem, db, id, first ? 0u : 1u);
}

// The bias -slope |d| (log2 domain) over a row of columns at distances d = d0 + Step c (Step 1: columns are
// queries, -1: columns are keys); nonneg, nonpos: d has one sign over the whole tile, and |d| needs no operation.  The
// distances are whole numbers, so that the products are exact to a rounding however steep the slope.
template <int Step>
struct Distance {
    float mul, d0;
    bool linear;
    __device__ __forceinline__ void set(float slope, int d, bool nonneg, bool nonpos) {
        linear = nonneg || nonpos;
        mul = nonneg || !nonpos ? -slope : slope;
        d0 = (float)d;
    }
    __device__ __forceinline__ float add(int c, float e) const {
        const float d = d0 + (float)(Step * c);
        return fmaf(mul, linear ? d : fabsf(d), e);
    }
};

// The cap's scale / cap (0 without it), and the factor that takes the raw scores -- with the cap their tanh
// -- to the log2 domain.
template <int F> __device__ __forceinline__ float cap_in_of(const Params<F> &p) {
    if constexpr (kHasCap<F>) return p.cap_in;
    else return 0.f;
}
template <int F> __device__ __forceinline__ float score_factor(const Params<F> &p) {
    if constexpr (kHasCap<F>) return p.cap_out;
    else return p.scale_log2;
}

// 32 H TMEM columns of this thread's lane -> registers.
template <int H>
__device__ __forceinline__ void load_cols(uint32_t taddr, uint32_t (&x)[H][32]) {
#pragma unroll
    for (int h = 0; h < H; ++h) tmem_ld32(taddr + 32 * h, x[h]);
#pragma unroll
    for (int h = 0; h < H; ++h) tmem_wait_ld(x[h]);
}

// Writes NCOLS (a multiple of 16) columns of this thread's row of an fp32 TMEM accumulator,
// times `mul`, as bf16 to dst (`store` false skips the write).  Zeros if !have.
template <int NCOLS>
__device__ __forceinline__ void store_rows(uint32_t tacc, bool have, bool store, float mul, __nv_bfloat16 *dst) {
    static_assert(NCOLS % 16 == 0, "16-column steps");
#pragma unroll
    for (int cc = 0; cc < NCOLS / 32; ++cc) {
        uint32_t v[32];
        if (have) {
            tmem_ld32(tacc + cc * 32, v);
            tmem_wait_ld(v);
        }
        if (store) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                pk[i] = have ? pack_bf16x2(__uint_as_float(v[2 * i]) * mul, __uint_as_float(v[2 * i + 1]) * mul) : 0u;
            uint4 *o = reinterpret_cast<uint4 *>(dst + cc * 32);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
        }
    }
    if constexpr (NCOLS % 32 != 0) {  // the last 16 columns
        constexpr int c0 = NCOLS / 32 * 32;
        uint32_t v[16];
        if (have) {
            tmem_ld16(tacc + c0, v);
            tmem_wait_ld16(v);
        }
        if (store) {
            uint32_t pk[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                pk[i] = have ? pack_bf16x2(__uint_as_float(v[2 * i]) * mul, __uint_as_float(v[2 * i + 1]) * mul) : 0u;
            uint4 *o = reinterpret_cast<uint4 *>(dst + c0);
            o[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            o[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
        }
    }
}

// The same columns as fp32.
template <int NCOLS>
__device__ __forceinline__ void store_rows_f32(uint32_t tacc, bool have, bool store, float *dst) {
#pragma unroll
    for (int cc = 0; cc < NCOLS / 16; ++cc) {
        uint32_t v[16];
        if (have) {
            tmem_ld16(tacc + cc * 16, v);
            tmem_wait_ld16(v);
        }
        if (store)
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4 *>(dst + cc * 16 + i) =
                    have ? make_float4(__uint_as_float(v[i]), __uint_as_float(v[i + 1]), __uint_as_float(v[i + 2]),
                                       __uint_as_float(v[i + 3]))
                         : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

// ================================================================== row term D = rowsum(dO * O)
// kTpr threads per row (d / 8 rounded up to a power of two), one 16-byte load of O and of dO each
// for the threads whose 8 columns lie inside d, then a shuffle reduction.
template <int D> constexpr int kRowThreads = D / 8 <= 4 ? 4 : (D / 8 <= 8 ? 8 : 16);
template <int D>
__device__ __forceinline__ void rowdot(const __nv_bfloat16 *o, const __nv_bfloat16 *dout, float *dterm,
                                       long long rows) {
    constexpr int kTpr = kRowThreads<D>;
    const long long gid = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long row = gid / kTpr;
    const int part = (int)(gid % kTpr);
    float acc = 0.f;
    if (row < rows && part * 8 < D) {
        const uint4 a = *reinterpret_cast<const uint4 *>(o + row * D + part * 8);
        const uint4 b = *reinterpret_cast<const uint4 *>(dout + row * D + part * 8);
        const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 fa = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&av[i]));
            const float2 fb = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&bv[i]));
            acc = fmaf(fa.x, fb.x, acc);
            acc = fmaf(fa.y, fb.y, acc);
        }
    }
#pragma unroll
    for (int off = kTpr / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(kFull, acc, off);
    if (row < rows && part == 0) dterm[row] = acc;
}
template <int D>
__global__ void __launch_bounds__(256) bwd_rowdot_kernel(const __nv_bfloat16 *o, const __nv_bfloat16 *dout,
                                                         float *dterm, long long rows) {
    rowdot<D>(o, dout, dterm, rows);
}

// The row term and, in the blocks after the first row_blocks, the intervals of two query tiles each.
template <int D>
__global__ void __launch_bounds__(256) bwd_rowdot_spans_kernel(const __nv_bfloat16 *o, const __nv_bfloat16 *dout,
                                                               float *dterm, long long rows, int row_blocks,
                                                               const BwdModParams p, int n_qt) {
    if ((int)blockIdx.x < row_blocks) {
        rowdot<D>(o, dout, dterm, rows);
        return;
    }
    __shared__ int2 part[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long tile = ((long long)blockIdx.x - row_blocks) * 2 + warp / 4;
    int2 s = make_int2(0, 0);
    if (tile < (long long)p.B * n_qt) {
        const int b = (int)(tile / n_qt), qt = (int)(tile % n_qt);
        s = bwd_row_span(p, b, qt * kT + ((int)threadIdx.x & 127), kv_end_for(p, b));
    }
    const bool some = s.x < s.y;
    const int lo = __reduce_min_sync(kFull, some ? s.x : 0x7fffffff), hi = __reduce_max_sync(kFull, some ? s.y : 0);
    if (lane == 0) part[warp] = make_int2(lo, hi);
    __syncthreads();
    if ((threadIdx.x & 127) == 0 && tile < (long long)p.B * n_qt) {
        int2 u = part[warp];
        for (int w = 1; w < 4; ++w) u = make_int2(min(u.x, part[warp + w].x), max(u.y, part[warp + w].y));
        p.spans[tile] = u;
    }
}

// ================================================================== dK / dV
// Modified forms: a streamed query tile's intervals, slope and whether every row sees all the CTA's keys
template <bool MOD> struct QuerySpans {};
template <> struct QuerySpans<true> {
    int4 lo[kStages][kT / 4], hi[kStages][kT / 4];
    float slope2[kStages];
    int inside[kStages];
    int first, last;  // query tiles that see one of the CTA's keys
};

template <int D>
struct alignas(1024) DkvTiles {
    __nv_bfloat16 k[kT * kBPad<D>];              // the CTA's 128 keys (kBBoxes boxes)
    __nv_bfloat16 v[kT * kBPad<D>];
    __nv_bfloat16 q[kStages][kT * kBPad<D>];     // streamed query tiles
    __nv_bfloat16 dout[kStages][kT * kBPad<D>];  // and their upstream gradients
    float nlse2[kStages][kT];             // minus the log2-domain LSE of each streamed query (0 past Nq)
    float dterm[kStages][kT];             // row term D of each streamed query (0 past Nq)
    uint64_t kv_full;
    uint64_t u_full[kStages], u_empty[kStages];
    uint64_t s_full, p_full, dp_full, ds_full, acc_done, drain;
    uint32_t tmem_base;
    int abort_flag;
};
template <int D, int F> struct DkvSmem : DkvTiles<D>, QuerySpans<kIsMod<F>> {};

// Query tiles a key tile [k0, k0+128) must visit: queries i >= k0 - delta can see its keys
// under the causal mask (query i sees key j iff j <= i + delta).
__device__ __forceinline__ void dkdv_range(const BwdParams &p, int k0, int kv_end, int delta, int &qi_start,
                                           int &nqt) {
    const int n_qt = (p.Nq + kT - 1) / kT;
    qi_start = 0;
    nqt = 0;
    if (k0 >= kv_end) return;
    if (p.causal) {
        const int first = k0 - delta;
        if (first >= p.Nq) return;
        qi_start = first > 0 ? first / kT : 0;
    }
    nqt = n_qt - qi_start;
}

template <int D, int F>
__device__ void dkdv_producer(DkvSmem<D, F> &sm, const Params<F> &p, const CUtensorMap *tmQ, const CUtensorMap *tmdO,
                              const CUtensorMap *tmK, const CUtensorMap *tmV, int b, int hkv, int bh_kv, int k0,
                              int qi_start, int nqt, int u0, int n, WaitCtx wc) {
    constexpr int kBoxes = kBBoxes<D>;
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
        prefetch_tensormap(tmQ);
        prefetch_tensormap(tmdO);
        mbar_arrive_expect_tx(&sm.kv_full, 2 * kBoxes * kBoxBytes);
#pragma unroll
        for (int i = 0; i < kBoxes; ++i) {
            tma_load_3d(sm.k + i * (kT * 64), tmK, &sm.kv_full, i * 64, k0, bh_kv);
            tma_load_3d(sm.v + i * (kT * 64), tmV, &sm.kv_full, i * 64, k0, bh_kv);
        }
    }
    // the row statistics of unit u's 128 queries, four per lane (plain loads, zeros past Nq); they
    // are loaded one unit ahead so their latency hides behind the ring wait
    auto load_stats = [&](int u, float (&l4)[4], float (&d4)[4]) {
        const int bh_q = b * p.Hq + hkv * p.group + (u0 + u) / nqt;
        const int q0 = (qi_start + (u0 + u) % nqt) * kT;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int row = q0 + lane * 4 + t;
            l4[t] = 0.f;
            d4[t] = 0.f;
            if (row < p.Nq) {
                l4[t] = p.lse[(size_t)bh_q * p.Nq + row];
                d4[t] = p.dterm[(size_t)bh_q * p.Nq + row];
            }
        }
    };
    float l4n[4], d4n[4];
    load_stats(0, l4n, d4n);
    int2 s4n[4] = {};
    float slope_n = 0.f;
    const int kv_end = kv_end_for(p, b);
    auto load_spans = [&](int u) {
        if constexpr (kIsMod<F>) {
#pragma unroll
            for (int t = 0; t < 4; ++t) s4n[t] = bwd_row_span(p, b, (qi_start + (u0 + u) % nqt) * kT + lane * 4 + t, kv_end);
            slope_n = p.slopes ? bias_slope(p.slopes[hkv * p.group + (u0 + u) / nqt]) : 0.f;
        }
    };
    if constexpr (kIsMod<F>) load_spans(0);
    int fills = 0;
    for (int u = 0; u < n; ++u) {
        const int slot = u % kStages, use = u / kStages;
        if (use > 0 && !__all_sync(kFull, mbar_wait(&sm.u_empty[slot], (uint32_t)((use - 1) & 1), wc, 60))) break;
        const int g = (u0 + u) / nqt, qi = qi_start + (u0 + u) % nqt;
        const int bh_q = b * p.Hq + hkv * p.group + g;
        const int q0 = qi * kT;
        *reinterpret_cast<float4 *>(&sm.nlse2[slot][lane * 4]) =
            make_float4(l4n[0] * -kLog2e, l4n[1] * -kLog2e, l4n[2] * -kLog2e, l4n[3] * -kLog2e);
        *reinterpret_cast<float4 *>(&sm.dterm[slot][lane * 4]) = make_float4(d4n[0], d4n[1], d4n[2], d4n[3]);
        if (u + 1 < n) load_stats(u + 1, l4n, d4n);
        if constexpr (kIsMod<F>) {
            sm.lo[slot][lane] = make_int4(s4n[0].x, s4n[1].x, s4n[2].x, s4n[3].x);
            sm.hi[slot][lane] = make_int4(s4n[0].y, s4n[1].y, s4n[2].y, s4n[3].y);
            bool all = true;
#pragma unroll
            for (int t = 0; t < 4; ++t) all = all && s4n[t].x <= k0 && s4n[t].y >= k0 + kT;
            all = __all_sync(kFull, all);
            if (lane == 0) {
                sm.inside[slot] = all ? 1 : 0;
                sm.slope2[slot] = slope_n;
            }
            if (u + 1 < n) load_spans(u + 1);
        }
        if (lane == 0) {
            mbar_arrive_expect_tx(&sm.u_full[slot], 2 * kBoxes * kBoxBytes);
#pragma unroll
            for (int i = 0; i < kBoxes; ++i) {
                tma_load_3d(sm.q[slot] + i * (kT * 64), tmQ, &sm.u_full[slot], i * 64, q0, bh_q);
                tma_load_3d(sm.dout[slot] + i * (kT * 64), tmdO, &sm.u_full[slot], i * 64, q0, bh_q);
            }
        } else {
            mbar_arrive(&sm.u_full[slot]);
        }
        ++fills;
    }
    if (lane == 0 && *wc.abort_flag) {
        // unwinding: let every copy still in flight land before the CTA exits
        WaitCtx drain{nullptr, wc.status};
        (void)mbar_wait(&sm.kv_full, 0, drain, 61);
        for (int f = (fills > kStages ? fills - kStages : 0); f < fills; ++f)
            (void)mbar_wait(&sm.u_full[f % kStages], (uint32_t)((f / kStages) & 1), drain, 62);
    }
}

template <int D, int F>
__device__ void dkdv_mma(DkvSmem<D, F> &sm, uint32_t tmem, int n, WaitCtx wc) {
    const uint32_t tS = tmem, tdP = tmem + 128, tdV = tmem + 256, tdK = tmem + 256 + kBPad<D>;
    bool ok = mbar_wait(&sm.kv_full, 0, wc, 63) && mbar_wait(&sm.u_full[0], 0, wc, 64);
    if (ok) {
        tc_fence_after_sync();
        mma_scores<D>(tS, sm.k, sm.q[0]);
        tc_commit(&sm.s_full);
        mma_scores<D>(tdP, sm.v, sm.dout[0]);
        tc_commit(&sm.dp_full);
        for (int j = 0; j < n; ++j) {
            const int slot = j % kStages;
            if (!(ok = mbar_wait(&sm.p_full, (uint32_t)(j & 1), wc, 65))) break;
            tc_fence_after_sync();
            mma_accum<D, F>(tdV, tS, sm.dout[slot], j == 0);  // dV += P^T dO
            if (j + 1 < n) {
                const int u = j + 1;
                if (!(ok = mbar_wait(&sm.u_full[u % kStages], (uint32_t)((u / kStages) & 1), wc, 66))) break;
                mma_scores<D>(tS, sm.k, sm.q[u % kStages]);  // S^T(j+1), after dV(j) read P^T(j)
                tc_commit(&sm.s_full);
            }
            if (!(ok = mbar_wait(&sm.ds_full, (uint32_t)(j & 1), wc, 67))) break;
            tc_fence_after_sync();
            mma_accum<D, F>(tdK, tdP, sm.q[slot], j == 0);  // dK += dS^T Q
            tc_commit(&sm.u_empty[slot]);
            if (j == n - 1) tc_commit(&sm.acc_done);
            if (j + 1 < n) {
                mma_scores<D>(tdP, sm.v, sm.dout[(j + 1) % kStages]);  // dP^T(j+1), after dK(j) read dS^T(j)
                tc_commit(&sm.dp_full);
            }
        }
    }
    tc_commit(&sm.drain);
    WaitCtx drain{nullptr, wc.status};
    (void)mbar_wait(&sm.drain, 0, drain, 68);
}

template <int D, int F>
__device__ void dkdv_compute(DkvSmem<D, F> &sm, const Params<F> &p, uint32_t tmem, int w, int bh_kv, int k0,
                             int kv_end, int delta, int qi_start, int nqt, int u0, int n, int split, int splits, WaitCtx wc) {
    constexpr int kC = kCols<F>, kH = kC / 32;
    const int r = threadIdx.x & 127;
    const uint32_t lane_base = tmem + ((uint32_t)(((threadIdx.x >> 5) & 3) * 32) << 16);
    const uint32_t tS = lane_base + (uint32_t)(w * kC);
    const uint32_t tdP = lane_base + 128u + (uint32_t)(w * kC);
    const int key = k0 + r;
    const bool key_ok = key < kv_end;
    // with the cap, the scores become tanh in place and the factor to the log2 domain is cap * log2(e)
    [[maybe_unused]] const TanhCap cap(cap_in_of<F>(p), 1.f);
    const float to_log2 = score_factor<F>(p);
    const uint64_t c2 = f32x2_pack(to_log2, to_log2);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
        const int slot = j % kStages;
        const int col0 = (qi_start + (u0 + j) % nqt) * kT + w * kC;  // query of this part's column 0
        // valid columns lo <= c < hi: query < Nq, key < kv_end, and key <= query + delta if causal
        int lo = 0, hi = min(kC, p.Nq - col0);
        if (p.causal) lo = max(0, key - delta - col0);
        if (!key_ok) hi = 0;
        bool need_mask = lo > 0 || hi < kC;

        // The columns' statistics are read before the score waits so that their latency hides
        // behind them.  The producer wrote them before arriving on the unit's full barrier; waiting
        // on that barrier (without arriving) orders these reads after its writes.  The slot cannot
        // be refilled before this step ends (the refill waits for dK(j), which needs this step's dS).
        if (!__all_sync(kFull, mbar_wait(&sm.u_full[slot], (uint32_t)((j / kStages) & 1), wc, 73))) {
            ok = false;
            break;
        }
        if constexpr (kIsMod<F>) need_mask = sm.inside[slot] == 0;
        constexpr int kAheadStats = kGroups<F> == 2 ? kC / 4 : 0;  // (four groups hide the latency, and lack the registers)
        float4 L4[kAheadStats + 1];
        const float4 *l2 = reinterpret_cast<const float4 *>(sm.nlse2[slot] + w * kC);
#pragma unroll
        for (int i = 0; i < kAheadStats; ++i) L4[i] = l2[i];
        if (!__all_sync(kFull, mbar_wait(&sm.s_full, (uint32_t)(j & 1), wc, 70))) {
            ok = false;
            break;
        }
        tc_fence_after_sync();
        uint32_t x[kH][32];
        load_cols(tS, x);
        if constexpr (kHasCap<F>) cap.apply(cap.tier(abs_max(x)), x);
        // column c is the query at position col0 + c + delta; under the causal mask the keys after it are
        // masked, so the linear form serves there too
        [[maybe_unused]] Distance<1> dist;
        if constexpr (kHasBias<F>) {
            const int first = col0 + delta;
            dist.set(sm.slope2[slot], first - key, p.causal || first >= k0 + kT - 1, first + kC - 1 <= k0);
        }
        // P^T = 2^(s * scale * log2e - lse2): bf16 pairs over the scores, fp32 kept in x
#pragma unroll
        for (int h = 0; h < kH; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 L = kAheadStats ? L4[(h * 32 + i) / 4] : l2[(h * 32 + i) / 4];
                const uint64_t x01 = f32x2_pack(__uint_as_float(x[h][i]), __uint_as_float(x[h][i + 1]));
                const uint64_t x23 = f32x2_pack(__uint_as_float(x[h][i + 2]), __uint_as_float(x[h][i + 3]));
                [[maybe_unused]] float g[4];  // 1 - tanh^2
                if constexpr (kHasCap<F>) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        g[t] = fmaf(-__uint_as_float(x[h][i + t]), __uint_as_float(x[h][i + t]), 1.f);
                }
                const uint64_t e01 = f32x2_fma(x01, c2, f32x2_pack(L.x, L.y));
                const uint64_t e23 = f32x2_fma(x23, c2, f32x2_pack(L.z, L.w));
                float e[4];
                f32x2_unpack(e01, e[0], e[1]);
                f32x2_unpack(e23, e[2], e[3]);
                if constexpr (kHasBias<F>) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) e[t] = dist.add(h * 32 + i + t, e[t]);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    float pv = ex2_approx(e[t]);
                    if constexpr (!kIsMod<F>) {
                        if (need_mask) {
                            const int c = h * 32 + i + t;
                            pv = (c >= lo && c < hi) ? pv : 0.f;
                        }
                    }
                    x[h][i + t] = __float_as_uint(pv);
                }
                if constexpr (kIsMod<F>) {
                    if (need_mask) {  // the columns' intervals, four queries at a time
                        const int4 a = sm.lo[slot][(w * kC + h * 32 + i) / 4], z = sm.hi[slot][(w * kC + h * 32 + i) / 4];
                        const int al[4] = {a.x, a.y, a.z, a.w}, zl[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                        for (int t = 0; t < 4; ++t)
                            if (key < al[t] || key >= zl[t]) x[h][i + t] = 0u;
                    }
                }
                pk[i / 2] = pack_bf16x2(__uint_as_float(x[h][i]), __uint_as_float(x[h][i + 1]));
                pk[i / 2 + 1] = pack_bf16x2(__uint_as_float(x[h][i + 2]), __uint_as_float(x[h][i + 3]));
                if constexpr (kHasCap<F>) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const float pg = __uint_as_float(x[h][i + t]) * g[t];
                        x[h][i + t] = need_mask && x[h][i + t] == 0u ? 0u : __float_as_uint(pg);  // masked: stays 0
                    }
                }
            }
            tmem_st16(tS + (uint32_t)(h * 16), pk);
        }
        tmem_wait_st();
        tc_fence_before_sync();
        mbar_arrive(&sm.p_full);

        float4 D4[kAheadStats + 1];
        const float4 *dd = reinterpret_cast<const float4 *>(sm.dterm[slot] + w * kC);
#pragma unroll
        for (int i = 0; i < kAheadStats; ++i) D4[i] = dd[i];
        if (!__all_sync(kFull, mbar_wait(&sm.dp_full, (uint32_t)(j & 1), wc, 71))) {
            ok = false;
            break;
        }
        tc_fence_after_sync();
        uint32_t y[kH][32];
        load_cols(tdP, y);
        // dS^T = P^T * (dP^T - D): bf16 pairs over dP^T
#pragma unroll
        for (int h = 0; h < kH; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 Dv = kAheadStats ? D4[(h * 32 + i) / 4] : dd[(h * 32 + i) / 4];
                float s0 = __uint_as_float(x[h][i]) * (__uint_as_float(y[h][i]) - Dv.x);
                float s1 = __uint_as_float(x[h][i + 1]) * (__uint_as_float(y[h][i + 1]) - Dv.y);
                float s2 = __uint_as_float(x[h][i + 2]) * (__uint_as_float(y[h][i + 2]) - Dv.z);
                float s3 = __uint_as_float(x[h][i + 3]) * (__uint_as_float(y[h][i + 3]) - Dv.w);
                if constexpr (kIsMod<F>) {
                    if (need_mask) {  // dP of a masked key may be anything
                        s0 = x[h][i] ? s0 : 0.f;
                        s1 = x[h][i + 1] ? s1 : 0.f;
                        s2 = x[h][i + 2] ? s2 : 0.f;
                        s3 = x[h][i + 3] ? s3 : 0.f;
                    }
                }
                pk[i / 2] = pack_bf16x2(s0, s1);
                pk[i / 2 + 1] = pack_bf16x2(s2, s3);
            }
            tmem_st16(tdP + (uint32_t)(h * 16), pk);
        }
        tmem_wait_st();
        tc_fence_before_sync();
        mbar_arrive(&sm.ds_full);
    }

    if (ok && n > 0) {
        if (!__all_sync(kFull, mbar_wait(&sm.acc_done, 0, wc, 72))) ok = false;
        else tc_fence_after_sync();
    }
    if (!ok) return;
    // dV, and dK (times scale), a warpgroup each or two; rows past Nkv are not stored
    const bool store = key < p.Nkv;
    const size_t row = (size_t)bh_kv * p.Nkv + (store ? key : 0);
    const bool is_k = w >= kGroups<F> / 2;
    const uint32_t acc = lane_base + 256u + (is_k ? (uint32_t)kBPad<D> : 0u);
    const float mul = is_k ? p.scale : 1.f;
    constexpr int c1 = kDqSplit<D>;  // of two: the second one's first column
    if constexpr (kIsMod<F>) {
        if (splits > 1) {  // a part of the queries: fp32 sums, added up by the reduction kernel
            const size_t part = (size_t)split * 2 + (is_k ? 1 : 0);
            float *out = p.kv_parts + (part * p.B * p.Hkv * p.Nkv + row) * D;
            if constexpr (kGroups<F> == 2) store_rows_f32<D>(acc, n > 0, store, out);
            else if (w & 1) store_rows_f32<D - c1>(acc + c1, n > 0, store, out + c1);
            else store_rows_f32<c1>(acc, n > 0, store, out);
            return;
        }
    }
    __nv_bfloat16 *dst = (is_k ? p.dk : p.dv) + row * D;
    if constexpr (kGroups<F> == 2) store_rows<D>(acc, n > 0, store, mul, dst);
    else if (w & 1) store_rows<D - c1>(acc + c1, n > 0, store, mul, dst + c1);
    else store_rows<c1>(acc, n > 0, store, mul, dst);
}

template <int D, int F>
__global__ void __launch_bounds__(kThreadsOf<F>, 1)
    bwd_dkdv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
                    const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const Params<F> p) {
    extern __shared__ uint8_t smem_raw[];
    DkvSmem<D, F> &sm =
        *reinterpret_cast<DkvSmem<D, F> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    int bh_kv, level, split = 0, splits = 1;
    bool shared_out = false;
    if constexpr (kIsMod<F>) shared_out = p.kv_target > 0;
    if (!shared_out) unit_of(p, p.B * p.Hkv, blockIdx.x, bh_kv, level);
    if constexpr (kIsMod<F>) {
        if (shared_out) {
            const int heads = p.B * p.Hkv;
            int at = (int)blockIdx.x;
            for (level = 0;; ++level) {  // key tiles in order across the heads, the longest shares first
                splits = tile_splits(level, p.kv_target, p.group, p.Nq, p.Nkv, p.causal != 0);
                if (at < splits * heads) break;
                at -= splits * heads;
            }
            bh_kv = at % heads;
            split = at / heads;
        }
    }
    const int b = bh_kv / p.Hkv, hkv = bh_kv % p.Hkv;
    const int k0 = level * kT;  // level 0 = key tile 0, seen by the most queries when causal
    const int kv_end = kv_end_for(p, b);
    const int delta = p.Nkv - p.Nq;
    int qi_start = 0, nqt = 0;
    if constexpr (!kIsMod<F>) {
        dkdv_range(p, k0, kv_end, delta, qi_start, nqt);
    }
    int n = nqt * p.group;  // steps: every query tile of every query head of the group

    if (threadIdx.x == 0) {
        if constexpr (kIsMod<F>) {
            sm.first = 0x7fffffff;
            sm.last = -1;
        }
        mbar_init(&sm.kv_full, 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm.u_full[s], 32);
            mbar_init(&sm.u_empty[s], 1);
        }
        mbar_init(&sm.s_full, 1);
        mbar_init(&sm.p_full, 128 * kGroups<F>);
        mbar_init(&sm.dp_full, 1);
        mbar_init(&sm.ds_full, 128 * kGroups<F>);
        mbar_init(&sm.acc_done, 1);
        mbar_init(&sm.drain, 1);
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp<F>) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sm.tmem_base;
    WaitCtx wc{&sm.abort_flag, p.status};
    int u0 = 0;  // first of the CTA's steps
    if constexpr (kIsMod<F>) {
        // the row-term kernel's results are complete from here on; the dQ kernel may start as CTAs leave
        griddep_wait();
        griddep_launch_dependents();
        const int n_qt = (p.Nq + kT - 1) / kT;
        int first = 0x7fffffff, last = -1;
        for (int qi = threadIdx.x; qi < n_qt; qi += kThreadsOf<F>) {
            const int2 s = p.spans[(size_t)b * n_qt + qi];
            if (s.x < k0 + kT && s.y > k0) {
                first = min(first, qi);
                last = qi;
            }
        }
        if (last >= 0) {
            atomicMin(&sm.first, first);
            atomicMax(&sm.last, last);
        }
        __syncthreads();
        if (sm.last >= 0) {
            qi_start = sm.first;
            nqt = sm.last - sm.first + 1;
        }
        const int all = nqt * p.group;
        u0 = (int)((long long)all * split / splits);
        n = (int)((long long)all * (split + 1) / splits) - u0;
    }

    // (each role inside the branch that sets its registers: code after a join gets the smaller limit)
    if (warp >= kProducerWarp<F>) {
        if constexpr (kSplitRegs<F>) setmaxnreg_dec<kRegsOther>();
        if (warp == kProducerWarp<F>) {
            if (n > 0) dkdv_producer<D, F>(sm, p, &tmQ, &tmdO, &tmK, &tmV, b, hkv, bh_kv, k0, qi_start, nqt, u0, n, wc);
        } else if (warp == kMmaWarp<F>) {
            if (lane == 0 && n > 0) dkdv_mma<D, F>(sm, tmem, n, wc);
        }
    } else {
        if constexpr (kSplitRegs<F>) setmaxnreg_inc<kRegsCompute>();
        dkdv_compute<D, F>(sm, p, tmem, warp >> 2, bh_kv, k0, kv_end, delta, qi_start, nqt, u0, n, split, splits, wc);
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp<F>) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ================================================================== dQ
template <bool MOD> struct KeySpan {};
template <> struct KeySpan<true> {
    int lo[4], hi[4];  // per warp of the first warpgroup: the union of its rows' intervals
};
template <int D>
struct alignas(1024) DqTiles {
    __nv_bfloat16 q[kT * kBPad<D>];  // the CTA's 128 queries
    __nv_bfloat16 dout[kT * kBPad<D>];
    __nv_bfloat16 k[kStages][kT * kBPad<D>];  // streamed key tiles
    __nv_bfloat16 v[kStages][kT * kBPad<D>];
    uint64_t qd_full;
    uint64_t u_full[kStages], u_empty[kStages];
    uint64_t s_full, s_free, dp_full, ds_full, acc_done, drain;
    uint32_t tmem_base;
    int abort_flag;
};
template <int D, int F> struct DqSmem : DqTiles<D>, KeySpan<kIsMod<F>> {};

template <int D, int F>
__device__ void dq_producer(DqSmem<D, F> &sm, const CUtensorMap *tmQ, const CUtensorMap *tmdO, const CUtensorMap *tmK,
                            const CUtensorMap *tmV, int bh, int bh_kv, int q0, int n, int j0, WaitCtx wc) {
    constexpr int kBoxes = kBBoxes<D>;
    prefetch_tensormap(tmK);
    prefetch_tensormap(tmV);
    mbar_arrive_expect_tx(&sm.qd_full, 2 * kBoxes * kBoxBytes);
#pragma unroll
    for (int i = 0; i < kBoxes; ++i) {
        tma_load_3d(sm.q + i * (kT * 64), tmQ, &sm.qd_full, i * 64, q0, bh);
        tma_load_3d(sm.dout + i * (kT * 64), tmdO, &sm.qd_full, i * 64, q0, bh);
    }
    int fills = 0;
    for (int u = 0; u < n; ++u) {
        const int slot = u % kStages, use = u / kStages;
        if (use > 0 && !mbar_wait(&sm.u_empty[slot], (uint32_t)((use - 1) & 1), wc, 80)) break;
        mbar_arrive_expect_tx(&sm.u_full[slot], 2 * kBoxes * kBoxBytes);
#pragma unroll
        for (int i = 0; i < kBoxes; ++i) {
            tma_load_3d(sm.k[slot] + i * (kT * 64), tmK, &sm.u_full[slot], i * 64, (j0 + u) * kT, bh_kv);
            tma_load_3d(sm.v[slot] + i * (kT * 64), tmV, &sm.u_full[slot], i * 64, (j0 + u) * kT, bh_kv);
        }
        ++fills;
    }
    if (*wc.abort_flag) {
        WaitCtx drain{nullptr, wc.status};
        (void)mbar_wait(&sm.qd_full, 0, drain, 81);
        for (int f = (fills > kStages ? fills - kStages : 0); f < fills; ++f)
            (void)mbar_wait(&sm.u_full[f % kStages], (uint32_t)((f / kStages) & 1), drain, 82);
    }
}

template <int D, int F>
__device__ void dq_mma(DqSmem<D, F> &sm, uint32_t tmem, int n, WaitCtx wc) {
    const uint32_t tS = tmem, tdP = tmem + 128, tdQ = tmem + 256;
    bool ok = mbar_wait(&sm.qd_full, 0, wc, 83) && mbar_wait(&sm.u_full[0], 0, wc, 84);
    if (ok) {
        tc_fence_after_sync();
        mma_scores<D>(tS, sm.q, sm.k[0]);
        tc_commit(&sm.s_full);
        mma_scores<D>(tdP, sm.dout, sm.v[0]);
        tc_commit(&sm.dp_full);
        for (int j = 0; j < n; ++j) {
            const int slot = j % kStages;
            if (j + 1 < n) {
                const int u = j + 1;
                if (!(ok = mbar_wait(&sm.s_free, (uint32_t)(j & 1), wc, 85))) break;
                if (!(ok = mbar_wait(&sm.u_full[u % kStages], (uint32_t)((u / kStages) & 1), wc, 86))) break;
                tc_fence_after_sync();
                mma_scores<D>(tS, sm.q, sm.k[u % kStages]);  // S(j+1): the warpgroups have read S(j)
                tc_commit(&sm.s_full);
            }
            if (!(ok = mbar_wait(&sm.ds_full, (uint32_t)(j & 1), wc, 87))) break;
            tc_fence_after_sync();
            mma_accum<D, F>(tdQ, tdP, sm.k[slot], j == 0);  // dQ += dS K
            tc_commit(&sm.u_empty[slot]);
            if (j == n - 1) tc_commit(&sm.acc_done);
            if (j + 1 < n) {
                mma_scores<D>(tdP, sm.dout, sm.v[(j + 1) % kStages]);  // dP(j+1), after dQ(j) read dS(j)
                tc_commit(&sm.dp_full);
            }
        }
    }
    tc_commit(&sm.drain);
    WaitCtx drain{nullptr, wc.status};
    (void)mbar_wait(&sm.drain, 0, drain, 88);
}

template <int D, int F>
__device__ void dq_compute(DqSmem<D, F> &sm, const Params<F> &p, uint32_t tmem, int w, int bh, int q0, int kv_end,
                           int delta, int n, int j0, int2 span, WaitCtx wc) {
    constexpr int kC = kCols<F>, kH = kC / 32;
    const int r = threadIdx.x & 127;
    const uint32_t lane_base = tmem + ((uint32_t)(((threadIdx.x >> 5) & 3) * 32) << 16);
    const uint32_t tS = lane_base + (uint32_t)(w * kC);
    const uint32_t tdP = lane_base + 128u + (uint32_t)(w * kC);
    const int row = q0 + r;
    const bool row_ok = row < p.Nq;
    const float lse2 = row_ok ? p.lse[(size_t)bh * p.Nq + row] * kLog2e : 0.f;
    const float drow = row_ok ? p.dterm[(size_t)bh * p.Nq + row] : 0.f;
    // keys < lim are valid for this row
    int lim = row_ok ? kv_end : 0;
    if (p.causal) lim = min(lim, row + delta + 1);
    if constexpr (kIsMod<F>) lim = span.y;
    [[maybe_unused]] const TanhCap cap(cap_in_of<F>(p), 1.f);
    const float to_log2 = score_factor<F>(p);
    const uint64_t c2 = f32x2_pack(to_log2, to_log2);
    [[maybe_unused]] float slope2 = 0.f;
    if constexpr (kHasBias<F>) slope2 = bias_slope(p.slopes[bh % p.Hq]);
    const uint64_t nl2 = f32x2_pack(-lse2, -lse2);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
        const int key0 = (j0 + j) * kT + w * kC;
        const int nvalid = lim - key0;  // columns c < nvalid are valid
        bool need_mask = nvalid < kC;
        [[maybe_unused]] int lo = 0;  // modified forms: and columns from lo on
        if constexpr (kIsMod<F>) {
            lo = span.x - key0;
            need_mask = __any_sync(kFull, need_mask || lo > 0);
        }
        if (!__all_sync(kFull, mbar_wait(&sm.s_full, (uint32_t)(j & 1), wc, 90))) {
            ok = false;
            break;
        }
        tc_fence_after_sync();
        uint32_t x[kH][32];
        load_cols(tS, x);
        tc_fence_before_sync();
        mbar_arrive(&sm.s_free);
        if constexpr (kHasCap<F>) cap.apply(cap.tier(abs_max(x)), x);
        [[maybe_unused]] Distance<-1> dist;
        if constexpr (kHasBias<F>) {
            const int at = q0 + delta;  // position of the tile's first query
            dist.set(slope2, row + delta - key0, p.causal || key0 + kC - 1 <= at, key0 >= at + kT - 1);
        }
#pragma unroll
        for (int h = 0; h < kH; ++h)
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const uint64_t x2 = f32x2_pack(__uint_as_float(x[h][i]), __uint_as_float(x[h][i + 1]));
                const uint64_t e2 = f32x2_fma(x2, c2, nl2);
                float e0, e1;
                f32x2_unpack(e2, e0, e1);
                if constexpr (kHasBias<F>) {
                    e0 = dist.add(h * 32 + i, e0);
                    e1 = dist.add(h * 32 + i + 1, e1);
                }
                float p0 = ex2_approx(e0), p1 = ex2_approx(e1);
                if constexpr (kHasCap<F>) {  // times 1 - tanh^2
                    p0 *= fmaf(-__uint_as_float(x[h][i]), __uint_as_float(x[h][i]), 1.f);
                    p1 *= fmaf(-__uint_as_float(x[h][i + 1]), __uint_as_float(x[h][i + 1]), 1.f);
                }
                if (need_mask) {
                    const int c = h * 32 + i;
                    p0 = c < nvalid && (!kIsMod<F> || c >= lo) ? p0 : 0.f;
                    p1 = c + 1 < nvalid && (!kIsMod<F> || c + 1 >= lo) ? p1 : 0.f;
                }
                x[h][i] = __float_as_uint(p0);
                x[h][i + 1] = __float_as_uint(p1);
            }

        if (!__all_sync(kFull, mbar_wait(&sm.dp_full, (uint32_t)(j & 1), wc, 91))) {
            ok = false;
            break;
        }
        tc_fence_after_sync();
        uint32_t y[kH][32];
        load_cols(tdP, y);
        // dS = P * (dP - D): bf16 pairs over dP
#pragma unroll
        for (int h = 0; h < kH; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                float s0 = __uint_as_float(x[h][i]) * (__uint_as_float(y[h][i]) - drow);
                float s1 = __uint_as_float(x[h][i + 1]) * (__uint_as_float(y[h][i + 1]) - drow);
                if constexpr (kIsMod<F>) {
                    if (need_mask) {  // dP of a masked key may be anything
                        s0 = x[h][i] ? s0 : 0.f;
                        s1 = x[h][i + 1] ? s1 : 0.f;
                    }
                }
                pk[i / 2] = pack_bf16x2(s0, s1);
            }
            tmem_st16(tdP + (uint32_t)(h * 16), pk);
        }
        if constexpr (kIsMod<F>) {
            // K rows past the sequence's keys may hold anything: dS is 0 there, and dS K needs finite values
            // (S(j) has been read, and the tile stays until dQ(j) completes)
            const int rows0 = kv_end - (j0 + j) * kT;
            if (rows0 < kT && kv_end < p.Nkv) {
                uint4 *tile = reinterpret_cast<uint4 *>(sm.k[j % kStages]);
                for (int box = 0; box < kBBoxes<D>; ++box)
                    for (int i = rows0 * 8 + (int)threadIdx.x; i < kT * 8; i += 128 * kGroups<F>)
                        tile[box * (kT * 8) + i] = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
            }
        }
        tmem_wait_st();
        tc_fence_before_sync();
        mbar_arrive(&sm.ds_full);
    }

    if (ok && n > 0) {
        if (!__all_sync(kFull, mbar_wait(&sm.acc_done, 0, wc, 92))) ok = false;
        else tc_fence_after_sync();
    }
    if (!ok) return;
    if (w > 1) return;
    // warpgroup 0 writes columns 0 .. kDqSplit - 1 of dQ, warpgroup 1 the rest (times scale)
    __nv_bfloat16 *dst = p.dq + ((size_t)bh * p.Nq + (row_ok ? row : 0)) * D + (w ? kDqSplit<D> : 0);
    if (w == 0) store_rows<kDqSplit<D>>(lane_base + 256u, n > 0, row_ok, p.scale, dst);
    else store_rows<D - kDqSplit<D>>(lane_base + 256u + (uint32_t)kDqSplit<D>, n > 0, row_ok, p.scale, dst);
}

template <int D, int F>
__global__ void __launch_bounds__(kThreadsOf<F>, 1)
    bwd_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
                  const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const Params<F> p) {
    extern __shared__ uint8_t smem_raw[];
    DqSmem<D, F> &sm = *reinterpret_cast<DqSmem<D, F> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    int bh, level;
    unit_of(p, p.B * p.Hq, blockIdx.x, bh, level);
    const int qt = p.units_per_head - 1 - level;  // level 0 = the last query tile (most keys if causal)
    const int b = bh / p.Hq;
    const int bh_kv = b * p.Hkv + (bh % p.Hq) / p.group;
    const int q0 = qt * kT;
    const int kv_end = kv_end_for(p, b);
    const int delta = p.Nkv - p.Nq;
    int limit = kv_end;
    if (p.causal) limit = min(limit, min(q0 + kT, p.Nq) + delta);
    int n = limit > 0 ? (limit + kT - 1) / kT : 0;
    int j0 = 0;  // modified forms: the first key tile that a row of the CTA sees
    int2 span = make_int2(0, 0);
    if constexpr (kIsMod<F>) {
        if (warp < kProducerWarp<F>) {
            span = bwd_row_span(p, b, q0 + ((int)threadIdx.x & 127), kv_end);
            const int lo = __reduce_min_sync(kFull, span.x < span.y ? span.x : 0x7fffffff);
            const int hi = __reduce_max_sync(kFull, span.x < span.y ? span.y : 0);
            if (warp < 4 && lane == 0) {
                sm.lo[warp] = lo;
                sm.hi[warp] = hi;
            }
        }
    }

    if (threadIdx.x == 0) {
        mbar_init(&sm.qd_full, 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm.u_full[s], 1);
            mbar_init(&sm.u_empty[s], 1);
        }
        mbar_init(&sm.s_full, 1);
        mbar_init(&sm.s_free, 128 * kGroups<F>);
        mbar_init(&sm.dp_full, 1);
        mbar_init(&sm.ds_full, 128 * kGroups<F>);
        mbar_init(&sm.acc_done, 1);
        mbar_init(&sm.drain, 1);
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp<F>) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sm.tmem_base;
    WaitCtx wc{&sm.abort_flag, p.status};
    if constexpr (kIsMod<F>) {
        const int lo = min(min(sm.lo[0], sm.lo[1]), min(sm.lo[2], sm.lo[3]));
        const int hi = max(max(sm.hi[0], sm.hi[1]), max(sm.hi[2], sm.hi[3]));
        j0 = hi > 0 ? lo / kT : 0;
        n = hi > 0 ? (hi + kT - 1) / kT - j0 : 0;
    }

    if (warp >= kProducerWarp<F>) {
        if constexpr (kSplitRegs<F>) setmaxnreg_dec<kRegsOther>();
        if (warp == kProducerWarp<F>) {
            if (lane == 0 && n > 0) dq_producer<D, F>(sm, &tmQ, &tmdO, &tmK, &tmV, bh, bh_kv, q0, n, j0, wc);
        } else if (warp == kMmaWarp<F>) {
            if (lane == 0 && n > 0) dq_mma<D, F>(sm, tmem, n, wc);
        }
    } else {
        if constexpr (kSplitRegs<F>) setmaxnreg_inc<kRegsCompute>();
        dq_compute<D, F>(sm, p, tmem, warp >> 2, bh, q0, kv_end, delta, n, j0, span, wc);
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp<F>) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
    // modified forms: this grid may have started before the dK/dV grid ended; its completion includes that
    if constexpr (kIsMod<F>) griddep_wait();
}

// dV and dK [B, Hkv, Nkv, D] of the key tiles with several CTAs from those CTAs' sums: four columns per thread, in
// the CTAs' order.
template <int D>
__global__ void __launch_bounds__(256) bwd_reduce_kernel(const BwdModParams p, unsigned rows) {
    const unsigned n4 = rows * (D / 4), i = blockIdx.x * 256 + threadIdx.x;  // (few key tiles: both below 2^31)
    if (i >= 2 * n4) return;
    const bool is_k = i >= n4;
    const unsigned at = is_k ? i - n4 : i;
    const int tile = (int)(at / (D / 4) % (unsigned)p.Nkv) / kT;
    const int splits = tile_splits(tile, p.kv_target, p.group, p.Nq, p.Nkv, p.causal != 0);
    griddep_wait();  // (launched as the dQ grid, whose end includes the dK/dV grid's, drains)
    if (splits == 1) return;
    const float4 *parts = reinterpret_cast<const float4 *>(p.kv_parts);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int s = 0; s < splits; ++s) {
        const float4 v = parts[(size_t)s * 2 * n4 + i];
        acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
    }
    const float f = is_k ? p.scale : 1.f;
    reinterpret_cast<uint2 *>(is_k ? p.dk : p.dv)[at] =
        make_uint2(pack_bf16x2(acc.x * f, acc.y * f), pack_bf16x2(acc.z * f, acc.w * f));
}

// Steps per CTA of the dK/dV kernel of the modified forms, 0 for a key tile's all.  Short sequences with few
// key/value heads leave the GPU empty at one CTA per key tile, and the causal mask makes those uneven; so the steps
// are shared out, a key tile's in equal shares of at most `target`: of the targets that cut the longest key tile
// (`steps`) into 1 to 16, and the shortest whose CTAs are resident at once, the one whose CTAs end first -- one wave
// after its longest share, more after their common work and, on average, half a share.  A CTA's start and end cost
// about 6 steps, and the addition of the sums 3.  (A target that kMaxSplits shares of the longest key tile do not reach
// is costed too low, as if its shares were that short; over 20000 sizes that never led to a longer longest share.)
// Measured, the whole backward, causal with a cap, us (shares / the same number of CTAs for each key tile; heads x queries with
// the key/value heads): d 64 2 x 16 (4) x 1000 53 / 57, 16 (4) x 2048 79 / 91, 16 (8) x 2048 81 / 91, 4 x 16 (4) x
// 1024 97 / 100, 8 (2) x 512 18.8 / 17.0; d 128 66 / 74, 96 / 115, 99 / 117, 123 / 133, 23.6 / 21.7.
struct DkdvPlan {
    int target, head_ctas, most;  // most: CTAs of one key tile
};
DkdvPlan dkdv_plan(int B, int Hkv, int group, int Nq, int Nkv, bool causal) {
    constexpr float kSms = 152.f, kStart = 6.f, kSums = 3.f;
    const int tiles = (Nkv + kT - 1) / kT;
    const long long heads = (long long)B * Hkv, steps = (long long)group * ((Nq + kT - 1) / kT);
    DkdvPlan pl{0, tiles, 1};
    if (heads * tiles >= 304 || steps < 4 || steps > 100000000) return pl;
    long long total = 0;
    for (int t = 0; t < tiles; ++t) {
        const int first = causal ? (t * kT - (Nkv - Nq)) / kT : 0;
        const long long n = (Nq + kT - 1) / kT - (first > 0 ? first : 0);
        total += n > 0 ? n * group : 0;
    }
    auto ctas_of = [&](int target) {  // of one head
        int n = 0;
        for (int t = 0; t < tiles; ++t) n += tile_splits(t, target, group, Nq, Nkv, causal);
        return n;
    };
    float best = (float)steps + kStart;
    if ((float)(heads * tiles) > kSms)
        best = fmaxf(best, ((float)(heads * total) + kStart * (float)(heads * tiles)) / kSms + 0.5f * (float)steps);
    auto consider = [&](int target) {
        const int ctas = ctas_of(target);
        const float all = (float)(heads * ctas);
        float cost = (float)target + kStart + kSums;
        if (all > kSms) cost = fmaxf(cost, ((float)(heads * total) + kStart * all) / kSms + 0.5f * (float)target + kSums);
        if (cost < best) {
            best = cost;
            pl = DkdvPlan{target, ctas, (int)((steps + target - 1) / target)};
            if (pl.most > kMaxSplits) pl.most = kMaxSplits;
        }
    };
    for (int k = 2; k <= kMaxSplits && 2 * k <= steps; ++k) consider((int)((steps + k - 1) / k));
    int lo = 2, hi = (int)steps;  // the shortest shares of one wave
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if ((float)(heads * ctas_of(mid)) <= kSms) hi = mid;
        else lo = mid + 1;
    }
    if (lo < steps) consider(lo);
    return pl;
}

int heads_per_chunk(double bytes_per_head, int n_heads) {
    // about 48 MB of streamed tiles per chunk: the chunk finishing and the one starting fit in
    // the 126 MB L2 together
    int h = (int)(48.0e6 / bytes_per_head);
    return h < 1 ? 1 : (h > n_heads ? n_heads : h);
}

// The register split draws on the launch allocation; a larger one would wait forever.
template <int F>
cudaError_t check_register_split(const void *kernel) {
    if (!kSplitRegs<F>) return cudaSuccess;
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    return (long)fa.numRegs * kThreadsOf<F> >= 128L * (2 * kRegsCompute + kRegsOther) ? cudaSuccess
                                                                                     : cudaErrorInvalidConfiguration;
}

template <int D, int F>
cudaError_t launch_bwd_d(const BwdArgs &a, cudaStream_t stream) {
    const long long rows = (long long)a.B * a.Hq * a.Nq;
    CUtensorMap tq, tdo, tk, tv;
    const int BHq = a.B * a.Hq, BHkv = a.B * a.Hkv;
    if (!encode_qkv_map(&tq, a.q, BHq, a.Nq, D) || !encode_qkv_map(&tdo, a.dout, BHq, a.Nq, D) ||
        !encode_qkv_map(&tk, a.k, BHkv, a.Nkv, D) || !encode_qkv_map(&tv, a.v, BHkv, a.Nkv, D))
        return cudaErrorInvalidValue;
    Params<F> p;
    p.lse = a.lse;
    p.dterm = a.dterm;
    p.dq = reinterpret_cast<__nv_bfloat16 *>(a.dq);
    p.dk = reinterpret_cast<__nv_bfloat16 *>(a.dk);
    p.dv = reinterpret_cast<__nv_bfloat16 *>(a.dv);
    p.kv_lens = a.kv_lens;
    p.status = a.status;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.group = a.Hq / a.Hkv;
    p.Nq = a.Nq;
    p.Nkv = a.Nkv;
    p.causal = a.causal;
    p.scale = a.scale;
    p.scale_log2 = a.scale * kLog2e;
    [[maybe_unused]] DkdvPlan plan{};
    if constexpr (kIsMod<F>) {
        p.key_begin = a.key_begin;
        p.key_end = a.key_end;
        p.slopes = a.slopes;
        p.cap_in = a.softcap > 0.f ? a.scale / a.softcap : 0.f;
        p.cap_out = a.softcap * kLog2e;
        p.spans = a.spans;
        plan = dkdv_plan(a.B, a.Hkv, p.group, a.Nq, a.Nkv, a.causal != 0);
        p.kv_target = plan.target;
        p.kv_parts = a.kv_parts;
    }

    {
        const int row_blocks = (int)((rows * kRowThreads<D> + 255) / 256);
        const __nv_bfloat16 *o = reinterpret_cast<const __nv_bfloat16 *>(a.o);
        const __nv_bfloat16 *dout = reinterpret_cast<const __nv_bfloat16 *>(a.dout);
        if constexpr (kIsMod<F>) {
            const int n_qt = (a.Nq + kT - 1) / kT;
            const int span_blocks = (int)(((long long)a.B * n_qt + 1) / 2);
            bwd_rowdot_spans_kernel<D><<<row_blocks + span_blocks, 256, 0, stream>>>(o, dout, a.dterm, rows, row_blocks,
                                                                                    p, n_qt);
        } else {
            bwd_rowdot_kernel<D><<<row_blocks, 256, 0, stream>>>(o, dout, a.dterm, rows);
        }
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }

    // dK/dV: one CTA per (batch, key/value head, key tile); streams Q and dO of the group's heads
    {
        Params<F> pk = p;
        pk.units_per_head = (a.Nkv + kT - 1) / kT;
        pk.heads_per_chunk = heads_per_chunk(2.0 * p.group * a.Nq * D * 2.0, BHkv);
        const size_t smem = sizeof(DkvSmem<D, F>) + 1024;
        static const cudaError_t split = check_register_split<F>(reinterpret_cast<const void *>(bwd_dkdv_kernel<D, F>));
        if (split != cudaSuccess) return split;
        cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void *>(bwd_dkdv_kernel<D, F>), (int)smem);
        if (e != cudaSuccess) return e;
        const unsigned grid = (unsigned)((size_t)pk.units_per_head * BHkv);
        if constexpr (kIsMod<F>) {
            e = launch_dependent(bwd_dkdv_kernel<D, F>, dim3((unsigned)plan.head_ctas * BHkv), kThreadsOf<F>, smem, stream, tq,
                                 tdo, tk, tv, pk);
        } else {
            bwd_dkdv_kernel<D, F><<<grid, kThreadsOf<F>, smem, stream>>>(tq, tdo, tk, tv, pk);
            e = cudaGetLastError();
        }
        if (e != cudaSuccess) return e;
    }
    // dQ: one CTA per (batch, query head, query tile); streams K and V of its key/value head
    {
        Params<F> pq = p;
        pq.units_per_head = (a.Nq + kT - 1) / kT;
        pq.heads_per_chunk = heads_per_chunk(2.0 * a.Nkv * D * 2.0 / p.group, BHq);
        const size_t smem = sizeof(DqSmem<D, F>) + 1024;
        static const cudaError_t split = check_register_split<F>(reinterpret_cast<const void *>(bwd_dq_kernel<D, F>));
        if (split != cudaSuccess) return split;
        cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void *>(bwd_dq_kernel<D, F>), (int)smem);
        if (e != cudaSuccess) return e;
        const unsigned grid = (unsigned)((size_t)pq.units_per_head * BHq);
        if constexpr (kIsMod<F>) {
            e = launch_dependent(bwd_dq_kernel<D, F>, dim3(grid), kThreadsOf<F>, smem, stream, tq, tdo, tk, tv, pq);
        } else {
            bwd_dq_kernel<D, F><<<grid, kThreadsOf<F>, smem, stream>>>(tq, tdo, tk, tv, pq);
            e = cudaGetLastError();
        }
        if (e != cudaSuccess) return e;
    }
    if constexpr (kIsMod<F>) {
        if (p.kv_target > 0) {
            const long long kv_rows = (long long)a.B * a.Hkv * a.Nkv;
            const cudaError_t e = launch_dependent(bwd_reduce_kernel<D>, dim3((unsigned)((kv_rows * (D / 2) + 255) / 256)),
                                                   256, 0, stream, static_cast<const BwdModParams &>(p), (unsigned)kv_rows);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace
}  // namespace attn
