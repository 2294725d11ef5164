// decode_fp4.cu -- paged decode over the 4-bit cache (fp4.cuh), with the modified scores of decode_scoremod.cu.
//
// The rows kernel's plan (decode_rows.cuh: tokens as the rows of the products, query heads as their columns, splits merged
// in a cluster or through the workspace), over pages of 9 d bytes a head that come by one bulk copy each:
//   S^T = K Q^T       a lane's codes of a token are neighbours in its row: 32 (d 128) or 16 dims, one or two blocks of the
//                     scales, read as one vector, and Q is held in that order of the dims;
//   O^T += V^T P^T    a block of 16 dims is one 8 x 8 matrix of ldmatrix, transposed: a lane gets four bytes, dims 2g and
//                     2g + 1 of token pairs (2t, 2t + 1) and (2t + 8, 2t + 9), the four registers of one operand.
// A byte of codes widens to one f16x2 register in one instruction and a product with the pair of block scales makes it the
// value (exact).  The scales of slots that are not seen are zeroed, so whatever they hold adds nothing.
#include "decode_rows.cuh"
#include "fp4.cuh"

namespace attn {
namespace {

constexpr int kFp4Slots = 4;  // pages in flight per warp

template <int D, int NT>
struct Fp4Smem {
    union {
        alignas(128) uint8_t kv[kRowWarps][kFp4Slots][2][9 * D];
        RowsRed<D, NT> red;
    } u;
    uint64_t full[kRowWarps][kFp4Slots];
    int abort_flag;
};

// Both halves of a word: the f16 value of byte `i` of e4m3 codes.
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}

// The dims of a lane's k-steps.  A row is cut into units of W dims, of which lane t takes W / 4 neighbours, 4 a k-step:
// one unit of 128, or units of 64 and one of the rest.
template <int D> constexpr int fp4_unit(int ks) { return D == 128 ? 128 : (D - ks / 4 * 64 >= 64 ? 64 : D % 64); }
template <int D> constexpr int fp4_base(int ks) { return D == 128 ? 0 : ks / 4 * 64; }
template <int D> constexpr int fp4_step(int ks) { return D == 128 ? ks : ks % 4; }

template <int D, int NT>
__global__ void __launch_bounds__(kRowWarps * 32, 4) decode_fp4_kernel(const uint8_t *__restrict__ k_pages,
                                                                       const uint8_t *__restrict__ v_pages,
                                                                       const RowsParams a) {
    constexpr int kSl = kFp4Slots;
    constexpr uint32_t kBlock = 9 * D;
    constexpr int KS = D / 16;  // k-steps of S^T, and 16-dim tiles of O^T
    constexpr float kThresh = 8.0f;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    using Smem = Fp4Smem<D, NT>;
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));

    const int split = blockIdx.x, b = blockIdx.z;
    const int kvh = (int)blockIdx.y / a.rgroups;
    const int row0 = ((int)blockIdx.y % a.rgroups) * 8 * NT;
    const int rows = min(8 * NT, a.group - row0);
    const int h0 = kvh * a.group + row0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const PageRange pr = rows_range<true>(a, b, split);
    float *ws = a.ws + (((size_t)b * a.H + h0) * a.ws_splits + a.ws_first + split) * (D + 4);
    const size_t ws_row = (size_t)a.ws_splits * (D + 4);
    if (pr.p0 >= pr.p1 && !a.cluster) return;  // nothing here (uniform over the CTA)
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

    // Page ids, 32 of this warp's pages at a time (lane l: page k0 + l); bit k % 32 of mapped: page k's id lies in the pool
    const int32_t *table = a.page_table + (size_t)b * a.max_pages + pr.p0 + warp;
    int my_pid = -1;
    uint32_t mapped = 0;
    auto issue = [&](int k) {
        if ((k & 31) == 0) my_pid = k + lane < nk ? table[kRowWarps * (k + lane)] : -1;
        const int pid = __shfl_sync(0xffffffffu, my_pid, k & 31);
        const bool ok = pid >= 0 && pid < a.num_pages;
        mapped = (mapped & ~(1u << (k & 31))) | ((ok ? 1u : 0u) << (k & 31));
        if (lane == 0) {
            uint64_t *bar = &sm.full[warp][k % kSl];
            if (ok) {
                const size_t at = ((size_t)pid * a.Hkv + kvh) * kBlock;
                mbar_arrive_expect_tx(bar, 2 * kBlock);
                bulk_load(sm.u.kv[warp][k % kSl][0], k_pages + at, kBlock, bar);
                bulk_load(sm.u.kv[warp][k % kSl][1], v_pages + at, kBlock, bar);
            } else {
                mbar_arrive(bar);
            }
        }
    };
    const int first = nk < kSl ? nk : kSl;
    for (int k = 0; k < first; ++k) issue(k);

    // Q as B fragments in the order of the codes, each head rounded to f16 after a 2^-sh of its own, which keeps it below
    // 2^15 (exact but for values under f16's range; sh 0 but for huge queries, at most 113); cc: per score column (heads
    // 2t, 2t + 1 of an n-tile) the factor of its products, to the cap's argument or, without a cap, to the log2 domain
    uint32_t qb[NT][KS][2];
    float cc[NT][2];
    {
        const float c = a.cap_in > 0.f ? a.cap_in : a.c;
        const __nv_bfloat16 *q = reinterpret_cast<const __nv_bfloat16 *>(a.q) + ((size_t)b * a.H + h0) * D;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float amax = 0.f;
            const __nv_bfloat16 *qr = q + (size_t)(8 * nt + g) * D;
            const bool have = 8 * nt + g < rows;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int x = fp4_base<D>(ks) + fp4_unit<D>(ks) / 4 * t + 4 * fp4_step<D>(ks);
                const uint2 u = have ? *reinterpret_cast<const uint2 *>(qr + x) : make_uint2(0u, 0u);
                qb[nt][ks][0] = u.x;
                qb[nt][ks][1] = u.y;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(qb[nt][ks][i] << 16)),
                                             fabsf(__uint_as_float(qb[nt][ks][i] & 0xffff0000u))));
            }
#pragma unroll
            for (int off = 1; off <= 2; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            const int e = (int)((__float_as_uint(amax) >> 23) & 0xffu) - 127;
            const int sh = e >= 15 ? min(e - 14, 113) : 0;
            const float f = __uint_as_float((uint32_t)(127 - sh) << 23), back = __uint_as_float((uint32_t)(127 + sh) << 23);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    qb[nt][ks][i] = pack_f16x2(__uint_as_float(qb[nt][ks][i] << 16) * f,
                                               __uint_as_float(qb[nt][ks][i] & 0xffff0000u) * f);
#pragma unroll
            for (int j = 0; j < 2; ++j) cc[nt][j] = c * __shfl_sync(0xffffffffu, back, 4 * (2 * t + j));
        }
    }
    float slope2[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 8 * nt + 2 * t + j;
            slope2[nt][j] = a.slopes && r < rows ? bias_slope(a.slopes[h0 + r]) : 0.f;
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

    int issued = first;
    bool failed = false;
    for (int k = 0; k < nk; ++k) {
        const int slot = k % kSl;
        if (!mbar_wait(&sm.full[warp][slot], (uint32_t)((k / kSl) & 1), wc, 150 + warp)) {
            failed = true;
            break;
        }
        if ((mapped >> (k & 31)) & 1u) {
            const int tok0 = (pr.p0 + warp + kRowWarps * k) * kRowPS;
            const int lo = pr.lo - tok0, hi = pr.hi - tok0;  // slots lo <= i < hi are seen
            const uint8_t *Kb = sm.u.kv[warp][slot][0];
            uint8_t *Vb = sm.u.kv[warp][slot][1];
            const bool ragged = hi < kRowPS || lo > 0;
            if (ragged) {
                for (int i = lane; i < kRowPS * KS; i += 32) {
                    const int r = i & 15;
                    if (r >= hi || r < lo) Vb[fp4_v_scale(D, r, i >> 4)] = 0;
                }
                __syncwarp();
            }
            // rows (tokens) g, g + 8, columns (heads) 2t, 2t + 1; two chains
            float sc[NT][4], sc2[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[nt][i] = sc2[nt][i] = 0.f;
            // one k-step: the f16 pairs of tokens g and g + 8 and their scales
            auto k_step = [&](int ks, uint32_t x0, uint32_t x1, uint32_t y0, uint32_t y1, uint32_t s0, uint32_t s1) {
                const uint32_t ka[4] = {f16x2_mul(x0, s0), f16x2_mul(y0, s1), f16x2_mul(x1, s0), f16x2_mul(y1, s1)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_16816_f16((ks & 1) ? sc2[nt] : sc[nt], ka, qb[nt][ks][0], qb[nt][ks][1]);
            };
            // two k-steps: a word of codes of each token
            auto k_word = [&](int ks, uint32_t w0, uint32_t w1, uint32_t s0, uint32_t s1) {
                uint32_t x[4], y[4];
                e2m1x8_to_f16x2x4(w0, x);
                e2m1x8_to_f16x2x4(w1, y);
                k_step(ks, x[0], x[1], y[0], y[1], s0, s1);
                k_step(ks + 1, x[2], x[3], y[2], y[3], s0, s1);
            };
            const uint8_t *k0 = Kb + fp4_k_codes(D, g, 0), *k1 = Kb + fp4_k_codes(D, g + 8, 0);
            const uint8_t *s0 = Kb + fp4_k_scale(D, g, 0), *s1 = Kb + fp4_k_scale(D, g + 8, 0);
            if constexpr (D == 128) {
                const uint4 w0 = *reinterpret_cast<const uint4 *>(k0 + 16 * t), w1 = *reinterpret_cast<const uint4 *>(k1 + 16 * t);
                const uint32_t p0 = e4m3_pair(*reinterpret_cast<const uint16_t *>(s0 + 2 * t));
                const uint32_t p1 = e4m3_pair(*reinterpret_cast<const uint16_t *>(s1 + 2 * t));
                const uint32_t a0 = prmt(p0, 0u, 0x1010u), a1 = prmt(p1, 0u, 0x1010u);
                const uint32_t b0 = prmt(p0, 0u, 0x3232u), b1 = prmt(p1, 0u, 0x3232u);
                k_word(0, w0.x, w1.x, a0, a1);
                k_word(2, w0.y, w1.y, a0, a1);
                k_word(4, w0.z, w1.z, b0, b1);
                k_word(6, w0.w, w1.w, b0, b1);
            } else {
#pragma unroll
                for (int u = 0; u < D / 64; ++u) {
                    const uint2 w0 = *reinterpret_cast<const uint2 *>(k0 + 32 * u + 8 * t);
                    const uint2 w1 = *reinterpret_cast<const uint2 *>(k1 + 32 * u + 8 * t);
                    const uint32_t a0 = e4m3_pair(s0[4 * u + t] * 0x101u), a1 = e4m3_pair(s1[4 * u + t] * 0x101u);
                    k_word(4 * u, w0.x, w1.x, a0, a1);
                    k_word(4 * u + 2, w0.y, w1.y, a0, a1);
                }
                constexpr int x = D / 64 * 32, n = D / 64 * 4;  // the rest: its byte, its first k-step and block
                if constexpr (D % 64 == 32) {
                    const uint32_t w0 = *reinterpret_cast<const uint32_t *>(k0 + x + 4 * t);
                    const uint32_t w1 = *reinterpret_cast<const uint32_t *>(k1 + x + 4 * t);
                    k_word(n, w0, w1, e4m3_pair(s0[n + (t >> 1)] * 0x101u), e4m3_pair(s1[n + (t >> 1)] * 0x101u));
                } else if constexpr (D % 64 == 16) {
                    const uint32_t w0 = *reinterpret_cast<const uint16_t *>(k0 + x + 2 * t);
                    const uint32_t w1 = *reinterpret_cast<const uint16_t *>(k1 + x + 2 * t);
                    uint32_t z[4];
                    e2m1x8_to_f16x2x4(w0 | w1 << 16, z);
                    k_step(n, z[0], z[1], z[2], z[3], e4m3_pair(s0[n] * 0x101u), e4m3_pair(s1[n] * 0x101u));
                }
            }
            uint32_t pb[NT][2];
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[nt][i] = (sc[nt][i] + sc2[nt][i]) * cc[nt][i & 1];
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
                pb[nt][0] = movmatrix_trans(pack_f16x2(p[0], p[1]));
                pb[nt][1] = movmatrix_trans(pack_f16x2(p[2], p[3]));
            }
            const uint32_t Vs = smem_u32(Vb);
            const uint8_t *sv = Vb + fp4_v_scale(D, 2 * t, 0);  // of the lane's quad of tokens: 4 bytes a block
#pragma unroll
            for (int n0 = 0; n0 < KS; n0 += 4) {
                uint32_t w[4];  // lane l: row l & 7 of block n0 + (l >> 3); past the last block: that one again
                ldsm_x4_trans(Vs + min(n0 + (lane >> 3), KS - 1) * 128 + (lane & 7) * 16, w);
#pragma unroll
                for (int i = 0; i < 4 && n0 + i < KS; ++i) {
                    const int nd = n0 + i;
                    uint32_t sa, sb, va[4];
                    e4m3x4_to_f16x2x2(*reinterpret_cast<const uint32_t *>(sv + 4 * nd), sa, sb);
                    e2m1x8_to_f16x2x4(w[i], va);
                    va[0] = f16x2_mul(va[0], sa);
                    va[1] = f16x2_mul(va[1], sa);
                    va[2] = f16x2_mul(va[2], sb);
                    va[3] = f16x2_mul(va[3], sb);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_16816_f16(o[nt][nd], va, pb[nt][0], pb[nt][1]);
                }
            }
        }
        // the slot is free: order this warp's reads and writes before the next bulk write
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
                (void)mbar_wait(&sm.full[warp][k % kSl], (uint32_t)((k / kSl) & 1), drain, 198);
        __syncwarp();
    }
    rows_finish<D, NT, true, true>(sm.u.red, &sm.abort_flag, a, o, m_ref, l, rows, h0, b, split, ws, ws_row);
}

// Pages per split: 64 (1024 tokens) where that fills the GPU several times over, down to 8 for small batches, whose
// latency is that of one split's pages.
int chunk_pages_for(int B, int H, int Hkv, int max_pages) {
    const int group = H / Hkv;
    const long long rows = (long long)B * Hkv * (group <= 8 ? 1 : (group + 15) / 16);
    int chunk = 64;
    while (chunk > 8 && rows * ((max_pages + chunk - 1) / chunk) < 4 * 152) chunk /= 2;
    return chunk;
}

template <int D, int NT>
cudaError_t launch_fp4_n(const DecodeMoreArgs &a, RowsParams p, cudaStream_t stream) {
    const size_t smem = sizeof(Fp4Smem<D, NT>) + 128;
    auto kernel = decode_fp4_kernel<D, NT>;
    cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void *>(kernel), (int)smem);
    if (e != cudaSuccess) return e;
    const uint8_t *k = static_cast<const uint8_t *>(a.k_pages), *v = static_cast<const uint8_t *>(a.v_pages);
    const dim3 grid(p.n_splits, p.Hkv * p.rgroups, p.B);
    if (p.cluster) {
        if (p.cluster > 8) e = ensure_large_clusters(reinterpret_cast<const void *>(kernel));
        if (e == cudaSuccess && cluster_fits(reinterpret_cast<const void *>(kernel), p.cluster, kRowWarps * 32, smem)) {
            RowsParams c = p;
            c.n_splits = p.cluster;
            c.chunk_pages = 0;
            return launch_cluster(kernel, dim3(p.cluster, grid.y, grid.z), kRowWarps * 32, smem, stream, k, v, c);
        }
        (void)cudaGetLastError();
        p.cluster = 0;  // no room for the cluster (a part of a GPU): the splits go through the workspace
    }
    kernel<<<grid, kRowWarps * 32, smem, stream>>>(k, v, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const unsigned blocks = (unsigned)(((long long)p.B * p.H + 3) / 4);
    return launch_dependent(decode_rows_merge_kernel<D, true>, dim3(blocks), 128, 0, stream, p);
}

template <int D>
cudaError_t launch_fp4_d(const DecodeMoreArgs &a, RowsParams p, cudaStream_t stream) {
    p.rgroups = p.group <= 8 ? 1 : (p.group + 15) / 16;
    return p.group <= 8 ? launch_fp4_n<D, 1>(a, p, stream) : launch_fp4_n<D, 2>(a, p, stream);
}

}  // namespace

size_t decode_fp4_workspace_bytes(int B, int H, int Hkv, int d, int max_pages, int page_size) {
    if (decode_workspace_bytes(B, H, Hkv, d, max_pages, page_size) == 0) return 0;  // unsupported sizes
    const size_t chunk = (size_t)chunk_pages_for(B, H, Hkv, max_pages);
    const size_t splits = ((size_t)max_pages + chunk - 1) / chunk;
    return (size_t)B * H * splits * (size_t)(d + 4) * sizeof(float);
}

cudaError_t launch_decode_fp4(const DecodeMoreArgs &a, cudaStream_t stream) {
    RowsParams p{};
    p.q = a.q;
    p.page_table = a.page_table;
    p.ctx_lens = a.ctx_lens;
    p.o = a.o;
    p.lse = a.lse;
    p.ws = static_cast<float *>(a.workspace);
    p.status = a.status;
    p.B = a.B;
    p.H = a.H;
    p.Hkv = a.Hkv;
    p.group = a.H / a.Hkv;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.chunk_pages = chunk_pages_for(a.B, a.H, a.Hkv, a.max_pages);
    p.n_splits = p.ws_splits = (a.max_pages + p.chunk_pages - 1) / p.chunk_pages;
    p.cluster = cluster_splits(a.B, a.H, a.Hkv, a.d, a.max_pages, true);
    const float kscale = a.scale * a.k_scale;
    p.c = kscale * kRowLog2e;
    p.v_scale = a.v_scale;
    p.cap_in = a.softcap > 0.f ? kscale / a.softcap : 0.f;
    p.cap_out = a.softcap * kRowLog2e;
    p.slopes = a.slopes;
    p.key_begin = a.key_begin;
    switch (a.d) {
        case 32: return launch_fp4_d<32>(a, p, stream);
        case 64: return launch_fp4_d<64>(a, p, stream);
        case 80: return launch_fp4_d<80>(a, p, stream);
        case 96: return launch_fp4_d<96>(a, p, stream);
        case 128: return launch_fp4_d<128>(a, p, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace attn
