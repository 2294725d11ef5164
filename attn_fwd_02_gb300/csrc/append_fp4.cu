// append_fp4.cu -- new tokens into the 4-bit paged cache (with the rotation of append_rope.cu on the way), and pages of
// that cache back as bf16.
//
// A block takes one pair of neighbouring positions 2m, 2m + 1 of a sequence, which share the bytes of the values' codes:
// a token that comes alone keeps the other nibble of each byte as it is, and no other block of the call writes there.  A
// thread takes 16 dims of a row, one block of the cache's scales; for a key it reads the 16 dims that they turn with as
// well (from L1 the second time), so that the block's maximum needs no exchange between threads.
//
// Neither memory nor the pipes are full (a quarter and a third to a half of the time): the chain position, angles, rows is what a
// block waits for, so what counts is the bytes that its threads ask for at once times the blocks that the registers allow.  Measured,
// up to 1024 new tokens of 8 sequences, ragged, 32 + 8 heads of 128, and their pages as bf16 (two calls, of which the second starts
// while the first drains), us:
//   query rows at once / blocks an SM   2 / 10 27.5, 4 / 10 28.1, 4 / 9 26.1, 4 / 8 25.1, 4 / 7 25.7, 5 / 8 25.9
//   before: the head dim at run time, the angles one by one   1 / 10 28.3, 2 / 10 27.8, 4 / 8 25.9; of that 64 threads a block 28.1, 256
//   29.0, the first query rows read before the angles 29.2
// and a division for each quotient 38 where the corrected ones took 29.8.  One token of 4 sequences: 6.0 us for the two calls, which
// is the host's time.
#include "fp4.cuh"
#include "rope.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 4;  // of the queries, in flight a thread

struct Fp4AppendParams {
    const uint4 *q, *k, *v;         // 16-byte vectors of 8 bf16
    long long qs[3], ks[3], vs[3];  // strides of batch, head and token, in vectors
    uint4 *q_out;
    uint8_t *k_pages, *v_pages;
    const float *cos_sin;           // null: no rotation
    const int32_t *page_table, *start_pos, *new_lens;  // new_lens may be null
    float k_inv, v_inv;             // 1 / scale
    int rope, max_pos, H, Hkv, N, pairs, max_pages, num_pages;
    RopeAxes axes;                  // positions null: the row of the table is the position in the cache
};

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 8) kv_append_fp4_kernel(const Fp4AppendParams p) {
    __shared__ __align__(16) float angles[2][kMaxRope];
    griddep_launch_dependents();
    griddep_wait();
    const int b = (int)(blockIdx.x / (unsigned)p.pairs);
    const int start = max(p.start_pos[b], 0);
    const long long pos0 = (long long)(start & ~1) + 2LL * (blockIdx.x % (unsigned)p.pairs);
    const int n_new = p.new_lens ? min(p.new_lens[b], p.N) : p.N;
    // the pair's tokens e: their place among the new ones, and whether they are there (uniform over the block)
    const int half = p.rope / 2;
    int tok[2];
    bool have[2];
    AxisRows at[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const long long t = pos0 + e - start;
        tok[e] = (int)t;
        have[e] = t >= 0 && t < n_new;
        if (have[e] && p.cos_sin) {
            if (p.axes.positions) {
                at[e] = axis_rows(p.axes, b, tok[e], p.max_pos);
            } else {
                at[e].ok = pos0 + e < p.max_pos;
#pragma unroll
                for (int a = 0; a < kMaxAxes; ++a) at[e].row[a] = (int)(pos0 + e);
            }
            have[e] = at[e].ok;  // past the rotation table: padding too
        }
    }
    {  // their angles, a thread a pair of dims
        static_assert(kThreads == kMaxRope, "two tokens' pairs");
        const int e = threadIdx.x / (kMaxRope / 2), pair = threadIdx.x % (kMaxRope / 2);
        if (e ? have[1] : have[0]) gather_pair(angles[e], p.cos_sin, p.axes, e ? at[1] : at[0], p.rope, pair);
    }
    if (!have[0] && !have[1]) return;
    const long long lp = pos0 / kFp4PS;
    int page = lp < p.max_pages ? p.page_table[(size_t)b * p.max_pages + lp] : -1;
    if (page >= p.num_pages) page = -1;
    __syncthreads();

    // Thread = (16-dim block j of a row, first row): it takes that block of every per_pass-th row.  The rows are those of the
    // tokens' keys, then the values' (a row for both tokens), then the tokens' queries.
    constexpr int vpr = D / 8, bpr = D / 16, per_pass = kThreads / bpr;
    const int j = threadIdx.x % bpr, r0 = threadIdx.x / bpr;
    if (r0 >= per_pass) return;
    const int e0 = have[0] ? 0 : 1, tokens = have[0] && have[1] ? 2 : 1;
    const int k_rows = page < 0 ? 0 : tokens * p.Hkv, kv_rows = page < 0 ? 0 : k_rows + p.Hkv;
    const int rows = kv_rows + (p.q ? tokens * p.H : 0);
    const int slot = (int)(pos0 % kFp4PS);  // even
    constexpr size_t block = (size_t)9 * D;
    // A row's 8 dims from vector w on, turned: fma(x, c, -(y s)) in the first half of the pairs, fma(y, c, x s) in the second.
    auto turn_pairs = [&](float (&x)[8], int w, const float *cs) {  // neighbours
        if (8 * w >= p.rope) return;
        const float *c = cs + 4 * w, *s = c + half;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // (rounded as the halves are, and as attn_rope_axes rounds)
            const float a = x[2 * i], e = x[2 * i + 1];
            x[2 * i] = __fmaf_rn(a, c[i], -__fmul_rn(e, s[i]));
            x[2 * i + 1] = __fmaf_rn(e, c[i], __fmul_rn(a, s[i]));
        }
    };
    auto turned = [&](const uint4 *row, int w, const float *cs, float (&x)[8]) {
        unpack8(row[w], x);
        if constexpr (INTER) {
            turn_pairs(x, w, cs);
        } else if (8 * w < p.rope) {
            const bool first = 8 * w < half;
            float y[8];
            unpack8(row[first ? w + half / 8 : w - half / 8], y);
            const float *c = cs + (first ? 8 * w : 8 * w - half);
            const uint64_t *c2 = reinterpret_cast<const uint64_t *>(c), *s2 = reinterpret_cast<const uint64_t *>(c + half);
            const uint64_t minus = first ? 0x8000000080000000ull : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f32x2_unpack(f32x2_fma(f32x2_pack(x[2 * i], x[2 * i + 1]), c2[i], f32x2_mul(f32x2_pack(y[2 * i], y[2 * i + 1]), s2[i] ^ minus)),
                             x[2 * i], x[2 * i + 1]);
        }
    };
    int row = r0;
    for (; row < kv_rows; row += per_pass) {
        if (row < k_rows) {
            const int second = row >= p.Hkv, e = e0 + second, h = row - second * p.Hkv;
            const uint4 *k = p.k + b * p.ks[0] + h * p.ks[1] + tok[e] * p.ks[2];
            uint8_t *kd = p.k_pages + ((size_t)page * p.Hkv + h) * block;
            float u[16], x[8];
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                turned(k, 2 * j + w, angles[e], x);
#pragma unroll
                for (int i = 0; i < 8; ++i) u[8 * w + i] = __fmul_rn(x[i], p.k_inv);
            }
            const uint32_t s = fp4_quotients(u), keep = s ? ~0u : 0u;
            float lo[8], hi[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) lo[i] = u[i], hi[i] = u[8 + i];
            kd[fp4_k_scale(D, slot + e, j)] = (uint8_t)s;
            *reinterpret_cast<uint2 *>(kd + fp4_k_codes(D, slot + e, j)) = make_uint2(f32x8_to_e2m1x8(lo) & keep, f32x8_to_e2m1x8(hi) & keep);
        } else {
            const int h = row - k_rows;
            const uint4 *v = p.v + b * p.vs[0] + h * p.vs[1] + 2 * j;
            uint8_t *vd = p.v_pages + ((size_t)page * p.Hkv + h) * block;
            uint4 *at = reinterpret_cast<uint4 *>(vd + fp4_v_codes(slot, j));
            uint4 old = make_uint4(0u, 0u, 0u, 0u);  // the codes of a token that is not there stay
            if (tokens == 1) old = *at;
            float u[2][16];
            uint32_t nonzero = ~0u;  // the nibbles of the tokens whose block has a scale
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint4 x0 = make_uint4(0u, 0u, 0u, 0u), x1 = x0;
                if (have[e]) x0 = v[tok[e] * p.vs[2]], x1 = v[tok[e] * p.vs[2] + 1];
                float x[2][8];
                unpack8(x0, x[0]);
                unpack8(x1, x[1]);
#pragma unroll
                for (int i = 0; i < 16; ++i) u[e][i] = __fmul_rn(x[i >> 3][i & 7], p.v_inv);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t s = fp4_quotients(u[e]);
                if (!s) nonzero &= e == 0 ? 0xf0f0f0f0u : 0x0f0f0f0fu;
                if (have[e]) vd[fp4_v_scale(D, slot + e, j)] = (uint8_t)s;
            }
            // byte x of the block: dim x of both tokens
            uint32_t bytes[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y[8];
#pragma unroll
                for (int n = 0; n < 4; ++n) y[2 * n] = u[0][4 * i + n], y[2 * n + 1] = u[1][4 * i + n];
                bytes[i] = f32x8_to_e2m1x8(y) & nonzero;
            }
            if (tokens == 1) {
                const uint32_t keep = e0 == 0 ? 0xf0f0f0f0u : 0x0f0f0f0fu;
                bytes[0] = (bytes[0] & ~keep) | (old.x & keep);
                bytes[1] = (bytes[1] & ~keep) | (old.y & keep);
                bytes[2] = (bytes[2] & ~keep) | (old.z & keep);
                bytes[3] = (bytes[3] & ~keep) | (old.w & keep);
            }
            *at = make_uint4(bytes[0], bytes[1], bytes[2], bytes[3]);
        }
    }
    // queries, kRows at once (in place too: a thread reads both halves of its pairs before it writes them)
    const int rot = p.rope / 16;
    const bool halves = !INTER && j < rot;  // x in the first half, its y in the second
    const int w0 = halves ? j : 2 * j, w1 = halves ? j + rot : 2 * j + 1;
    for (; row < rows; row += kRows * per_pass) {
        uint4 xv[kRows], yv[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int at = min(row + i * per_pass, rows - 1) - kv_rows, second = at >= p.H;
            const uint4 *q = p.q + b * p.qs[0] + (at - second * p.H) * p.qs[1] + tok[e0 + second] * p.qs[2];
            xv[i] = q[w0];
            yv[i] = q[w1];
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int at = row + i * per_pass - kv_rows, second = at >= p.H, e = e0 + second, h = at - second * p.H;
            if (at >= rows - kv_rows) break;
            uint4 *to = p.q_out + (((size_t)b * p.H + h) * p.N + tok[e]) * vpr;
            float x[8], y[8];
            unpack8(xv[i], x);
            unpack8(yv[i], y);
            if (INTER) {
                turn_pairs(x, w0, angles[e]);
                turn_pairs(y, w1, angles[e]);
            } else if (halves) {
                const float *c = angles[e] + 8 * j;
                const uint64_t *c2 = reinterpret_cast<const uint64_t *>(c), *s2 = reinterpret_cast<const uint64_t *>(c + half);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const uint64_t a = f32x2_pack(x[2 * n], x[2 * n + 1]), o = f32x2_pack(y[2 * n], y[2 * n + 1]);
                    f32x2_unpack(f32x2_fma(a, c2[n], f32x2_mul(o, s2[n] ^ 0x8000000080000000ull)), x[2 * n], x[2 * n + 1]);
                    f32x2_unpack(f32x2_fma(o, c2[n], f32x2_mul(a, s2[n])), y[2 * n], y[2 * n + 1]);
                }
            }
            to[w0] = pack8(x);
            to[w1] = pack8(y);
        }
    }
}

// ---------------------------------------------------------------- pages as bf16
struct UnpackParams {
    const uint8_t *k_pages, *v_pages;
    const int32_t *page_ids;
    uint4 *k_out, *v_out;
    float k_scale, v_scale;
    int n, Hkv, d, num_pages;
};

// A pair of codes, widened to f16, times their block's scale (exact: 6 bits, multiples of 2^-10 below 2^12) and the tensor's, as
// bf16.
__device__ __forceinline__ uint32_t scaled_pair(uint32_t h2, uint32_t block2, uint64_t scale2) {
    const uint32_t v = f16x2_mul(h2, block2);
    const __half2 h = *reinterpret_cast<const __half2 *>(&v);
    float x, y;
    f32x2_unpack(f32x2_mul(f32x2_pack(__low2float(h), __high2float(h)), scale2), x, y);
    return pack_bf16x2(x, y);
}

// One CTA a page's keys or values (blockIdx.y).  A thread takes 8 dims of two tokens that share the values' bytes, so that its
// vectors of the output are neighbours of the next lanes', and reads kAtOnce such pieces before it writes the first.
// Bound by memory from about 1000 pages of 8 heads on (11.8 us, 7.1 TB/s from L2); 250 pages with 1 / 2 / 4 pieces at once 6.3 / 4.9 / 4.6 us.
constexpr int kAtOnce = 4;
template <int D>
__global__ void __launch_bounds__(256) kv_unpack_fp4_kernel(const UnpackParams p) {
    constexpr int kVpr = D / 8, kPerHead = kVpr * 8;
    griddep_launch_dependents();
    griddep_wait();
    const int page = p.page_ids[blockIdx.x];
    if (page < 0 || page >= p.num_pages) return;
    const bool value = blockIdx.y != 0;
    const float f = value ? p.v_scale : p.k_scale;
    const uint64_t scale = f32x2_pack(f, f);
    const uint8_t *pages = (value ? p.v_pages : p.k_pages) + (size_t)page * p.Hkv * (9 * D);
    uint4 *out = (value ? p.v_out : p.k_out) + (size_t)blockIdx.x * p.Hkv * kFp4PS * kVpr;
    const int items = p.Hkv * kPerHead;
    for (int e0 = threadIdx.x; e0 < items; e0 += 256 * kAtOnce) {
        // vector w of tokens `token`, `token` + 1: the values' codes of both, or each token's of the keys; their two scales
        uint32_t c[kAtOnce][2], s[kAtOnce][2];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int e = min(e0 + 256 * i, items - 1);
            const int w = e % kVpr, token = 2 * (e / kVpr % 8), h = e / kPerHead;
            const uint8_t *src = pages + (size_t)h * (9 * D);
            if (value) {
                const uint2 v = *reinterpret_cast<const uint2 *>(src + fp4_v_codes(token, w / 2) + (w & 1) * 8);
                const uint32_t two = *reinterpret_cast<const uint16_t *>(src + fp4_v_scale(D, token, w / 2));
                c[i][0] = v.x, c[i][1] = v.y;
                s[i][0] = two & 0xffu, s[i][1] = two >> 8;
            } else {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    c[i][t] = *reinterpret_cast<const uint32_t *>(src + fp4_k_codes(D, token + t, 0) + 4 * w);
                    s[i][t] = src[fp4_k_scale(D, token + t, w / 2)];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int e = e0 + 256 * i;
            if (e >= items) break;
            const int w = e % kVpr, token = 2 * (e / kVpr % 8), h = e / kPerHead;
            uint4 *dst = out + ((size_t)h * kFp4PS + token) * kVpr + w;
            uint32_t r[2][4], x[2][4];
            e2m1x8_to_f16x2x4(c[i][0], x[0]);
            e2m1x8_to_f16x2x4(c[i][1], x[1]);
#pragma unroll
            for (int n = 0; n < 4; ++n) {  // (values: dims 2n, 2n + 1, each with both tokens)
                const uint32_t a = x[n >> 1][2 * (n & 1)], b = x[n >> 1][2 * (n & 1) + 1];
                r[0][n] = value ? __byte_perm(a, b, 0x5410) : x[0][n];
                r[1][n] = value ? __byte_perm(a, b, 0x7632) : x[1][n];
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint32_t b2 = e4m3_pair(s[i][t] * 0x101u);
                dst[t * kVpr] = make_uint4(scaled_pair(r[t][0], b2, scale), scaled_pair(r[t][1], b2, scale),
                                           scaled_pair(r[t][2], b2, scale), scaled_pair(r[t][3], b2, scale));
            }
        }
    }
}

template <int D>
cudaError_t launch_append_d(const Fp4AppendParams &p, dim3 grid, bool interleaved, cudaStream_t stream) {
    return interleaved ? launch_dependent(kv_append_fp4_kernel<D, true>, grid, kThreads, 0, stream, p)
                       : launch_dependent(kv_append_fp4_kernel<D, false>, grid, kThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_kv_append_fp4(const RopeAppendArgs &a, cudaStream_t stream) {
    Fp4AppendParams p;
    p.q = static_cast<const uint4 *>(a.q);
    p.k = static_cast<const uint4 *>(a.k_new);
    p.v = static_cast<const uint4 *>(a.v_new);
    for (int i = 0; i < 3; ++i) {
        p.qs[i] = a.q_strides[i] / 8;
        p.ks[i] = a.k_strides[i] / 8;
        p.vs[i] = a.v_strides[i] / 8;
    }
    p.q_out = static_cast<uint4 *>(a.q_out);
    p.k_pages = static_cast<uint8_t *>(a.k_pages);
    p.v_pages = static_cast<uint8_t *>(a.v_pages);
    p.cos_sin = a.cos_sin;
    p.page_table = a.page_table;
    p.start_pos = a.start_pos;
    p.new_lens = a.new_lens;
    p.k_inv = 1.f / a.k_scale;
    p.v_inv = 1.f / a.v_scale;
    p.rope = a.cos_sin ? a.rope_dim : 0;
    p.max_pos = a.max_pos;
    p.H = a.H;
    p.Hkv = a.Hkv;
    p.N = a.Nnew;
    p.pairs = a.Nnew / 2 + 1;  // the positions may start at an odd one
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.axes = a.axes;
    const dim3 grid((unsigned)((long long)a.B * p.pairs));
    const bool inter = a.interleaved != 0;
    switch (a.d) {
        case 32: return launch_append_d<32>(p, grid, inter, stream);
        case 64: return launch_append_d<64>(p, grid, inter, stream);
        case 80: return launch_append_d<80>(p, grid, inter, stream);
        case 96: return launch_append_d<96>(p, grid, inter, stream);
        case 128: return launch_append_d<128>(p, grid, inter, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_kv_unpack_fp4(const void *k_pages, const void *v_pages, float k_scale, float v_scale,
                                 const int32_t *page_ids, int n, void *k_out, void *v_out, int Hkv, int d, int num_pages,
                                 cudaStream_t stream) {
    const UnpackParams p{static_cast<const uint8_t *>(k_pages), static_cast<const uint8_t *>(v_pages), page_ids,
                         static_cast<uint4 *>(k_out), static_cast<uint4 *>(v_out), k_scale, v_scale, n, Hkv, d, num_pages};
    const dim3 grid((unsigned)n, 2);
    switch (d) {
        case 32: return launch_dependent(kv_unpack_fp4_kernel<32>, grid, 256, 0, stream, p);
        case 64: return launch_dependent(kv_unpack_fp4_kernel<64>, grid, 256, 0, stream, p);
        case 80: return launch_dependent(kv_unpack_fp4_kernel<80>, grid, 256, 0, stream, p);
        case 96: return launch_dependent(kv_unpack_fp4_kernel<96>, grid, 256, 0, stream, p);
        case 128: return launch_dependent(kv_unpack_fp4_kernel<128>, grid, 256, 0, stream, p);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace attn
