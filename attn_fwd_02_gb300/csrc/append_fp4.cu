// append_fp4.cu -- new tokens into the 4-bit paged cache (with the rotation of append_rope.cu on the way), and pages of
// that cache back as bf16.
//
// A block takes one pair of neighbouring positions 2m, 2m + 1 of a sequence, which share the bytes of the values' codes:
// a token that comes alone keeps the other nibble of each byte as it is, and no other block of the call writes there.  A
// thread takes 16 dims of a row, one block of the cache's scales; for a key it reads the 16 dims that they turn with as
// well (from L1 the second time), so that the block's maximum needs no exchange between threads.
#include "fp4.cuh"
#include "rope.cuh"

namespace attn {
namespace {

constexpr int kThreads = 128;

struct Fp4AppendParams {
    const uint4 *q, *k, *v;         // 16-byte vectors of 8 bf16
    long long qs[3], ks[3], vs[3];  // strides of batch, head and token, in vectors
    uint4 *q_out;
    uint8_t *k_pages, *v_pages;
    const float *cos_sin;           // null: no rotation
    const int32_t *page_table, *start_pos, *new_lens;  // new_lens may be null
    float k_inv, v_inv;             // 1 / scale
    int rope, max_pos, H, Hkv, N, pairs, d, max_pages, num_pages;
    RopeAxes axes;                  // positions null: the row of the table is the position in the cache
};

template <bool INTER>
__global__ void __launch_bounds__(kThreads) kv_append_fp4_kernel(const Fp4AppendParams p) {
    __shared__ float angles[2][kMaxRope];
    const int b = (int)(blockIdx.x / (unsigned)p.pairs);
    const int start = max(p.start_pos[b], 0);
    const long long pos0 = (long long)(start & ~1) + 2LL * (blockIdx.x % (unsigned)p.pairs);
    const int n_new = p.new_lens ? min(p.new_lens[b], p.N) : p.N;
    // the pair's tokens e: their place among the new ones, and whether they are there (uniform over the block)
    int tok[2];
    bool have[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const long long t = pos0 + e - start;
        tok[e] = (int)t;
        have[e] = t >= 0 && t < n_new;
        if (have[e] && p.cos_sin) {
            AxisRows rows;
            if (p.axes.positions) {
                rows = axis_rows(p.axes, b, tok[e], p.max_pos);
            } else {
                rows.ok = pos0 + e < p.max_pos;
#pragma unroll
                for (int a = 0; a < kMaxAxes; ++a) rows.row[a] = (int)(pos0 + e);
            }
            have[e] = rows.ok;  // past the rotation table: padding too
            if (rows.ok) gather_angles(angles[e], p.cos_sin, p.axes, rows, p.rope, threadIdx.x, kThreads);
        }
    }
    if (!have[0] && !have[1]) return;
    const long long lp = pos0 / kFp4PS;
    int page = lp < p.max_pages ? p.page_table[(size_t)b * p.max_pages + lp] : -1;
    if (page >= p.num_pages) page = -1;
    __syncthreads();

    // Thread = (16-dim block j of a row, first row): it takes that block of every per_pass-th row.
    const int vpr = p.d / 8, bpr = p.d / 16, half = p.rope / 2;
    const int per_pass = kThreads / bpr;
    const int j = threadIdx.x % bpr, r0 = threadIdx.x / bpr;
    if (r0 >= per_pass) return;
    // A row's 8 dims from vector w on, turned: x c - y s in the first half of the pairs, y c + x s in the second.
    auto turned = [&](const uint4 *row, int w, const float *cs, float (&x)[8]) {
        unpack8(row[w], x);
        if (8 * w >= p.rope) return;
        if constexpr (INTER) {
            const float *c = cs + 4 * w, *s = c + half;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = x[2 * i] * c[i] - x[2 * i + 1] * s[i];
                x[2 * i + 1] = x[2 * i + 1] * c[i] + x[2 * i] * s[i];
                x[2 * i] = u;
            }
        } else {
            const bool first = 8 * w < half;
            float y[8];
            unpack8(row[first ? w + half / 8 : w - half / 8], y);
            const float *c = cs + (first ? 8 * w : 8 * w - half), *s = c + half;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = first ? x[i] * c[i] - y[i] * s[i] : x[i] * c[i] + y[i] * s[i];
        }
    };
    // 16 values times 1 / scale
    auto load_block = [&](const uint4 *row, const float *cs, float inv, bool turn, float (&u)[16]) {
        float x[2][8];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if (turn) turned(row, 2 * j + w, cs, x[w]);
            else unpack8(row[2 * j + w], x[w]);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[8 * w + i] = __fmul_rn(x[w][i], inv);
        }
    };
    if (p.q) {
        // (in place too: a thread reads both halves of its pairs before it writes them)
        const int rot = p.rope / 16;
        const bool turns = !INTER && j < rot;
        const int w0 = turns ? j : 2 * j, w1 = turns ? j + rot : 2 * j + 1;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (!have[e]) continue;
            const uint4 *q = p.q + b * p.qs[0] + tok[e] * p.qs[2];
            uint4 *out = p.q_out + ((size_t)b * p.H * p.N + tok[e]) * vpr;
            for (int h = r0; h < p.H; h += per_pass) {
                float x[8], y[8];
                const uint4 *row = q + h * p.qs[1];
                uint4 *to = out + (size_t)h * p.N * vpr;
                if (turns) {
                    unpack8(row[w0], x);
                    unpack8(row[w1], y);
                    const float *c = angles[e] + 8 * j, *s = c + half;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float u = x[i] * c[i] - y[i] * s[i];
                        y[i] = y[i] * c[i] + x[i] * s[i];
                        x[i] = u;
                    }
                } else if (INTER) {
                    turned(row, w0, angles[e], x);
                    turned(row, w1, angles[e], y);
                } else {
                    unpack8(row[w0], x);
                    unpack8(row[w1], y);
                }
                to[w0] = pack8(x);
                to[w1] = pack8(y);
            }
        }
    }
    if (page < 0) return;
    const int slot = (int)(pos0 % kFp4PS);  // even
    const size_t block = (size_t)9 * p.d;
    for (int h = r0; h < p.Hkv; h += per_pass) {
        uint8_t *kd = p.k_pages + ((size_t)page * p.Hkv + h) * block, *vd = p.v_pages + ((size_t)page * p.Hkv + h) * block;
        float u[16];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (!have[e]) continue;
            uint32_t codes[2];
            load_block(p.k + b * p.ks[0] + h * p.ks[1] + tok[e] * p.ks[2], angles[e], p.k_inv, p.cos_sin != nullptr, u);
            kd[fp4_k_scale(p.d, slot + e, j)] = (uint8_t)fp4_block(u, codes);
            *reinterpret_cast<uint2 *>(kd + fp4_k_codes(p.d, slot + e, j)) = make_uint2(codes[0], codes[1]);
        }
        // values: nibble e of byte x holds dim x of token e
        uint4 *at = reinterpret_cast<uint4 *>(vd + fp4_v_codes(slot, j));
        uint32_t bytes[4] = {0u, 0u, 0u, 0u};
        if (!have[0] || !have[1]) {
            const uint4 old = *at;
            const uint32_t keep = have[0] ? 0xf0f0f0f0u : 0x0f0f0f0fu;
            bytes[0] = old.x & keep, bytes[1] = old.y & keep, bytes[2] = old.z & keep, bytes[3] = old.w & keep;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (!have[e]) continue;
            uint32_t codes[2];
            load_block(p.v + b * p.vs[0] + h * p.vs[1] + tok[e] * p.vs[2], nullptr, p.v_inv, false, u);
            vd[fp4_v_scale(p.d, slot + e, j)] = (uint8_t)fp4_block(u, codes);
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // nibbles 4i .. 4i + 3 into the bytes of a word
                const uint32_t n = codes[i >> 1] >> (16 * (i & 1));
                const uint32_t w = (n & 0xfu) | (n & 0xf0u) << 4 | (n & 0xf00u) << 8 | (n & 0xf000u) << 12;
                bytes[i] |= w << (4 * e);
            }
        }
        *at = make_uint4(bytes[0], bytes[1], bytes[2], bytes[3]);
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

// Eight codes' f16 words, low half first, times f (the block's scale times the tensor's) as bf16.
__device__ __forceinline__ uint32_t scaled_pair(uint32_t h2, float s, float scale) {
    const __half2 h = *reinterpret_cast<const __half2 *>(&h2);
    return pack_bf16x2(__fmul_rn(__low2float(h) * s, scale), __fmul_rn(__high2float(h) * s, scale));
}

// A thread takes 16 dims of two tokens (a byte of the values' codes holds both); z: keys, values.
__global__ void __launch_bounds__(256) kv_unpack_fp4_kernel(const UnpackParams p) {
    const int bpr = p.d / 16, per_head = bpr * 8;
    const bool value = blockIdx.y != 0;
    const long long total = (long long)p.n * p.Hkv * per_head;
    for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < total; e += (long long)gridDim.x * 256) {
        const int j = (int)(e % bpr), pair = (int)(e / bpr % 8);
        const long long row = e / per_head;  // page * Hkv + head
        const int page = p.page_ids[row / p.Hkv];
        if (page < 0 || page >= p.num_pages) continue;
        const uint8_t *src = (value ? p.v_pages : p.k_pages) + ((size_t)page * p.Hkv + row % p.Hkv) * (size_t)(9 * p.d);
        uint4 *dst = (value ? p.v_out : p.k_out) + ((size_t)row * kFp4PS + 2 * pair) * (size_t)(p.d / 8) + 2 * j;
        const float scale = value ? p.v_scale : p.k_scale;
        uint32_t out[2][8];
        if (value) {
            const uint4 w = *reinterpret_cast<const uint4 *>(src + fp4_v_codes(2 * pair, j));
            const float s0 = e4m3_to_float(src[fp4_v_scale(p.d, 2 * pair, j)]);
            const float s1 = e4m3_to_float(src[fp4_v_scale(p.d, 2 * pair + 1, j)]);
            const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t r[4];  // dims 4i .. 4i + 3, a pair of tokens each
                e2m1x8_to_f16x2x4(ws[i], r);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t lo = __byte_perm(r[2 * h], r[2 * h + 1], 0x5410), hi = __byte_perm(r[2 * h], r[2 * h + 1], 0x7632);
                    out[0][2 * i + h] = scaled_pair(lo, s0, scale);
                    out[1][2 * i + h] = scaled_pair(hi, s1, scale);
                }
            }
        } else {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint2 w = *reinterpret_cast<const uint2 *>(src + fp4_k_codes(p.d, 2 * pair + t, j));
                const float s = e4m3_to_float(src[fp4_k_scale(p.d, 2 * pair + t, j)]);
                uint32_t r[2][4];
                e2m1x8_to_f16x2x4(w.x, r[0]);
                e2m1x8_to_f16x2x4(w.y, r[1]);
#pragma unroll
                for (int i = 0; i < 8; ++i) out[t][i] = scaled_pair(r[i >> 2][i & 3], s, scale);
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            dst[t * (p.d / 8)] = make_uint4(out[t][0], out[t][1], out[t][2], out[t][3]);
            dst[t * (p.d / 8) + 1] = make_uint4(out[t][4], out[t][5], out[t][6], out[t][7]);
        }
    }
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
    p.d = a.d;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.axes = a.axes;
    const unsigned grid = (unsigned)((long long)a.B * p.pairs);
    if (a.interleaved) kv_append_fp4_kernel<true><<<grid, kThreads, 0, stream>>>(p);
    else kv_append_fp4_kernel<false><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kv_unpack_fp4(const void *k_pages, const void *v_pages, float k_scale, float v_scale,
                                 const int32_t *page_ids, int n, void *k_out, void *v_out, int Hkv, int d, int num_pages,
                                 cudaStream_t stream) {
    int sms = 0;
    const cudaError_t e = current_sm_count(&sms);
    if (e != cudaSuccess) return e;
    const UnpackParams p{static_cast<const uint8_t *>(k_pages), static_cast<const uint8_t *>(v_pages), page_ids,
                         static_cast<uint4 *>(k_out), static_cast<uint4 *>(v_out), k_scale, v_scale, n, Hkv, d, num_pages};
    const long long want = ((long long)n * Hkv * (d / 2) + 255) / 256, most = (long long)sms * 8;
    kv_unpack_fp4_kernel<<<dim3((unsigned)(want < most ? want : most), 2), 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace attn
