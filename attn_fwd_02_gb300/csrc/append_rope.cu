// append_rope.cu -- rotary position embedding of new queries and keys on their way into the paged
// KV cache.
//
// Token t of sequence b sits at position p = start_pos[b] + t.  The first r dims of its query and
// key rows are r / 2 pairs (x, y), each turned by the angle of its position:
//     x' = x cos - y sin,   y' = y cos + x sin,
// with cos and sin read from a table of fp32 rows (cos of the r / 2 pairs, then their sin), so any
// rule for the angles fits.  Pair i is dims (i, i + r / 2), or (2i, 2i + 1) when interleaved.  The
// rotated key and the value go to slot p % 16 of page page_table[b][p / 16], the rotated query to a
// contiguous [B, H, Nnew, d] tensor, as the decode and the chunked prefill read it.
//
// Memory-bound: every element is read and written once.  One block takes one token, so the position,
// the page and the table row are looked up once per block; a thread moves 16 elements at a time (two
// 16-byte vectors, the two halves of eight pairs), all in registers, so a contiguous query tensor may
// be rotated in place.  The rotation runs in fp32 and is rounded once, to bf16 or to the cache's e4m3.
#include <cuda_fp8.h>

#include "launch.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kPS = 16;

struct RopeParams {
    const uint4 *q, *k, *v;     // 16-byte vectors of 8 bf16
    long long qs[3], ks[3], vs[3];  // strides of batch, head and token, in vectors
    uint4 *q_out;
    void *k_pages, *v_pages;
    const float *cos_sin;
    const int32_t *page_table, *start_pos, *new_lens;  // new_lens may be null
    float k_inv, v_inv;         // 1 / scale of an e4m3 cache
    int rope, max_pos, H, Hkv, N, d, max_pages, num_pages;
};

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}
// e4m3 nearest-even of f * inv, saturating at +-448, as the unrotated append converts.
__device__ __forceinline__ uint2 quant8(const float (&f)[8], float inv) {
    uint32_t out[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = make_float2(__fmul_rn(f[2 * i], inv), __fmul_rn(f[2 * i + 1], inv));
        out[i >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3) << (16 * (i & 1));
    }
    return make_uint2(out[0], out[1]);
}

template <bool INTER, bool FP8>
__global__ void __launch_bounds__(128) kv_append_rope_kernel(const RopeParams p) {
    const int b = (int)(blockIdx.x / (unsigned)p.N), t = (int)(blockIdx.x % (unsigned)p.N);
    if (p.new_lens && t >= p.new_lens[b]) return;  // padding
    const long long pos = (long long)max(p.start_pos[b], 0) + t;
    if (pos >= p.max_pos) return;  // past the rotation table: padding too
    const long long lp = pos / kPS;
    const int page = lp < p.max_pages ? p.page_table[(size_t)b * p.max_pages + lp] : -1;
    const bool mapped = page >= 0 && page < p.num_pages;
    const float *cs = p.cos_sin + (size_t)pos * p.rope;

    const int vpr = p.d / 8;         // vectors per row
    const int ipr = p.d / 16;        // items (two vectors) per row
    const int rot = p.rope / 16;     // items of a row that turn
    const int rows = (p.q ? p.H : 0) + 2 * p.Hkv;
    for (int e = threadIdx.x; e < rows * ipr; e += blockDim.x) {
        const int i = e % ipr;
        int row = e / ipr;
        const uint4 *src;
        int kind;  // 0 query, 1 key, 2 value
        int head = row - 2 * p.Hkv;
        if (row < p.Hkv) {
            kind = 1, head = row;
            src = p.k + b * p.ks[0] + head * p.ks[1] + t * p.ks[2];
        } else if (row < 2 * p.Hkv) {
            kind = 2, head = row - p.Hkv;
            src = p.v + b * p.vs[0] + head * p.vs[1] + t * p.vs[2];
        } else {
            kind = 0;
            src = p.q + b * p.qs[0] + head * p.qs[1] + t * p.qs[2];
        }
        if (kind != 0 && !mapped) continue;  // past the table's capacity, or an unmapped page
        const bool turn = kind != 2 && i < rot;
        // vectors of this item: the two halves of eight pairs, or two neighbours
        const int v0 = (turn && !INTER) ? i : 2 * i;
        const int v1 = (turn && !INTER) ? i + rot : 2 * i + 1;
        float x[8], y[8];
        unpack8(src[v0], x);
        unpack8(src[v1], y);
        if (turn) {
            const float4 *c4 = reinterpret_cast<const float4 *>(cs + 8 * i);
            const float4 *s4 = reinterpret_cast<const float4 *>(cs + p.rope / 2 + 8 * i);
            const float4 ca = c4[0], cb = c4[1], sa = s4[0], sb = s4[1];
            const float c[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
            const float s[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
            if constexpr (INTER) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float u = x[2 * j] * c[j] - x[2 * j + 1] * s[j];
                    x[2 * j + 1] = x[2 * j + 1] * c[j] + x[2 * j] * s[j];
                    x[2 * j] = u;
                    const float w = y[2 * j] * c[4 + j] - y[2 * j + 1] * s[4 + j];
                    y[2 * j + 1] = y[2 * j + 1] * c[4 + j] + y[2 * j] * s[4 + j];
                    y[2 * j] = w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float u = x[j] * c[j] - y[j] * s[j];
                    y[j] = y[j] * c[j] + x[j] * s[j];
                    x[j] = u;
                }
            }
        }
        if (kind == 0) {
            uint4 *dst = p.q_out + (((size_t)b * p.H + head) * p.N + t) * vpr;
            dst[v0] = pack8(x);
            dst[v1] = pack8(y);
        } else {
            const size_t at = (((size_t)page * p.Hkv + head) * kPS + (size_t)(pos % kPS)) * vpr;
            void *pool = kind == 1 ? p.k_pages : p.v_pages;
            if constexpr (FP8) {
                const float inv = kind == 1 ? p.k_inv : p.v_inv;
                uint2 *dst = static_cast<uint2 *>(pool) + at;
                dst[v0] = quant8(x, inv);
                dst[v1] = quant8(y, inv);
            } else {
                uint4 *dst = static_cast<uint4 *>(pool) + at;
                dst[v0] = pack8(x);
                dst[v1] = pack8(y);
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv_append_rope(const RopeAppendArgs &a, cudaStream_t stream) {
    RopeParams p;
    p.q = static_cast<const uint4 *>(a.q);
    p.k = static_cast<const uint4 *>(a.k_new);
    p.v = static_cast<const uint4 *>(a.v_new);
    for (int i = 0; i < 3; ++i) {
        p.qs[i] = a.q_strides[i] / 8;
        p.ks[i] = a.k_strides[i] / 8;
        p.vs[i] = a.v_strides[i] / 8;
    }
    p.q_out = static_cast<uint4 *>(a.q_out);
    p.k_pages = a.k_pages;
    p.v_pages = a.v_pages;
    p.cos_sin = a.cos_sin;
    p.page_table = a.page_table;
    p.start_pos = a.start_pos;
    p.new_lens = a.new_lens;
    p.k_inv = 1.f / a.k_scale;
    p.v_inv = 1.f / a.v_scale;
    p.rope = a.rope_dim;
    p.max_pos = a.max_pos;
    p.H = a.H;
    p.Hkv = a.Hkv;
    p.N = a.Nnew;
    p.d = a.d;
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    const unsigned grid = (unsigned)((long long)a.B * a.Nnew);
    if (a.kv_fp8) {
        if (a.interleaved) kv_append_rope_kernel<true, true><<<grid, 128, 0, stream>>>(p);
        else kv_append_rope_kernel<false, true><<<grid, 128, 0, stream>>>(p);
    } else {
        if (a.interleaved) kv_append_rope_kernel<true, false><<<grid, 128, 0, stream>>>(p);
        else kv_append_rope_kernel<false, false><<<grid, 128, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace attn
