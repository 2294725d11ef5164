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
// Memory-bound: every element is read and written once.  One block takes one token.  A thread moves 16
// elements of a row at a time (two 16-byte vectors, the two halves of eight pairs), all in registers, so a
// contiguous query tensor may be rotated in place; it takes the same item of several rows, so its sines and
// cosines are loaded once, and its first rows are in flight before the position, the page and the angles are
// known (the chain of those loads is what a decode step waits for).  The rotation runs in fp32 and is rounded
// once, to bf16 or to the cache's e4m3.  Measured (32 query and 8 key/value heads, d 128): 8 x 1024 tokens,
// half of them padding, 14.8 us (5.49 TB/s; 17.4 with the loads after the look-ups, 15.3 with 64 threads a
// block, 23 with 256 before); 128 tokens into an e4m3 cache 2.3 us (3.0).
#include <cuda_fp8.h>

#include "launch.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kPS = 16;
constexpr int kThreads = 128;
constexpr int kAhead = 2;  // query rows a thread has in flight before it knows its position

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
__global__ void __launch_bounds__(kThreads) kv_append_rope_kernel(const RopeParams p) {
    const int b = (int)(blockIdx.x / (unsigned)p.N), t = (int)(blockIdx.x % (unsigned)p.N);
    if (p.new_lens && t >= p.new_lens[b]) return;  // padding
    // Thread = (item of a row, first row): an item is two vectors -- the two halves of eight pairs, or two
    // neighbours where nothing turns -- and the thread takes that item of every per_pass-th row, so its sines
    // and cosines are loaded once.
    const int vpr = p.d / 8;         // vectors per row
    const int ipr = p.d / 16;        // items per row
    const int rot = p.rope / 16;     // items of a row that turn
    const int per_pass = kThreads / ipr;
    const int i = threadIdx.x % ipr, r0 = threadIdx.x / ipr;
    if (r0 >= per_pass) return;
    const bool turns = i < rot;
    const int t0 = (turns && !INTER) ? i : 2 * i, t1 = (turns && !INTER) ? i + rot : 2 * i + 1;  // its vectors
    // the first rows' loads start before the position, the page and the angles are known
    const uint4 *q = p.q + b * p.qs[0] + t * p.qs[2];
    const uint4 *k = p.k + b * p.ks[0] + t * p.ks[2], *v = p.v + b * p.vs[0] + t * p.vs[2];
    uint4 x0[kAhead], y0[kAhead], kx, ky, vx, vy;
    if (p.q) {
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
            const int h = r0 + n * per_pass;
            if (h < p.H) {
                x0[n] = q[h * p.qs[1] + t0];
                y0[n] = q[h * p.qs[1] + t1];
            }
        }
    }
    if (r0 < p.Hkv) {
        kx = k[r0 * p.ks[1] + t0];
        ky = k[r0 * p.ks[1] + t1];
        vx = v[r0 * p.vs[1] + 2 * i];
        vy = v[r0 * p.vs[1] + 2 * i + 1];
    }
    const long long pos = (long long)max(p.start_pos[b], 0) + t;
    if (pos >= p.max_pos) return;  // past the rotation table: padding too
    const long long lp = pos / kPS;
    const int page = lp < p.max_pages ? p.page_table[(size_t)b * p.max_pages + lp] : -1;
    float c[8], s[8];
    if (turns) {
        const float *cs = p.cos_sin + (size_t)pos * p.rope + 8 * i;
        const float4 *c4 = reinterpret_cast<const float4 *>(cs), *s4 = reinterpret_cast<const float4 *>(cs + p.rope / 2);
        const float4 ca = c4[0], cb = c4[1], sa = s4[0], sb = s4[1];
        c[0] = ca.x, c[1] = ca.y, c[2] = ca.z, c[3] = ca.w, c[4] = cb.x, c[5] = cb.y, c[6] = cb.z, c[7] = cb.w;
        s[0] = sa.x, s[1] = sa.y, s[2] = sa.z, s[3] = sa.w, s[4] = sb.x, s[5] = sb.y, s[6] = sb.z, s[7] = sb.w;
    }
    // one item: its values, the destination row (a query's or a page slot's), whether it turns, and the
    // cache's factor
    auto put = [&](uint4 xv, uint4 yv, void *dst, bool turn, bool page_row, float inv) {
        float x[8], y[8];
        unpack8(xv, x);
        unpack8(yv, y);
        if (turn) {
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
        const int v0 = turn ? t0 : 2 * i, v1 = turn ? t1 : 2 * i + 1;
        if (FP8 && page_row) {
            static_cast<uint2 *>(dst)[v0] = quant8(x, inv);
            static_cast<uint2 *>(dst)[v1] = quant8(y, inv);
        } else {
            static_cast<uint4 *>(dst)[v0] = pack8(x);
            static_cast<uint4 *>(dst)[v1] = pack8(y);
        }
    };
    if (p.q) {
        uint4 *qo = p.q_out + ((size_t)b * p.H * p.N + t) * vpr;
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
            const int h = r0 + n * per_pass;
            if (h < p.H) put(x0[n], y0[n], qo + (size_t)h * p.N * vpr, turns, false, 1.f);
        }
        for (int h = r0 + kAhead * per_pass; h < p.H; h += per_pass)
            put(q[h * p.qs[1] + t0], q[h * p.qs[1] + t1], qo + (size_t)h * p.N * vpr, turns, false, 1.f);
    }
    if (page < 0 || page >= p.num_pages) return;  // past the table's capacity, or an unmapped page
    constexpr size_t kElem = FP8 ? 8 : 16;        // bytes of a page vector
    const size_t slot = ((size_t)page * p.Hkv * kPS + (size_t)(pos % kPS)) * vpr;  // of head 0
    uint8_t *kd = static_cast<uint8_t *>(p.k_pages), *vd = static_cast<uint8_t *>(p.v_pages);
    for (int h = r0; h < p.Hkv; h += per_pass) {
        const size_t at = (slot + (size_t)h * kPS * vpr) * kElem;
        if (h != r0) {
            kx = k[h * p.ks[1] + t0];
            ky = k[h * p.ks[1] + t1];
            vx = v[h * p.vs[1] + 2 * i];
            vy = v[h * p.vs[1] + 2 * i + 1];
        }
        put(kx, ky, kd + at, turns, true, p.k_inv);
        put(vx, vy, vd + at, false, true, p.v_inv);
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
        if (a.interleaved) kv_append_rope_kernel<true, true><<<grid, kThreads, 0, stream>>>(p);
        else kv_append_rope_kernel<false, true><<<grid, kThreads, 0, stream>>>(p);
    } else {
        if (a.interleaved) kv_append_rope_kernel<true, false><<<grid, kThreads, 0, stream>>>(p);
        else kv_append_rope_kernel<false, false><<<grid, kThreads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace attn
