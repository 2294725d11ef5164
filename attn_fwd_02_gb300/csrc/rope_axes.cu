// rope_axes.cu -- rotary position embedding of queries and keys by positions with several axes, outside the cache: a
// training step's or a vision tower's, and its gradient.
//
// Pair i of a token, (x, y), turns by the angle whose cosine c and sine s stand in column i of row
// positions[axis(i)][token]:  x' = x c - y s, y' = y c + x s.  The gradient is the transposed rotation of the gradient:
// dx = dx' c + dy' s, dy = dy' c - dx' s (right for tables with a factor on c and s too).
//
// Memory-bound: every element is read and written once.  A block takes kTokens tokens of one sequence, gathers their
// angles into shared memory, and turns the rows of all heads, 16 elements (8 pairs) a thread at a time, held in registers,
// so that a view may be turned in place.
#include "rope.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;

struct RopeOnlyParams {
    const uint4 *q, *k;
    uint4 *q_out, *k_out;
    long long qs[3], ks[3], qo[3], ko[3];  // strides of batch, head and token, in vectors of 8
    const float *cos_sin;
    int rope, max_pos, H, Hkv, N, d, blocks;
    float sign;  // of the sines: -1 for the gradient
    RopeAxes axes;
};

template <bool INTER>
__global__ void __launch_bounds__(kThreads) rope_axes_kernel(const RopeOnlyParams p) {
    __shared__ __align__(16) float angles[kTokens][kMaxRope];
    __shared__ int inside[kTokens];
    const int b = (int)(blockIdx.x / (unsigned)p.blocks), t0 = (int)(blockIdx.x % (unsigned)p.blocks) * kTokens;
    const int tokens = min(kTokens, p.N - t0);
    for (int t = threadIdx.x >> 6; t < tokens; t += kThreads / 64) {
        const AxisRows rows = axis_rows(p.axes, b, t0 + t, p.max_pos);
        if (rows.ok) gather_angles(angles[t], p.cos_sin, p.axes, rows, p.rope, threadIdx.x & 63, 64);
        if ((threadIdx.x & 63) == 0) inside[t] = rows.ok;
    }
    __syncthreads();
    const int ipr = p.d / 16, rot = p.rope / 16, half = p.rope / 2;
    const int per_token = (p.H + p.Hkv) * ipr;
    for (int e = threadIdx.x; e < tokens * per_token; e += kThreads) {
        const int i = e % ipr, row = e / ipr % (p.H + p.Hkv), t = e / per_token;
        const bool is_k = row >= p.H, turns = i < rot;
        const int h = is_k ? row - p.H : row;
        const long long *si = is_k ? p.ks : p.qs, *so = is_k ? p.ko : p.qo;
        const uint4 *src = (is_k ? p.k : p.q) + b * si[0] + h * si[1] + (t0 + t) * si[2];
        uint4 *dst = (is_k ? p.k_out : p.q_out) + b * so[0] + h * so[1] + (t0 + t) * so[2];
        const int w0 = turns && !INTER ? i : 2 * i, w1 = turns && !INTER ? i + rot : 2 * i + 1;
        uint4 xv = src[w0], yv = src[w1];
        if (!inside[t]) {
            xv = yv = make_uint4(0u, 0u, 0u, 0u);
        } else if (turns) {
            float x[8], y[8];
            unpack8(xv, x);
            unpack8(yv, y);
            const float *c = angles[t] + 8 * i, *s = c + half;
            if constexpr (INTER) {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float s0 = p.sign * s[n], s1 = p.sign * s[4 + n];
                    const float u = x[2 * n] * c[n] - x[2 * n + 1] * s0;
                    x[2 * n + 1] = x[2 * n + 1] * c[n] + x[2 * n] * s0;
                    x[2 * n] = u;
                    const float v = y[2 * n] * c[4 + n] - y[2 * n + 1] * s1;
                    y[2 * n + 1] = y[2 * n + 1] * c[4 + n] + y[2 * n] * s1;
                    y[2 * n] = v;
                }
            } else {
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const float sn = p.sign * s[n];
                    const float u = x[n] * c[n] - y[n] * sn;
                    y[n] = y[n] * c[n] + x[n] * sn;
                    x[n] = u;
                }
            }
            xv = pack8(x);
            yv = pack8(y);
        }
        dst[w0] = xv;
        dst[w1] = yv;
    }
}

}  // namespace

cudaError_t launch_rope_axes(const RopeArgs &a, cudaStream_t stream) {
    RopeOnlyParams p;
    p.q = static_cast<const uint4 *>(a.q);
    p.k = static_cast<const uint4 *>(a.k);
    p.q_out = static_cast<uint4 *>(a.q_out);
    p.k_out = static_cast<uint4 *>(a.k_out);
    for (int i = 0; i < 3; ++i) {
        p.qs[i] = a.q_strides[i] / 8;
        p.ks[i] = a.k_strides[i] / 8;
        p.qo[i] = a.q_out_strides[i] / 8;
        p.ko[i] = a.k_out_strides[i] / 8;
    }
    p.cos_sin = a.cos_sin;
    p.rope = a.rope_dim;
    p.max_pos = a.max_pos;
    p.H = a.H;
    p.Hkv = a.k ? a.Hkv : 0;
    p.N = a.N;
    p.d = a.d;
    p.blocks = (a.N + kTokens - 1) / kTokens;
    p.sign = a.back ? -1.f : 1.f;
    p.axes = a.axes;
    const unsigned grid = (unsigned)((long long)a.B * p.blocks);
    if (a.interleaved) rope_axes_kernel<true><<<grid, kThreads, 0, stream>>>(p);
    else rope_axes_kernel<false><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace attn
