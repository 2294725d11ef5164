// rope_axes.cu -- rotary position embedding of queries and keys by positions with several axes, outside the cache: a
// training step's or a vision tower's, and its gradient.
//
// Pair i of a token, (x, y), turns by the angle whose cosine c and sine s stand in column i of row
// positions[axis(i)][token]:  x' = x c - y s, y' = y c + x s.  The gradient is the transposed rotation of the gradient:
// dx = dx' c + dy' s, dy = dy' c - dx' s (right for tables with a factor on c and s too).
//
// Memory-bound: every element is read and written once.  A block takes one token, gathers its angles into shared memory, and turns
// the rows of all heads, 16 elements (8 pairs) a thread at a time, held in registers, so that a view may be turned in place.  What
// counts is how much of its life a block has loads in flight, and how little it does besides: its first rows are read before the
// angles are there, blocks are small, the head dim is a template's and a thread looks up one pair's angle.  Measured, 8 x 1024
// tokens, 16 + 16 heads of 80, forward / 2 x 16384 tokens, 32 + 8 heads of 128, gradients into strided views, us: 16.9 / 100.7
// (6.7 TB/s); with the head dim at run time and the angles one by one 18.6 / 106.4, of that four tokens and 256 threads a block
// 19.4 / 111, without the early reads 20.2 / 110, two rows in flight a thread 20.9 / 115, four 24.9 / 135.  Now 128 threads a block
// 19.4 / 109.5; registers held to 24 blocks an SM 17.3 / 99.1, to 28 20.9 / 109.
#include "rope.cuh"

namespace attn {
namespace {

constexpr int kThreads = 64;

struct RopeOnlyParams {
    const uint4 *q, *k;
    uint4 *q_out, *k_out;
    long long qs[3], ks[3], qo[3], ko[3];  // strides of batch, head and token, in vectors of 8
    const float *cos_sin;
    int rope, max_pos, H, heads, N;  // heads: of queries and keys
    float sign;                      // of the sines: -1 for the gradient
    RopeAxes axes;
};

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_axes_kernel(const RopeOnlyParams p) {
    __shared__ __align__(16) float angles[kMaxRope];
    griddep_launch_dependents();
    griddep_wait();
    const int b = (int)(blockIdx.x / (unsigned)p.N), t = (int)(blockIdx.x % (unsigned)p.N);
    // Thread = (item i of a row, first row): two vectors of 8, the two halves of 8 pairs, or neighbours where nothing turns or
    // the pairs are neighbours themselves.  Its rows are every kPass-th of the heads, each read one ahead of its use, the first
    // one before the angles.
    constexpr int kItems = D / 16, kPass = kThreads / kItems;
    const int i = threadIdx.x % kItems, half = p.rope / 2, rot = p.rope / 16;
    const bool turns = i < rot;
    const int w0 = turns && !INTER ? i : 2 * i, w1 = turns && !INTER ? i + rot : 2 * i + 1;
    int h = threadIdx.x < kPass * kItems ? threadIdx.x / kItems : p.heads;
    const uint4 *q = p.q + b * p.qs[0] + t * p.qs[2], *k = p.k + b * p.ks[0] + t * p.ks[2] - p.H * p.ks[1];  // (its heads count from H on)
    uint4 xv, yv;
    auto fetch = [&] {
        if (h >= p.heads) return;
        const uint4 *src = h >= p.H ? k + h * p.ks[1] : q + h * p.qs[1];
        xv = src[w0];
        yv = src[w1];
    };
    fetch();
    const AxisRows rows = axis_rows(p.axes, b, t, p.max_pos);
    if (rows.ok) gather_pair(angles, p.cos_sin, p.axes, rows, p.rope, threadIdx.x, p.sign);
    __syncthreads();
    uint4 *qo = p.q_out + b * p.qo[0] + t * p.qo[2], *ko = p.k_out + b * p.ko[0] + t * p.ko[2] - p.H * p.ko[1];
    const float *c = angles + 8 * i;
    const uint64_t *c2 = reinterpret_cast<const uint64_t *>(c), *s2 = reinterpret_cast<const uint64_t *>(c + half);
    while (h < p.heads) {
        uint4 *dst = h >= p.H ? ko + h * p.ko[1] : qo + h * p.qo[1];
        uint4 xn = xv, yn = yv;
        h += kPass;
        fetch();
        if (!rows.ok) {
            xn = yn = make_uint4(0u, 0u, 0u, 0u);
        } else if (turns) {
            float x[8], y[8];
            unpack8(xn, x);
            unpack8(yn, y);
#pragma unroll
            for (int m = 0; m < 4; ++m) {  // pairs 2m, 2m + 1 of the item: (a, e) of each
                float (&z)[8] = INTER && m >= 2 ? y : x;
                const int at = INTER ? 4 * (m & 1) : 2 * m;
                float &a0 = z[at], &a1 = z[INTER ? at + 2 : at + 1];
                float &e0 = INTER ? z[at + 1] : y[at], &e1 = INTER ? z[at + 3] : y[at + 1];
                const uint64_t a = f32x2_pack(a0, a1), e = f32x2_pack(e0, e1);
                const uint64_t minus = s2[m] ^ 0x8000000080000000ull;
                // (rounded as the appends round it)
                f32x2_unpack(f32x2_fma(a, c2[m], f32x2_mul(e, minus)), a0, a1);
                f32x2_unpack(f32x2_fma(e, c2[m], f32x2_mul(a, s2[m])), e0, e1);
            }
            xn = pack8(x);
            yn = pack8(y);
        }
        dst[w0] = xn;
        dst[w1] = yn;
    }
}

template <int D>
cudaError_t launch_rope_d(const RopeOnlyParams &p, dim3 grid, bool interleaved, cudaStream_t stream) {
    return interleaved ? launch_dependent(rope_axes_kernel<D, true>, grid, kThreads, 0, stream, p)
                       : launch_dependent(rope_axes_kernel<D, false>, grid, kThreads, 0, stream, p);
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
    p.heads = a.H + (a.k ? a.Hkv : 0);
    p.N = a.N;
    p.sign = a.back ? -1.f : 1.f;
    p.axes = a.axes;
    const dim3 grid((unsigned)((long long)a.B * a.N));
    const bool inter = a.interleaved != 0;
    switch (a.d) {
        case 32: return launch_rope_d<32>(p, grid, inter, stream);
        case 64: return launch_rope_d<64>(p, grid, inter, stream);
        case 80: return launch_rope_d<80>(p, grid, inter, stream);
        case 96: return launch_rope_d<96>(p, grid, inter, stream);
        case 128: return launch_rope_d<128>(p, grid, inter, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace attn
