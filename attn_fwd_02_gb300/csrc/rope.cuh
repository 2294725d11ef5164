// rope.cuh -- what the kernels that rotate share: vectors of 8 bf16, and positions with several axes.
//
// With several axes (time, height, width) pair i of a token turns by the angle of column i in row positions[axis(i)][token]
// of the table of cosines and sines.  A token's pairs may thus read any of its axes' rows; a block gathers them into
// shared memory once per token, whatever the pattern of the axes, and the rows of all heads read them from there.
#pragma once

#include "launch.h"
#include "sm103_ptx.cuh"

namespace attn {

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

// A token's rows of the table, one per axis; ok: all of them lie in it.
struct AxisRows {
    int row[kMaxAxes];
    bool ok;
};
__device__ __forceinline__ AxisRows axis_rows(const RopeAxes &x, int b, int t, int max_pos) {
    AxisRows r;
    r.ok = true;
    const int32_t *p = x.positions + b * x.batch_stride + t;
#pragma unroll
    for (int a = 0; a < kMaxAxes; ++a) {
        r.row[a] = a < x.axes ? p[a * x.axis_stride] : 0;
        r.ok = r.ok && (unsigned)r.row[a] < (unsigned)max_pos;
    }
    return r;
}
__device__ __forceinline__ int axis_row(const RopeAxes &x, const AxisRows &r, int pair) {
    const int a = (int)(x.pair_axis[pair >> 5] >> (2 * (pair & 31))) & 3;
    return a < 2 ? (a == 0 ? r.row[0] : r.row[1]) : (a == 2 ? r.row[2] : r.row[3]);
}
// Pair `i` of a token (past the last one: none): its cosine and, times `sign`, its sine, to where the cosines of all pairs and
// then their sines stand.
__device__ __forceinline__ void gather_pair(float *to, const float *cos_sin, const RopeAxes &x, const AxisRows &r, int rope, int i,
                                            float sign = 1.f) {
    if (i >= rope / 2) return;
    const float *row = cos_sin + (size_t)axis_row(x, r, i) * rope + i;
    to[i] = row[0];
    to[rope / 2 + i] = row[rope / 2] * sign;
}

}  // namespace attn
