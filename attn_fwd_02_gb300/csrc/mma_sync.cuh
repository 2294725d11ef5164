// mma_sync.cuh -- warp-level products for the decode kernels, whose few rows leave a 128-row tcgen05
// tile nearly empty: ldmatrix, mma.sync m16n8k16, and the swizzled page-block layout.
#pragma once

#include <stdint.h>
#include <string.h>

namespace attn {

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// d (+)= a b: a 16x16 bf16 (row-major fragment), b 16x8 bf16 (column-major fragment), d 16x8 fp32.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same product over f16 fragments.
__device__ __forceinline__ void mma_16816_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Byte permute: byte i of the result is byte (sel >> 4i) & 7 of {hi:lo}.
__device__ __forceinline__ uint32_t prmt(uint32_t lo, uint32_t hi, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(lo), "r"(hi), "r"(sel));
    return r;
}

// A query head is rounded to f16 after a division by 2^query_shift: of its largest magnitude amax, 2^15 or more comes down below
// 2^15, and less than 2^-7 up to [1, 2), as far as c, the factor of its products, times that power stays a normal fp32 number (past
// that every score is 0 beside 1).  So all values are exact but those under f16's range, which are off by 2^-18 of amax at most.
// From low = query_low(c), -126 or more, to 113; 0 for magnitudes in between.  (With a branch, and c's exponent taken in the kernel, the 4-bit decode of 32
// sequences of up to 8192 tokens took 38.5 us instead of 38.0; so, with low from the host, it takes no longer than without.)
__host__ __device__ inline int query_low(float c) {
    uint32_t u;
    memcpy(&u, &c, 4);
    const int low = 1 - (int)(u >> 23 & 0xffu);  // -126 less c's exponent
    return low < -126 ? -126 : (low > 0 ? 0 : low);
}
__device__ __forceinline__ int query_shift(float amax, int low) {
    const int e = (int)((__float_as_uint(amax) >> 23) & 0xffu) - 127;
    return e >= -7 ? max(min(e - 14, 113), 0) : max(e, low);
}

// Byte offset of the 16-byte chunk holding column col (a multiple of 8) of row r in a page block
// stored as 128-byte-swizzled boxes of 16 rows x 64 bf16 columns.
__device__ __forceinline__ uint32_t swz_off(int r, int col) {
    return (uint32_t)((col >> 6) * (16 * 128) + r * 128 + ((((col & 63) >> 3) ^ (r & 7)) << 4));
}

}  // namespace attn
