// kv4_device.cuh - conversions of the 4-bit cache format (e2m1 codes, e4m3 scales) and the
// fp16 tensor-core step that reads it.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace pbsa {

// e4m3, round to nearest even, saturating at 448.
__device__ __forceinline__ uint8_t e4m3_from_float(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return (uint8_t)(r & 0xffu);
}

// Two e4m3 bytes (low byte first) as a half2: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}

__device__ __forceinline__ float e4m3_to_float(uint8_t v) {
    const uint32_t r = e4m3x2_to_half2(v);
    return __half2float(__ushort_as_half((unsigned short)(r & 0xffffu)));
}

// Two e2m1 codes, `lo` in the low nibble: round to nearest even, saturating at 6.
__device__ __forceinline__ uint32_t e2m1x2_from_float(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\t"
        "cvt.u32.u8 %0, t;\n\t}"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r;
}

// The eight codes of a word as four half2, byte by byte (low nibble in the low half): exact.
__device__ __forceinline__ void e2m1x8_to_half2x4(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t"
        "mov.b32 {t0, t1, t2, t3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, t0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, t1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, t2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, t3;\n\t}"
        : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
        : "r"(w));
}

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// d += A B: A 16 x 16 (rows x contraction), B 16 x 8, fp16 operands, fp32 sums.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit elements held two to a lane (row = lane / 4).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

}  // namespace pbsa
