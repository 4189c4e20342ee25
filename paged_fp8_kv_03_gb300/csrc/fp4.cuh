// Device code of the 4-bit cache: E2M1 codes, E4M3 block scales and the
// addresses of their tiles.
#pragma once

#include <cuda_fp4.h>

#include "fp4.h"

namespace pkv {

// Waits until the kernels ahead in the stream have ended and their writes are
// seen; lets the next kernel be brought onto the GPU (it waits in turn).
__device__ __forceinline__ void grid_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void launch_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Byte offset in a pool of the tile holding row `row` of pool page `page`.
__device__ __forceinline__ int64_t fp4_tile_offset(int64_t page, int h, int row, int hkv, int page_size)
{
    return ((page * hkv + h) * (page_size >> 4) + (row >> 4)) * kFp4Tile;
}

// Bulk copy of contiguous bytes (a multiple of 16, both ends 16-byte aligned)
// into shared memory, completing on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar,
                                          uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

// a + b rounded, and exactly what that loses (Knuth's two-sum).  Long sums of like
// terms keep it: rounded the same way every time, they drift by up to 2^-24 a term.
__device__ __forceinline__ float two_sum(float a, float b, float &rest)
{
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    rest = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
    return s;
}

__device__ __forceinline__ float e4m3_value(uint8_t c)
{
    const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half *>(&h));
}

// The four bytes of a word (8 codes) as four f16 pairs, exact: byte i gives
// (low nibble, high nibble).
__device__ __forceinline__ void e2m1x8_to_f16x8(uint32_t w, uint32_t (&p)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
        : "r"(w));
}

// Eight fp32 values -> eight E2M1 codes (round to nearest even, saturating to
// +-6), first value in the lowest nibble.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float (&x)[8])
{
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return w;
}

}  // namespace pkv
