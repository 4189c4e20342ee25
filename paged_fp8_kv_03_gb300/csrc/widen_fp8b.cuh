// The block-scaled FP8 cache's rows as 16-bit ones: for the copies of its prefill, and for
// the attention that takes them from the cache itself.
#pragma once

#include "fp8b.h"
#include "prefill.cuh"

namespace pkv {

__device__ __forceinline__ float scale_of(uint32_t x)    // 2^(x - 127)
{
    return __uint_as_float(x == 0 ? 0x00400000u : x << 23);
}

// What V's codes of a block with byte x are multiplied by, in units of 2^(ref - 127).
__device__ __forceinline__ float scale_of_v(uint32_t x, int ref)
{
    return __int_as_float(max(static_cast<int>(x) - ref + 127, 1) << 23);
}

// Eight codes of K as bf16 (exact: 4 significant bits).
__device__ __forceinline__ uint4 widen_k(uint2 c, float scale)
{
    uint32_t k[4];
    e4m3x4_to_f16x4(c.x, k[0], k[1]);
    e4m3x4_to_f16x4(c.y, k[2], k[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = f16x2_to_f32x2(k[e]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * scale, f.y * scale);
        k[e] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(k[0], k[1], k[2], k[3]);
}

// Eight codes of V as f16; NaNs become zeros, and a bit each of `nans`.
__device__ __forceinline__ uint4 widen_v(uint2 c, float scale, uint32_t &nans)
{
    const uint32_t n0 = __vcmpeq4(c.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu), n1 = __vcmpeq4(c.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    nans = 0;
    if ((n0 | n1) != 0) {
        c.x &= ~n0;
        c.y &= ~n1;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            nans |= ((n0 >> (8 * e)) & 1u) << e | ((n1 >> (8 * e)) & 1u) << (4 + e);
    }
    uint32_t v[4];
    e4m3x4_to_f16x4(c.x, v[0], v[1]);
    e4m3x4_to_f16x4(c.y, v[2], v[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = f16x2_to_f32x2(v[e]);
        v[e] = f32x2_to_f16x2(f.x * scale, f.y * scale);
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// True where one of 16 codes is a NaN.
__device__ __forceinline__ bool any_nan(const uint4 &c)
{
    auto carry = [](uint32_t x) { return (x & 0x7F7F7F7Fu) + 0x01010101u; };
    return ((carry(c.x) | carry(c.y) | carry(c.z) | carry(c.w)) & 0x80808080u) != 0;
}

// Two codes (bytes 2 i and 2 i + 1 of x) as bf16 in units of 2^-120: exponent and mantissa
// where bf16 has them, the smallest codes as its subnormal numbers.
template <int i>
__device__ __forceinline__ uint32_t bf16_bits(uint32_t x)
{
    const uint32_t w = __byte_perm(x, 0u, i ? 0x3424 : 0x1404);
    return (w & 0x80008000u) | ((w >> 4) & 0x07F007F0u);
}

// 16 codes as 16-bit values, whatever their scale; V: and NaNs' bits.
struct EightPairs {
    uint32_t v[8], nans;
};

template <bool kV>
__device__ __forceinline__ EightPairs widen_rare(uint4 c, float scale)
{
    uint32_t n0 = 0, n1 = 0;
    const uint4 lo = kV ? widen_v(make_uint2(c.x, c.y), scale, n0) : widen_k(make_uint2(c.x, c.y), scale);
    const uint4 hi = kV ? widen_v(make_uint2(c.z, c.w), scale, n1) : widen_k(make_uint2(c.z, c.w), scale);
    return EightPairs{{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}, n0 | n1 << 8};
}

// Where a block of 16 tokens lies: row y of page and kv head z, or z < 0 where no query of the
// chunk sees one of them.
struct BlockPlace {
    int z, y;
};

__device__ __forceinline__ BlockPlace block_place(const PrefillArgs &a, const KeyTiles &seen, int b, int h, int lp, int L, int t)
{
    BlockPlace p = {-1, 0};
    if (t >= L || (t >= seen.sinks && t + kBlock <= seen.from))
        return p;
    int pg, row;
    if (!seq_token_page(a, b, lp, t, pg, row)) {
        if (a.err)
            atomicOr(a.err, PKV_DEVERR_PAGE);
        return p;
    }
    p.z = pg * a.hkv + h;
    p.y = row;
    return p;
}

// What a lane has of a warp's quarter of a key tile (32 tokens, two blocks), of K or of V: 16
// dims, 16 part .., of rows 4 j + sub.  Their codes lie in the tile's second half, 128-byte
// swizzled; blocks of which no query sees a token (exponent < 0) do not, and rows that none sees are zeros.
struct QuarterTile {
    uint4 codes[8];
};

__device__ __forceinline__ void take_quarter(const KeyTiles &seen, const uint8_t *tile, const volatile int *exps, int key0, int L,
                                             int w, int lane, QuarterTile &q)
{
    const int sub = lane >> 3, part = lane & 7;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int row = 32 * w + 4 * j + sub, t = key0 + row;
        q.codes[j] = make_uint4(0u, 0u, 0u, 0u);
        if (exps[2 * w + (j >> 2)] >= 0 && t < L && (t < seen.sinks || t >= seen.from))
            q.codes[j] = *reinterpret_cast<const uint4 *>(tile + 16384 + row * 128 + ((part ^ (row & 7)) << 4));
    }
}

// Stores the quarter as 16-bit rows into the tile as TMA would have left it: two halves of 64
// dims, rows of 128 bytes, 128-byte swizzle.  Lanes of the second half write their two
// pieces in the other order, so that eight lanes' pieces have banks of their own.  V: records
// NaNs, and says if there is one.
//
// The conversions are few warps' alone, so their instructions count: two codes of V are a
// conversion to f16 and a product (the scale is an f16 down to 2^-24), two of K moves of their
// bits and a product (up to a scale of 2^7).  Other scales, and NaNs, go the copies' way.  A
// loop of two rows: unrolled over eight, its code and the softmax's do not fit the instruction
// cache, and warps wait for instructions most of the time (4.6 us a key tile instead of 3.1).
template <bool kV>
__device__ __forceinline__ bool store_quarter(const PrefillArgs &a, QuarterTile &q, const volatile int *exps, uint8_t *tile,
                                              int64_t copy_row, int w, int v_ref, int lane)
{
    const int sub = lane >> 3, part = lane & 7, half = part >> 2;
    uint32_t marks[4] = {0u, 0u, 0u, 0u};                // V: NaNs of rows 2 i and 2 i + 1, 16 bits each
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {                        // two rows
        const int x = max(exps[2 * w + (i >> 1)], 0), d = kV ? x - v_ref : x - 127;
        // 2^d as f16 (subnormal numbers below 2^-14), 2^(120 + d) as bf16; twice
        uint32_t two = kV ? (d >= -14 ? static_cast<uint32_t>(d + 15) << 10 : 1u << max(d + 24, 0))
                          : static_cast<uint32_t>(min(d + 247, 254)) << 7;
        two |= two << 16;
        const bool fast = kV ? d >= -24 : d <= 7;
        uint8_t *to = tile + half * 16384 + (32 * w + 8 * i + sub) * 128;
        const int chunk = 2 * (part & 3) + half;         // its first piece: even or odd
        uint32_t mark = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint4 c = q.codes[j];
            EightPairs y;
            if (__builtin_expect(fast && !any_nan(c), 1)) {
                if (kV) {
                    e4m3x4_to_f16x4(c.x, y.v[0], y.v[1]);
                    e4m3x4_to_f16x4(c.y, y.v[2], y.v[3]);
                    e4m3x4_to_f16x4(c.z, y.v[4], y.v[5]);
                    e4m3x4_to_f16x4(c.w, y.v[6], y.v[7]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const __half2 p =
                            __hmul2(*reinterpret_cast<const __half2 *>(&y.v[e]), *reinterpret_cast<const __half2 *>(&two));
                        y.v[e] = *reinterpret_cast<const uint32_t *>(&p);
                    }
                } else {
                    const uint32_t code[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        y.v[e] = e & 1 ? bf16_bits<1>(code[e >> 1]) : bf16_bits<0>(code[e >> 1]);
                        const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&y.v[e]),
                                                         *reinterpret_cast<const __nv_bfloat162 *>(&two));
                        y.v[e] = *reinterpret_cast<const uint32_t *>(&p);
                    }
                }
            } else {
                y = kV ? widen_rare<true>(c, scale_of_v(x, v_ref)) : widen_rare<false>(c, scale_of(x));
                mark |= y.nans << (16 * j);
            }
            // (rows 8 i + 4 j + sub)
            const uint4 lo = make_uint4(y.v[0], y.v[1], y.v[2], y.v[3]), hi = make_uint4(y.v[4], y.v[5], y.v[6], y.v[7]);
            const int swizzled = (chunk ^ (4 * j + sub)) << 4;
            *reinterpret_cast<uint4 *>(to + 512 * j + swizzled) = half ? hi : lo;
            *reinterpret_cast<uint4 *>(to + 512 * j + (swizzled ^ 16)) = half ? lo : hi;
        }
#pragma unroll
        for (int j = 0; j < 6; ++j)
            q.codes[j] = q.codes[j + 2];
        if (kV) {
            marks[0] = marks[1];
            marks[1] = marks[2];
            marks[2] = marks[3];
            marks[3] = mark;
        }
    }
    bool some = false;
    if (kV) {
        some = __any_sync(kAll, (marks[0] | marks[1] | marks[2] | marks[3]) != 0);
        if (some)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                reinterpret_cast<uint16_t *>(nan_value_rows(a) + (copy_row + 32 * w + 4 * j + sub) * 16)[part] =
                    static_cast<uint16_t>(marks[j >> 1] >> (16 * (j & 1)));
    }
    return some;
}

}  // namespace pkv
