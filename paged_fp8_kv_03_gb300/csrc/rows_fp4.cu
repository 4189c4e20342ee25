// kv_append_fp4 and kv_read_fp4: rows of K and V into the 4-bit cache and
// back.
//
// A row of 128 values is 8 blocks of 16.  A block holds E2M1 codes e and one
// E4M3 scale s; with the kv head's scale k a value is e s k.  Written:
//   s = E4M3(amax / (6 k))   so that the block's largest value lands on 6 or
//                            within 1/16 of it (it saturates there),
//   code = E2M1(x / (s k)),
// the products 6 k and s k and both quotients rounded to fp32 (IEEE), both
// conversions to nearest, ties to even (a bound on either side of x / (s k)
// mostly settles the code without the division).  e s has 6 significant bits, so f16,
// bf16 and fp32 all hold it exactly.
//
// What bounds them: the bytes, 256 or 512 of the row and 72 of the cache each
// way.  Reading back, a thread owns 16 bytes of a row (8 bf16 or 4 fp32
// values), of K and of V, so a warp writes 512 contiguous bytes an instruction
// (with 32 a thread, half of every sector waits for a second instruction: 5.0
// instead of 6.2 TB/s).  Appending, it owns 32 bytes (16 or 8 values; a block is
// one or two lanes), because what a block's scale costs is paid once a thread
// and instructions are as much of a limit as bytes (128K bf16 tokens of 8 heads:
// 114 us, 6.0 TB/s; fp32: 186 us, 6.6 TB/s).  In calls large enough a thread
// takes the same place in several consecutive tokens: reading back, their loads are
// in flight together; appending, the next one's while one is quantised.
#include "fp4.cuh"

namespace pkv {

namespace {

constexpr int kRowThreads = 256;

// The bytes of a row that a thread owns.
template <bool kBf16, int kBytes>
struct Part {
    static constexpr int kVals = kBytes / (kBf16 ? 2 : 4);
    static constexpr int kPerRow = kHeadDim / kVals;       // threads a row
    static constexpr int kLanes = 16 / kVals;              // lanes a block
};

// Where a thread works: its token group (kTokens tokens), kv head and part.
struct RowPlace {
    int64_t token;
    int h, part;
    bool in;
};

template <typename P>
__device__ __forceinline__ RowPlace row_place(const Fp4RowArgs &a, int tokens)
{
    RowPlace p;
    const uint32_t i = blockIdx.x * kRowThreads + threadIdx.x;     // (a slab of tokens keeps it within 32 bits)
    p.part = i % P::kPerRow;
    const uint32_t row = i / P::kPerRow, g = row / static_cast<uint32_t>(a.hkv);
    p.h = static_cast<int>(row - g * a.hkv);
    p.token = static_cast<int64_t>(blockIdx.y) * a.slab + static_cast<int64_t>(g) * tokens;
    p.in = static_cast<int64_t>(g) * tokens < a.slab && p.token < a.num_tokens;
    return p;
}

// Byte offset of the row at `slot` in a pool: its tile, and its row in it.
__device__ __forceinline__ int64_t slot_tile(const Fp4RowArgs &a, int64_t slot, int h, int &r)
{
    const int64_t page = slot >> a.page_log2;
    r = static_cast<int>(slot & (a.page_size - 1));
    const int64_t tile = fp4_tile_offset(page, h, r, a.hkv, a.page_size);
    r &= 15;
    return tile;
}

// x / d correctly rounded, from y = RN(1 / d): one Newton step on x y gives a
// faithful quotient, and a second one then the correctly rounded one
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000",
// 1990), as long as nothing under- or overflows.  (Remainders with the sign
// turned: that way -0 stays -0.)
__device__ __forceinline__ float divide(float x, float d, float y)
{
    const float q0 = __fmul_rn(x, y);
    const float q1 = __fmaf_rn(-__fmaf_rn(q0, d, -x), y, q0);
    return __fmaf_rn(-__fmaf_rn(q1, d, -x), y, q1);
}

// A kv head's scale k and what quantising divides by: 6 k.
struct HeadScale {
    float k, k6, inv_k6;
    bool plain;                                            // out of the range in which divide() is safe
    bool few_bits;                                         // k is a bf16 value
};

__device__ __forceinline__ HeadScale head_scale(float k)
{
    HeadScale h;
    h.k = k;
    h.k6 = __fmul_rn(6.f, k);
    h.inv_k6 = __frcp_rn(h.k6);
    h.few_bits = (__float_as_uint(k) & 0xFFFFu) == 0;
    h.plain = !(k >= 0x1p-60f && k <= 0x1p60f);
    return h;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The larger magnitude (with some sign) of each pair; a NaN wins.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Quantises a thread's part of a row (32 bytes; fp32: with the neighbouring
// lane that has the block's other half) and stores codes and scale.
template <bool kBf16>
__device__ __forceinline__ void quantise_part(const uint4 (&u)[2], const HeadScale &hs, uint8_t *tile, int r, int part,
                                              bool store)
{
    using P = Part<kBf16, 32>;
    const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
    uint32_t m[8], top;                                    // largest |x| as its bits; a NaN's exceed all others'
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m[i] = kBf16 ? w[i] : w[i] & 0x7FFFFFFFu;
#pragma unroll
    for (int n = 4; n > 0; n >>= 1)
#pragma unroll
        for (int i = 0; i < n; ++i)
            m[i] = kBf16 ? max_abs_bf16x2(m[i], m[i + n]) : max(m[i], m[i + n]);
    if (kBf16)
        top = max_u16x2(m[0] & 0x7FFF7FFFu, (m[0] << 16) & 0x7FFF0000u) & 0xFFFF0000u;
    else
        top = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
    const float amax = __uint_as_float(top);
    uint8_t scale = 0x7F;
    uint32_t c[2] = {0u, 0u};
    if (top <= 0x7F800000u) {
        // (amax = Inf, or a quotient past the largest fp32, is beyond divide(); a
        // subnormal amax gives scale 0 either way)
        const bool huge = hs.plain || !(amax < 0x1p60f);
        float ratio;
        if (huge)
            ratio = __fdiv_rn(amax, hs.k6);
        else
            ratio = divide(amax, hs.k6, hs.inv_k6);
        scale = static_cast<uint8_t>(__nv_cvt_float_to_fp8(ratio, __NV_SATFINITE, __NV_E4M3));
        const float step = __fmul_rn(e4m3_value(scale), hs.k);
        float q[8];
        auto value = [&](int i) {
            return __uint_as_float(kBf16 ? ((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16) : w[i & 7]);
        };
        if (scale == 0) {
            // nothing of the block is left: its codes stay 0
        } else if (huge || scale == 0x7E) {                // a saturated scale: x / step may be anything
#pragma unroll 1
            for (int i = 0; i < P::kVals; i += 8) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    q[j] = __fdiv_rn(i ? value(j + P::kVals - 8) : value(j), step);
                c[i >> 3] = f32x8_to_e2m1x8(q);
            }
        } else {
            // The quotient lies between x y (1 - 2^-20) and x y (1 + 2^-20) (their
            // roundings and the quotient's are off by less than 2^-22), so where both
            // have the same code, it has that too.  Where they differ, in one warp of 700,
            // it is divided; and always where k has so few bits that a bf16 x is often
            // exactly halfway between two codes (16K bf16 tokens of 8 heads: 18 us,
            // dividing always 20; after most comparisons 5 us more).
            const float y = __frcp_rn(step);
            uint32_t differ = hs.few_bits;
            if (differ == 0) {
                const float less = __fmul_rn(y, 1.f - 0x1p-20f), more = __fmul_rn(y, 1.f + 0x1p-20f);
#pragma unroll
                for (int i = 0; i < P::kVals / 8; ++i) {
                    float lo[8], hi[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        lo[j] = __fmul_rn(value(8 * i + j), less);
                        hi[j] = __fmul_rn(value(8 * i + j), more);
                    }
                    c[i] = f32x8_to_e2m1x8(hi);
                    differ |= c[i] ^ f32x8_to_e2m1x8(lo);
                }
            }
            if (differ != 0) {
#pragma unroll
                for (int i = 0; i < P::kVals / 8; ++i) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        q[j] = divide(value(8 * i + j), step, y);
                    c[i] = f32x8_to_e2m1x8(q);
                }
            }
        }
    }
    if (store) {
        if (kBf16)
            *reinterpret_cast<uint2 *>(tile + r * 64 + part * 8) = make_uint2(c[0], c[1]);
        else
            *reinterpret_cast<uint32_t *>(tile + r * 64 + part * 4) = c[0];
        if (part % P::kLanes == 0)
            tile[kFp4Codes + r * 8 + part / P::kLanes] = scale;
    }
}

template <bool kBf16, bool kMany>
__global__ void __launch_bounds__(kRowThreads, kBf16 ? 3 : 4) kv_append_fp4_kernel(const Fp4RowArgs a)
{
    using P = Part<kBf16, 32>;
    const int tokens = kMany ? a.tokens : 1;
    const RowPlace p = row_place<P>(a, tokens);
    const HeadScale ks = head_scale(__ldg(a.k_scale + p.h)), vs = head_scale(__ldg(a.v_scale + p.h));
    // the next token's loads are on their way while one is quantised
    struct Token {
        int64_t slot;
        uint4 k[2], v[2];
    };
    auto load = [&](int i) {
        Token x;
        const int64_t t = p.token + i;
        const bool in = p.in && t < a.num_tokens;
        x.slot = in ? __ldg(a.slots + t) : -1;
        const int64_t at = ((t * a.hkv + p.h) * P::kPerRow + p.part) * 2;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x.k[j] = in ? __ldg(static_cast<const uint4 *>(a.k_in) + at + j) : make_uint4(0, 0, 0, 0);
            x.v[j] = in ? __ldg(static_cast<const uint4 *>(a.v_in) + at + j) : make_uint4(0, 0, 0, 0);
        }
        return x;
    };
    Token next = load(0);
#pragma unroll 1
    for (int i = 0; i < tokens; ++i) {                    // (lanes of a block share their token, so its slot)
        const Token x = next;
        if (i + 1 < tokens)
            next = load(i + 1);
        const bool store = x.slot >= 0 && x.slot < a.num_slots;
        if (x.slot >= a.num_slots && a.err && p.part == 0)
            atomicOr(a.err, PKV_DEVERR_SLOT);
        int r = 0;
        const int64_t tile = store ? slot_tile(a, x.slot, p.h, r) : 0;
        quantise_part<kBf16>(x.k, ks, a.k_cache + tile, r, p.part, store);
        quantise_part<kBf16>(x.v, vs, a.v_cache + tile, r, p.part, store);
    }
}

// A thread's codes (8 or 4, lowest first) and its block's scale as 16 bytes of
// a row.
template <bool kBf16>
__device__ __forceinline__ uint4 values_part(uint32_t codes, uint8_t scale, float k)
{
    using P = Part<kBf16, 16>;
    const float s = e4m3_value(scale);
    uint32_t p[4];
    e2m1x8_to_f16x8(codes, p);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < P::kVals / 2; ++j) {
        const float2 f = f16x2_to_f32x2(p[j]);
        const float lo = f.x * s * k, hi = f.y * s * k;     // e s is exact: one rounding
        if (kBf16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
            w[j] = *reinterpret_cast<const uint32_t *>(&b);
        } else {
            w[2 * (j & 1)] = __float_as_uint(lo);
            w[2 * (j & 1) + 1] = __float_as_uint(hi);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool kBf16, int kTokens>
__global__ void __launch_bounds__(kRowThreads) kv_read_fp4_kernel(const Fp4RowArgs a)
{
    using P = Part<kBf16, 16>;
    const RowPlace p = row_place<P>(a, kTokens);
    if (!p.in)
        return;
    const float ks = __ldg(a.k_scale + p.h), vs = __ldg(a.v_scale + p.h);
    int64_t slot[kTokens];
    uint32_t kc[kTokens], vc[kTokens];
    uint8_t kb[kTokens], vb[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i)
        slot[i] = p.token + i < a.num_tokens ? __ldg(a.slots + p.token + i) : -1;
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        kc[i] = vc[i] = 0;
        kb[i] = vb[i] = 0;
        if (slot[i] >= 0 && slot[i] < a.num_slots) {
            int r;
            const int64_t tile = slot_tile(a, slot[i], p.h, r);
            const int64_t at = tile + r * 64 + p.part * (P::kVals / 2), sc = tile + kFp4Codes + r * 8 + p.part / P::kLanes;
            kc[i] = kBf16 ? *reinterpret_cast<const uint32_t *>(a.k_cache + at)
                          : *reinterpret_cast<const uint16_t *>(a.k_cache + at);
            vc[i] = kBf16 ? *reinterpret_cast<const uint32_t *>(a.v_cache + at)
                          : *reinterpret_cast<const uint16_t *>(a.v_cache + at);
            kb[i] = a.k_cache[sc];
            vb[i] = a.v_cache[sc];
        }
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        if (slot[i] < 0)
            continue;
        if (slot[i] >= a.num_slots && a.err && p.part == 0)
            atomicOr(a.err, PKV_DEVERR_SLOT);
        const int64_t at = ((p.token + i) * a.hkv + p.h) * P::kPerRow + p.part;
        static_cast<uint4 *>(a.k_out)[at] = values_part<kBf16>(kc[i], kb[i], ks);
        static_cast<uint4 *>(a.v_out)[at] = values_part<kBf16>(vc[i], vb[i], vs);
    }
}

typedef void (*RowKernel)(const Fp4RowArgs);

// A thread takes `tokens` tokens in `many` where that still fills the GPU with
// threads, else one.  tokens = 0: as many as give `resident` threads an SM equal
// shares, in rounds of at most 10 (append of bf16 rows of 8 heads: 16K tokens, 9 a thread
// in one round, 18.0 us, one a thread 19.2; 128K, 9 a thread, 114 us, 72 in one round 118;
// 4K, 3 a thread 6.7 us, one 5.4).
cudaError_t launch_rows(RowKernel one, RowKernel many, int tokens, int resident, int per_row, const Fp4RowArgs &args,
                        cudaStream_t stream)
{
    if (args.num_tokens == 0)
        return cudaSuccess;
    Fp4RowArgs a = args;
    const int64_t threads = a.num_tokens * a.hkv * per_row, sms = device_sm_count();
    if (tokens == 0) {
        const int64_t share = (threads + sms * resident - 1) / (sms * resident), rounds = (share + 9) / 10;
        tokens = static_cast<int>((share + rounds - 1) / rounds);
        if (tokens < 4)
            tokens = 1;
    } else if (threads < sms * 2048 * tokens) {
        tokens = 1;
    }
    a.tokens = tokens;
    // tokens a slab: its threads count in 32 bits, and whole groups
    int64_t slab = ((int64_t(1) << 30) / (static_cast<int64_t>(a.hkv) * per_row) + tokens) / tokens * tokens;
    if (slab > a.num_tokens)
        slab = (a.num_tokens + tokens - 1) / tokens * tokens;
    const int64_t slabs = (a.num_tokens + slab - 1) / slab;
    if (slabs > 65535)
        return cudaErrorInvalidValue;
    a.slab = slab;
    const int64_t blocks = (slab / tokens * a.hkv * per_row + kRowThreads - 1) / kRowThreads;
    (tokens > 1 ? many : one)<<<dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(slabs)), kRowThreads, 0,
                                stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append_fp4(const Fp4RowArgs &a, cudaStream_t stream)
{
    return a.bf16 ? launch_rows(kv_append_fp4_kernel<true, false>, kv_append_fp4_kernel<true, true>, 0, 768,
                                Part<true, 32>::kPerRow, a, stream)
                  : launch_rows(kv_append_fp4_kernel<false, false>, kv_append_fp4_kernel<false, true>, 16, 0,
                                Part<false, 32>::kPerRow, a, stream);
}

cudaError_t launch_kv_read_fp4(const Fp4RowArgs &a, cudaStream_t stream)
{
    return a.bf16 ? launch_rows(kv_read_fp4_kernel<true, 1>, kv_read_fp4_kernel<true, 4>, 4, 0,
                                Part<true, 16>::kPerRow, a, stream)
                  : launch_rows(kv_read_fp4_kernel<false, 1>, kv_read_fp4_kernel<false, 4>, 4, 0,
                                Part<false, 16>::kPerRow, a, stream);
}

}  // namespace pkv
