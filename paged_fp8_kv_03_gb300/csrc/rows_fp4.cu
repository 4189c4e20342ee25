// kv_append_fp4 and kv_read_fp4: rows of K and V into the 4-bit cache and
// back.
//
// A row of 128 values is 8 blocks of 16.  A block holds E2M1 codes e and one
// E4M3 scale s; with the kv head's scale k a value is e s k.  Written:
//   s = E4M3(amax / (6 k))   so that the block's largest value lands on 6 or
//                            within 1/16 of it (it saturates there),
//   code = E2M1(x / (s k)),
// the products 6 k and s k and both quotients rounded to fp32 (IEEE), both
// conversions to nearest, ties to even.  e s has 6 significant bits, so f16,
// bf16 and fp32 all hold it exactly.
//
// One thread owns one block of one (token, kv head) row, of K and of V.
#include "fp4.cuh"

namespace pkv {

namespace {

constexpr int kBlocks = kHeadDim / 16;

template <bool kBf16>
__device__ __forceinline__ void load_block(const void *base, int64_t elem, float (&x)[16])
{
    if (kBf16) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(base) + elem);
        const uint4 u[2] = {__ldg(p), __ldg(p + 1)};
        const uint32_t *w = reinterpret_cast<const uint32_t *>(u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + elem);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = __ldg(p + i);
            x[4 * i] = v.x;
            x[4 * i + 1] = v.y;
            x[4 * i + 2] = v.z;
            x[4 * i + 3] = v.w;
        }
    }
}

// 16 values -> 8 bytes of codes and the scale byte.
__device__ __forceinline__ uint2 quantise_block(const float (&x)[16], float k, uint8_t &scale)
{
    float amax = 0.f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        amax = fmaxf(amax, fabsf(x[i]));
        nan |= x[i] != x[i];
    }
    scale = static_cast<uint8_t>(
        nan ? 0x7F : __nv_cvt_float_to_fp8(__fdiv_rn(amax, 6.f * k), __NV_SATFINITE, __NV_E4M3));
    if ((scale & 0x7F) == 0 || nan)
        return make_uint2(0u, 0u);
    const float step = __fmul_rn(e4m3_value(scale), k);
    float q[2][8];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        q[i >> 3][i & 7] = __fdiv_rn(x[i], step);
    return make_uint2(f32x8_to_e2m1x8(q[0]), f32x8_to_e2m1x8(q[1]));
}

template <bool kBf16>
__global__ void __launch_bounds__(256) kv_append_fp4_kernel(const Fp4RowArgs a)
{
    const int64_t total = a.num_tokens * a.hkv * kBlocks;
    for (int64_t c = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; c < total;
         c += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int part = static_cast<int>(c % kBlocks);
        const int64_t row = c / kBlocks;
        const int h = static_cast<int>(row % a.hkv);
        const int64_t slot = __ldg(a.slots + row / a.hkv);
        if (slot < 0)
            continue;
        if (slot >= a.num_slots) {
            if (a.err && part == 0)
                atomicOr(a.err, PKV_DEVERR_SLOT);
            continue;
        }
        const int64_t page = slot / a.page_size;
        const int r = static_cast<int>(slot - page * a.page_size);
        const int64_t tile = fp4_tile_offset(page, h, r, a.hkv, a.page_size);
        const int64_t codes = tile + (r & 15) * 64 + part * 8, scales = tile + kFp4Codes + (r & 15) * 8 + part;
        float x[16];
        load_block<kBf16>(a.k_in, row * kHeadDim + part * 16, x);
        *reinterpret_cast<uint2 *>(a.k_cache + codes) = quantise_block(x, __ldg(a.k_scale + h), a.k_cache[scales]);
        load_block<kBf16>(a.v_in, row * kHeadDim + part * 16, x);
        *reinterpret_cast<uint2 *>(a.v_cache + codes) = quantise_block(x, __ldg(a.v_scale + h), a.v_cache[scales]);
    }
}

// One block of a row: its 16 values times k to the output.
template <bool kBf16>
__device__ __forceinline__ void store_block(void *out, int64_t elem, uint2 codes, uint8_t scale, float k)
{
    const float s = e4m3_value(scale);
    float v[16];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t p[4];
        e2m1x8_to_f16x8(i ? codes.y : codes.x, p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = f16x2_to_f32x2(p[j]);
            v[8 * i + 2 * j] = f.x * s * k;                 // e s is exact: one rounding
            v[8 * i + 2 * j + 1] = f.y * s * k;
        }
    }
    if (kBf16) {
        uint4 *p = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + elem);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t *>(&b);
            }
            p[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(out) + elem);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
}

template <bool kBf16>
__global__ void __launch_bounds__(256) kv_read_fp4_kernel(const Fp4RowArgs a)
{
    const int64_t total = a.num_tokens * a.hkv * kBlocks;
    for (int64_t c = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; c < total;
         c += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int part = static_cast<int>(c % kBlocks);
        const int64_t row = c / kBlocks;
        const int h = static_cast<int>(row % a.hkv);
        const int64_t slot = __ldg(a.slots + row / a.hkv);
        if (slot < 0)
            continue;
        const bool in = slot < a.num_slots;
        if (!in && a.err && part == 0)
            atomicOr(a.err, PKV_DEVERR_SLOT);
        uint2 kc = make_uint2(0u, 0u), vc = make_uint2(0u, 0u);
        uint8_t ks = 0, vs = 0;
        if (in) {
            const int64_t page = slot / a.page_size;
            const int r = static_cast<int>(slot - page * a.page_size);
            const int64_t tile = fp4_tile_offset(page, h, r, a.hkv, a.page_size);
            const int64_t codes = tile + (r & 15) * 64 + part * 8, scales = tile + kFp4Codes + (r & 15) * 8 + part;
            kc = *reinterpret_cast<const uint2 *>(a.k_cache + codes);
            vc = *reinterpret_cast<const uint2 *>(a.v_cache + codes);
            ks = a.k_cache[scales];
            vs = a.v_cache[scales];
        }
        store_block<kBf16>(a.k_out, row * kHeadDim + part * 16, kc, ks, __ldg(a.k_scale + h));
        store_block<kBf16>(a.v_out, row * kHeadDim + part * 16, vc, vs, __ldg(a.v_scale + h));
    }
}

unsigned row_blocks(const Fp4RowArgs &a)
{
    const int64_t total = a.num_tokens * a.hkv * kBlocks;
    int64_t blocks = (total + 255) / 256;
    const int64_t cap = static_cast<int64_t>(device_sm_count()) * 16;
    return static_cast<unsigned>(blocks > cap ? cap : blocks);
}

}  // namespace

cudaError_t launch_kv_append_fp4(const Fp4RowArgs &a, cudaStream_t stream)
{
    if (a.num_tokens == 0)
        return cudaSuccess;
    if (a.bf16)
        kv_append_fp4_kernel<true><<<row_blocks(a), 256, 0, stream>>>(a);
    else
        kv_append_fp4_kernel<false><<<row_blocks(a), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv_read_fp4(const Fp4RowArgs &a, cudaStream_t stream)
{
    if (a.num_tokens == 0)
        return cudaSuccess;
    if (a.bf16)
        kv_read_fp4_kernel<true><<<row_blocks(a), 256, 0, stream>>>(a);
    else
        kv_read_fp4_kernel<false><<<row_blocks(a), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace pkv
