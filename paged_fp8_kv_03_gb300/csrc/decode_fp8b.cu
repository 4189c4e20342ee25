// paged_gqa_decode_fp8b: grouped-query decode attention over the block-scaled FP8
// cache, with an optional window and sinks.
//   s_t = sm_scale q . (code_K 2^ek)_t,  w = softmax(s),  o = sum_t w_t (code_V 2^ev)_t
//
// One CTA a (sequence, query head): its warps take the visible tokens in turns, a
// lane four dims, and join their (max, sum, accumulator) states at the end.
#include "fp8b.h"
#include "split.cuh"

namespace pkv {

namespace {

constexpr int kSimpleWarps = 8;

__device__ __forceinline__ float exp_of(const uint8_t *exps, int64_t at)
{
    const uint32_t x = __ldg(exps + at);
    return __uint_as_float(x == 0 ? 0x00400000u : x << 23);
}

__device__ __forceinline__ float4 row_values(uint32_t w, float f)
{
    uint32_t lo, hi;
    e4m3x4_to_f16x4(w, lo, hi);
    const float2 a = f16x2_to_f32x2(lo), b = f16x2_to_f32x2(hi);
    return make_float4(a.x * f, a.y * f, b.x * f, b.y * f);
}

__global__ void __launch_bounds__(32 * kSimpleWarps) paged_gqa_decode_fp8b_kernel(const Fp8bDecodeArgs da)
{
    const CacheAttnArgs &a = da.a;
    __shared__ float4 acc_s[kSimpleWarps][32];
    __shared__ float2 ml_s[kSimpleWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.x / a.hq, i = blockIdx.x % a.hq, h = i / a.group;
    const Sight sg = sight_of(a, b);
    if (i == 0 && threadIdx.x == 0)
        flag_sequence(a, b, sg);
    const int64_t row = static_cast<int64_t>(b) * a.hq + i;
    const uint2 qw = __ldg(reinterpret_cast<const uint2 *>(a.q + row * kHeadDim) + lane);
    const float q[4] = {__uint_as_float(qw.x << 16), __uint_as_float(qw.x & 0xFFFF0000u), __uint_as_float(qw.y << 16),
                        __uint_as_float(qw.y & 0xFFFF0000u)};
    float m = -INFINITY, l = 0.f;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = warp; k < 16 * sg.tiles; k += kSimpleWarps) {
        const int t = 16 * tile_at(sg, k >> 4) + (k & 15);
        if (t >= sg.len || (t < sg.from && t >= sg.sinks))
            continue;
        const int tile = tile_number(a, sg, b, h, k >> 4);
        float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
        if (tile >= 0) {
            const int64_t at = (static_cast<int64_t>(tile) * 16 + (k & 15)) * kHeadDim + 4 * lane;
            kv = row_values(__ldg(reinterpret_cast<const uint32_t *>(a.k_cache + at)), exp_of(da.k_exp, tile));
            vv = row_values(__ldg(reinterpret_cast<const uint32_t *>(a.v_cache + at)), exp_of(da.v_exp, tile));
        }
        float s = q[0] * kv.x + q[1] * kv.y + q[2] * kv.z + q[3] * kv.w;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            s += __shfl_xor_sync(kEvery, s, o);
        s *= a.sm_scale_log2;
        const float mn = fmaxf(m, s);
        const float f = m == mn ? 1.f : exp2f(m - mn), p = exp2f(s - mn);
        m = mn;
        l = l * f + p;
        A = make_float4(A.x * f + p * vv.x, A.y * f + p * vv.y, A.z * f + p * vv.z, A.w * f + p * vv.w);
    }
    acc_s[warp][lane] = A;
    if (lane == 0)
        ml_s[warp] = make_float2(m, l);
    __syncthreads();
    if (warp != 0)
        return;
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < kSimpleWarps; ++w)
        M = fmaxf(M, ml_s[w].x);
    A = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < kSimpleWarps; ++w) {
        if (ml_s[w].y == 0.f)
            continue;
        const float f = exp2f(ml_s[w].x - M);
        const float4 v = acc_s[w][lane];
        L += f * ml_s[w].y;
        A = make_float4(A.x + f * v.x, A.y + f * v.y, A.z + f * v.z, A.w + f * v.w);
    }
    const float inv = sg.len == 0 ? 0.f : 1.f / L;
    store4(a, row, 4 * lane, make_float4(A.x * inv, A.y * inv, A.z * inv, A.w * inv));
}

}  // namespace

cudaError_t launch_paged_decode_fp8b(const Fp8bDecodeArgs &da, cudaStream_t stream)
{
    paged_gqa_decode_fp8b_kernel<<<static_cast<unsigned>(da.a.batch * da.a.hq), 32 * kSimpleWarps, 0, stream>>>(da);
    return cudaGetLastError();
}

}  // namespace pkv
