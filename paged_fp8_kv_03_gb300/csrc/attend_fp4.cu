// Attention over the 4-bit cache, for decode (one query a sequence) and for
// chunked prefill (a chunk of queries a sequence):
//   s_t = sm_scale k_scale q . (e s)_t,  w = softmax(s),  o = v_scale sum_t w_t (e s)_t
// over the tokens t that the query's position p, its window and the sinks
// leave visible.
//
// One CTA per (query row, kv head); its warps take the visible tokens in
// turns, a lane holds 4 dims, and the warps' (max, sum, accumulator) states
// are joined in shared memory.
#include "fp4.cuh"

namespace pkv {

namespace {

constexpr int kAttWarps = 8;

__device__ __forceinline__ float4 row_values(const uint8_t *tile, int r, int lane)
{
    const uint32_t c = *reinterpret_cast<const uint16_t *>(tile + r * 64 + lane * 2);
    uint32_t p[4];
    e2m1x8_to_f16x8(c, p);
    const float s = e4m3_value(tile[kFp4Codes + r * 8 + (lane >> 2)]);
    const float2 a = f16x2_to_f32x2(p[0]), b = f16x2_to_f32x2(p[1]);
    return make_float4(a.x * s, a.y * s, b.x * s, b.y * s);
}

__global__ void __launch_bounds__(32 * kAttWarps) attend_fp4_kernel(const Fp4AttnArgs a)
{
    __shared__ float red[kAttWarps][PKV_MAX_GROUP][kHeadDim];
    __shared__ float red_m[kAttWarps][PKV_MAX_GROUP], red_l[kAttWarps][PKV_MAX_GROUP];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x % a.hkv;
    const int row = blockIdx.x / a.hkv;
    int b = row, L = __ldg(a.seq_lens + (a.cu_q ? 0 : row)), p;
    const bool first = threadIdx.x == 0 && h == 0;
    int lp;
    if (a.cu_q == nullptr) {
        lp = seq_page_log2(a, b);
        const long long cap = lp < 0 ? 0 : min(static_cast<long long>(a.max_pages) << lp, static_cast<long long>(a.max_len));
        const int Lc = L < 0 ? 0 : (L > cap ? static_cast<int>(cap) : L);
        if (first && a.err && (lp < 0 || Lc != L))
            atomicOr(a.err, lp < 0 ? PKV_DEVERR_PAGESIZE : PKV_DEVERR_SEQLEN);
        L = Lc;
        p = L - 1;
    } else {
        for (b = 0; b < a.batch && !(row >= __ldg(a.cu_q + b) && row < __ldg(a.cu_q + b + 1)); ++b) {
        }
        if (b == a.batch)
            return;
        const int q0 = __ldg(a.cu_q + b), n = __ldg(a.cu_q + b + 1) - q0;
        L = __ldg(a.seq_lens + b);
        lp = seq_page_log2(a, b);
        if (q0 < 0 || q0 + n > a.total_q || n > a.max_q_len || L < n || L > a.max_len || lp < 0 ||
            static_cast<long long>(L) > (static_cast<long long>(a.max_pages) << lp)) {
            if (first && a.err)
                atomicOr(a.err, lp < 0 ? PKV_DEVERR_PAGESIZE : PKV_DEVERR_SEQLEN);
            return;
        }
        p = L - n + row - q0;
    }
    const int from = a.win.window == 0 ? 0 : max(0, p - a.win.window + 1);
    const int sinks = min(a.win.sinks, from);
    const int count = p + 1 - from + sinks;
    float4 q[PKV_MAX_GROUP], acc[PKV_MAX_GROUP];
    float m[PKV_MAX_GROUP], l[PKV_MAX_GROUP];
#pragma unroll
    for (int g = 0; g < PKV_MAX_GROUP; ++g) {
        q[g] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (g < a.group) {
            const uint2 u = *reinterpret_cast<const uint2 *>(
                a.q + (static_cast<int64_t>(row) * a.hq + h * a.group + g) * kHeadDim + 4 * lane);
            q[g] = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                               __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
        }
        acc[g] = make_float4(0.f, 0.f, 0.f, 0.f);
        m[g] = -INFINITY;
        l[g] = 0.f;
    }
    const float scale = __ldg(a.k_scale + h) * a.sm_scale_log2;
    for (int i = warp; i < count; i += kAttWarps) {
        const int t = i < sinks ? i : i - sinks + from;
        int phys, r;
        float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
        if (seq_token_page(a, b, lp, t, phys, r)) {
            const int64_t tile = fp4_tile_offset(phys, h, r, a.hkv, a.page_size);
            k = row_values(a.k_cache + tile, r & 15, lane);
            v = row_values(a.v_cache + tile, r & 15, lane);
        } else if (lane == 0 && a.err) {
            atomicOr(a.err, PKV_DEVERR_PAGE);
        }
#pragma unroll
        for (int g = 0; g < PKV_MAX_GROUP; ++g) {
            if (g >= a.group)
                break;
            float s = q[g].x * k.x + q[g].y * k.y + q[g].z * k.z + q[g].w * k.w;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                s += __shfl_xor_sync(0xffffffffu, s, o);
            s *= scale;
            const float mn = fmaxf(m[g], s);
            const float f = exp2f(m[g] - mn), w = exp2f(s - mn);
            m[g] = mn;
            l[g] = l[g] * f + w;
            acc[g].x = acc[g].x * f + w * v.x;
            acc[g].y = acc[g].y * f + w * v.y;
            acc[g].z = acc[g].z * f + w * v.z;
            acc[g].w = acc[g].w * f + w * v.w;
        }
    }
    for (int g = 0; g < a.group; ++g) {
        *reinterpret_cast<float4 *>(&red[warp][g][4 * lane]) = acc[g];
        if (lane == 0) {
            red_m[warp][g] = m[g];
            red_l[warp][g] = l[g];
        }
    }
    __syncthreads();
    const float vs = __ldg(a.v_scale + h);
    for (int e = threadIdx.x; e < a.group * kHeadDim; e += blockDim.x) {
        const int g = e / kHeadDim, d = e % kHeadDim;
        float M = -INFINITY, s = 0.f, o = 0.f;
        for (int w = 0; w < kAttWarps; ++w)
            M = fmaxf(M, red_m[w][g]);
        for (int w = 0; w < kAttWarps; ++w) {
            const float f = red_m[w][g] == -INFINITY ? 0.f : exp2f(red_m[w][g] - M);
            s += f * red_l[w][g];
            o += f * red[w][g][d];
        }
        o = count > 0 ? o * vs / s : 0.f;
        const int64_t at = (static_cast<int64_t>(row) * a.hq + h * a.group + g) * kHeadDim + d;
        if (a.out_f32)
            static_cast<float *>(a.out)[at] = o;
        else
            static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(o);
    }
}

}  // namespace

cudaError_t launch_attend_fp4(const Fp4AttnArgs &a, cudaStream_t stream)
{
    const int64_t rows = a.cu_q ? a.total_q : a.batch;
    attend_fp4_kernel<<<static_cast<unsigned>(rows * a.hkv), 32 * kAttWarps, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace pkv
