// kv_append_fp8b and kv_read_fp8b: rows of K and V into the block-scaled FP8
// cache and back.
//
// A block (16 tokens of a kv head) holds E4M3 codes and one power of two 2^e.
// A call's new rows of a block give
//   e_new = the smallest e with amax <= 448 * 2^e   (amax: their largest finite |x|),
// and the block's e is e_new if the call writes the block's row 0 (it begins the
// block), else max(e_old, e_new).  New rows: code = E4M3(x * 2^-e), a product that is
// exact, so one rounding (nearest, ties to even; +-Inf saturates, NaN stays).
// Where e grows, the rows that the block held before are rounded to it once more:
// code' = E4M3(code * 2^(e_old - e)), which changes none that stays a normal E4M3
// number.
//
// Who works for a block: the warp that finds the block's first token in the call.
// A token is the first if none of the 31 before it has its block; the block's
// other tokens are among the 31 behind it.  So a block's tokens need not be next
// to one another nor in order, only within 32 of the call's.
//
// What bounds them: the bytes, 256 or 512 a row of the call and 128 of the cache.
#include "fp8b.h"

namespace pkv {

namespace {

constexpr unsigned kWarp = 0xffffffffu;
constexpr int kAppendThreads = 256, kReach = 32;

// The exponent of a block whose largest |value| has these bits (finite).
__device__ __forceinline__ int block_exponent(uint32_t top)
{
    // 448 = 1.75 * 2^8
    const int e = static_cast<int>(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return min(max(e, kExpMin), kExpMax);                  // (0 and subnormals: kExpMin)
}

__device__ __forceinline__ float two_to(int e)             // -126 .. 127
{
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d)
{
    uint32_t w;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(w)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return w;
}

// Four codes as values.
__device__ __forceinline__ void from_e4m3x4(uint32_t w, float (&v)[4])
{
    uint32_t lo, hi;
    e4m3x4_to_f16x4(w, lo, hi);
    const float2 a = f16x2_to_f32x2(lo), b = f16x2_to_f32x2(hi);
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
}

// 8 values of a row, as they lie in memory.
template <bool kBf16>
struct Eight {
    uint4 u[kBf16 ? 1 : 2];
};

template <bool kBf16>
__device__ __forceinline__ void load_eight(const void *rows, int64_t at, Eight<kBf16> &x)
{
    const uint4 *p = kBf16 ? reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(rows) + at)
                           : reinterpret_cast<const uint4 *>(static_cast<const float *>(rows) + at);
#pragma unroll
    for (int i = 0; i < (kBf16 ? 1 : 2); ++i)
        x.u[i] = __ldg(p + i);
}

template <bool kBf16>
__device__ __forceinline__ void values_of(const Eight<kBf16> &x, float (&v)[8])
{
    const uint32_t *w = reinterpret_cast<const uint32_t *>(x.u);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = kBf16 ? __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16) : __uint_as_float(w[i]);
}

// A block's new rows in one call.
struct Members {
    int count;                                             // rows found (at most 16)
    uint32_t rows;                                         // a bit a row of the block
    uint8_t token[kBlock], row[kBlock];                    // beyond the first one's token; row of the block
};

// One block of K or of V (the whole warp): its new rows' tokens are t0 + m.token[i].
template <bool kBf16>
__device__ __forceinline__ void append_block(const Fp8bRowArgs &a, const void *rows, uint8_t *cache, uint8_t *exps, int64_t t0,
                                             int64_t slot, int h, const Members &m, int lane)
{
    const int64_t page = slot >> a.page_log2;
    const int row0 = static_cast<int>(slot & (a.page_size - 1)) & ~(kBlock - 1);
    uint8_t *block = cache + ((page * a.hkv + h) * a.page_size + row0) * kHeadDim;
    uint8_t *exp = exps + (page * a.hkv + h) * (a.page_size / kBlock) + row0 / kBlock;
    const bool begins = m.rows & 1u;
    const int old = begins ? kExpMin : min(static_cast<int>(*exp) - kExpBias, kExpMax);
    const int part = lane & 15, half = lane >> 4;          // 8 dims of two rows at a time
    Eight<kBf16> x[kBlock / 2];
#pragma unroll
    for (int i = 0; i < kBlock / 2; ++i) {
        const int k = 2 * i + half;
        if (k < m.count)
            load_eight<kBf16>(rows, ((t0 + m.token[k]) * a.hkv + h) * kHeadDim + 8 * part, x[i]);
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kBlock / 2; ++i) {
        if (2 * i + half < m.count) {
            float v[8];
            values_of<kBf16>(x[i], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t bits = __float_as_uint(v[j]) & 0x7FFFFFFFu;
                top = max(top, bits < 0x7F800000u ? bits : 0u);
            }
        }
    }
    top = __reduce_max_sync(kWarp, top);
    const int e = max(block_exponent(top), old);
    const float down = two_to(-e);
#pragma unroll
    for (int i = 0; i < kBlock / 2; ++i) {
        const int k = 2 * i + half;
        if (k < m.count) {
            float v[8];
            values_of<kBf16>(x[i], v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] *= down;
            *reinterpret_cast<uint2 *>(block + m.row[k] * kHeadDim + 8 * part) =
                make_uint2(to_e4m3x4(v[0], v[1], v[2], v[3]), to_e4m3x4(v[4], v[5], v[6], v[7]));
        }
    }
    if (!begins && e > old) {                              // the rows that were there, to the larger power of two
        const float f = two_to(max(old - e, -126));
        for (int r = lane >> 3; r < kBlock; r += 4) {
            if ((m.rows >> r) & 1u)
                continue;
            uint4 *p = reinterpret_cast<uint4 *>(block + r * kHeadDim) + (lane & 7);
            uint4 u = *p;
            uint32_t *w = reinterpret_cast<uint32_t *>(&u);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v[4];
                from_e4m3x4(w[j], v);
                w[j] = to_e4m3x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
            }
            *p = u;
        }
    }
    if (lane == 0 && (begins || e > old))
        *exp = static_cast<uint8_t>(e + kExpBias);
}

// A CTA looks at `tokens` of the call's tokens; the blocks that these begin in the
// call, times heads, times K and V, are shared among its warps and those of the
// gridDim.y CTAs beside it.
template <bool kBf16>
__global__ void __launch_bounds__(kAppendThreads) kv_append_fp8b_kernel(const Fp8bRowArgs a, int tokens)
{
    __shared__ Members members[kBlock];
    __shared__ int64_t slots[kBlock];
    __shared__ int place[kBlock + 1];                      // tokens that come first, and how many
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * tokens;
    auto slot_at = [&](int64_t t) { return t >= 0 && t < a.num_tokens ? __ldg(a.slots + t) : int64_t(-1); };
    for (int i = warp; i < tokens; i += kAppendThreads / 32) {
        const int64_t t = first + i, slot = slot_at(t);
        const int64_t behind = slot_at(t + lane), before = slot_at(t - kReach + 1 + lane);   // (lane 31: t itself)
        const bool in = slot >= 0 && slot < a.num_slots;
        if (slot >= a.num_slots && lane == 0 && blockIdx.y == 0 && a.err)
            atomicOr(a.err, PKV_DEVERR_SLOT);
        const bool again = lane < kReach - 1 && before >= 0 && before / kBlock == slot / kBlock;
        const bool mine = in && behind >= 0 && behind / kBlock == slot / kBlock;
        const uint32_t mask = __ballot_sync(kWarp, mine);
        const bool leads = in && !__any_sync(kWarp, again);
        if (leads) {
            const int rank = __popc(mask & ((1u << lane) - 1u));
            const int row = static_cast<int>(behind & (kBlock - 1));
            const uint32_t rows = __reduce_or_sync(kWarp, mine ? 1u << row : 0u);
            if (mine && rank < kBlock) {                   // (more: a slot occurs twice)
                members[i].token[rank] = static_cast<uint8_t>(lane);
                members[i].row[rank] = static_cast<uint8_t>(row);
            }
            if (lane == 0) {
                members[i].count = min(__popc(mask), kBlock);
                members[i].rows = rows;
            }
        }
        if (lane == 0)
            slots[i] = leads ? slot : -1;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int n = 0;
        for (int i = 0; i < tokens; ++i)
            if (slots[i] >= 0)
                place[n++] = i;
        place[kBlock] = n;
    }
    __syncthreads();
    const int items = place[kBlock] * a.hkv * 2;
    for (int k = blockIdx.y * (kAppendThreads / 32) + warp; k < items; k += gridDim.y * (kAppendThreads / 32)) {
        const int i = place[k / (2 * a.hkv)], rest = k % (2 * a.hkv);
        const int h = rest >> 1;
        if (rest & 1)
            append_block<kBf16>(a, a.v_in, a.v_cache, a.v_exp, first + i, slots[i], h, members[i], lane);
        else
            append_block<kBf16>(a, a.k_in, a.k_cache, a.k_exp, first + i, slots[i], h, members[i], lane);
    }
}

// 16 bytes of a row of K and of V a thread.
template <bool kBf16>
__global__ void __launch_bounds__(256) kv_read_fp8b_kernel(const Fp8bRowArgs a)
{
    constexpr int kVals = kBf16 ? 8 : 4, kPerRow = kHeadDim / kVals;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int part = static_cast<int>(i % kPerRow);
    const int64_t row = i / kPerRow, t = row / a.hkv;
    const int h = static_cast<int>(row - t * a.hkv);
    if (t >= a.num_tokens)
        return;
    const int64_t slot = __ldg(a.slots + t);
    if (slot < 0)
        return;
    const bool in = slot < a.num_slots;
    if (!in && a.err)
        atomicOr(a.err, PKV_DEVERR_SLOT);
    const int64_t page = slot >> a.page_log2, r = slot & (a.page_size - 1);
    const int64_t at = ((page * a.hkv + h) * a.page_size + r) * kHeadDim + part * kVals;
    const int64_t x_at = (page * a.hkv + h) * (a.page_size / kBlock) + r / kBlock;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const uint8_t *cache = kv ? a.v_cache : a.k_cache, *exps = kv ? a.v_exp : a.k_exp;
        void *out = kv ? a.v_out : a.k_out;
        uint32_t w[kVals / 4];
        float f = 0.f;
#pragma unroll
        for (int j = 0; j < kVals / 4; ++j)
            w[j] = in ? __ldg(reinterpret_cast<const uint32_t *>(cache + at) + j) : 0u;
        if (in) {
            const uint32_t x = __ldg(exps + x_at);
            f = __uint_as_float(x == 0 ? 0x00400000u : x << 23);   // 2^(x - 127)
        }
        float v[kVals];
#pragma unroll
        for (int j = 0; j < kVals / 4; ++j) {
            float y[4];
            from_e4m3x4(w[j], y);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[4 * j + k] = y[k] * f;
        }
        if constexpr (kBf16) {
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                o[j] = *reinterpret_cast<const uint32_t *>(&b);
            }
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + row * kHeadDim + part * kVals) =
                make_uint4(o[0], o[1], o[2], o[3]);
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(out) + row * kHeadDim + part * kVals) =
                make_float4(v[0], v[1], v[2], v[3]);
        }
    }
}

}  // namespace

cudaError_t launch_kv_append_fp8b(const Fp8bRowArgs &a, bool bf16, cudaStream_t stream)
{
    const int tokens = a.num_tokens <= 512 ? 1 : (a.num_tokens <= 4096 ? 4 : kBlock);
    const int64_t grid = (a.num_tokens + tokens - 1) / tokens;
    const int share = tokens == 1 ? (2 * a.hkv + kAppendThreads / 32 - 1) / (kAppendThreads / 32) : 1;
    const dim3 g(static_cast<unsigned>(grid), static_cast<unsigned>(share > 64 ? 64 : share));
    if (bf16)
        kv_append_fp8b_kernel<true><<<g, kAppendThreads, 0, stream>>>(a, tokens);
    else
        kv_append_fp8b_kernel<false><<<g, kAppendThreads, 0, stream>>>(a, tokens);
    return cudaGetLastError();
}

cudaError_t launch_kv_read_fp8b(const Fp8bRowArgs &a, bool bf16, cudaStream_t stream)
{
    const int64_t threads = a.num_tokens * a.hkv * (kHeadDim / (bf16 ? 8 : 4));
    const int64_t grid = (threads + 255) / 256;
    if (bf16)
        kv_read_fp8b_kernel<true><<<static_cast<unsigned>(grid), 256, 0, stream>>>(a);
    else
        kv_read_fp8b_kernel<false><<<static_cast<unsigned>(grid), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace pkv
