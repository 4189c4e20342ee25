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
// Who works for a block: the warp that finds the block's first token in the call
// among the few that it looks at.  A token is the first if none of the 31 before it has
// its block; the block's other tokens are among the 31 behind it.  So a block's tokens
// need not be next to one another nor in order, only within 32 of the call's.
// (Sixteen tokens that are a whole block's rows, as most of a prompt's are, need no
// search.)  A warp loads the block's rows of one kv head, of K or of V, at once.
//
// What bounds them: the bytes, 256 or 512 a row of the call and 128 of the cache.
#include "fp8b.h"
#include "grid.cuh"

namespace pkv {

namespace {

constexpr unsigned kWarp = 0xffffffffu;
constexpr int kRowThreads = 256;

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

__device__ __forceinline__ float two_to_minus(int e)       // e: -117 .. 127 (2^-127 is a subnormal number)
{
    return e == 127 ? __uint_as_float(0x00400000u) : two_to(-e);
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
        x.u[i] = p[i];
}

template <bool kBf16>
__device__ __forceinline__ void values_of(const Eight<kBf16> &x, float (&v)[8])
{
    const uint32_t *w = reinterpret_cast<const uint32_t *>(x.u);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = kBf16 ? __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16) : __uint_as_float(w[i]);
}

// The bits of the largest |value| of eight, sign aside (bf16: in the high half of
// either half's place, see top_bits).
template <bool kBf16>
__device__ __forceinline__ uint32_t max_bits(const Eight<kBf16> &x, uint32_t top)
{
    const uint32_t *w = reinterpret_cast<const uint32_t *>(x.u);
#pragma unroll
    for (int i = 0; i < (kBf16 ? 4 : 8); ++i) {
        if (kBf16)
            asm("max.u16x2 %0, %1, %2;" : "=r"(top) : "r"(top), "r"(w[i] & 0x7FFF7FFFu));
        else
            top = max(top, w[i] & 0x7FFFFFFFu);
    }
    return top;
}

// The fp32 bits of what max_bits has left.
template <bool kBf16>
__device__ __forceinline__ uint32_t top_bits(uint32_t top)
{
    return kBf16 ? max(top << 16, top & 0xFFFF0000u) : top;
}

// The same of the finite ones, by each value.
template <bool kBf16>
__device__ __forceinline__ uint32_t finite_bits(const Eight<kBf16> &x, uint32_t top)
{
    float v[8];
    values_of<kBf16>(x, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t bits = __float_as_uint(v[j]) & 0x7FFFFFFFu;
        top = max(top, bits < 0x7F800000u ? bits : 0u);
    }
    return top;
}

// One block of K or of V (the whole warp).  Its `count` new rows: lane k (and 16 + k) has
// the token and the row of the k-th, `rows` a bit a row; kFull: all 16, token k in row k.
template <bool kBf16, bool kFull>
__device__ __forceinline__ void append_block(const Fp8bRowArgs &a, const void *in, uint8_t *cache, uint8_t *exps, int64_t t0,
                                             int64_t slot, int h, int count, int token, int row, uint32_t rows, int lane)
{
    const int64_t page = slot >> a.page_log2;
    const int row0 = static_cast<int>(slot & (a.page_size - 1)) & ~(kBlock - 1);
    uint8_t *block = cache + ((page * a.hkv + h) * a.page_size + row0) * kHeadDim;
    uint8_t *exp = exps + (page * a.hkv + h) * (a.page_size / kBlock) + row0 / kBlock;
    const bool begins = kFull || (rows & 1u);
    const int part = lane & 15, half = lane >> 4;          // 8 dims of two rows at a time
    Eight<kBf16> x[kBlock / 2];
#pragma unroll
    for (int i = 0; i < kBlock / 2; ++i) {
        const int k = 2 * i + half, t = kFull ? k : __shfl_sync(kWarp, token, k);
        if (kFull || k < count)
            load_eight<kBf16>(in, ((t0 + t) * a.hkv + h) * kHeadDim + 8 * part, x[i]);
    }
    // (a byte above an appended block's largest keeps its meaning; 255, which has none, counts as 254)
    const int old = begins ? kExpMin : min(static_cast<int>(*exp), 254) - kExpBias;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kBlock / 2; ++i)
        if (kFull || 2 * i + half < count)
            top = max_bits<kBf16>(x[i], top);
    top = __reduce_max_sync(kWarp, top_bits<kBf16>(top));
    if (top >= 0x7F800000u) {                              // an infinity or a NaN
        top = 0;
#pragma unroll
        for (int i = 0; i < kBlock / 2; ++i)
            if (kFull || 2 * i + half < count)
                top = finite_bits<kBf16>(x[i], top);
        top = __reduce_max_sync(kWarp, top);
    }
    const int e = max(block_exponent(top), old);
    const float down = two_to_minus(e);
#pragma unroll
    for (int i = 0; i < kBlock / 2; ++i) {
        const int k = 2 * i + half, r = kFull ? k : __shfl_sync(kWarp, row, k);
        if (kFull || k < count) {
            float v[8];
            values_of<kBf16>(x[i], v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] *= down;
            *reinterpret_cast<uint2 *>(block + r * kHeadDim + 8 * part) =
                make_uint2(to_e4m3x4(v[0], v[1], v[2], v[3]), to_e4m3x4(v[4], v[5], v[6], v[7]));
        }
    }
    if (!begins && e > old) {                              // the rows that were there, to the larger power of two
        const float f = two_to(max(old - e, -126));
        for (int r = lane >> 3; r < kBlock; r += 4) {
            if ((rows >> r) & 1u)
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

// Position of the k-th set bit (k < popcount).
__device__ __forceinline__ int nth_bit(uint64_t m, int k)
{
    int at = 0;
#pragma unroll
    for (int w = 32; w > 0; w >>= 1) {
        const int n = __popcll(m & ((uint64_t(1) << w) - 1));
        if (k >= n) {
            k -= n;
            m >>= w;
            at += w;
        }
    }
    return at;
}

// A warp looks at `tokens` (at most 16) of the call's tokens, for one kv head's K or V.
template <bool kBf16>
__global__ void __launch_bounds__(kRowThreads, kBf16 ? 4 : 2) kv_append_fp8b_kernel(const Fp8bRowArgs a, int tokens)
{
    grid_wait();
    const int lane = threadIdx.x & 31;
    const uint32_t id = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5), per = 2 * a.hkv;
    const uint32_t group = id / per, rest = id - group * per;
    const int h = static_cast<int>(rest >> 1);
    const int64_t first = static_cast<int64_t>(group) * tokens;
    if (first >= a.num_tokens)
        return;
    const void *in = rest & 1 ? a.v_in : a.k_in;
    uint8_t *cache = rest & 1 ? a.v_cache : a.k_cache, *exps = rest & 1 ? a.v_exp : a.k_exp;
    auto slot_at = [&](int64_t t) { return t >= 0 && t < a.num_tokens ? a.slots[t] : int64_t(-1); };
    const int64_t s = slot_at(first + lane), s0 = __shfl_sync(kWarp, s, 0);
    if (tokens == kBlock && s0 >= 0 && s0 < a.num_slots && (s0 & (kBlock - 1)) == 0 &&
        __all_sync(kWarp, lane >= kBlock || s == s0 + lane)) {
        append_block<kBf16, true>(a, in, cache, exps, first, s0, h, kBlock, 0, 0, 0xFFFFu, lane);
        return;
    }
    const int64_t before = slot_at(first - 32 + lane), behind = slot_at(first + 32 + lane);
    const bool mine = lane < tokens && s >= 0;             // (beyond the call: -1)
    if (mine && s >= a.num_slots && rest == 0 && a.err)
        atomicOr(a.err, PKV_DEVERR_SLOT);
    // (no token: a block of its own)
    const int64_t block = s >= 0 ? s / kBlock : -1 - lane;
    const uint32_t same = __match_any_sync(kWarp, block);
    uint32_t leaders = __ballot_sync(kWarp, mine && s < a.num_slots && (same & ((1u << lane) - 1u)) == 0);
    while (leaders != 0) {
        const int L = __ffs(leaders) - 1;
        leaders &= leaders - 1;
        const int64_t slot = __shfl_sync(kWarp, s, L), b = slot / kBlock;
        if (__any_sync(kWarp, lane > L && before >= 0 && before / kBlock == b))
            continue;                                      // begun by an earlier token
        const uint32_t lo = __shfl_sync(kWarp, same, L);
        const uint32_t hi = __ballot_sync(kWarp, lane < L && behind >= 0 && behind / kBlock == b);
        const uint64_t members = static_cast<uint64_t>(hi) << 32 | lo;
        const int count = min(__popcll(members), kBlock);  // (more: a slot occurs twice)
        const uint32_t rows = __reduce_or_sync(kWarp, ((lo >> lane) & 1u ? 1u << (s & (kBlock - 1)) : 0u) |
                                                          ((hi >> lane) & 1u ? 1u << (behind & (kBlock - 1)) : 0u));
        const int token = (lane & 15) < count ? nth_bit(members, lane & 15) : L;
        const int from_s = __shfl_sync(kWarp, static_cast<int>(s & (kBlock - 1)), token & 31);
        const int from_behind = __shfl_sync(kWarp, static_cast<int>(behind & (kBlock - 1)), token & 31);
        append_block<kBf16, false>(a, in, cache, exps, first, slot, h, count, token, token < 32 ? from_s : from_behind, rows,
                                   lane);
    }
}

// 16 bytes of a row of K and of V of kTokens tokens a thread, whose loads are in flight
// together.
template <bool kBf16, int kTokens>
__global__ void __launch_bounds__(kRowThreads) kv_read_fp8b_kernel(const Fp8bRowArgs a)
{
    grid_wait();
    constexpr int kVals = kBf16 ? 8 : 4, kPerRow = kHeadDim / kVals;
    const uint32_t i = blockIdx.x * kRowThreads + threadIdx.x, row = i / kPerRow, part = i % kPerRow;
    const uint32_t group = row / static_cast<uint32_t>(a.hkv), h = row - group * a.hkv;
    const int64_t token = static_cast<int64_t>(group) * kTokens;
    if (token >= a.num_tokens)
        return;
    int64_t slot[kTokens];
    uint32_t w[kTokens][2][kVals / 4], x[kTokens][2];
#pragma unroll
    for (int n = 0; n < kTokens; ++n)
        slot[n] = token + n < a.num_tokens ? a.slots[token + n] : -1;
#pragma unroll
    for (int n = 0; n < kTokens; ++n) {
        const bool in = slot[n] >= 0 && slot[n] < a.num_slots;
        const int64_t page = slot[n] >> a.page_log2, at = (page * a.hkv + h) * a.page_size + (slot[n] & (a.page_size - 1));
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint8_t *src = (kv ? a.v_cache : a.k_cache) + at * kHeadDim + part * kVals;
            if (kBf16) {
                const uint2 u = in ? *reinterpret_cast<const uint2 *>(src) : make_uint2(0u, 0u);
                w[n][kv][0] = u.x;
                w[n][kv][kVals / 4 - 1] = u.y;
            } else {
                w[n][kv][0] = in ? *reinterpret_cast<const uint32_t *>(src) : 0u;
            }
            x[n][kv] = in ? (kv ? a.v_exp : a.k_exp)[at / kBlock] : kExpBias;
        }
    }
#pragma unroll
    for (int n = 0; n < kTokens; ++n) {
        if (slot[n] < 0)
            continue;
        if (slot[n] >= a.num_slots && a.err)
            atomicOr(a.err, PKV_DEVERR_SLOT);
        const int64_t to = (((token + n) * a.hkv + h) * kHeadDim + part * kVals);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            void *out = kv ? a.v_out : a.k_out;
            const float f = __uint_as_float(x[n][kv] == 0 ? 0x00400000u : x[n][kv] << 23);   // 2^(x - 127)
            float v[kVals];
#pragma unroll
            for (int j = 0; j < kVals / 4; ++j) {
                float y[4];
                from_e4m3x4(w[n][kv][j], y);
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
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out) + to) = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
                *reinterpret_cast<float4 *>(static_cast<float *>(out) + to) = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv_append_fp8b(const Fp8bRowArgs &a, bool bf16, cudaStream_t stream)
{
    // tokens a warp looks at: a block's 16 where that leaves enough warps
    int tokens = kBlock;
    while (tokens > 1 && a.num_tokens * 2 * a.hkv < static_cast<int64_t>(device_sm_count()) * 16 * tokens)
        tokens /= 2;
    const int64_t warps = (a.num_tokens + tokens - 1) / tokens * 2 * a.hkv;
    const int64_t grid = (warps + kRowThreads / 32 - 1) / (kRowThreads / 32);
    if (warps > UINT32_MAX - kRowThreads)
        return cudaErrorInvalidValue;
    return launch_with(bf16 ? kv_append_fp8b_kernel<true> : kv_append_fp8b_kernel<false>, dim3(static_cast<unsigned>(grid)),
                       kRowThreads, 0, 1, true, stream, a, tokens);
}

typedef void (*ReadKernel)(const Fp8bRowArgs);

// Several tokens a thread where that still fills the GPU with threads.  Threads count in
// 32 bits: longer calls are several launches.
cudaError_t launch_kv_read_fp8b(const Fp8bRowArgs &args, bool bf16, cudaStream_t stream)
{
    constexpr int kMany = 4;
    const int64_t per_token = static_cast<int64_t>(args.hkv) * (bf16 ? 16 : 32);
    const bool many = args.num_tokens * per_token >= static_cast<int64_t>(device_sm_count()) * 2048 * kMany;
    const ReadKernel kernel = bf16 ? (many ? kv_read_fp8b_kernel<true, kMany> : kv_read_fp8b_kernel<true, 1>)
                                   : (many ? kv_read_fp8b_kernel<false, kMany> : kv_read_fp8b_kernel<false, 1>);
    const int64_t most = (int64_t(1) << 31) / per_token / kMany * kMany;
    if (most < 1)
        return cudaErrorInvalidValue;
    for (int64_t t = 0; t < args.num_tokens; t += most) {
        Fp8bRowArgs a = args;
        a.num_tokens = args.num_tokens - t < most ? args.num_tokens - t : most;
        a.slots += t;
        a.k_out = static_cast<uint8_t *>(args.k_out) + t * args.hkv * kHeadDim * (bf16 ? 2 : 4);
        a.v_out = static_cast<uint8_t *>(args.v_out) + t * args.hkv * kHeadDim * (bf16 ? 2 : 4);
        const int64_t threads = (a.num_tokens + (many ? kMany : 1) - 1) / (many ? kMany : 1) * per_token;
        const cudaError_t e = launch_with(kernel, dim3(static_cast<unsigned>((threads + kRowThreads - 1) / kRowThreads)),
                                          kRowThreads, 0, 1, true, stream, a);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace pkv
