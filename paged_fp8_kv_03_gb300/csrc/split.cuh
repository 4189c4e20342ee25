// What the windowed decode kernels share, whatever the cache's format: which
// tokens a query sees, the list of units and the places in it, bounded waits, the
// query as MMA fragment, output rows, and the cluster's shared memory.
#pragma once

#include "attn.h"

namespace pkv {

constexpr unsigned kEvery = 0xffffffffu;
constexpr uint64_t kLimitNs = 2000000000ull;

// What one sequence shows its query: tokens [0, sinks) and [from, len), as
// tiles 0 .. first - 1 and then first + skip .. (tiles in all).
struct Sight {
    int len, sinks, from, first, skip, tiles;
};

__device__ __forceinline__ Sight sight_of(const CacheAttnArgs &a, int b)
{
    Sight s;
    const int lp = seq_page_log2(a, b);
    const long long cap = lp < 0 ? 0 : static_cast<long long>(a.max_pages) << lp;
    const int most = cap < a.max_len ? static_cast<int>(cap) : a.max_len;
    const int L = a.seq_lens[b];
    s.len = L < 0 ? 0 : min(L, most);
    s.from = a.win.window == 0 ? 0 : max(0, s.len - a.win.window);
    s.sinks = min(a.win.sinks, s.from);
    s.first = (s.sinks + 15) >> 4;
    s.skip = max(s.from >> 4, s.first) - s.first;
    s.tiles = ((s.len + 15) >> 4) - s.skip;
    return s;
}

// Tile of the sequence that is tile i of its visible ones.
__device__ __forceinline__ int tile_at(const Sight &s, int i)
{
    return i < s.first ? i : i + s.skip;
}

struct Place {
    int b, h, unit;
};

__device__ __forceinline__ Place place_of(const int *start, int batch, int x)
{
    const int per_head = start[batch];
    Place p;
    p.h = x / per_head;
    const int rem = x - p.h * per_head;
    int lo = 0, hi = batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= rem)
            lo = mid;
        else
            hi = mid - 1;
    }
    p.b = lo;
    p.unit = rem - start[lo];
    return p;
}

// Bounded wait by a whole warp.
static __device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int *stop, int32_t *err, int lane)
{
    uint64_t t0 = 0;
    for (uint32_t it = 0;; ++it) {
        if (__all_sync(kEvery, mbar_try_wait(bar, parity)))
            return true;
        if ((it & 15u) == 15u) {
            int quit = 0;
            if (lane == 0) {
                if (t0 == 0)
                    t0 = global_timer_ns();
                if (*stop) {
                    quit = 1;
                } else if (global_timer_ns() - t0 > kLimitNs) {
                    *stop = 1;
                    if (err)
                        atomicOr(err, PKV_DEVERR_TIMEOUT);
                    quit = 1;
                }
            }
            if (__shfl_sync(kEvery, quit, 0))
                return false;
        }
    }
}

// The list's position of position x of the same list with one more, empty unit
// after every segment: an empty one counts as the next segment's first.
__device__ __forceinline__ int real_position(const int *start, int batch, int hkv, int x)
{
    const int per_head = start[batch], wide = per_head + batch;
    const int h = x / wide;
    if (h >= hkv)
        return per_head * hkv;
    const int rem = x - h * wide;
    int lo = 0, hi = batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] + mid <= rem)
            lo = mid;
        else
            hi = mid - 1;
    }
    return h * per_head + min(rem - lo, start[lo + 1]);
}

__device__ __forceinline__ bool wait_stage(uint32_t bar, uint32_t parity, volatile int *stop, int32_t *err, int lane)
{
    return __all_sync(kEvery, mbar_try_wait(bar, parity)) || wait_slow(bar, parity, stop, err, lane);
}

__device__ __forceinline__ void lds128(uint32_t at, uint32_t (&r)[4])
{
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void lds64(uint32_t at, uint32_t (&r)[2])
{
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at));
}
__device__ __forceinline__ uint32_t lds16(uint32_t at)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Two E4M3 bytes (low 16 bits) -> f16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t s)
{
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(s)));
    return d;
}

// Two fp32 values in one 64-bit register pair; each half rounds like the
// scalar operation.
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t r)
{
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
    return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// 16 consecutive dims of one output row.
__device__ __forceinline__ void store16(const CacheAttnArgs &a, int64_t row, int d, const float (&v)[16])
{
    if (a.out_f32) {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + row * kHeadDim + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
        uint4 *p = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + row * kHeadDim + d);
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
    }
}

__device__ __forceinline__ void store4(void *out, bool f32, int64_t row, int d, float4 v)
{
    if (f32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(out) + row * kHeadDim + d) = v;
    } else {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(out) + row * kHeadDim + d) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
    }
}

__device__ __forceinline__ void store4(const CacheAttnArgs &a, int64_t row, int d, float4 v)
{
    store4(a.out, a.out_f32 != 0, row, d, v);
}

// a 2^d 2^e / l for a whole number e.  Either power may lie beyond fp32's range where the
// result does not (a large weight that meets tiny values, beside a tiny one that meets large
// ones): the whole part of both is multiplied in two halves, exactly.
struct Quotient {
    float rest, low, high;
    __device__ __forceinline__ Quotient(float d, float e, float l)
    {
        const float near = rintf(d);
        rest = ex2_approx(d - near) / l;
        // (a is below 2^60: with 2^-252 nothing is left of it, with 2^254 more than fp32 holds)
        const int whole = static_cast<int>(fminf(fmaxf(near + e, -252.f), 254.f)), half = whole >> 1;
        low = __int_as_float((half + 127) << 23);
        high = __int_as_float((whole - half + 127) << 23);
    }
    __device__ __forceinline__ float operator()(float a) const { return a * rest * low * high; }
    __device__ __forceinline__ float4 operator()(float4 a) const
    {
        return make_float4((*this)(a.x), (*this)(a.y), (*this)(a.z), (*this)(a.w));
    }
};

// All threads of the cluster (one CTA: of the CTA).
__device__ __forceinline__ void cluster_sync(int ctas)
{
    if (ctas > 1)
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    else
        __syncthreads();
}

// The float at address `at` of this CTA's shared memory in CTA `cta` of the
// cluster (own: in this one).
__device__ __forceinline__ float cluster_load(uint32_t at, int cta, bool own)
{
    float v;
    if (own) {
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    } else {
        uint32_t there;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(cta));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(there) : "memory");
    }
    return v;
}

// The same for four floats, 16-byte aligned.
__device__ __forceinline__ float4 cluster_load4(uint32_t at, int cta, bool own)
{
    float4 v;
    if (own) {
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    } else {
        uint32_t there;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(cta));
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                     : "r"(there)
                     : "memory");
    }
    return v;
}

// Q as B fragment: head r, dims 32c + 4 kk + {0, 1} and {2, 3}, brought to [1, 2)
// by a power of two, so that f16 holds all bits of what is at least 2^-17 of the
// row's largest |q|, and the rest to 2^-25 of that; f0, f1 turn unscaled scores of
// heads 2c, 2c + 1 into exponents of 2.
struct Query {
    uint32_t q[8][2];
    float f0, f1;
};

__device__ __forceinline__ void load_rows(const CacheAttnArgs &a, int b, int h, int r, int c, uint4 (&raw)[4])
{
    const int64_t row = static_cast<int64_t>(b) * a.hq + static_cast<int64_t>(h) * a.group + (r < a.group ? r : 0);
    const uint4 *src = reinterpret_cast<const uint4 *>(a.q + row * kHeadDim + 32 * c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        raw[i] = src[i];
}

__device__ __forceinline__ void make_query(const CacheAttnArgs &a, const uint4 (&raw)[4], float k_scale, int r, int c,
                                           Query &o)
{
    const uint32_t *w = reinterpret_cast<const uint32_t *>(raw);
    uint32_t top = 0;                                      // largest |q|, as its bits
#pragma unroll
    for (int i = 0; i < 16; ++i)
        top = max(top, max((w[i] << 16) & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
    top = max(top, __shfl_xor_sync(kEvery, top, 1));
    top = max(top, __shfl_xor_sync(kEvery, top, 2));
    const int ex = min(max(static_cast<int>(top >> 23), 1), 253);
    const float down = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);
    const float up = __uint_as_float(static_cast<uint32_t>(ex) << 23) * (k_scale * a.sm_scale_log2);
    const bool on = r < a.group;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        o.q[i >> 1][i & 1] = f32x2_to_f16x2(on ? __uint_as_float(w[i] << 16) * down : 0.f,
                                            on ? __uint_as_float(w[i] & 0xFFFF0000u) * down : 0.f);
    o.f0 = __shfl_sync(kEvery, up, 8 * c);
    o.f1 = __shfl_sync(kEvery, up, 8 * c + 4);
}

// Units of a segment of which every token is visible: past the sinks and the
// window's first tile, before the last tokens.
struct Inner {
    int lo;
    uint32_t n;
};

__device__ __forceinline__ Inner inner_units(const Sight &s)
{
    const int lo = (s.from > 0 ? s.first + 2 : 1) >> 1, hi = ((s.len >> 4) - s.skip) >> 1;
    return Inner{lo, hi > lo ? static_cast<uint32_t>(hi - lo) : 0u};
}

// Tile number in the pools of visible tile i of segment (b, h); -1: its page
// lies outside the pool (flagged), -2: there is no such tile.
__device__ __forceinline__ int tile_number(const CacheAttnArgs &a, const Sight &s, int b, int h, int i)
{
    if (i >= s.tiles)
        return -2;
    int phys, row;
    if (!seq_token_page(a, b, seq_page_log2(a, b), 16 * tile_at(s, i), phys, row)) {
        if (a.err)
            atomicOr(a.err, PKV_DEVERR_PAGE);
        return -1;
    }
    return (phys * a.hkv + h) * (a.page_size >> 4) + (row >> 4);
}

__device__ __forceinline__ void flag_sequence(const CacheAttnArgs &a, int b, const Sight &s)
{
    if (a.err == nullptr)
        return;
    if (seq_page_log2(a, b) < 0)
        atomicOr(a.err, PKV_DEVERR_PAGESIZE);
    else if (a.seq_lens[b] != s.len)
        atomicOr(a.err, PKV_DEVERR_SEQLEN);
}

}  // namespace pkv
