// What the prefill attention kernels share: bounded waits, operand descriptors,
// paired fp32 arithmetic, and which keys a chunk of queries sees.
#pragma once

#include "fp4.cuh"
#include "tcgen05.cuh"

namespace pkv {

constexpr int kRows = 128;                       // M: rows of a query tile
constexpr int kKeys = 128;                       // keys per tile
constexpr int kMaxKv = INT32_MAX - (kKeys - 1);  // longest sequence: 32 bits hold it rounded up to whole key tiles
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr unsigned kAll = 0xffffffffu;

// Bounded wait, one thread.  honour_abort = false for drains.
__device__ __forceinline__ bool pwait(uint32_t bar, uint32_t parity, volatile int *abort_flag, int32_t *err,
                                      bool honour_abort = true)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity))
            return true;
        if ((it & 15u) == 0) {
            if (honour_abort && *abort_flag)
                return false;
            if (global_timer_ns() - t0 > kWaitNs) {
                *abort_flag = 1;
                if (err)
                    atomicOr(err, PKV_DEVERR_TIMEOUT);
                return false;
            }
        }
    }
}

// Bounded wait by a whole warp; the result is warp-uniform.
__device__ __forceinline__ bool wwait(uint32_t bar, uint32_t parity, volatile int *abort_flag, int32_t *err,
                                      int lane)
{
    uint64_t t0 = 0;
    for (uint32_t it = 0;; ++it) {
        if (__all_sync(kAll, mbar_try_wait(bar, parity)))
            return true;
        if ((it & 15u) == 15u) {
            int stop = 0;
            if (lane == 0) {
                if (*abort_flag) {
                    stop = 1;
                } else if (t0 == 0) {
                    t0 = global_timer_ns();
                } else if (global_timer_ns() - t0 > kWaitNs) {
                    *abort_flag = 1;
                    if (err)
                        atomicOr(err, PKV_DEVERR_TIMEOUT);
                    stop = 1;
                }
            }
            if (__shfl_sync(kAll, stop, 0))
                return false;
        }
    }
}

// Descriptors are built once per ring stage; a K step then only advances the
// start-address field (bytes / 16, the low bits of the descriptor), so the
// issuing thread spends its time issuing, not rebuilding 64-bit descriptors.
// K-major operand (128 rows x 128 dims, 128B swizzle; the query tile as A and
// a K tile as B of S = Q K^T): K step s of 16 dims starts (s / 4) * 16 KB +
// (s % 4) * 32 B into the tile.
__device__ __forceinline__ uint64_t kmajor_base(uint32_t tile)
{
    return tc::smem_desc_sw128(tile, 16, 1024);
}
__device__ __forceinline__ uint64_t kmajor_step(uint64_t base, int s)
{
    return base + static_cast<uint64_t>(((s >> 2) * 16384 + (s & 3) * 32) >> 4);
}

// V as the B operand of O += P V: rows = keys (the K dimension), 128 dims (N)
// contiguous in two 64-dim column blocks 16 KB apart; K step s = keys 16s..16s+15
// starts s * 2 KB into the tile.
__device__ __forceinline__ uint64_t vmn_base(uint32_t tile)
{
    return tc::smem_desc_sw128(tile, 16384, 1024);
}
__device__ __forceinline__ uint64_t vmn_step(uint64_t base, int s)
{
    return base + static_cast<uint64_t>((s * 2048) >> 4);
}

// Packed pairs of fp32 (one 64-bit register pair): the paired add and fma
// run two lanes of fp32 arithmetic per instruction, each rounded exactly as
// the scalar operation, so results equal the scalar code bit for bit.
__device__ __forceinline__ uint64_t f2_pack(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float2 f2_unpack(uint64_t r)
{
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
    return v;
}

__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t f2_sub(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// max(a, b, c) in one instruction (exact, like two fmaxf).
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// True in exactly one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, e;\n\t}"
        : "=r"(p));
    return p != 0;
}

// Checks a sequence's sizes; false (and PKV_DEVERR_SEQLEN when `report`) when
// the chunk or its length are inconsistent.
__device__ __forceinline__ bool sequence_ok(const PrefillArgs &a, int b, int q0, int q1, int L, bool report)
{
    const int n = q1 - q0;
    const int lp = seq_page_log2(a, b);
    const bool ok = q0 >= 0 && n >= 0 && q1 <= a.total_q && n <= a.max_q_len && L >= n &&
                    L <= min(a.max_kv_len, kMaxKv) && lp >= 0 &&
                    static_cast<int64_t>(L) <= (static_cast<int64_t>(a.max_pages) << lp);
    if (!ok && report && a.err)
        atomicOr(a.err, lp < 0 ? PKV_DEVERR_PAGESIZE : PKV_DEVERR_SEQLEN);
    return ok;
}

// What turns raw scores into exponents of 2.  A product too small for fp32 is its
// smallest number instead of 0, which would make NaN of a hidden key's -inf.
__device__ __forceinline__ float score_factor(const PrefillArgs &a, int h)
{
    const float f = __ldg(a.k_scale + h) * a.sm_scale_log2;
    return f == 0.f ? __uint_as_float(1u) : f;
}

// Sums over a long context are kept in levels, so that no chain of additions grows
// with it; the last level lies where the result will, in the row's place in the
// output.  What the thread that works for a row (or half of one) keeps of it, in
// shared memory, where it takes no registers from the scores' loop:
struct MovedRow {
    uint4 *out;                                            // the place; nullptr: a padding row
    float m, l;                                            // reference and sum of what has been moved there
};

// Key tiles of a sequence that some query of its chunk sees, under a window of
// the 4-bit cache's calls: tiles 0 .. first - 1 (sinks) and then first + skip ..
// (keys from `from` on).  Without a window: all of them (first = skip = 0).
struct KeyTiles {
    int from, sinks;                                     // keys t >= from or t < sinks are seen by someone
    int first, skip;
};

template <bool kWin>
__device__ __forceinline__ KeyTiles key_tiles(const Fp4Window &w, int first_pos)
{
    KeyTiles k = {0, 0, 0, 0};
    if (kWin && w.window > 0) {
        k.from = max(0, first_pos - w.window + 1);
        k.sinks = min(w.sinks, k.from);
        k.first = (k.sinks + kKeys - 1) / kKeys;
        k.skip = max(k.from / kKeys, k.first) - k.first;
    }
    return k;
}

// Key tiles that a query tile, or a pair of them, may visit: without a window all of
// the longest sequence's, with one the sinks' and those that 2 tokens_per_tile +
// window - 1 keys touch.
inline int64_t most_key_tiles(const PrefillArgs &a, const Fp4Window &w)
{
    const int64_t all = (static_cast<int64_t>(a.max_kv_len) + kKeys - 1) / kKeys;
    if (w.window == 0)
        return all;
    const int64_t seen = (static_cast<int64_t>(w.sinks) + kKeys - 1) / kKeys +
                         (static_cast<int64_t>(w.window) + 2 * a.tokens_per_tile) / kKeys + 2;
    return seen < all ? seen : all;
}

// NaN blocks of the 4-bit cache's V.  A weight of zero times a NaN is a NaN, so
// the widening kernel writes zeros for them and records where they were; the
// attention puts NaNs into the outputs of the rows that see them.
__device__ __forceinline__ uint32_t *nan_tiles(const PrefillArgs &a)
{
    return reinterpret_cast<uint32_t *>(a.v16 + a.rows_cap * kHeadDim);
}

__device__ __forceinline__ uint8_t *nan_rows(const PrefillArgs &a)
{
    return reinterpret_cast<uint8_t *>(nan_tiles(a) + a.rows_cap / kKeys);
}

// Blocks of 16 dims (a bit each) in which a row at position p sees a NaN: nt
// key tiles, the i-th one is key_tile(i) of the sequence and copy_tile(i) of the
// copy, which starts at tile `tile0` (the whole warp).
template <bool kWin, typename KeyTile, typename CopyTile>
__device__ __forceinline__ uint32_t nan_blocks(const PrefillArgs &a, const Fp4Window &w, int tile0, int nt, int p, int lane,
                                               KeyTile key_tile, CopyTile copy_tile)
{
    const uint32_t *tiles = nan_tiles(a);
    bool some = false;
    for (int i = lane; i < nt; i += 32)
        some = some || __ldg(tiles + tile0 + copy_tile(i)) != 0;
    uint32_t hit = 0;
    if (__any_sync(kAll, some)) {
#pragma unroll 1
        for (int i = 0; i < nt; ++i) {
            const int64_t tile = tile0 + copy_tile(i);
            const uint32_t word = __ldg(tiles + tile);
            if (word == 0)
                continue;
#pragma unroll 1
            for (int k = 0; k < kKeys; ++k) {
                const int t = key_tile(i) * kKeys + k;
                if ((word >> (8 * (k >> 5)) & 0xFFu) != 0 && t <= p && (!kWin || t > p - w.window || t < w.sinks))
                    hit |= __ldg(nan_rows(a) + tile * kKeys + k);
            }
        }
    }
    return hit;
}

// 128-row tiles of sequence b's widened region (all its kv heads): zero for a
// sequence with an empty or inconsistent chunk.
template <bool kWin>
__device__ __forceinline__ long long region_tiles(const PrefillArgs &a, const Fp4Window &w, int b)
{
    const int q0 = __ldg(a.cu_q + b), q1 = __ldg(a.cu_q + b + 1);
    const int L = __ldg(a.seq_lens + b);
    if (q1 - q0 <= 0 || !sequence_ok(a, b, q0, q1, L, false))
        return 0;
    return static_cast<long long>(a.hkv) * ((L + kKeys - 1) / kKeys - key_tiles<kWin>(w, L - (q1 - q0)).skip);
}

}  // namespace pkv
