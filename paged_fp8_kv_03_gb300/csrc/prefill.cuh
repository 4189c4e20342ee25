// What the prefill attention kernels share: bounded waits, operand descriptors,
// paired fp32 arithmetic, and which keys a chunk of queries sees.
#pragma once

#include <math.h>

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
template <bool kBlocks>
__device__ __forceinline__ float score_factor(const PrefillArgs &a, int h)
{
    const float f = (kBlocks ? 1.f : __ldg(a.k_scale + h)) * a.sm_scale_log2;
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
__device__ __forceinline__ KeyTiles key_tiles(const KeyWindow &w, int first_pos)
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

// The share of a query tile's nt key tiles (or of a pair's) that CTA `part` of `split`
// has: at least two each, so that both tiles of a pair have one (they visit as many, but
// for one); `parts` CTAs share them.
struct KeyShare {
    int parts, begin, end;
};

__device__ __forceinline__ KeyShare key_share(int nt, int part, int split)
{
    KeyShare s;
    s.parts = max(1, min(split, nt >> 1));
    s.begin = static_cast<int>(static_cast<long long>(nt) * part / s.parts);
    s.end = static_cast<int>(static_cast<long long>(nt) * (part + 1) / s.parts);
    return s;
}

// The state (O, then m and l) that such a CTA leaves of row `row` of its `tiles` query tiles.
__device__ __forceinline__ float *split_row(const PrefillArgs &a, int tiles, unsigned block, unsigned part, int row)
{
    return a.partials + ((static_cast<int64_t>(block) * a.split + part) * (tiles * kRows) + row) * kPartialStride;
}

// For such CTAs' kernels, which mask as under a window: one that hides nothing.
constexpr int kNoWindow = 1 << 30;

// Key tiles that a query tile, or a pair of them, may visit: without a window all of
// the longest sequence's, with one the sinks' and those that 2 tokens_per_tile +
// window - 1 keys touch.
inline int64_t most_key_tiles(const PrefillArgs &a, const KeyWindow &w)
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
// (kBlocks: written while this kernel may be on the GPU already, see grid.cuh.  By ordinary loads
// the attention's loop, which hangs on what stands behind it, takes longer: 4096 of 16384 tokens 1281 us, so 1260.)
template <bool kWin, bool kBlocks, typename KeyTile, typename CopyTile>
__device__ __forceinline__ uint32_t nan_blocks(const PrefillArgs &a, const KeyWindow &w, int tile0, int nt, int p, int lane,
                                               KeyTile key_tile, CopyTile copy_tile)
{
    const uint32_t *tiles = nan_tiles(a);
    auto load = [](auto *p) { return kBlocks ? __ldcg(p) : __ldg(p); };
    bool some = false;
    for (int i = lane; i < nt; i += 32)
        some = some || load(tiles + tile0 + copy_tile(i)) != 0;
    uint32_t hit = 0;
    if (__any_sync(kAll, some)) {
#pragma unroll 1
        for (int i = 0; i < nt; ++i) {
            const int64_t tile = tile0 + copy_tile(i);
            const uint32_t word = load(tiles + tile);
            if (word == 0)
                continue;
#pragma unroll 1
            for (int k = 0; k < kKeys; ++k) {
                const int t = key_tile(i) * kKeys + k;
                if ((word >> (8 * (k >> 5)) & 0xFFu) != 0 && t <= p && (!kWin || t > p - w.window || t < w.sinks))
                    hit |= load(nan_rows(a) + tile * kKeys + k);
            }
        }
    }
    return hit;
}

// The block-scaled FP8 cache's copies record single NaNs of V, behind the words above
// (which are zeros there): a word a tile, then 16 bytes a row, a bit a dim.
__device__ __forceinline__ uint32_t *nan_value_tiles(const PrefillArgs &a)
{
    return nan_tiles(a) + a.rows_cap / kKeys;
}

__device__ __forceinline__ uint8_t *nan_value_rows(const PrefillArgs &a)
{
    return reinterpret_cast<uint8_t *>(nan_value_tiles(a) + a.rows_cap / kKeys);
}

// What they do to the outputs: puts NaNs into the rows of tokens t0 .. t1 - 1 of a chunk, which have
// been written, where they see one (the whole CTA of `threads`).
template <bool kWin>
__device__ __forceinline__ void put_nans_of(const PrefillArgs &a, const KeyWindow &w, int b, int h, int t0, int t1, int threads)
{
    const int q0 = a.cu_q[b], n = a.cu_q[b + 1] - q0, L = a.seq_lens[b];
    const int off0 = a.tile_off[b], off1 = a.tile_off[b + 1];
    const KeyTiles seq_kt = key_tiles<kWin>(w, L - n), kt = key_tiles<kWin>(w, L - n + t0);
    const int64_t tile0 = off0 + h * ((off1 - off0) / a.hkv);
    const int nt = (L - n + t1 - 1) / kKeys + 1 - kt.skip;
    auto key_tile = [&](int i) { return !kWin || i < kt.first ? i : i + kt.skip; };
    auto copy_tile = [&](int i) {
        const int t = key_tile(i);
        return !kWin || t < seq_kt.first ? t : t - seq_kt.skip;
    };
    bool some = false;
    for (int i = threadIdx.x; i < nt; i += threads)
        some = some || nan_value_tiles(a)[tile0 + copy_tile(i)] != 0;
    if (!__syncthreads_or(some))
        return;
    const uint32_t *rows = reinterpret_cast<const uint32_t *>(nan_value_rows(a));
    // a thread a (token, 32 dims)
    for (int x = threadIdx.x; x < 4 * (t1 - t0); x += threads) {
        const int t = t0 + (x >> 2), p = L - n + t, j = x & 3;
        uint32_t hit = 0;
#pragma unroll 1
        for (int i = 0; i < nt; ++i) {
            const int64_t tile = tile0 + copy_tile(i);
            const uint32_t word = nan_value_tiles(a)[tile];
            if (word == 0)
                continue;
#pragma unroll 1
            for (int k = 0; k < kKeys; ++k) {
                const int key = key_tile(i) * kKeys + k;
                if ((word >> (8 * (k >> 5)) & 0xFFu) != 0 && key <= p && (!kWin || key > p - w.window || key < w.sinks))
                    hit |= rows[(tile * kKeys + k) * 4 + j];
            }
        }
        const int64_t row = (static_cast<int64_t>(q0) + t) * a.hq + static_cast<int64_t>(h) * a.group;
#pragma unroll 1
        for (int d = 0; hit != 0 && d < 32; ++d)
            for (int g = 0; ((hit >> d) & 1u) && g < a.group; ++g) {
                if (a.out_f32)
                    static_cast<float *>(a.out)[(row + g) * kHeadDim + 32 * j + d] = NAN;
                else
                    static_cast<__nv_bfloat16 *>(a.out)[(row + g) * kHeadDim + 32 * j + d] = __float2bfloat16_rn(NAN);
            }
    }
}

// Those of an attention CTA's query tiles (`tiles` of them).  Out of line, and from the block's
// number on, so that the attention's loop keeps nothing for it.
template <bool kWin>
__device__ __noinline__ void put_nans(const PrefillArgs &a, const KeyWindow &w, int tiles, int threads)
{
    const int per = (a.max_tiles + tiles - 1) / tiles;
    const int bh = blockIdx.x / per, first = (per - 1 - (static_cast<int>(blockIdx.x) - bh * per)) * tiles;
    const int b = bh / a.hkv, h = bh - b * a.hkv;
    const int n = a.cu_q[b + 1] - a.cu_q[b];
    put_nans_of<kWin>(a, w, b, h, first * a.tokens_per_tile, min(n, (first + tiles) * a.tokens_per_tile), threads);
}

// 128-row tiles of sequence b's widened region (all its kv heads): zero for a
// sequence with an empty or inconsistent chunk.
template <bool kWin>
__device__ __forceinline__ long long region_tiles(const PrefillArgs &a, const KeyWindow &w, int b)
{
    const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1];
    const int L = a.seq_lens[b];
    if (q1 - q0 <= 0 || !sequence_ok(a, b, q0, q1, L, false))
        return 0;
    return static_cast<long long>(a.hkv) * ((L + kKeys - 1) / kKeys - key_tiles<kWin>(w, L - (q1 - q0)).skip);
}

}  // namespace pkv
