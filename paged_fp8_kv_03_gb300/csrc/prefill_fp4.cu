// paged_prefill_fp4: the widening of the 4-bit cache to 16-bit copies (K as bf16,
// V as f16: e s has 6 significant bits, exact in both), and the attention over
// them with a bf16 output, on the 5th-generation tensor cores.
//
// What bounds the attention.  A tile of 128 rows (tokens x query heads of the group) and
// 128 keys costs the tensor cores 2 x 128^3 multiply-adds and the softmax 128^2
// exponentials.  One f16 part of P is enough under a bf16 output's 2^-8 (the
// weights are rounded once, 2^-11 each), so the products are two thirds of
// those that a second part would need, and the softmax must keep up with
// them: per score a half each of max, fma, add and conversion, and one
// exponential at a quarter of an SMSP's issue rate or less.
//
// So one CTA takes two query tiles, A and B, of the same kv head.  Each has its
// own softmax warpgroup (one row a thread: no exchange between warps), its own
// scores in TMEM and its own accumulator, and while the tensor cores work for
// one tile the other's softmax runs; each K and V tile brought on chip serves
// both.  P overwrites the first half of its scores' columns in two steps, so
// that the products with V start on the first 64 keys while the last 64 are
// still being exponentiated.
//   warp 0      TMA: two query tiles, then K and V tiles into 2-stage rings
//   warp 1      tcgen05.mma, in the order  S_A(j+1) after O_A += P_A(j) V(j),
//               S_B(j+1) after O_B += P_B(j) V(j)
//   warps 2-5   softmax and output of tile A,  warps 6-9 of tile B
// The tensor cores add with truncation, up to 2^-23 of the sum an addition of 16
// keys, so a chain of additions must not grow with the context: every kFold2 key
// tiles (1024 additions, 2^-13) a row's accumulator is added in fp32 to what earlier
// folds have left, the sum's bf16 rounding is kept in the row's place in the output,
// and the chain goes on from the rest, which fp32 holds exactly and which is at
// most 2^-8 of the sum.  (512K tokens of V of one sign, 128 of them two thirds of
// the sum: 6.8e-5 too small, in one chain 1.07e-3.)
// Every wait is bounded (2 s): on expiry the CTA sets PKV_DEVERR_TIMEOUT,
// drains its own copies and MMAs, frees TMEM and exits.
#include <math.h>
#include <mutex>

#include "context.h"
#include "prefill.cuh"

namespace pkv {

namespace {

constexpr int kStages2 = 2;                      // K and V rings
constexpr int kWarp0 = 2;                        // first softmax warp
constexpr int kThreads2 = 32 * (kWarp0 + 8);
// P = 2^(score - m) with a reference m that is kLift below the row's maximum (log2
// units) when it is set, and moves only when it is exceeded by more than kMoveMax: P <=
// 2^15.9 is within f16, and moving it costs a pass over the accumulator.  The lift keeps small
// weights off f16's lower end, where 2^-25 is lost: 2^-27 of the largest weight a key, for
// 128K keys 2^-10 of all, under the output's 2^-8.  (A lift of 6 takes 3% longer with 16K
// keys, 6% with a window.)  Beyond them it grows with the keys' logarithm, so that all
// of them (up to 2^27 keys) still lose 2^-10 at most.
constexpr float kMoveMax = 15.9f, kLift = 2.f;
// Key tiles of one tensor-core accumulation (1024 additions, as in decode).
constexpr int kFold2 = 128;
constexpr uint32_t kScoreCol = 128, kOutCol = 256;   // tile x: scores at 128 x, accumulator at 256 + 128 x

// Shared memory, offsets from a 1024-byte aligned base.  Operand tiles are
// [2 column blocks][128 rows][128 bytes] with the 128-byte swizzle.
struct P2 {
    static constexpr int kTile = 32768;
    static constexpr int kQ = 0;                           // query tiles A and B
    static constexpr int kK = 2 * kTile;
    static constexpr int kV = kK + kStages2 * kTile;
    static constexpr int kBars = kV + kStages2 * kTile;
    enum {
        Q_FULL, Q_READY = Q_FULL + 2, K_FULL = Q_READY + 2, K_EMPTY = K_FULL + kStages2, V_FULL = K_EMPTY + kStages2,
        V_EMPTY = V_FULL + kStages2, S_FULL = V_EMPTY + kStages2, P_FULL = S_FULL + 2, PV_DONE = P_FULL + 4,
        DRAIN = PV_DONE + 2, kNumBars = DRAIN + 1
    };
    static constexpr int kTmem = kBars + kNumBars * 8;
    static constexpr int kFlag = kTmem + 4;
    static constexpr int kMoved = (kFlag + 4 + 15) / 16 * 16;   // MovedRow [2][kRows]
    static constexpr int kEnd = kMoved + 2 * kRows * static_cast<int>(sizeof(MovedRow));
    static constexpr size_t bytes(bool folds) { return static_cast<size_t>(folds ? kEnd : kFlag + 4) + 1024; }
};
static_assert(P2::bytes(true) <= 232448, "prefill tile buffers exceed the shared memory of one CTA");

// ---------------------------------------------------------------------- widening
// The 16-bit copies' regions are laid out as the FP8 widening kernel's: tile_off
// is the prefix sum of the sequences' 128-row tiles (a region past the workspace
// is flagged), K and V of a sequence's kv head in consecutive rows, zero rows up
// to a whole tile.  Keys that no query sees under the window get no tile, or
// zero rows in a tile others are seen of.  A NaN block of V is widened to zeros
// and recorded.
//
// Bytes bound it: 144 of the cache to 512 of the copies a row.  A CTA takes a
// tile (or a quarter of one, where there are few), so what the tile belongs to is
// found once; a thread takes 8 values of kRowsEach of its rows, of K and of V, 16
// lanes write a row's 256 bytes.
template <int kRowsEach>
__global__ void __launch_bounds__(256) kv_widen_fp4_kernel(const PrefillArgs a, const Fp4Window win)
{
    constexpr int kPieces = 8 / kRowsEach;               // CTAs' steps a tile
    static_assert(kPieces == 1 || kPieces == 4, "a tile's word has a byte a piece");
    extern __shared__ int off[];                         // [batch + 1], then 8 warp sums
    int *warp_sum = off + a.batch + 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long cap_tiles = a.rows_cap / kKeys;
    const int most = static_cast<int>(cap_tiles + 1);    // sums saturate just past the workspace
    {
        const int chunk = (a.batch + 255) / 256;
        const int b0 = min(a.batch, tid * chunk), b1 = min(a.batch, b0 + chunk);
        long long local = 0;
        for (int b = b0; b < b1; ++b)
            local += region_tiles<true>(a, win, b);
        const int loc = static_cast<int>(local < most ? local : most);
        int incl = loc;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kAll, incl, o);
            if (lane >= o)
                incl = min(incl + v, most);
        }
        if (lane == 31)
            warp_sum[warp] = incl;
        __syncthreads();
        int base = 0;
        for (int w = 0; w < warp; ++w)
            base = min(base + warp_sum[w], most);
        int run = min(base + incl - loc, most);
        for (int b = b0; b < b1; ++b) {
            off[b] = run;
            run = static_cast<int>(min(run + region_tiles<true>(a, win, b), static_cast<long long>(most)));
        }
        if (tid == 255)
            off[a.batch] = min(base + incl, most);
        __syncthreads();
        if (blockIdx.x == 0)
            for (int b = tid; b <= a.batch; b += 256) {
                a.tile_off[b] = off[b];
                if (b < a.batch && off[b + 1] > cap_tiles && off[b + 1] > off[b] && a.err)
                    atomicOr(a.err, PKV_DEVERR_SEQLEN);  // its region does not fit the workspace
            }
    }
    const int part = tid & 15;                           // dims 8 part .. 8 part + 7
    const int tiles = static_cast<int>(min(static_cast<long long>(off[a.batch]), cap_tiles));
    for (int piece = blockIdx.x; piece < tiles * kPieces; piece += gridDim.x) {
        const int tile = piece / kPieces, first = (piece % kPieces) * 16 * kRowsEach + (tid >> 4);   // first row
        int lo = 0, hi = a.batch - 1;                    // the sequence whose region holds the tile
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (off[mid] <= tile)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int b = lo;
        if (off[b + 1] > cap_tiles)
            continue;                                    // region past the workspace: flagged above
        const int L = __ldg(a.seq_lens + b), lp = seq_page_log2(a, b);
        const KeyTiles kt = key_tiles<true>(win, L - (__ldg(a.cu_q + b + 1) - __ldg(a.cu_q + b)));
        const int per_head = (off[b + 1] - off[b]) / a.hkv;
        const int h = (tile - off[b]) / per_head, vt = (tile - off[b]) - h * per_head;
        const int key0 = (vt < kt.first ? vt : vt + kt.skip) * kKeys;
        uint32_t kc[kRowsEach], vc[kRowsEach];
        uint8_t ks[kRowsEach], vs[kRowsEach];
        uint32_t nans = 0;                               // V's, a bit a row
#pragma unroll
        for (int i = 0; i < kRowsEach; ++i) {
            const int t = key0 + first + 16 * i;
            kc[i] = vc[i] = 0;
            ks[i] = vs[i] = 0;
            if (t < L && (t < kt.sinks || t >= kt.from)) {
                int pg, row;
                if (seq_token_page(a, b, lp, t, pg, row)) {
                    const int64_t at = fp4_tile_offset(pg, h, row, a.hkv, a.page_size);
                    const int64_t codes = at + (row & 15) * 64 + 4 * part, scale = at + kFp4Codes + (row & 15) * 8 + (part >> 1);
                    kc[i] = __ldg(reinterpret_cast<const uint32_t *>(a.k_cache + codes));
                    vc[i] = __ldg(reinterpret_cast<const uint32_t *>(a.v_cache + codes));
                    ks[i] = __ldg(a.k_cache + scale);
                    vs[i] = __ldg(a.v_cache + scale);
                    if ((vs[i] & 0x7F) == 0x7F) {
                        vs[i] = 0;
                        nans |= 1u << i;
                    }
                } else if (part == 0 && a.err) {
                    atomicOr(a.err, PKV_DEVERR_PAGE);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kRowsEach; ++i) {
            const int64_t at = (static_cast<int64_t>(tile) * kKeys + first + 16 * i) * kHeadDim + 8 * part;
            const __half2 sk = __float2half2_rn(e4m3_value(ks[i])), sv = __float2half2_rn(e4m3_value(vs[i]));
            uint32_t k[4], v[4];
            e2m1x8_to_f16x8(kc[i], k);
            e2m1x8_to_f16x8(vc[i], v);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 kf = __half22float2(__hmul2(*reinterpret_cast<const __half2 *>(&k[e]), sk));
                const __nv_bfloat162 kb = __floats2bfloat162_rn(kf.x, kf.y);
                const __half2 vh = __hmul2(*reinterpret_cast<const __half2 *>(&v[e]), sv);
                k[e] = *reinterpret_cast<const uint32_t *>(&kb);
                v[e] = *reinterpret_cast<const uint32_t *>(&vh);
            }
            *reinterpret_cast<uint4 *>(a.k16 + at) = make_uint4(k[0], k[1], k[2], k[3]);
            *reinterpret_cast<uint4 *>(a.v16 + at) = make_uint4(v[0], v[1], v[2], v[3]);
        }
        const bool any = __syncthreads_or(static_cast<int>(nans)) != 0;
        if (tid == 0) {
            if (kPieces == 1)
                nan_tiles(a)[tile] = any ? 0x01010101u : 0u;
            else
                reinterpret_cast<uint8_t *>(nan_tiles(a) + tile)[piece % kPieces] = any;
        }
        if (any) {
#pragma unroll
            for (int i = 0; i < kRowsEach; ++i) {
                // even lanes of a row's 16 stand for its blocks
                uint32_t x = __ballot_sync(kAll, (nans >> i) & 1u) >> (lane & 16) & 0x5555u;
                x = (x | x >> 1) & 0x3333u;
                x = (x | x >> 2) & 0x0F0Fu;
                x = (x | x >> 4) & 0xFFu;
                if (part == 0)
                    nan_rows(a)[static_cast<int64_t>(tile) * kKeys + first + 16 * i] = static_cast<uint8_t>(x);
            }
        }
    }
}

// ---------------------------------------------------------------------- attention
__device__ __forceinline__ void bf16x8(const uint4 &u, float (&v)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = __uint_as_float((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
}

// What a softmax thread of the folding kernel keeps in shared memory.
__device__ __forceinline__ volatile MovedRow &moved_row()
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    return reinterpret_cast<volatile MovedRow *>(smem + P2::kMoved)[threadIdx.x - 32 * kWarp0];
}

// Adds a row's accumulator and its sum l of the weights (m: their reference) to what
// earlier folds have left (old): the bf16 rounding of the accumulators' sum goes
// to the output, the rest back into the accumulator, the last time all of it.
// Returns the sum of all.  Out of line, for the loop around it.
__device__ __noinline__ float fold(uint32_t o_tm, float m, float l, bool old, bool last)
{
    volatile MovedRow &st = moved_row();
    uint4 *dst = st.out;
    const float back = old ? ex2_approx(st.m - m) : 0.f;
    l = old ? st.l * back + l : l;
    st.m = m;
    st.l = l;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
        uint4 was[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            was[i] = old && dst ? dst[2 * c + i] : make_uint4(0, 0, 0, 0);
        uint32_t o[16];
        tc::ld16(o_tm + 16 * c, o);
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float y[8];
            bf16x8(was[i], y);
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t &o0 = o[8 * i + 2 * e], &o1 = o[8 * i + 2 * e + 1];
                const float s0 = __uint_as_float(o0) + y[2 * e] * back;
                const float s1 = __uint_as_float(o1) + y[2 * e + 1] * back;
                const __nv_bfloat162 b = __floats2bfloat162_rn(s0, s1);
                w[e] = last ? 0u : *reinterpret_cast<const uint32_t *>(&b);
                o0 = __float_as_uint(s0 - __uint_as_float(w[e] << 16));
                o1 = __float_as_uint(s1 - __uint_as_float(w[e] & 0xFFFF0000u));
            }
            if (dst && !last)
                dst[2 * c + i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        tc::st16(o_tm + 16 * c, o);
    }
    tc::wait_st();
    return l;
}

// The lift where a row visits nt key tiles: one more from 1025, 2049, .. on.
template <bool kFolds>
__device__ __forceinline__ float lift_of(int nt)
{
    return kFolds ? kLift + static_cast<float>(min(max(22 - __clz(nt - 1), 0), 10)) : kLift;
}

// kFolds: for calls in which a query tile may visit more than kFold2 key tiles.
template <bool kWin, bool kFolds>
__global__ void __launch_bounds__(kThreads2, 1)
    paged_prefill_pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                              const __grid_constant__ CUtensorMap tm_v, const PrefillArgs a, const Fp4Window win)
{
    // (sequence, kv head)-major, heaviest pairs of tiles first within each
    const int pairs = (a.max_tiles + 1) >> 1;
    const int bh = blockIdx.x / pairs;
    const int qp = pairs - 1 - (blockIdx.x - bh * pairs);
    const int b = bh / a.hkv;
    const int h = bh - b * a.hkv;
    const int G = a.group, tpt = a.tokens_per_tile;
    const int q0 = __ldg(a.cu_q + b), q1 = __ldg(a.cu_q + b + 1);
    const int n = q1 - q0;
    const int L = __ldg(a.seq_lens + b);
    if (!sequence_ok(a, b, q0, q1, L, qp == 0 && h == 0 && threadIdx.x == 0))
        return;
    const int off0 = __ldg(a.tile_off + b), off1 = __ldg(a.tile_off + b + 1);
    const KeyTiles seq_kt = key_tiles<kWin>(win, L - n);
    if (off1 > a.rows_cap / 128 || off1 - off0 != a.hkv * ((L + kKeys - 1) / kKeys - seq_kt.skip))
        return;
    const int row0 = off0 * 128 + h * (off1 - off0) / a.hkv * 128;   // first row of this kv head's copy
    const int t0 = qp * 2 * tpt;                         // first token of the pair in the chunk
    if (t0 >= n)
        return;
    const int nv0 = min(tpt, n - t0), nv1 = max(0, min(tpt, n - t0 - tpt));   // tokens of A and of B
    const int pos0 = L - n + t0;                         // position of the first one
    const KeyTiles kt = key_tiles<kWin>(win, pos0);      // what some row of the pair sees
    const int nt0 = (pos0 + nv0 - 1) / kKeys + 1 - kt.skip;   // key tiles that A visits
    const int nt1 = nv1 > 0 ? (pos0 + tpt + nv1 - 1) / kKeys + 1 - kt.skip : 0;
    const int nt = max(nt0, nt1);
    // the i-th one, and where it lies in the sequence's copy
    auto key_tile = [&](int i) { return !kWin || i < kt.first ? i : i + kt.skip; };
    auto copy_tile = [&](int i) {
        const int t = key_tile(i);
        return !kWin || t < seq_kt.first ? t : t - seq_kt.skip;
    };

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_addr(smem);
    auto bar = [&](int i) { return sb + P2::kBars + 8u * i; };
    uint64_t *bar_ptr = reinterpret_cast<uint64_t *>(smem + P2::kBars);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + P2::kTmem);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + P2::kFlag);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < P2::kNumBars; ++i)
            mbar_init(bar(i), i >= P2::Q_READY && i < P2::K_FULL ? 4 : (i >= P2::P_FULL && i < P2::PV_DONE ? 4 : 1));
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(tslot, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = *tslot;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA
        if (lane == 0) {
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
            const uint64_t pol = l2_policy_evict_first();
            const int nq = nv1 > 0 ? 2 : 1;
            for (int x = 0; x < nq; ++x) {
                mbar_arrive_expect_tx(bar(P2::Q_FULL + x), 2u * 128u * G * tpt);
                tma_load_3d(sb + P2::kQ + x * P2::kTile, &tm_q, 0, h * G, q0 + t0 + x * tpt, bar(P2::Q_FULL + x), pol);
                tma_load_3d(sb + P2::kQ + x * P2::kTile + 16384, &tm_q, 64, h * G, q0 + t0 + x * tpt,
                            bar(P2::Q_FULL + x), pol);
            }
            uint32_t karmed[kStages2] = {}, varmed[kStages2] = {};
            bool ok = true;
            for (int t = 0; ok && t < nt; ++t) {
                const int s = t % kStages2;
                const int row = row0 + copy_tile(t) * kKeys;
                if (t >= kStages2 && !pwait(bar(P2::K_EMPTY + s), ((t / kStages2) - 1) & 1, abort_flag, a.err)) {
                    ok = false;
                    break;
                }
                // (test facility: the withheld CTA never arms or loads its first K tile)
                if (t > 0 || static_cast<int>(blockIdx.x) != a.withhold_block) {
                    mbar_arrive_expect_tx(bar(P2::K_FULL + s), P2::kTile);
                    karmed[s] = static_cast<uint32_t>(t / kStages2) + 1;
                    tma_load_3d_plain(sb + P2::kK + s * P2::kTile, &tm_k, 0, row, 0, bar(P2::K_FULL + s));
                    tma_load_3d_plain(sb + P2::kK + s * P2::kTile + 16384, &tm_k, 64, row, 0, bar(P2::K_FULL + s));
                }
                if (t >= kStages2 && !pwait(bar(P2::V_EMPTY + s), ((t / kStages2) - 1) & 1, abort_flag, a.err)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(bar(P2::V_FULL + s), P2::kTile);
                varmed[s] = static_cast<uint32_t>(t / kStages2) + 1;
                tma_load_3d_plain(sb + P2::kV + s * P2::kTile, &tm_v, 0, row, 0, bar(P2::V_FULL + s));
                tma_load_3d_plain(sb + P2::kV + s * P2::kTile + 16384, &tm_v, 64, row, 0, bar(P2::V_FULL + s));
            }
            // No copy may still be landing when the CTA leaves.
            for (int x = 0; x < nq; ++x)
                pwait(bar(P2::Q_FULL + x), 0, abort_flag, a.err, false);
            for (int s = 0; s < kStages2; ++s) {
                if (karmed[s])
                    pwait(bar(P2::K_FULL + s), (karmed[s] - 1) & 1, abort_flag, a.err, false);
                if (varmed[s])
                    pwait(bar(P2::V_FULL + s), (varmed[s] - 1) & 1, abort_flag, a.err, false);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issue
        // The whole warp runs this converged; one elected lane issues.
        const uint32_t id_qk = tc::idesc_bf16_f32(kRows, kKeys, false);
        const uint32_t id_pv = tc::idesc_f16_f32(kRows, kHeadDim, true);
        uint64_t qdesc[2], kdesc[kStages2], vdesc[kStages2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            qdesc[i] = kmajor_base(sb + P2::kQ + i * P2::kTile);
#pragma unroll
        for (int i = 0; i < kStages2; ++i) {
            kdesc[i] = kmajor_base(sb + P2::kK + i * P2::kTile);
            vdesc[i] = vmn_base(sb + P2::kV + i * P2::kTile);
        }
        const bool leader = elect_one();
        bool ok = true;
        // scores of tile x against key tile j
        auto score = [&](int x, int j, bool last) {
            const int s = j % kStages2;
            if (!wwait(bar(P2::K_FULL + s), (j / kStages2) & 1, abort_flag, a.err, lane))
                return false;
            tc::fence_after();
            if (leader) {
#pragma unroll
                for (int d = 0; d < 8; ++d)             // dims 16d..16d+15
                    tc::mma_ss(tm + kScoreCol * x, kmajor_step(qdesc[x], d), kmajor_step(kdesc[s], d), id_qk, d > 0);
                tc::commit(bar_ptr + P2::S_FULL + x);
                if (last)
                    tc::commit(bar_ptr + P2::K_EMPTY + s);
            }
            __syncwarp();
            return true;
        };
        // O += P V of tile x, key tile j: keys 16d..16d+15 of P in columns 8d ..
        auto output = [&](int x, int j, bool last) {
            const int s = j % kStages2;
            if (!wwait(bar(P2::V_FULL + s), (j / kStages2) & 1, abort_flag, a.err, lane))
                return false;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (!wwait(bar(P2::P_FULL + 2 * x + half), j & 1, abort_flag, a.err, lane))
                    return false;
                tc::fence_after();
                if (leader) {
#pragma unroll
                    for (int d = 4 * half; d < 4 * half + 4; ++d)
                        tc::mma_ts(tm + kOutCol + kScoreCol * x, tm + kScoreCol * x + 8 * d, vmn_step(vdesc[s], d),
                                   id_pv, j > 0 || d > 0 ? 1u : 0u);
                    if (half == 1) {
                        tc::commit(bar_ptr + P2::PV_DONE + x);
                        if (last)
                            tc::commit(bar_ptr + P2::V_EMPTY + s);
                    }
                }
                __syncwarp();
            }
            return true;
        };
        ok = wwait(bar(P2::Q_READY), 0, abort_flag, a.err, lane) && score(0, 0, nt1 == 0);
        if (ok && nt1 > 0)
            ok = wwait(bar(P2::Q_READY + 1), 0, abort_flag, a.err, lane) && score(1, 0, true);
        for (int j = 0; ok && j < nt; ++j) {
            if (j < nt0)
                ok = output(0, j, j >= nt1) && (j + 1 >= nt0 || score(0, j + 1, j + 1 >= nt1));
            if (ok && j < nt1)
                ok = output(1, j, true) && (j + 1 >= nt1 || score(1, j + 1, true));
        }
        // Every MMA issued has finished before TMEM is released.
        if (leader) {
            tc::commit(bar_ptr + P2::DRAIN);
            pwait(bar(P2::DRAIN), 0, abort_flag, a.err, false);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax + output
        const int x = (warp - kWarp0) >> 2;              // the warpgroup's tile
        const int qtr = warp & 3;                        // TMEM lane quarter of this warp
        const int row = qtr * 32 + lane;
        const int nvx = x ? nv1 : nv0, ntx = x ? nt1 : nt0;
        const int tl = row / G;
        const int g = row - tl * G;
        const bool valid = row < G * tpt && tl < nvx;
        const int p_row = pos0 + x * tpt + (valid ? tl : nvx - 1);   // padding rows mirror the last row
        const float sl2 = score_factor(a, h);
        const uint32_t s_tm = tm + (static_cast<uint32_t>(qtr * 32) << 16) + kScoreCol * x;
        const uint32_t o_tm = s_tm + kOutCol;
        float m = -INFINITY, l = 0.f;
        if (kFolds) {
            const int64_t orow = (static_cast<int64_t>(q0) + t0 + x * tpt + tl) * a.hq + h * G + g;
            moved_row().out =
                valid ? reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + orow * kHeadDim) : nullptr;
        }
        bool ok = ntx > 0 && wwait(bar(P2::Q_FULL + x), 0, abort_flag, a.err, lane);
        if (ok) {
            // rows past the G x tpt that the copy fills are zeroed
            if (row >= G * tpt) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint4 *qrow = reinterpret_cast<uint4 *>(smem + P2::kQ + x * P2::kTile + half * 16384 + row * 128);
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        qrow[c] = make_uint4(0, 0, 0, 0);
                }
            }
            fence_proxy_async_smem();     // generic-proxy writes -> visible to the tensor cores
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(P2::Q_READY + x));
        }
        for (int j = 0; ok && j < ntx; ++j) {
            // (S_{j-1} came behind PV_{j-2}: so PV_DONE's phase is that of PV_{j-1})
            if (kFolds && j > 0 && j % kFold2 == 0) {
                if (!wwait(bar(P2::PV_DONE + x), (j - 1) & 1, abort_flag, a.err, lane)) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                fold(o_tm, m, l, j > kFold2, false);
                l = 0.f;
            }
            if (!wwait(bar(P2::S_FULL + x), j & 1, abort_flag, a.err, lane)) {
                ok = false;
                break;
            }
            tc::fence_after();
            uint32_t v[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                tc::ld32(s_tm + 32 * c, v[c]);
            tc::wait_ld();
            // hidden keys become -inf: after the row's position, or before its
            // window and behind the sinks
            const int key0 = key_tile(j) * kKeys;
            const int vis = p_row - key0;
            if (vis < kKeys - 1) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (vis < 32 * c + 31) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (32 * c + k > vis)
                                v[c][k] = __float_as_uint(-INFINITY);
                    }
            }
            if (kWin) {
                const int out = vis - win.window, snk = win.sinks - key0;
                if (out >= 0 && snk < kKeys) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (out >= 32 * c && snk < 32 * c + 32) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (32 * c + k <= out && 32 * c + k >= snk)
                                    v[c][k] = __float_as_uint(-INFINITY);
                        }
                }
            }
            float mx[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                mx[k] = max3(__uint_as_float(v[0][2 * k]), __uint_as_float(v[0][2 * k + 1]), -INFINITY);
#pragma unroll
            for (int k = 8; k < 64; ++k)
                mx[k & 7] = max3(mx[k & 7], __uint_as_float(v[k >> 4][2 * (k & 15)]),
                                 __uint_as_float(v[k >> 4][2 * (k & 15) + 1]));
            const float top = fmaxf(max3(mx[0], mx[1], mx[2]), max3(max3(mx[3], mx[4], mx[5]), mx[6], mx[7])) * sl2;
            const bool need = top > m + kMoveMax;
            if (__any_sync(kAll, need)) {
                const float mn = need ? top - lift_of<kFolds>(ntx) : m;
                const float f = need ? ex2_approx(m - mn) : 1.f;
                m = mn;
                l *= f;
                if (j > 0) {                               // the accumulator holds tiles 0 .. j-1
                    if (!wwait(bar(P2::PV_DONE + x), (j - 1) & 1, abort_flag, a.err, lane)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        uint32_t o[16];
                        tc::ld16(o_tm + 16 * c, o);
                        tc::wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tc::st16(o_tm + 16 * c, o);
                    }
                    tc::wait_st();
                }
            }
            // P = 2^(s sl2 - m) as f16 pairs over the scores' first 64 columns
            // (a row that has seen nothing yet: every P is 2^-inf)
            const float ms = kWin && m == -INFINITY ? 0.f : m;
            const uint64_t sl2x2 = f2_pack(sl2, sl2), nmm = f2_pack(-ms, -ms);
            uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t ph[32];
#pragma unroll
                for (int q = 0; q < 32; ++q) {
                    const int c = 2 * half + (q >> 4), k = 2 * (q & 15);
                    const float2 y = f2_unpack(
                        f2_fma(f2_pack(__uint_as_float(v[c][k]), __uint_as_float(v[c][k + 1])), sl2x2, nmm));
                    const float p0 = ex2_approx(y.x), p1 = ex2_approx(y.y);
                    ls[q & 3] = f2_add(ls[q & 3], f2_pack(p0, p1));
                    ph[q] = f32x2_to_f16x2(p0, p1);
                }
                tc::st32(s_tm + 32 * half, ph);
                tc::wait_st();
                tc::fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(P2::P_FULL + 2 * x + half));
            }
            const float2 s0 = f2_unpack(f2_add(ls[0], ls[1])), s1 = f2_unpack(f2_add(ls[2], ls[3]));
            l += (s0.x + s0.y) + (s1.x + s1.y);
        }
        if (ok && wwait(bar(P2::PV_DONE + x), (ntx - 1) & 1, abort_flag, a.err, lane)) {
            tc::fence_after();
            if (kFolds && ntx > kFold2)
                l = fold(o_tm, m, l, true, true);
            const float inv = __ldg(a.v_scale + h) / l;
            const uint32_t nans = nan_blocks<kWin>(a, win, row0 / kKeys, ntx, p_row, lane, key_tile, copy_tile);
            const int64_t orow = (static_cast<int64_t>(q0) + t0 + x * tpt + tl) * a.hq + h * G + g;
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + orow * kHeadDim);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                tc::ld32(o_tm + 32 * c, o);
                tc::wait_ld();
                if (!valid)
                    continue;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t w[4];
                    const float f = (nans >> (2 * c + (k >> 1))) & 1u ? NAN : inv;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(o[8 * k + 2 * e]) * f,
                                                                        __uint_as_float(o[8 * k + 2 * e + 1]) * f);
                        w[e] = *reinterpret_cast<const uint32_t *>(&b2);
                    }
                    dst[4 * c + k] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
    }

    tc::fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after();
        tc::tmem_dealloc(tm, 512);
    }
}

std::mutex g_pair_mu;
unsigned long long g_pair_ctx[64][4] = {};   // per device and kernel: the context its limit was raised in

}  // namespace

// The widening launch of the 4-bit calls.
cudaError_t launch_widen_fp4(const PrefillArgs &a, const Fp4Window &win, cudaStream_t stream)
{
    const int64_t tiles = a.rows_cap / kKeys, most = static_cast<int64_t>(device_sm_count()) * 8;
    const size_t smem = (static_cast<size_t>(a.batch) + 1 + 8) * sizeof(int);
    if (tiles * 4 <= most)                               // (CTA 0 always lays out the regions)
        kv_widen_fp4_kernel<2><<<static_cast<unsigned>(tiles < 1 ? 1 : tiles * 4), 256, smem, stream>>>(a, win);
    else
        kv_widen_fp4_kernel<8><<<static_cast<unsigned>(tiles < most ? tiles : most), 256, smem, stream>>>(a, win);
    return cudaGetLastError();
}

// The attention launch alone: the widening kernel has been enqueued before.
cudaError_t launch_prefill_pair(const PrefillArgs &a, const Fp4Window &win, const CUtensorMap &tm_q,
                                const CUtensorMap &tm_k16, const CUtensorMap &tm_v16, cudaStream_t stream)
{
    // The folding kernel takes longer even where it folds nothing (4096 of 16384 tokens, 64
    // query heads: 1172 us instead of 1153), and where it does (2048 of 131072: 6.01 ms, in
    // one chain 5.74; 1024 of 524288: 12.4 and 11.8).
    const bool folds = most_key_tiles(a, win) > kFold2;
    const int which = (win.window > 0 ? 1 : 0) + (folds ? 2 : 0);
    const auto kernel = win.window > 0 ? (folds ? paged_prefill_pair_kernel<true, true> : paged_prefill_pair_kernel<true, false>)
                                       : (folds ? paged_prefill_pair_kernel<false, true> : paged_prefill_pair_kernel<false, false>);
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    {
        unsigned long long ctx = 0;
        const bool known = current_context_id(&ctx);
        std::lock_guard<std::mutex> lk(g_pair_mu);
        if (!known || g_pair_ctx[dev][which] != ctx) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(P2::bytes(folds)));
            if (e != cudaSuccess)
                return e;
            g_pair_ctx[dev][which] = known ? ctx : 0;
        }
    }
    const int64_t grid = static_cast<int64_t>(a.batch) * a.hkv * ((a.max_tiles + 1) / 2);
    kernel<<<static_cast<unsigned>(grid), kThreads2, P2::bytes(folds), stream>>>(tm_q, tm_k16, tm_v16, a, win);
    return cudaGetLastError();
}

}  // namespace pkv
