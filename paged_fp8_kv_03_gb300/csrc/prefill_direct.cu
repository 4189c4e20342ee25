// Prefill attention over the block-scaled FP8 cache itself, where few rows have a long past:
// instead of 16-bit copies that one launch writes and another reads (768 bytes a key and head
// where the codes are 256), eight more warps widen the codes in shared memory.
//
// One CTA has two query tiles, A and B, of one kv head and a share of their keys, and leaves
// their rows' sums; prefill_join_fp8b_kernel adds them up.  20 warps:
//   warp 0       TMA: the query tiles
//   warp 1       tcgen05.mma, in the order  S_A(j+1) after O_A += P_A(j) V(j),
//                S_B(j+1) after O_B += P_B(j) V(j)
//   warps 2, 3   TMA: K's codes, and V's, into the second half of the tiles that they become
//   warps 4-7    softmax of tile A,  warps 8-11 of tile B, a row a thread
//   warps 12-15  widen K's tiles in place,  warps 16-19 V's
// A key tile takes 3.1 us, where attention over copies takes 1.3: the widening's instructions
// and the softmax's share the issue slots (56% used), and their code the instruction cache.
// What it saves is the copies: 9 x 32 tokens of 32 query and 8 kv heads past 8192 116 us, else
// 160; 16 tokens of 64 and 8 past 131072 177 and 257.
// A kernel of its own: as an instance of the one that reads copies, that one's other
// instances took 2% longer.
// Every wait is bounded (2 s): on expiry the CTA sets PKV_DEVERR_TIMEOUT, drains its own copies
// and MMAs, frees TMEM and exits.
#include <math.h>
#include <mutex>

#include "context.h"
#include "prefill.cuh"
#include "widen_fp8b.cuh"

namespace pkv {

namespace {

constexpr int kStages2 = 2;                      // K and V rings
// A warpgroup that issues copies and products, two of softmax, one that widens K and one for V,
// and the registers a thread of each (640 threads have 96 to share).
constexpr int kWarpS = 4, kThreadsS = 32 * 20, kRegsIssue = 32, kRegsSoftmax = 160, kRegsWiden = 64;
static_assert(kRegsIssue + 2 * kRegsSoftmax + 2 * kRegsWiden <= 5 * 96, "the warpgroups' registers");
template <int kRegs>
__device__ __forceinline__ void fewer_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void more_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// P = 2^(score - m), with m kLift below the row's maximum when it is set, moved when that
// exceeds it by more than kMoveMax: P is within f16, and what its lower end loses is 2^-27 of the
// largest weight a key: of the output, that much of this weight times the sum of |v|, which is under
// its 2^-8 unless small weights meet values larger by as much.  (Decode refers its weights to what they
// contribute; here the row's one reference comes from the scores.)
constexpr float kMoveMax = 15.9f, kLift = 2.f;
constexpr uint32_t kScoreCol = 128, kOutCol = 256;   // tile x: scores at 128 x, accumulator at 256 + 128 x

// Shared memory, offsets from a 1024-byte aligned base.
struct D {
    static constexpr int kTile = 32768;
    static constexpr int kQ = 0;                           // query tiles A and B
    static constexpr int kK = 2 * kTile;
    static constexpr int kV = kK + kStages2 * kTile;
    static constexpr int kBars = kV + kStages2 * kTile;
    enum {
        Q_FULL, Q_READY = Q_FULL + 2, K_FULL = Q_READY + 2, K_EMPTY = K_FULL + kStages2, V_FULL = K_EMPTY + kStages2,
        V_EMPTY = V_FULL + kStages2, S_FULL = V_EMPTY + kStages2, P_FULL = S_FULL + 2, PV_DONE = P_FULL + 4,
        DRAIN = PV_DONE + 2, CODES = DRAIN + 1, TAKEN = CODES + 2 * kStages2, kNumBars = TAKEN + 2
    };
    static constexpr int kTmem = kBars + kNumBars * 8;
    static constexpr int kFlag = kTmem + 4;
    static constexpr int kFactor = kFlag + 4;              // its entry of v_refs
    static constexpr int kExps = kFactor + 4;              // exponents of K's and V's stages' blocks
    static constexpr size_t kBytes = kExps + 2 * kStages2 * 8 * 4 + 1024;
};
static_assert(D::kBytes <= 232448, "prefill tile buffers exceed the shared memory of one CTA");

__global__ void __launch_bounds__(kThreadsS, 1)
    paged_prefill_direct_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                                const __grid_constant__ CUtensorMap tm_v, const PrefillArgs a, const KeyWindow win)
{
    // (sequence, kv head)-major, heaviest pairs of tiles first within each
    const int pairs = (a.max_tiles + 1) >> 1;
    const int bh = blockIdx.x / pairs;
    const int qp = pairs - 1 - (blockIdx.x - bh * pairs);
    const int b = bh / a.hkv;
    const int h = bh - b * a.hkv;
    const int G = a.group, tpt = a.tokens_per_tile;
    grid_wait();                                         // ahead of all that is read (every CTA, so that this ends after it)
    const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1];
    const int n = q1 - q0;
    const int L = a.seq_lens[b];
    if (!sequence_ok(a, b, q0, q1, L, qp == 0 && h == 0 && threadIdx.x == 0))
        return;
    const int off0 = a.tile_off[b], off1 = a.tile_off[b + 1];
    const KeyTiles seq_kt = key_tiles<true>(win, L - n);
    if (off1 > a.rows_cap / 128 || off1 - off0 != a.hkv * ((L + kKeys - 1) / kKeys - seq_kt.skip))
        return;
    const int row0 = off0 * 128 + h * (off1 - off0) / a.hkv * 128;   // first row of this kv head's copy
    const int t0 = qp * 2 * tpt;                         // first token of the pair in the chunk
    if (t0 >= n)
        return;
    const int nv0 = min(tpt, n - t0), nv1 = max(0, min(tpt, n - t0 - tpt));   // tokens of A and of B
    const int pos0 = L - n + t0;                         // position of the first one
    const KeyTiles kt = key_tiles<true>(win, pos0);      // what some row of the pair sees
    const int all0 = (pos0 + nv0 - 1) / kKeys + 1 - kt.skip;  // key tiles that A visits
    const int all1 = nv1 > 0 ? (pos0 + tpt + nv1 - 1) / kKeys + 1 - kt.skip : 0;
    const KeyShare share = key_share(max(all0, all1), blockIdx.y, a.split);
    if (static_cast<int>(blockIdx.y) >= share.parts)
        return;
    const int nt0 = min(all0, share.end) - share.begin;
    const int nt1 = nv1 > 0 ? min(all1, share.end) - share.begin : 0;
    const int nt = max(nt0, nt1);
    // the i-th one, and where it lies in the sequence's copy
    auto key_tile = [&](int j) {
        const int i = share.begin + j;
        return i < kt.first ? i : i + kt.skip;
    };
    auto copy_tile = [&](int i) {
        const int t = key_tile(i);
        return t < seq_kt.first ? t : t - seq_kt.skip;
    };

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_addr(smem);
    auto bar = [&](int i) { return sb + D::kBars + 8u * i; };
    uint64_t *bar_ptr = reinterpret_cast<uint64_t *>(smem + D::kBars);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + D::kTmem);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + D::kFlag);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < D::kNumBars; ++i)
            mbar_init(bar(i), (i >= D::Q_READY && i < D::K_FULL) || (i >= D::P_FULL && i < D::PV_DONE) || i >= D::TAKEN ||
                                      (i >= D::K_FULL && i < D::K_EMPTY) || (i >= D::V_FULL && i < D::V_EMPTY)
                                  ? 4 : (i >= D::CODES ? 8 : 1));
        *abort_flag = 0;
        *reinterpret_cast<volatile float *>(smem + D::kFactor) = __ldcg(a.v_refs + bh);
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

    if (warp < kWarpS) {
        fewer_registers<kRegsIssue>();
        if (warp == 0) {
            // ------------------------------------------------------------ TMA
            if (lane == 0) {
                const uint64_t pol = l2_policy_evict_first();
                const int nq = nv1 > 0 ? 2 : 1;
                for (int x = 0; x < nq; ++x) {
                    mbar_arrive_expect_tx(bar(D::Q_FULL + x), 2u * 128u * G * tpt);
                    tma_load_3d(sb + D::kQ + x * D::kTile, &tm_q, 0, h * G, q0 + t0 + x * tpt, bar(D::Q_FULL + x), pol);
                    tma_load_3d(sb + D::kQ + x * D::kTile + 16384, &tm_q, 64, h * G, q0 + t0 + x * tpt,
                                bar(D::Q_FULL + x), pol);
                }
                // No copy may still be landing when the CTA leaves.
                for (int x = 0; x < nq; ++x)
                    pwait(bar(D::Q_FULL + x), 0, abort_flag, a.err, false);
            }
        } else if (warp >= 2) {
            // ------------------------------------------------------------ TMA: K's codes, or V's, from the cache
            // A lane a block of 16 keys; into the second half of the tile that they become.
            const bool is_v = warp == 3;
            const int lp = seq_page_log2(a, b), codes = D::CODES + (is_v ? kStages2 : 0);
            const int empty = is_v ? D::V_EMPTY : D::K_EMPTY;
            const uint8_t *exps = is_v ? a.v_exp : a.k_exp;
            const CUtensorMap *map = is_v ? &tm_v : &tm_k;
            auto place = [&](int t) {
                return t < nt && lane < 8 ? block_place(a, seq_kt, b, h, lp, L, key_tile(t) * kKeys + kBlock * lane)
                                          : BlockPlace{-1, 0};
            };
            auto exponent = [&](const BlockPlace &p) {
                return p.z >= 0 ? static_cast<int>(exps[(static_cast<int64_t>(p.z) * a.page_size + p.y) / kBlock]) : -1;
            };
            BlockPlace now = place(0), next = place(1);
            int x = exponent(now), t = 0;
            for (; t < nt; ++t) {
                const int s = t % kStages2;
                if (t >= kStages2 && !wwait(bar(empty + s), ((t / kStages2) - 1) & 1, abort_flag, a.err, lane))
                    break;
                if (lane < 8) {
                    *(reinterpret_cast<volatile int *>(smem + D::kExps) + 8 * (2 * s + is_v) + lane) = x;
                    mbar_arrive_expect_tx(bar(codes + s), now.z >= 0 ? kBlock * kHeadDim : 0);
                    if (now.z >= 0)
                        tma_load_3d_plain(sb + (is_v ? D::kV : D::kK) + s * D::kTile + 16384 + lane * kBlock * kHeadDim, map, 0,
                                          now.y, now.z, bar(codes + s));
                }
                __syncwarp();
                now = next;
                x = exponent(now);
                next = place(t + 2);
            }
            // No copy may still be landing when the CTA leaves.
            if (lane == 0)
                for (int s = 0; s < kStages2 && s < t; ++s)
                    pwait(bar(codes + s), ((t - 1 - s) / kStages2) & 1, abort_flag, a.err, false);
            __syncwarp();
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issue
            // The whole warp runs this converged; one elected lane issues.
            const uint32_t id_qk = tc::idesc_bf16_f32(kRows, kKeys, false);
            const uint32_t id_pv = tc::idesc_f16_f32(kRows, kHeadDim, true);
            uint64_t qdesc[2], kdesc[kStages2], vdesc[kStages2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                qdesc[i] = kmajor_base(sb + D::kQ + i * D::kTile);
#pragma unroll
            for (int i = 0; i < kStages2; ++i) {
                kdesc[i] = kmajor_base(sb + D::kK + i * D::kTile);
                vdesc[i] = vmn_base(sb + D::kV + i * D::kTile);
            }
            const bool leader = elect_one();
            bool ok = true;
            // scores of tile x against key tile j
            auto score = [&](int x, int j, bool last) {
                const int s = j % kStages2;
                if (!wwait(bar(D::K_FULL + s), (j / kStages2) & 1, abort_flag, a.err, lane))
                    return false;
                tc::fence_after();
                if (leader) {
#pragma unroll
                    for (int d = 0; d < 8; ++d)             // dims 16d..16d+15
                        tc::mma_ss(tm + kScoreCol * x, kmajor_step(qdesc[x], d), kmajor_step(kdesc[s], d), id_qk, d > 0);
                    tc::commit(bar_ptr + D::S_FULL + x);
                    if (last)
                        tc::commit(bar_ptr + D::K_EMPTY + s);
                }
                __syncwarp();
                return true;
            };
            // O += P V of tile x, key tile j: keys 16d..16d+15 of P in columns 8d ..
            auto output = [&](int x, int j, bool last) {
                const int s = j % kStages2;
                if (!wwait(bar(D::V_FULL + s), (j / kStages2) & 1, abort_flag, a.err, lane))
                    return false;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!wwait(bar(D::P_FULL + 2 * x + half), j & 1, abort_flag, a.err, lane))
                        return false;
                    tc::fence_after();
                    if (leader) {
#pragma unroll
                        for (int d = 4 * half; d < 4 * half + 4; ++d)
                            tc::mma_ts(tm + kOutCol + kScoreCol * x, tm + kScoreCol * x + 8 * d, vmn_step(vdesc[s], d),
                                       id_pv, j > 0 || d > 0 ? 1u : 0u);
                        if (half == 1) {
                            tc::commit(bar_ptr + D::PV_DONE + x);
                            if (last)
                                tc::commit(bar_ptr + D::V_EMPTY + s);
                        }
                    }
                    __syncwarp();
                }
                return true;
            };
            ok = wwait(bar(D::Q_READY), 0, abort_flag, a.err, lane) && score(0, 0, nt1 == 0);
            if (ok && nt1 > 0)
                ok = wwait(bar(D::Q_READY + 1), 0, abort_flag, a.err, lane) && score(1, 0, true);
            for (int j = 0; ok && j < nt; ++j) {
                if (j < nt0)
                    ok = output(0, j, j >= nt1) && (j + 1 >= nt0 || score(0, j + 1, j + 1 >= nt1));
                if (ok && j < nt1)
                    ok = output(1, j, true) && (j + 1 >= nt1 || score(1, j + 1, true));
            }
            // Every MMA issued has finished before TMEM is released.
            if (leader) {
                tc::commit(bar_ptr + D::DRAIN);
                pwait(bar(D::DRAIN), 0, abort_flag, a.err, false);
            }
            __syncwarp();
        }
    } else if (warp >= kWarpS + 8) {
        // ------------------------------------------------------------ K and V tiles' codes, widened in place
        // Four warps for K's, four for V's, each for 32 keys of every tile.
        fewer_registers<kRegsWiden>();
        const bool is_v = warp >= kWarpS + 12;
        const int w = warp & 3;
        const int ref = (__float_as_int(*reinterpret_cast<volatile float *>(smem + D::kFactor)) >> 23) & 0xFF;
        const int codes = D::CODES + (is_v ? kStages2 : 0), full = is_v ? D::V_FULL : D::K_FULL, taken = D::TAKEN + is_v;
        uint8_t *ring = smem + (is_v ? D::kV : D::kK);
        for (int t = 0; t < nt; ++t) {
            const int s = t % kStages2, tile = row0 / kKeys + copy_tile(t);
            const volatile int *exps = reinterpret_cast<const volatile int *>(smem + D::kExps) + 8 * (2 * s + is_v);
            if (!wwait(bar(codes + s), (t / kStages2) & 1, abort_flag, a.err, lane))
                break;
            QuarterTile q;
            take_quarter(seq_kt, ring + s * D::kTile, exps, key_tile(t) * kKeys, L, w, lane, q);
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(taken));
            if (!wwait(bar(taken), t & 1, abort_flag, a.err, lane))   // (what they write lies over the codes)
                break;
            bool some = false;
            if (is_v)
                some = store_quarter<true>(a, q, exps, ring + s * D::kTile, static_cast<int64_t>(tile) * kKeys, w, ref, lane);
            else
                store_quarter<false>(a, q, exps, ring + s * D::kTile, 0, w, ref, lane);
            fence_proxy_async_smem();
            __syncwarp();
            // (test facility: the withheld CTA's first K tile never is full)
            if (lane == 0 && (is_v || t > 0 || static_cast<int>(blockIdx.x) != a.withhold_block))
                mbar_arrive(bar(full + s));
            if (is_v && lane == 0) {                     // (CTAs of one kv head that have the tile store the same)
                reinterpret_cast<uint8_t *>(nan_value_tiles(a) + tile)[w] = some;
                if (some)
                    *const_cast<volatile float *>(a.v_refs + bh) = __int_as_float(ref << 23 | static_cast<int>(0x80000000u));
            }
        }
    } else {
        // ------------------------------------------------------------ softmax + output
        more_registers<kRegsSoftmax>();
        const int x = (warp - kWarpS) >> 2;              // the warpgroup's tile
        const int qtr = warp & 3;                        // TMEM lane quarter of this warp
        const int row = qtr * 32 + lane;
        const int nvx = x ? nv1 : nv0, ntx = x ? nt1 : nt0;
        const int tl = row / G;
        const bool valid = row < G * tpt && tl < nvx;
        const int p_row = pos0 + x * tpt + (valid ? tl : nvx - 1);   // padding rows mirror the last row
        const float sl2 = score_factor<true>(a, h);
        const uint32_t s_tm = tm + (static_cast<uint32_t>(qtr * 32) << 16) + kScoreCol * x;
        const uint32_t o_tm = s_tm + kOutCol;
        float m = -INFINITY, l = 0.f;
        bool ok = ntx > 0 && wwait(bar(D::Q_FULL + x), 0, abort_flag, a.err, lane);
        if (ok) {
            // rows past the G x tpt that the copy fills are zeroed
            if (row >= G * tpt) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint4 *qrow = reinterpret_cast<uint4 *>(smem + D::kQ + x * D::kTile + half * 16384 + row * 128);
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        qrow[c] = make_uint4(0, 0, 0, 0);
                }
            }
            fence_proxy_async_smem();     // generic-proxy writes -> visible to the tensor cores
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(D::Q_READY + x));
        }
        for (int j = 0; ok && j < ntx; ++j) {
            if (!wwait(bar(D::S_FULL + x), j & 1, abort_flag, a.err, lane)) {
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
            {
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
                // (keys may differ much in size, so that rows move often: the warp's other rows move along)
                const bool moves = top > m + kLift;
                const float mn = moves ? top - kLift : m;
                const float f = moves ? ex2_approx(m - mn) : 1.f;
                m = mn;
                l *= f;
                if (j > 0) {                               // the accumulator holds tiles 0 .. j-1
                    if (!wwait(bar(D::PV_DONE + x), (j - 1) & 1, abort_flag, a.err, lane)) {
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
            const float ms = m == -INFINITY ? 0.f : m;
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
                    mbar_arrive(bar(D::P_FULL + 2 * x + half));
            }
            const float2 s0 = f2_unpack(f2_add(ls[0], ls[1])), s1 = f2_unpack(f2_add(ls[2], ls[3]));
            l += (s0.x + s0.y) + (s1.x + s1.y);
        }
        if (ok && wwait(bar(D::PV_DONE + x), (ntx - 1) & 1, abort_flag, a.err, lane)) {
            tc::fence_after();
            float *to = split_row(a, 2, blockIdx.x, blockIdx.y, x * kRows + row);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                tc::ld32(o_tm + 32 * c, o);
                tc::wait_ld();
                if (valid)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        reinterpret_cast<uint4 *>(to + 32 * c)[k] =
                            make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            }
            if (valid)
                *reinterpret_cast<float2 *>(to + kHeadDim) = make_float2(m, l);
        }
    }

    tc::fence_before();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after();
        tc::tmem_dealloc(tm, 512);
    }
}

std::mutex g_direct_mu;
unsigned long long g_direct_ctx[64] = {};        // per device: the context the kernel's limit was raised in

}  // namespace

// The attention launch alone: the references' launch is ahead of it, the join's behind.
cudaError_t launch_prefill_direct(const PrefillArgs &a, const KeyWindow &win, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                                  const CUtensorMap &tm_v, cudaStream_t stream)
{
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    {
        unsigned long long ctx = 0;
        const bool known = current_context_id(&ctx);
        std::lock_guard<std::mutex> lk(g_direct_mu);
        if (!known || g_direct_ctx[dev] != ctx) {
            // (a warpgroup waits for registers that others give up: those of the launch must do)
            cudaFuncAttributes f;
            e = cudaFuncGetAttributes(&f, paged_prefill_direct_kernel);
            if (e == cudaSuccess && f.numRegs * kThreadsS < 128 * (kRegsIssue + 2 * kRegsSoftmax + 2 * kRegsWiden))
                e = cudaErrorInvalidConfiguration;
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(paged_prefill_direct_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(D::kBytes));
            if (e != cudaSuccess)
                return e;
            g_direct_ctx[dev] = known ? ctx : 0;
        }
    }
    const dim3 grid(static_cast<unsigned>(a.batch * a.hkv * ((a.max_tiles + 1) / 2)), static_cast<unsigned>(a.split));
    return launch_with(paged_prefill_direct_kernel, grid, kThreadsS, D::kBytes, 1, true, stream, tm_q, tm_k, tm_v, a, win);
}

}  // namespace pkv
