// paged_gqa_decode_fp8b: grouped-query decode attention over the block-scaled FP8
// cache, with an optional window and sinks.
//   s_t = sm_scale q . (code_K 2^ek)_t,  w = softmax(s),  o = sum_t w_t (code_V 2^ev)_t
//
// What bounds it: every visible row is read once, 128 bytes of K and 128 of V, so the
// floor is the HBM's.  At that rate an SM gets a block of K and V (4096 bytes) about
// every 180 cycles.
//
// Work split.  As the 4-bit cache's decode: the visible blocks of a (sequence, kv head)
// segment are cut in units of two, the segments lie end to end in one list, every
// warp takes an equal range of it, a second kernel joins what the pieces of cut
// segments leave; short work runs in one launch, a cluster of CTAs a segment.
//
// Each warp feeds itself: a ring of its own in shared memory, filled by TMA tensor
// loads, a block (16 rows of 128 bytes) each, with the 128-byte swizzle, so that
// both operands are read 16 bytes a lane without bank conflicts.  The blocks' bytes x
// come with the tile numbers, looked up half a batch ahead, and wait beside the unit
// in shared memory.  The order of the contracted index is free as long as both
// operands agree on it:
//   S^T[t][g] = K[t][:] . Q[g][:]    A = K: lane (r, c) takes dims 32c .. 32c+31 of rows r, r + 8
//   O^T[d][g] += V^T[d][t] P^T[t][g]  A = V^T: lane (r, c) takes dims 16r .. 16r+15 of tokens 2c,
//                                    2c + 1 and both + 8; two tokens' bytes are interleaved before
//                                    they are widened, so that a conversion gives a pair of tokens
// Codes are exact in f16, and stay unscaled: ek goes into the factor of a block's
// scores, ev into the exponent of its weights, which are rounded to f16 in one part
// (bf16 output) or two.  So what the tensor cores get is P = 2^(s + ev - n), and the
// reference n is taken from the largest contribution, s + ev, so that a weight is not
// lost to another one that meets smaller values.  The sum of the weights has its
// own reference m, from the largest s.  Both move only when exceeded by more than 15.9.
// n is kept less a whole number e, the larger ev of the unit that moved it last: exponents
// are then small wherever the values lie, and no bits of s are lost to ev.
//
// Every wait on an mbarrier is bounded (2 s): on expiry the kernel raises
// PKV_DEVERR_TIMEOUT, stops issuing copies, drains those in flight, returns.
#include <math.h>

#include "fp8b.h"
#include "list.cuh"

namespace pkv {

namespace {

constexpr int kTile = kBlock * kHeadDim;                   // bytes of a block's K or V codes
constexpr int kUnitBytes = 4 * kTile;                      // K 0, K 1, V 0, V 1
// A weight P is 2^(s + ev - n) with a reference n that is a lift below the largest s + ev so
// far (log2 units) when it is set, and moves only when it is exceeded by more than
// kMoveMax: P up to 2^15.9 is within f16.  The lift keeps small contributions off f16's
// lower end, where 2^-25 is lost: of the largest contribution 2^-27 a token in one
// part, 2^-10 of it for 128K tokens, under a bf16 output's 2^-8; 2^-37 in two.  (With more
// tokens in sight the lift of one part grows with their logarithm, up to 2^27 tokens.)
constexpr float kMoveMax = 15.9f;
template <int kParts>
__device__ __forceinline__ float lift_of(int tiles)
{
    return kParts == 1 ? 2.f + static_cast<float>(min(max(19 - __clz(tiles - 1), 0), 10)) : 12.f;
}
// Units after which a piece's accumulator is added into an fp32 copy: the tensor
// cores add with truncation, up to 2^-23 of the sum an addition.  1024 additions (512
// units of one part) may leave 2^-13 under a bf16 output's 2^-8, 64 (16 units of two
// parts) 2^-17 under an fp32 one.
template <int kParts>
constexpr int kFoldUnits = kParts == 1 ? 512 : 16;

// The list's kernel.  Two CTAs an SM with rings of three units bring as much at once as
// three with rings of two, and still do where not every SM has its second (32 x 4096 tokens, a
// segment a CTA, 46.8 us; three by two 55.1; 64 sequences of 512 to 131072 tokens 438 and 440).
constexpr int kListWarps = kFp8bListWarps, kListThreads = 32 * kListWarps, kListCtas = 2, kStages = 3;
struct ListSmem {                                          // the rings, [warps][kStages][kUnitBytes], come first,
    static constexpr int kFull = kListWarps * kStages * kUnitBytes;   // from a 1024-byte aligned base
    static constexpr int kScales = kFull + kListWarps * kStages * 8;  // float4 [warps][kStages]: 2^ek, ev of either block
    static constexpr int kFlag = kScales + kListWarps * kStages * 16;
    static constexpr int kSums = kFlag + 16;
    static constexpr int kHow = kSums + 16;                // int [warps]: ListRange::how
    static constexpr int kStart = kHow + 16;               // int [batch + 1]
    static size_t bytes(int batch) { return static_cast<size_t>(kStart) + 4u * (batch + 1) + 1024u; }
};
static_assert(kListWarps == kSplitWarps && kListWarps <= 4, "a CTA's warps share 16 bytes of each");

// What one thread sets up.  (As a lambda in a kernel with tensor maps it stops nvcc 13.0
// with an internal error.)
struct ListInit {
    uint8_t *smem;
    __device__ __forceinline__ void operator()() const
    {
        *reinterpret_cast<volatile int *>(smem + ListSmem::kFlag) = 0;
        const uint32_t bars = smem_addr(smem) + ListSmem::kFull;
        for (int i = 0; i < kListWarps * kStages; ++i)
            mbar_init(bars + 8 * i, 1);
        fence_barrier_init();
    }
};

// ListRange::how of a CTA that has a segment to itself.
constexpr int kWholeSegment = INT32_MAX;

// The cluster's kernel.
constexpr int kClusterWarps = 4, kClusterStages = 3;
struct ClusterSmem {                                       // [warps][kClusterStages][kUnitBytes] first
    static constexpr int kWarp = kClusterStages * kUnitBytes;
    static constexpr int kFull = kClusterWarps * kWarp;
    static constexpr int kFlag = kFull + kClusterWarps * kClusterStages * 8;
    static constexpr int kBytes = kFlag + 16 + 1024;
};

__device__ __forceinline__ uint8_t *aligned_smem(uint8_t *raw)
{
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
}

// Where a lane (r, c) reads within a block's swizzled rows (16-byte chunk i of row t
// lies at chunk i ^ (t & 7)).
struct LaneOffsets {
    uint32_t k0, k1;         // K row r: chunks 2c, 2c + 1 (row r + 8: 1024 further)
    uint32_t v0, v1;         // V rows 2c, 2c + 1: chunk r (rows + 8: 1024 further)
};

__device__ __forceinline__ LaneOffsets lane_offsets(int r, int c)
{
    LaneOffsets o;
    o.k0 = r * kHeadDim + (((2 * c) ^ r) << 4);
    o.k1 = r * kHeadDim + (((2 * c + 1) ^ r) << 4);
    o.v0 = 2 * c * kHeadDim + ((r ^ (2 * c)) << 4);
    o.v1 = (2 * c + 1) * kHeadDim + ((r ^ (2 * c + 1)) << 4);
    return o;
}

struct RawK {
    uint32_t k[2][2][4];     // rows r, r + 8: dims 32c .. 32c + 15, and the next 16
};
struct RawV {
    uint32_t v[4][4];        // rows 2c, 2c + 1, 2c + 8, 2c + 9: dims 16r .. 16r + 15
};

__device__ __forceinline__ void load_k(uint32_t kt, const LaneOffsets &o, RawK &x)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        lds128(kt + o.k0 + 1024 * j, x.k[j][0]);
        lds128(kt + o.k1 + 1024 * j, x.k[j][1]);
    }
}

__device__ __forceinline__ void load_v(uint32_t vt, const LaneOffsets &o, RawV &x)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        lds128(vt + o.v0 + 1024 * j, x.v[2 * j]);
        lds128(vt + o.v1 + 1024 * j, x.v[2 * j + 1]);
    }
}

// Unscaled scores of two blocks: lane (r, c) gets tokens r (y[.][0]) and r + 8 (y[.][1]), each
// for heads 2c, 2c + 1.
__device__ __forceinline__ void scores(const RawK (&x)[2], const uint32_t (&q)[8][2], uint64_t (&y)[2][2])
{
    float d[2][4] = {};
#pragma unroll
    for (int w = 0; w < 8; ++w)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x4(x[j].k[0][w >> 2][w & 3], a0, a2);
            e4m3x4_to_f16x4(x[j].k[1][w >> 2][w & 3], a1, a3);
            mma_16816(d[j], a0, a1, a2, a3, q[w][0], q[w][1]);
        }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        y[j][0] = pack2(d[j][0], d[j][1]);
        y[j][1] = pack2(d[j][2], d[j][3]);
    }
}

// acc += V^T P^T for a block; b: the weights of its 16 tokens (B fragment) in
// kParts f16 parts.
template <int kParts>
__device__ __forceinline__ void accumulate(const RawV &x, const uint32_t (&b)[kParts][2], float (&acc)[8][4])
{
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint32_t p[2][4];                                  // tokens 2c, 2c + 1; both + 8: dims 4w .. 4w + 3
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            e4m3x4_to_f16x4(__byte_perm(x.v[2 * j][w], x.v[2 * j + 1][w], 0x5140), p[j][0], p[j][1]);
            e4m3x4_to_f16x4(__byte_perm(x.v[2 * j][w], x.v[2 * j + 1][w], 0x7362), p[j][2], p[j][3]);
        }
#pragma unroll
        for (int part = 0; part < kParts; ++part)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                mma_16816(acc[2 * w + i], p[0][2 * i], p[0][2 * i + 1], p[1][2 * i], p[1][2 * i + 1], b[part][0], b[part][1]);
    }
}

// A piece's running state: lane (r, c) holds dims 16r .. 16r + 15 of heads 2c,
// 2c + 1 (acc[i][j]: dim 2i of head 2c + j, acc[i][2 + j]: dim 2i + 1), the heads' references
// of weights (m) and contributions (n + e), and the weights' sums (both heads') over
// its own tokens.
struct State {
    float m0, m1, n0, n1, e, acc[8][4];
    uint64_t sum;
};

__device__ __forceinline__ void clear(State &s)
{
    s.m0 = s.m1 = s.n0 = s.n1 = -INFINITY;
    s.e = 0.f;
    s.sum = 0ull;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s.acc[i][k] = 0.f;
}

// The heads' sums over all tokens, in every lane.
__device__ __forceinline__ void whole_sums(const State &s, float (&l)[2])
{
    const float2 v = unpack2(s.sum);
    l[0] = v.x;
    l[1] = v.y;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        l[0] += __shfl_xor_sync(kEvery, l[0], o);
        l[1] += __shfl_xor_sync(kEvery, l[1], o);
    }
}

// One unit: the 32 tokens of unit `unit` at shared address st; sc: 2^ek and ev of
// either block.  done() is called when the unit has been read.
template <int kParts, typename Done>
__device__ __forceinline__ void take_unit(uint32_t st, const float4 &sc, const LaneOffsets &o, const Query &qu, const Sight &sg,
                                          const Inner &inner, int unit, int lane, State &s, Done done)
{
    const int r = lane >> 2, c = lane & 3;
    uint64_t y[2][2];
    {
        RawK x[2];
        load_k(st, o, x[0]);
        load_k(st + kTile, o, x[1]);
        scores(x, qu.q, y);
    }
    RawV xv[2];
    load_v(st + 2 * kTile, o, xv[0]);
    load_v(st + 3 * kTile, o, xv[1]);
    done();
    uint32_t seen = kEvery;                                // the visible ones of the unit's tokens
    const float ek[2] = {sc.x, sc.z}, ev[2] = {sc.y, sc.w};
    float2 z[2][2], zn[2][2];                              // exponents of the weights, and of what meets V
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint64_t f = pack2(qu.f0 * ek[j], qu.f1 * ek[j]), nm = pack2(-s.m0, -s.m1);
        const uint64_t d = pack2(s.m0 - s.n0 + (ev[j] - s.e), s.m1 - s.n1 + (ev[j] - s.e));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint64_t v = fma2(y[j][k], f, nm);
            z[j][k] = unpack2(v);
            zn[j][k] = unpack2(add2(v, d));
            top = max3(max3(top, z[j][k].x, z[j][k].y), zn[j][k].x, zn[j][k].y);
        }
    }
    const bool edge = static_cast<uint32_t>(unit - inner.lo) >= inner.n;
    if (edge || __any_sync(kEvery, !(top <= kMoveMax))) {
        // an edge of the sequence or of its window, or a reference moves
        if (edge) {
            const int ti = 2 * unit + (lane >> 4);
            const int t = 16 * tile_at(sg, ti) + (lane & 15);
            seen = __ballot_sync(kEvery, ti < sg.tiles && t < sg.len && (t < sg.sinks || t >= sg.from));
            if (seen != kEvery) {                          // codes of unseen tokens may be anything
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const bool on = (seen >> (16 * j + 2 * c + (k & 1) + 8 * (k >> 1))) & 1u;
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            xv[j].v[k][w] = on ? xv[j].v[k][w] : 0u;
                    }
            }
        }
        float t0 = -INFINITY, t1 = -INFINITY, c0 = -INFINITY, c1 = -INFINITY;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 w = unpack2(y[j][k]);
                const bool on = (seen >> (16 * j + 8 * k + r)) & 1u;
                z[j][k].x = on ? w.x * (qu.f0 * ek[j]) : -INFINITY;
                z[j][k].y = on ? w.y * (qu.f1 * ek[j]) : -INFINITY;
                t0 = fmaxf(t0, z[j][k].x);
                t1 = fmaxf(t1, z[j][k].y);
                c0 = fmaxf(c0, z[j][k].x + (ev[j] - s.e));
                c1 = fmaxf(c1, z[j][k].y + (ev[j] - s.e));
            }
        if (__any_sync(kEvery, c0 > s.n0 + kMoveMax || c1 > s.n1 + kMoveMax)) {
            const float e = fmaxf(ev[0], ev[1]);
            s.n0 += s.e - e;
            s.n1 += s.e - e;
            s.e = e;
            c0 = fmaxf(fmaxf(z[0][0].x, z[0][1].x) + (ev[0] - e), fmaxf(z[1][0].x, z[1][1].x) + (ev[1] - e));
            c1 = fmaxf(fmaxf(z[0][0].y, z[0][1].y) + (ev[0] - e), fmaxf(z[1][0].y, z[1][1].y) + (ev[1] - e));
        }
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
            t0 = fmaxf(t0, __shfl_xor_sync(kEvery, t0, d));
            t1 = fmaxf(t1, __shfl_xor_sync(kEvery, t1, d));
            c0 = fmaxf(c0, __shfl_xor_sync(kEvery, c0, d));
            c1 = fmaxf(c1, __shfl_xor_sync(kEvery, c1, d));
        }
        const float lift = lift_of<kParts>(sg.tiles);
        const float m0 = t0 > s.m0 + kMoveMax ? t0 : s.m0, m1 = t1 > s.m1 + kMoveMax ? t1 : s.m1;
        const float n0 = c0 > s.n0 + kMoveMax ? c0 - lift : s.n0, n1 = c1 > s.n1 + kMoveMax ? c1 - lift : s.n1;
        s.sum = fma2(s.sum, pack2(m0 == s.m0 ? 1.f : ex2_approx(s.m0 - m0), m1 == s.m1 ? 1.f : ex2_approx(s.m1 - m1)), 0ull);
        const float g0 = n0 == s.n0 ? 1.f : ex2_approx(s.n0 - n0), g1 = n1 == s.n1 ? 1.f : ex2_approx(s.n1 - n1);
        s.m0 = m0;
        s.m1 = m1;
        s.n0 = n0;
        s.n1 = n1;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            s.acc[k][0] *= g0;
            s.acc[k][1] *= g1;
            s.acc[k][2] *= g0;
            s.acc[k][3] *= g1;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                zn[j][k] = make_float2(z[j][k].x + (ev[j] - s.e) - s.n0, z[j][k].y + (ev[j] - s.e) - s.n1);
                z[j][k] = make_float2(z[j][k].x - s.m0, z[j][k].y - s.m1);
            }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        s.sum = add2(s.sum, add2(pack2(ex2_approx(z[j][0].x), ex2_approx(z[j][0].y)),
                                 pack2(ex2_approx(z[j][1].x), ex2_approx(z[j][1].y))));
        const float p0 = ex2_approx(zn[j][0].x), p1 = ex2_approx(zn[j][0].y);
        const float p2 = ex2_approx(zn[j][1].x), p3 = ex2_approx(zn[j][1].y);
        const uint32_t ha = f32x2_to_f16x2(p0, p1), hb = f32x2_to_f16x2(p2, p3);
        uint32_t b[kParts][2];
        b[0][0] = transpose8x8(ha);
        b[0][1] = transpose8x8(hb);
        if constexpr (kParts == 2) {
            const float2 va = f16x2_to_f32x2(ha), vb = f16x2_to_f32x2(hb);
            b[1][0] = transpose8x8(f32x2_to_f16x2(p0 - va.x, p1 - va.y));
            b[1][1] = transpose8x8(f32x2_to_f16x2(p2 - vb.x, p3 - vb.y));
        }
        accumulate<kParts>(xv[j], b, s.acc);
    }
}

// A lane's 16 dims of head 2c + j.
__device__ __forceinline__ void lane_dims(const State &s, int j, float (&v)[16])
{
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        v[2 * k] = s.acc[k][j];
        v[2 * k + 1] = s.acc[k][j + 2];
    }
}

// A state's row of one head: 128 dims, m, sum, n, e.
__device__ __forceinline__ void store_state(float *row, const State &s, const float (&l)[2], int j, int r)
{
    float v[16];
    lane_dims(s, j, v);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        reinterpret_cast<float4 *>(row + 16 * r)[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    if (r == 0)
        *reinterpret_cast<float4 *>(row + kRowM) = make_float4(j ? s.m1 : s.m0, l[j], j ? s.n1 : s.n0, s.e);
}

// The bytes x of a tile's blocks of K (low) and V: of a tile outside the pool (it reads
// as zeros), or of none, those of 1 and of the smallest scale.
__device__ __forceinline__ uint32_t tile_bytes(const Fp8bDecodeArgs &da, int t)
{
    if (t < 0)
        return kExpBias | (kExpMin + kExpBias) << 8;
    return da.k_exp[t] | static_cast<uint32_t>(da.v_exp[t]) << 8;
}

// 2^ek and ev.
__device__ __forceinline__ float2 tile_scales(uint32_t bytes)
{
    const uint32_t k = bytes & 0xFFu;
    return make_float2(__uint_as_float(k == 0 ? 0x00400000u : k << 23), static_cast<float>(static_cast<int>(bytes >> 8) - kExpBias));
}

// One block of K (or V) into shared memory; t < 0: zeros.
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *tm, int t, int per_page_log2, int zeros, uint32_t bar,
                                          uint64_t policy)
{
    const int z = t < 0 ? zeros : t >> per_page_log2, y = t < 0 ? 0 : (t & ((1 << per_page_log2) - 1)) * kBlock;
    tma_load_3d(dst, tm, 0, y, z, bar, policy);
}

// ---------------------------------------------------------------------- the list
template <int kParts>
__device__ __forceinline__ void work_list(const Fp8bDecodeArgs &da, const CUtensorMap &tm_k, const CUtensorMap &tm_v, uint8_t *smem,
                                          int warp, int lane, int worker, int lo, int n)
{
    const CacheAttnArgs &a = da.a;
    const int *start = reinterpret_cast<const int *>(smem + ListSmem::kStart);
    volatile int *stop = reinterpret_cast<volatile int *>(smem + ListSmem::kFlag);
    const uint32_t ring = smem_addr(smem) + warp * kStages * kUnitBytes;
    const uint32_t full = smem_addr(smem) + ListSmem::kFull + warp * kStages * 8;
    const uint32_t scales = smem_addr(smem) + ListSmem::kScales + warp * kStages * 16;
    const uint64_t policy = l2_policy_evict_first();
    const int zeros = static_cast<int>(a.num_pages * a.hkv), per_page = a.pool_log2 - 4;
    // tile numbers, 16 units at a time, half a batch ahead, and their bytes a quarter:
    // lane 2i + j has tile j of unit i
    auto look_up = [&](int u0) -> int {
        const int u = u0 + (lane >> 1);
        if (u >= n)
            return -2;
        const Place p = place_of(start, a.batch, lo + u);
        return tile_number(a, sight_of(a, p.b), p.b, p.h, 2 * p.unit + (lane & 1));
    };
    // (read where it is needed: a register less in the loop)
    auto how = [&]() { return *reinterpret_cast<volatile int *>(smem + ListSmem::kHow + 4 * warp); };
    int now = look_up(0), next = -2;
    uint32_t bytes_now = 0, bytes_next = 0;
    auto issue = [&](int u) {                              // unit u into stage u % kStages
        const int i = u & 15, s = u % kStages;
        if (i == 0 && u > 0) {
            now = next;
            bytes_now = bytes_next;
        }
        if (i == 8)
            next = look_up(u + 8);
        if (i == 12)
            bytes_next = tile_bytes(da, next);
        // (lanes 0, 1 bring K, lanes 2, 3 V)
        const int t = __shfl_sync(kEvery, now, 2 * i + (lane & 1));
        const bool two = __shfl_sync(kEvery, now, 2 * i + 1) != -2;
        if (lane < 4 && (worker != da.withhold || u != 0)) {
            const uint32_t bar = full + 8 * s;
            // (bytes that land before they are announced are only counted early)
            if (lane == 0)
                mbar_arrive_expect_tx(bar, two ? 4 * kTile : 2 * kTile);
            if (t != -2)
                load_tile(ring + s * kUnitBytes + lane * kTile, lane < 2 ? &tm_k : &tm_v, t, per_page, zeros, bar, policy);
        }
    };
    auto put_scales = [&](int u) {
        const int i = u & 15;
        if ((lane >> 1) == i) {
            const float2 v = tile_scales(bytes_now);
            asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(scales + (u % kStages) * 16 + (lane & 1) * 8), "f"(v.x), "f"(v.y)
                         : "memory");
        }
        __syncwarp();
    };
    for (int v = 0; v < kStages && v < n; ++v)
        issue(v);
    bytes_now = tile_bytes(da, now);
    bool dead = false;
    const int r = lane >> 2, c = lane & 3;
    const LaneOffsets offsets = lane_offsets(r, c);
    int stage = 0;
    uint32_t parity = 0;
    int u = 0;
    while (u < n && !dead) {
        const Place p = place_of(start, a.batch, lo + u);
        const Sight sg = sight_of(a, p.b);
        const Inner inner = inner_units(sg);
        const int units = start[p.b + 1] - start[p.b];
        const int take = min(units - p.unit, n - u);
        const bool whole = p.unit == 0 && take == units;
        if (lane == 0) {                                   // who holds the segment's first and last unit
            int2 *j = da.joins + p.b * a.hkv + p.h;
            if (p.unit == 0)
                j->x = whole || how() == kWholeSegment ? -1 : worker;
            if (p.unit == 0 && !whole && how() != kWholeSegment)
                da.firsts[worker] = p.b * a.hkv + p.h;
            if (p.unit + take == units)
                j->y = how() == ListRange::SPREAD ? worker : ~worker;
        }
        Query qu;
        {
            uint4 raw[4];
            load_rows(a, p.b, p.h, r, c, raw);
            make_query(a, raw, 1.f, r, c, qu);
        }
        if (u == 0) {
            for (int v = 0; v < kStages && v < n; ++v)
                put_scales(v);
        }
        const int64_t slot = static_cast<int64_t>(worker) + p.h * a.batch + p.b;
        State s;
        clear(s);
        float mf0 = -INFINITY, mf1 = -INFINITY, nf0 = -INFINITY, nf1 = -INFINITY, ef = 0.f;   // references of what has been folded
        uint64_t sums = 0ull;                              // and its sums
        for (int i = 0; i < take && !dead;) {              // (folded between loops)
            const int end = min(take, i + kFoldUnits<kParts>);
#pragma unroll 1
            for (; i < end; ++i) {
                if (!wait_stage(full + 8 * stage, parity, stop, a.err, lane)) {
                    dead = true;
                    break;
                }
                uint32_t sc[4];
                lds128(scales + 16 * stage, sc);
                const float4 scf = make_float4(__uint_as_float(sc[0]), __uint_as_float(sc[1]), __uint_as_float(sc[2]),
                                               __uint_as_float(sc[3]));
                take_unit<kParts>(ring + stage * kUnitBytes, scf, offsets, qu, sg, inner, p.unit + i, lane, s, [&]() {
                    if (u + i + kStages < n) {             // the unit just read makes room
                        fence_proxy_async_smem();
                        __syncwarp();
                        issue(u + i + kStages);
                        put_scales(u + i + kStages);
                    }
                });
                if (++stage == kStages) {
                    stage = 0;
                    parity ^= 1u;
                }
            }
            if (!dead && take >= kFoldUnits<kParts>) {
                // the piece's own slot of the workspace holds the accumulator's copy (each lane its own elements)
                const bool old = i > kFoldUnits<kParts>, last = i == take;
                const float g0 = old ? ex2_approx((nf0 - s.n0) + (ef - s.e)) : 0.f;
                const float g1 = old ? ex2_approx((nf1 - s.n1) + (ef - s.e)) : 0.f;
                if (slot >= da.num_slots) {
                    if (a.err && lane == 0)
                        atomicOr(a.err, PKV_DEVERR_INTERNAL);
                } else {
                    // what a sum's rounding loses stays in the lanes, unless it is the last one
                    float *at0 = da.partials + slot * a.group * kPartialStride;
                    auto add = [&](float *at, float v, float g) {
                        float rest;
                        const float sum = two_sum(old ? *at * g : 0.f, v, rest);
                        if (!last)
                            *at = sum;
                        return last ? sum : rest;
                    };
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (2 * c + j >= a.group)
                            continue;
                        const float g = j ? g1 : g0;
                        float *at = at0 + (2 * c + j) * kPartialStride + 16 * r;
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            float &v = s.acc[k >> 1][2 * (k & 1) + j];
                            v = add(at + k, v, g);
                        }
                    }
                    const float2 was = unpack2(sums), now = unpack2(s.sum);
                    float2 rest;
                    sums = pack2(two_sum(old ? was.x * ex2_approx(mf0 - s.m0) : 0.f, now.x, rest.x),
                                 two_sum(old ? was.y * ex2_approx(mf1 - s.m1) : 0.f, now.y, rest.y));
                    s.sum = last ? sums : pack2(rest.x, rest.y);
                }
                mf0 = s.m0;
                mf1 = s.m1;
                nf0 = s.n0;
                nf1 = s.n1;
                ef = s.e;
            }
        }
        if (dead)
            break;
        u += take;

        // ---- end of piece: heads 2c, 2c + 1; dims 16 r ..
        float l[2];
        whole_sums(s, l);
        const int64_t row0 = static_cast<int64_t>(p.b) * a.hq + static_cast<int64_t>(p.h) * a.group;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int g = 2 * c + j;
            if (g >= a.group)
                continue;
            if (whole) {
                const Quotient f(j ? s.n1 - s.m1 : s.n0 - s.m0, s.e, l[j]);
                float v[16];
                lane_dims(s, j, v);
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    v[k] = f(v[k]);
                store16(a, row0 + g, 16 * r, v);
            } else if (how() >= 0) {                       // over the ring, which nothing more is brought into
                store_state(reinterpret_cast<float *>(smem + warp * kStages * kUnitBytes) + g * kPartialStride, s, l, j, r);
            } else if (slot < da.num_slots) {
                store_state(da.partials + (slot * a.group + g) * kPartialStride, s, l, j, r);
            } else if (a.err && r == 0) {
                atomicOr(a.err, PKV_DEVERR_INTERNAL);
            }
        }
    }
    // After an abort: no copy may land in this ring once the warp has left.
    if (dead && lane == 0)
        for (int s = 0; s < kStages; ++s) {
            // the stages' last fill: of the units issued before the wait that ran out
            const uint64_t t0 = global_timer_ns();
            const uint32_t par = s >= stage ? parity : parity ^ 1u;
            while (!mbar_try_wait(full + 8 * s, par) && global_timer_ns() - t0 < kLimitNs) {
            }
        }
}

// Every sequence has about as many units as the others, at least one for each warp, and
// the segments, one a CTA, fill the SMs about evenly (whole CTA).  Then a CTA takes a
// segment, and nothing is left to join: 32 x 4096 tokens of 8 kv heads 46.8 us, cut into equal
// ranges 49.9.
__device__ __forceinline__ bool segment_a_cta(const CacheAttnArgs &a, const int *start)
{
    const int segments = a.batch * a.hkv, sms = static_cast<int>(gridDim.x) / kListCtas;
    bool like = segments > sms && segments <= sms * kListCtas && 5 * ((segments + sms - 1) / sms * sms) <= 6 * segments;
    for (int b = threadIdx.x; b < a.batch && like; b += kListThreads) {
        const int units = start[b + 1] - start[b];
        like = units >= kListWarps && 10ll * units * a.batch <= 11ll * start[a.batch];
    }
    return __syncthreads_and(like) != 0;
}

// Joins the states of a CTA's warps, which share a segment, and writes its rows.
__device__ __noinline__ void join_segment(void *out, bool f32, int64_t row0, int group, const uint8_t *smem, int warp, int lane)
{
    auto state = [&](int w, int g) {
        return reinterpret_cast<const float *>(smem + w * kStages * kUnitBytes) + g * kPartialStride;
    };
    for (int g = warp; g < group; g += kListWarps) {
        auto ref = [&](int w) { return Reference{state(w, g)[kRowRef], state(w, g)[kRowRef + 1]}; };
        float M = -INFINITY, L = 0.f;
        Reference N = {-INFINITY, 0.f};
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kListWarps; ++w) {
            M = fmaxf(M, state(w, g)[kRowM]);
            N = larger(ref(w), N);
        }
#pragma unroll
        for (int w = 0; w < kListWarps; ++w) {
            const float4 v = *reinterpret_cast<const float4 *>(state(w, g) + 4 * lane);
            const float e = ex2_approx(ref(w).over(N));
            L += ex2_approx(state(w, g)[kRowM] - M) * state(w, g)[kRowM + 1];
            A = make_float4(A.x + e * v.x, A.y + e * v.y, A.z + e * v.z, A.w + e * v.w);
        }
        store4(out, f32, row0 + g, 4 * lane, Quotient(N.n - M, N.e, L)(A));
    }
}

template <int kParts>
__global__ void __launch_bounds__(kListThreads, kListCtas)
    paged_gqa_decode_fp8b_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                                 const Fp8bDecodeArgs da)
{
    const CacheAttnArgs &a = da.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = aligned_smem(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int *start = reinterpret_cast<int *>(smem + ListSmem::kStart);
    int *sums = reinterpret_cast<int *>(smem + ListSmem::kSums);
    if (tid < 2)
        prefetch_tensormap(tid ? &tm_v : &tm_k);
    grid_wait();
    const bool no_empty = list_starts<kListWarps>(a, start, sums, ListInit{smem});
    zero_rows<kListThreads>(da, start);
    launch_dependents();

    ListRange range;
    if (segment_a_cta(a, start)) {
        const int segment = static_cast<int>(blockIdx.x), b = segment % a.batch, h = segment / a.batch;
        range = ListRange{segment < a.batch * a.hkv, segment * kListWarps + warp, 0, 0, kWholeSegment};
        if (lane == 0)
            da.firsts[range.worker] = -1;
        if (range.on) {
            const int units = start[b + 1] - start[b], lo = units * warp / kListWarps;
            range.lo = h * start[a.batch] + start[b] + lo;
            range.n = units * (warp + 1) / kListWarps - lo;
        }
    } else {
        range = list_range<kListWarps>(da, start, no_empty, warp, lane);
    }
    if (range.on) {
        volatile int *how = reinterpret_cast<volatile int *>(smem + ListSmem::kHow + 4 * warp);
        if (lane == 0)
            how[0] = range.how;
        __syncwarp();
        work_list<kParts>(da, tm_k, tm_v, smem, warp, lane, range.worker, range.lo, range.n);
        if (how[0] >= 0) {                                 // the warps' states lie in shared memory
            __syncthreads();
            if (how[0] == kWholeSegment)
                join_segment(a.out, a.out_f32 != 0,
                             static_cast<int64_t>(blockIdx.x % a.batch) * a.hq + static_cast<int64_t>(blockIdx.x / a.batch) * a.group,
                             a.group, smem, warp, lane);
            else if (how[0] < da.num_slots)                // the segment begins before and ends behind the CTA's ranges
                join_warps<true, kListWarps, kStages * kUnitBytes>(
                    da.partials + static_cast<int64_t>(how[0]) * a.group * kPartialStride, a.group, smem, warp, lane);
            else if (a.err && lane == 0)
                atomicOr(a.err, PKV_DEVERR_INTERNAL);
        }
    }
}

// ---------------------------------------------------------------------- the cluster
// One cluster of da.cluster CTAs a segment.  Its warps share the segment's
// units evenly, leave their states in shared memory and join them there.
template <int kParts>
__global__ void __launch_bounds__(32 * kClusterWarps, 2)
    paged_gqa_decode_fp8b_cluster_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                                         const Fp8bDecodeArgs da)
{
    using S = ClusterSmem;
    const CacheAttnArgs &a = da.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = aligned_smem(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, c = lane & 3;
    volatile int *stop = reinterpret_cast<volatile int *>(smem + S::kFlag);
    const int rank = static_cast<int>(blockIdx.x) % da.cluster, seg = static_cast<int>(blockIdx.x) / da.cluster;
    const int b = seg / a.hkv, h = seg % a.hkv;
    if (tid < 2)
        prefetch_tensormap(tid ? &tm_v : &tm_k);
    launch_dependents();
    grid_wait();
    const Sight sg = sight_of(a, b);
    // the query rows: on their way while the tiles are looked up
    uint4 raw[4];
    load_rows(a, b, h, r, c, raw);
    if (tid == 0) {
        *stop = 0;
        for (int i = 0; i < kClusterWarps * kClusterStages; ++i)
            mbar_init(smem_addr(smem) + S::kFull + 8 * i, 1);
        fence_barrier_init();
        if (rank == 0 && h == 0)
            flag_sequence(a, b, sg);
    }
    const int units = (sg.tiles + 1) >> 1, workers = da.cluster * kClusterWarps, at = rank * kClusterWarps + warp;
    const int lo = units * at / workers;
    const int n = units * (at + 1) / workers - lo;
    // tile numbers as in the list: lane 2i + j has tile j of unit i of the 16 at hand
    auto look_up = [&](int u0) -> int {
        const int u = u0 + (lane >> 1);
        return u < n ? tile_number(a, sg, b, h, 2 * (lo + u) + (lane & 1)) : -2;
    };
    int now = look_up(0), next = -2;
    uint32_t bytes_next = 0;
    __syncthreads();
    const uint32_t ring = smem_addr(smem) + warp * S::kWarp;
    const uint32_t full = smem_addr(smem) + S::kFull + warp * kClusterStages * 8;
    const uint64_t policy = l2_policy_evict_first();
    const int zeros = static_cast<int>(a.num_pages * a.hkv), my = lane >> 1;
    // units from .. to - 1 (of the 16 at hand) into their stages, by the lanes that have their tiles
    auto issue = [&](int from, int to) {
        if ((from & 15) == 0 && from > 0)
            now = next;
        if ((from & 15) == 8)
            next = look_up(from + 8);
        if ((from & 15) == 12)
            bytes_next = tile_bytes(da, next);
        const int u = (from & ~15) + my, stage = u % kClusterStages;
        const uint32_t have = __ballot_sync(kEvery, now != -2), bar = full + 8 * stage;
        // (test facility: the withheld warp never loads its first unit)
        const bool on = u >= from && u < to &&
                        !(u == 0 && static_cast<int>(blockIdx.x) * kClusterWarps + warp == da.withhold);
        if (on && !(lane & 1))
            mbar_arrive_expect_tx(bar, 2 * kTile * __popc((have >> lane) & 3u));
        __syncwarp();
        if (on && now != -2) {
            const uint32_t dst = ring + stage * kUnitBytes + (lane & 1) * kTile;
            load_tile(dst, &tm_k, now, a.pool_log2 - 4, zeros, bar, policy);
            load_tile(dst + 2 * kTile, &tm_v, now, a.pool_log2 - 4, zeros, bar, policy);
        }
        __syncwarp();
    };
    issue(0, min(n, kClusterStages));
    float2 mine = tile_scales(tile_bytes(da, now));

    const LaneOffsets offsets = lane_offsets(r, c);
    const Inner inner = inner_units(sg);
    Query qu;
    make_query(a, raw, 1.f, r, c, qu);
    State s;
    clear(s);
    bool dead = false;
    int stage = 0;
    uint32_t parity = 0;
#pragma unroll 1
    for (int u = 0; u < n; ++u) {
        const int i = u & 15;
        if (i == 0 && u > 0)
            mine = tile_scales(bytes_next);
        const float4 sc = make_float4(__shfl_sync(kEvery, mine.x, 2 * i), __shfl_sync(kEvery, mine.y, 2 * i),
                                      __shfl_sync(kEvery, mine.x, 2 * i + 1), __shfl_sync(kEvery, mine.y, 2 * i + 1));
        if (!wait_stage(full + 8 * stage, parity, stop, a.err, lane)) {
            dead = true;
            if (lane == 0)                                 // no copy may land in what the states overwrite
                for (int v = u; v < min(n, u + kClusterStages); ++v) {
                    const uint64_t t0 = global_timer_ns();
                    while (!mbar_try_wait(full + 8 * (v % kClusterStages), (v / kClusterStages) & 1) &&
                           global_timer_ns() - t0 < kLimitNs) {
                    }
                }
            break;
        }
        take_unit<kParts>(ring + stage * kUnitBytes, sc, offsets, qu, sg, inner, lo + u, lane, s, [&]() {
            if (u + kClusterStages < n) {                  // the unit just read makes room
                fence_proxy_async_smem();
                __syncwarp();
                issue(u + kClusterStages, u + kClusterStages + 1);
            }
        });
        if (++stage == kClusterStages) {
            stage = 0;
            parity ^= 1u;
        }
    }
    __syncwarp();
    float *state = reinterpret_cast<float *>(smem + warp * S::kWarp);   // over the ring
    if (n > 0 && !dead) {
        float l[2];
        whole_sums(s, l);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (2 * c + j < a.group)
                store_state(state + (2 * c + j) * kPartialStride, s, l, j, r);
    } else if (lane < a.group) {
        *reinterpret_cast<float4 *>(state + lane * kPartialStride + kRowM) = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    }

    // ---- join (at most 32 states, one a lane), in worker order: CTA k takes the
    // heads k, k + CTAs, ..; of several CTAs each warp 32 dims of all of them, of
    // one CTA a warp every fourth head
    cluster_sync(da.cluster);
    const bool one = da.cluster == 1;
    for (int g = one ? warp : rank; g < a.group; g += one ? kClusterWarps : da.cluster) {
        const uint32_t mine0 = smem_addr(smem) + g * kPartialStride * 4;       // warp 0's state of this head, this CTA
        float m = -INFINITY, l = 0.f;
        Reference ref = {-INFINITY, 0.f};
        if (lane < workers) {
            const float4 v = cluster_load4(mine0 + (lane & 3) * S::kWarp + kRowM * 4, lane >> 2, one);
            m = v.x;
            l = v.y;
            ref = Reference{v.z, v.w};
        }
        float M = m;
        Reference N = ref;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            M = fmaxf(M, __shfl_xor_sync(kEvery, M, o));
            N = larger(Reference{__shfl_xor_sync(kEvery, N.n, o), __shfl_xor_sync(kEvery, N.e, o)}, N);
        }
        N = Reference{__shfl_sync(kEvery, N.n, 0), __shfl_sync(kEvery, N.e, 0)};
        // (m = -inf: no units, l = 0, or only tokens whose scores are NaN, l = NaN)
        float sum = m == -INFINITY ? l : ex2_approx(m - M) * l;
        // (not 0 where there is a state: a NaN of V in it is seen whatever its weight)
        const float e = m == -INFINITY ? 0.f : fmaxf(ex2_approx(ref.over(N)), 0x1p-126f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(kEvery, sum, o);
        const Quotient f(units == 0 ? 0.f : N.n - M, N.e, units == 0 ? 1.f : sum);   // (of no units: of zeros)
        const int64_t row = static_cast<int64_t>(b) * a.hq + static_cast<int64_t>(h) * a.group + g;
        // (what a warp without units left is read, but not used)
        if (one) {
            float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kClusterWarps; ++i) {
                const float ei = __shfl_sync(kEvery, e, i);
                const float4 v =
                    *reinterpret_cast<const float4 *>(smem + i * S::kWarp + (g * kPartialStride + 4 * lane) * 4);
                A.x += ei != 0.f ? ei * v.x : 0.f;
                A.y += ei != 0.f ? ei * v.y : 0.f;
                A.z += ei != 0.f ? ei * v.z : 0.f;
                A.w += ei != 0.f ? ei * v.w : 0.f;
            }
            store4(a, row, 4 * lane, f(A));
        } else {
            const int d = 32 * warp + lane;
            float A = 0.f;
            float v[32];                                   // all on their way together: one round trip
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i] = i < workers ? cluster_load(mine0 + (i & 3) * S::kWarp + 4 * d, i >> 2, false) : 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float ei = __shfl_sync(kEvery, e, i);
                A += ei != 0.f ? ei * v[i] : 0.f;
            }
            if (a.out_f32)
                static_cast<float *>(a.out)[row * kHeadDim + d] = f(A);
            else
                static_cast<__nv_bfloat16 *>(a.out)[row * kHeadDim + d] = __float2bfloat16_rn(f(A));
        }
    }
    cluster_sync(da.cluster);                              // no CTA leaves while its states are read
}

}  // namespace

size_t decode_fp8b_smem(int batch)
{
    return ListSmem::bytes(batch);
}

size_t decode_fp8b_cluster_smem()
{
    return ClusterSmem::kBytes;
}

const void *decode_fp8b_kernel(bool two_parts, bool cluster)
{
    if (cluster)
        return two_parts ? reinterpret_cast<const void *>(&paged_gqa_decode_fp8b_cluster_kernel<2>)
                         : reinterpret_cast<const void *>(&paged_gqa_decode_fp8b_cluster_kernel<1>);
    return two_parts ? reinterpret_cast<const void *>(&paged_gqa_decode_fp8b_kernel<2>)
                     : reinterpret_cast<const void *>(&paged_gqa_decode_fp8b_kernel<1>);
}

int decode_fp8b_threads(bool cluster)
{
    return cluster ? 32 * kClusterWarps : kListThreads;
}

// CTAs a segment for the cluster kernel, 0: the list.  (`units`: of the longest sequence,
// `slots`: resident CTAs.)  Where all are resident at once, the fewest (1, 2, 4, 8) that
// leave a warp at most kClusterStages units, else the most; where they are not, 1.
// A cluster spares the list's start and join, 3 to 4 us (8 kv heads, 32 x 512 tokens 8.9 us, by
// the list 12.7; 32 x 1024 14.7 and 18.3; 8 x 2048 in fours 11.2 and 14.5; 4 x 4096 in eights 11.0 and
// 14.0), but shares a segment's units among its own warps only: what one long sequence among
// short ones takes is its own units' time, 0.85 us one of a warp's 32 tokens.  So a warp has
// 12 of them at most (32 x 1400: 17.3 and 21.1; with 16, 32 x 2048 of equal length 24.4 and 28.7, but
// spread over 128 .. 2048 20.5 and 16.6), 8 where a quarter of the slots and more are empty (1 x 8192:
// 11.7 and 11.9; 2 x 8192 14.4 and 14.2; 2 x 10000 16.4 and 15.0).  More segments than CTAs run in rounds,
// the last of which should be well filled (64 x 1024, 1.7 rounds: 28.4 and 33.1; 40 x 2048, 1.1
// rounds: 42.9 and 36.0) or short (75 x 500: 20.3 and 24.1), and rounds of less than two units a warp
// few (128 x 128, 3.4 rounds: 16.8 and 17.4; 256 x 128, 6.7 rounds: 28.7 and 25.9).
int decode_fp8b_cluster(long long units, long long segments, int slots)
{
    auto each = [&](int c) { return (units + c * kClusterWarps - 1) / (c * kClusterWarps); };
    if (segments > slots) {
        const long long rounds = (segments + slots - 1) / slots;
        const bool filled = 3 * rounds * slots <= 4 * segments || each(1) <= 4;
        return each(1) <= 12 && filled && (each(1) >= 2 || rounds <= 4) ? 1 : 0;
    }
    int best = 1;
    while (best < 8 && segments * best * 2 <= slots && each(best) > kClusterStages)
        best *= 2;
    return each(best) <= (4 * segments * best >= 3ll * slots ? 12 : 8) ? best : 0;
}

cudaError_t launch_paged_decode_fp8b(const Fp8bDecodeArgs &da, const CUtensorMap &tm_k, const CUtensorMap &tm_v, int ctas,
                                     cudaStream_t stream, const char **site)
{
    *site = "block-scaled decode kernel launch";
    const bool two = da.a.out_f32;
    if (da.cluster > 0) {
        const dim3 grid(static_cast<unsigned>(da.a.batch * da.a.hkv * da.cluster));
        return launch_with(two ? paged_gqa_decode_fp8b_cluster_kernel<2> : paged_gqa_decode_fp8b_cluster_kernel<1>, grid,
                           32 * kClusterWarps, ClusterSmem::kBytes, da.cluster, true, stream, tm_k, tm_v, da);
    }
    cudaError_t e = launch_with(two ? paged_gqa_decode_fp8b_kernel<2> : paged_gqa_decode_fp8b_kernel<1>,
                                dim3(static_cast<unsigned>(ctas)), kListThreads, decode_fp8b_smem(da.a.batch), 1, true,
                                stream, tm_k, tm_v, da);
    if (e != cudaSuccess)
        return e;
    *site = "block-scaled join kernel launch";
    return launch_join<true>(da, ctas, stream);
}

}  // namespace pkv
