// paged_gqa_decode_fp4: grouped-query decode attention over the 4-bit cache,
// with an optional window and sinks.
//   s_t = sm_scale k_scale q . (e s)_t,  w = softmax(s),  o = v_scale sum_t w_t (e s)_t
//
// What bounds it: every visible row is read once, 72 bytes of K and 72 of V,
// so the floor is the HBM's.  At that rate an SM gets a 16-token tile (2304
// bytes) about every 100 cycles, and an SMSP has about 760 cycles for two of
// them.  Their 4096 codes each cost it 128 conversions to f16 pairs (2 cycles of the
// ALU pipe), as many multiplications with a scale (2 cycles of the FMA pipe) and 34
// mma.sync m16n8k16 (8 cycles of the tensor pipe, and about as many issue slots as
// five other instructions): that alone measures 610 cycles, with the reads from
// shared memory and the softmax 650.  So HBM and issue slots are both nearly
// full, and everything beside those instructions has to be few.
//
// Work split.  The visible tokens of a (sequence, kv head) segment are cut in
// units of two 16-token tiles (a window leaves the tiles of the sinks and
// those of the window).  The segments lie end to end in one list, kv head by
// kv head; every worker (a warp) takes an equal contiguous range of it,
// whatever the lengths.  A range cuts segments into pieces: a whole segment
// is written out, other pieces leave a (max, sum, accumulator) state in
// workspace slot worker + rank of the segment, and a second kernel (a
// programmatic dependent launch) joins them in worker order.  A CTA whose four
// ranges lie within one segment joins their states itself.
// Short work (few units for every warp) runs in one launch instead: a cluster
// of CTAs a segment, whose warps join their states in shared memory.
//
// The list's kernel has three CTAs an SM of four warps, and each warp feeds itself: it
// looks up its units' pages half a batch ahead and brings the tiles in by bulk
// copies, a tile of K and one of V each 1152 contiguous bytes, into a
// ring of its own, 18 KB deep, so that an SM has 221 KB on their way.  Four CTAs an
// SM with shorter rings took 13% longer, and producer warps beside 12 that
// compute 36%: they take issue slots from the same SMSPs.
// The codes go from shared memory straight into mma.sync
// fragments, because the order of the contracted index is free as long as
// both operands agree on it:
//   S^T[t][g] = K[t][:] . Q[g][:]    A = K: lane (r, c) takes the 32 dims 32c .. 32c+31 of row r,
//                                    16 bytes of codes and two scales
//   O^T[d][g] += V^T[d][t] P^T[t][g]  A = V^T: lane (r, c) takes the 16 dims of block r of 4 tokens;
//                                    two tokens' nibbles are interleaved before they are widened,
//                                    so that a conversion gives a pair of tokens
// Codes times their block scale are exact in f16 (6 significant bits).  The
// weights leave the S^T fragment as B operand through two 8x8 transposes.
// Heads are columns of both results, so the running maximum and sum of a head
// sit in the lanes that hold its accumulator and a rescale needs no exchange;
// the reference that takes the maximum's place is moved only when a score exceeds it
// by more than 15.9 (log2 units, so a weight of 2^15.9).
//
// Every wait on an mbarrier is bounded (2 s): on expiry the kernel raises
// PKV_DEVERR_TIMEOUT, stops issuing copies, drains those in flight, returns.
#include <math.h>

#include "fp4.cuh"

namespace pkv {

namespace {

constexpr unsigned kEvery = 0xffffffffu;
constexpr int kUnitBytes = 4 * kFp4Tile;                   // K tile 0, K tile 1, V tile 0, V tile 1
// A weight is 2^(score - m) with a reference m that is a lift below the largest
// score so far (log2 units) when it is set, and moves only when a score exceeds it
// by more than kMoveMax: weights up to 2^15.9 are within f16.  The lift keeps small weights off
// f16's lower end, where 2^-25 is lost: of the largest weight 2^-27 a token in one part,
// 2^-10 of all for 128K tokens, under a bf16 output's 2^-8; 2^-37 in two.
constexpr float kMoveMax = 15.9f;
// (With more than 128K tokens in sight the lift of one part grows with their logarithm,
// so that 2^-10 of all stays the most, up to 2^27 tokens.)
template <int kParts>
__device__ __forceinline__ float lift_of(int tiles)
{
    return kParts == 1 ? 2.f + static_cast<float>(min(max(19 - __clz(tiles - 1), 0), 10)) : 12.f;
}
// Units after which a piece's accumulator is added into an fp32 copy: the
// tensor cores add with truncation, up to 2^-23 of the sum an addition.  1024
// additions (512 units of one part) may leave 2^-13 under a bf16 output's 2^-8.
// Under an fp32 one 64 (16 units of two parts) may leave 2^-17, and measure
// 1e-6 over 8K to 60K tokens, what a plain fp32 computation has; 256 measured 3e-6.
template <int kParts>
constexpr int kFoldUnits = kParts == 1 ? 512 : 16;
constexpr uint64_t kLimitNs = 2000000000ull;

// The list's kernel: every warp is a worker with its own ring, whose stages are
// filled and waited for in pairs (one by one, the copies' issue and the waits cost
// 4% more of the whole).
constexpr int kListWarps = kFp4DecodeWorkers, kListThreads = 32 * kListWarps, kListCtas = 3, kStages = 4;
struct ListSmem {                                          // the rings, [warps][kStages][kUnitBytes], come first
    static constexpr int kFull = kListWarps * kStages * kUnitBytes;
    static constexpr int kFlag = kFull + kListWarps * kStages * 8;
    static constexpr int kSums = kFlag + 16;
    static constexpr int kHow = kSums + 16;                // int [warps]: slot of the CTA's one state, or one of
    static constexpr int kStart = kHow + 16;               // these; int [batch + 1]
    enum { SPREAD = -1, ADJACENT = -2 };
    static size_t bytes(int batch) { return static_cast<size_t>(kStart) + 4u * (batch + 1); }
};

// The cluster's kernel: a warp's units are all on their way at once.
constexpr int kClusterWarps = 4;
constexpr int kClusterUnits = 6;
struct ClusterSmem {                                       // [warps][kClusterUnits][kUnitBytes] first
    static constexpr int kWarp = kClusterUnits * kUnitBytes;
    static constexpr int kFull = kClusterWarps * kWarp;
    static constexpr int kFlag = kFull + kClusterWarps * kClusterUnits * 8;
    static constexpr int kBytes = kFlag + 16;
};

// What one sequence shows its query: tokens [0, sinks) and [from, len), as
// tiles 0 .. first - 1 and then first + skip .. (tiles in all).
struct Sight {
    int len, sinks, from, first, skip, tiles;
};

__device__ __forceinline__ Sight sight_of(const Fp4AttnArgs &a, int b)
{
    Sight s;
    const int lp = seq_page_log2(a, b);
    const long long cap = lp < 0 ? 0 : static_cast<long long>(a.max_pages) << lp;
    const int most = cap < a.max_len ? static_cast<int>(cap) : a.max_len;
    const int L = __ldg(a.seq_lens + b);
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
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int *stop, int32_t *err, int lane)
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

// Row n of a fragment is token order(n) of its tile (8 + order(n - 8) for the
// upper half): adjacent lanes' K rows then differ in parity (conflict-free
// 16-byte reads) and a quad's V rows pair up even and odd (2-way).
__device__ __forceinline__ int order(int n)
{
    return n ^ ((n >> 1) & 1);
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
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Where a lane (r, c) reads within a tile.
struct LaneOffsets {
    uint32_t k, ks;          // K row order(r): its 16 bytes, its two scales (row + 8: 512, 64 further)
    uint32_t v0, v1, s0, s1; // V rows order(2c), order(2c + 1): block r's 8 bytes, its scale
};

__device__ __forceinline__ LaneOffsets lane_offsets(int r, int c)
{
    LaneOffsets o;
    o.k = order(r) * 64 + 16 * c;
    o.ks = kFp4Codes + order(r) * 8 + 2 * c;
    o.v0 = order(2 * c) * 64 + 8 * r;
    o.v1 = order(2 * c + 1) * 64 + 8 * r;
    o.s0 = kFp4Codes + order(2 * c) * 8 + r;
    o.s1 = kFp4Codes + order(2 * c + 1) * 8 + r;
    return o;
}

struct RawK {
    uint32_t k[2][4], s[2];   // rows order(r), order(r) + 8
};
struct RawV {
    uint32_t v[4][2], s[2];   // rows order(2c), order(2c + 1), and both + 8; scale bytes of each pair
};

__device__ __forceinline__ void load_k(uint32_t kt, const LaneOffsets &o, RawK &x)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        lds128(kt + o.k + 512 * j, x.k[j]);
        x.s[j] = lds16(kt + o.ks + 64 * j);
    }
}

__device__ __forceinline__ void load_v(uint32_t vt, const LaneOffsets &o, RawV &x)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        lds64(vt + o.v0 + 512 * j, x.v[2 * j]);
        lds64(vt + o.v1 + 512 * j, x.v[2 * j + 1]);
        x.s[j] = lds8(vt + o.s1 + 64 * j) * 256u + lds8(vt + o.s0 + 64 * j);
    }
}

// Unscaled scores of a tile: lane (r, c) gets tokens order(r) (y[0]) and
// order(r) + 8 (y[1]), each for heads 2c, 2c + 1.
__device__ __forceinline__ void scores(const RawK &x, const uint32_t (&q)[8][2], uint64_t (&y)[2])
{
    __half2 s[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t p = e4m3x2_to_f16x2(x.s[j]);
        s[j][0] = __low2half2(*reinterpret_cast<const __half2 *>(&p));
        s[j][1] = __high2half2(*reinterpret_cast<const __half2 *>(&p));
    }
    float d[4] = {};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint32_t a[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            e2m1x8_to_f16x8(x.k[j][w], a[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&a[j][i]), s[j][w >> 1]);
                a[j][i] = *reinterpret_cast<const uint32_t *>(&v);
            }
        }
        mma_16816(d, a[0][0], a[1][0], a[0][1], a[1][1], q[2 * w][0], q[2 * w][1]);
        mma_16816(d, a[0][2], a[1][2], a[0][3], a[1][3], q[2 * w + 1][0], q[2 * w + 1][1]);
    }
    y[0] = pack2(d[0], d[1]);
    y[1] = pack2(d[2], d[3]);
}

// acc += V^T P^T for a tile; b: the weights of its 16 tokens (B fragment) in
// kParts f16 parts.
template <int kParts>
__device__ __forceinline__ void accumulate(const RawV &x, const uint32_t (&b)[kParts][2], float (&acc)[8][4])
{
    const uint32_t s0 = e4m3x2_to_f16x2(x.s[0]), s1 = e4m3x2_to_f16x2(x.s[1]);
    constexpr uint32_t kLow = 0x0F0F0F0Fu;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        uint32_t e[2][4], o[2][4];                         // even, odd dims of the block; pair 0, pair 1
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint32_t t0 = x.v[2 * p][w], t1 = x.v[2 * p + 1][w];
            e2m1x8_to_f16x8((t0 & kLow) | ((t1 << 4) & ~kLow), e[p]);
            e2m1x8_to_f16x8(((t0 >> 4) & kLow) | (t1 & ~kLow), o[p]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e[p][i] = mul_f16x2(e[p][i], p ? s1 : s0);
                o[p][i] = mul_f16x2(o[p][i], p ? s1 : s0);
            }
        }
#pragma unroll
        for (int part = 0; part < kParts; ++part)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mma_16816(acc[4 * w + i], e[0][i], o[0][i], e[1][i], o[1][i], b[part][0], b[part][1]);
    }
}

// 16 consecutive dims of one output row.
__device__ __forceinline__ void store16(const Fp4AttnArgs &a, int64_t row, int d, const float (&v)[16])
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

__device__ __forceinline__ void store4(const Fp4AttnArgs &a, int64_t row, int d, float4 v)
{
    if (a.out_f32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + row * kHeadDim + d) = v;
    } else {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + row * kHeadDim + d) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
    }
}

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

// kParts: f16 parts of a softmax weight.  One (rounded to f16, 2^-11) is enough
// under a bf16 output's 2^-8; two keep an fp32 output to 2^-21.  The sum that
// normalises them is of the fp32 weights.

// A piece's running state: lane (r, c) holds dims 16r .. 16r + 15 of heads 2c,
// 2c + 1 (acc[i][j]: dim 2i of head 2c + j, acc[i][2 + j]: dim 2i + 1), their
// maxima, and their sums (both heads') over its own tokens.
struct State {
    float m0, m1, acc[8][4];
    uint64_t sum;
};

__device__ __forceinline__ void clear(State &s)
{
    s.m0 = s.m1 = -INFINITY;
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

// Q as B fragment: head r, dims 32c + 4 kk + {0, 1} and {2, 3}, brought to [1, 2)
// by a power of two, so that f16 holds all bits of what is at least 2^-17 of the
// row's largest |q|, and the rest to 2^-25 of that; f0, f1 turn unscaled scores of
// heads 2c, 2c + 1 into exponents of 2.
struct Query {
    uint32_t q[8][2];
    float f0, f1;
};

__device__ __forceinline__ void load_rows(const Fp4AttnArgs &a, int b, int h, int r, int c, uint4 (&raw)[4])
{
    const int64_t row = static_cast<int64_t>(b) * a.hq + static_cast<int64_t>(h) * a.group + (r < a.group ? r : 0);
    const uint4 *src = reinterpret_cast<const uint4 *>(a.q + row * kHeadDim + 32 * c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        raw[i] = __ldg(src + i);
}

__device__ __forceinline__ void make_query(const Fp4AttnArgs &a, const uint4 (&raw)[4], float k_scale, int r, int c,
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

// One unit: the 32 tokens of unit `unit` at shared address st.  done() is
// called when the unit has been read.
template <int kParts, typename Done>
__device__ __forceinline__ void take_unit(uint32_t st, const LaneOffsets &o, const Query &qu, const Sight &sg,
                                          const Inner &inner, int unit, int lane, State &s, Done done)
{
    const int r = lane >> 2, c = lane & 3;
    uint64_t y[2][2];
    {
        RawK x[2];
        load_k(st, o, x[0]);
        load_k(st + kFp4Tile, o, x[1]);
        scores(x[0], qu.q, y[0]);
        scores(x[1], qu.q, y[1]);
    }
    RawV xv[2];
    load_v(st + 2 * kFp4Tile, o, xv[0]);
    load_v(st + 3 * kFp4Tile, o, xv[1]);
    done();
    uint32_t seen = kEvery;                                // the visible ones of the unit's tokens
    float2 z[2][2];
    const uint64_t f = pack2(qu.f0, qu.f1), nm = pack2(-s.m0, -s.m1);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k)
            z[j][k] = unpack2(fma2(y[j][k], f, nm));
    const bool edge = static_cast<uint32_t>(unit - inner.lo) >= inner.n;
    const float top = fmaxf(max3(fmaxf(z[0][0].x, z[0][0].y), z[0][1].x, z[0][1].y),
                            max3(fmaxf(z[1][0].x, z[1][0].y), z[1][1].x, z[1][1].y));
    if (edge || __any_sync(kEvery, !(top <= kMoveMax))) {
        // an edge of the sequence or of its window, or the maximum moves
        if (edge) {
            const int ti = 2 * unit + (lane >> 4);
            const int t = 16 * tile_at(sg, ti) + (lane & 15);
            seen = __ballot_sync(kEvery, ti < sg.tiles && t < sg.len && (t < sg.sinks || t >= sg.from));
            if (seen != kEvery) {                          // values of unseen tokens may be anything
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t v = seen >> (16 * j + 8 * k);
                        xv[j].s[k] &= ((v >> order(2 * c)) & 1u ? 0x00FFu : 0u) |
                                      ((v >> order(2 * c + 1)) & 1u ? 0xFF00u : 0u);
                    }
            }
        }
        float t0 = -INFINITY, t1 = -INFINITY;
        float2 w[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                w[j][k] = unpack2(y[j][k]);
                const bool on = (seen >> (16 * j + 8 * k + order(r))) & 1u;
                w[j][k].x = on ? w[j][k].x * qu.f0 : -INFINITY;
                w[j][k].y = on ? w[j][k].y * qu.f1 : -INFINITY;
                t0 = fmaxf(t0, w[j][k].x);
                t1 = fmaxf(t1, w[j][k].y);
            }
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
            t0 = fmaxf(t0, __shfl_xor_sync(kEvery, t0, d));
            t1 = fmaxf(t1, __shfl_xor_sync(kEvery, t1, d));
        }
        const float lift = lift_of<kParts>(sg.tiles);
        const float n0 = t0 > s.m0 + kMoveMax ? t0 - lift : s.m0;
        const float n1 = t1 > s.m1 + kMoveMax ? t1 - lift : s.m1;
        const float g0 = n0 == s.m0 ? 1.f : ex2_approx(s.m0 - n0), g1 = n1 == s.m1 ? 1.f : ex2_approx(s.m1 - n1);
        s.m0 = n0;
        s.m1 = n1;
        s.sum = fma2(s.sum, pack2(g0, g1), 0ull);
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
            for (int k = 0; k < 2; ++k)
                z[j][k] = make_float2(w[j][k].x - s.m0, w[j][k].y - s.m1);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float p0 = ex2_approx(z[j][0].x), p1 = ex2_approx(z[j][0].y);
        const float p2 = ex2_approx(z[j][1].x), p3 = ex2_approx(z[j][1].y);
        s.sum = add2(s.sum, add2(pack2(p0, p1), pack2(p2, p3)));
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

// A state's row of one head: 128 dims, then maximum and sum.
__device__ __forceinline__ void store_state(float *row, const State &s, const float (&l)[2], int j, int r)
{
    float v[16];
    lane_dims(s, j, v);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        reinterpret_cast<float4 *>(row + 16 * r)[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    if (r == 0)
        *reinterpret_cast<float2 *>(row + kHeadDim) = make_float2(j ? s.m1 : s.m0, l[j]);
}

// Tile number in the pools of visible tile i of segment (b, h); -1: its page
// lies outside the pool (flagged), -2: there is no such tile.
__device__ __forceinline__ int tile_number(const Fp4AttnArgs &a, const Sight &s, int b, int h, int i)
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

// A tile that reads as zeros: the scales of its K and V (the whole warp; st:
// the unit's address, j: the tile's place in it).
__device__ __forceinline__ void zero_tile(uint32_t st, int j, int lane)
{
    const uint32_t at = st + j * kFp4Tile + kFp4Codes + 4 * lane;
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(0u) : "memory");
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + 2 * kFp4Tile), "r"(0u) : "memory");
}

__device__ __forceinline__ void flag_sequence(const Fp4AttnArgs &a, int b, const Sight &s)
{
    if (a.err == nullptr)
        return;
    if (seq_page_log2(a, b) < 0)
        atomicOr(a.err, PKV_DEVERR_PAGESIZE);
    else if (__ldg(a.seq_lens + b) != s.len)
        atomicOr(a.err, PKV_DEVERR_SEQLEN);
}

// ---------------------------------------------------------------------- the list
__device__ __forceinline__ float *warp_state(uint8_t *smem, int warp)
{
    return reinterpret_cast<float *>(smem + warp * kStages * kUnitBytes);
}

// Joins the states of a CTA's warps, whose ranges all lie within one segment,
// into one (out: [group][kPartialStride]).  Out of line, for the loop above it (in
// line, the mixed batch takes 0.5% longer).
__device__ __noinline__ void join_warps(float *out, int group, uint8_t *smem, int warp, int lane)
{
    for (int g = warp; g < group; g += kListWarps) {
        float m[kListWarps], l[kListWarps], M = -INFINITY, L = 0.f;
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kListWarps; ++w) {
            const float2 ml = *reinterpret_cast<const float2 *>(warp_state(smem, w) + g * kPartialStride + kHeadDim);
            m[w] = ml.x;
            l[w] = ml.y;
            M = fmaxf(M, ml.x);
        }
#pragma unroll
        for (int w = 0; w < kListWarps; ++w) {
            const float e = ex2_approx(m[w] - M);
            const float4 v = *reinterpret_cast<const float4 *>(warp_state(smem, w) + g * kPartialStride + 4 * lane);
            L += e * l[w];
            A.x += e * v.x;
            A.y += e * v.y;
            A.z += e * v.z;
            A.w += e * v.w;
        }
        float *row = out + g * kPartialStride;
        *reinterpret_cast<float4 *>(row + 4 * lane) = A;
        if (lane == 0)
            *reinterpret_cast<float2 *>(row + kHeadDim) = make_float2(M, L);
    }
}

template <int kParts>
__device__ __forceinline__ void work_list(const Fp4DecodeArgs &da, uint8_t *smem, int warp, int lane, int worker, int lo,
                                          int n)
{
    const Fp4AttnArgs &a = da.a;
    const int *start = reinterpret_cast<const int *>(smem + ListSmem::kStart);
    volatile int *stop = reinterpret_cast<volatile int *>(smem + ListSmem::kFlag);
    const uint32_t ring = smem_addr(smem) + warp * kStages * kUnitBytes;
    const uint32_t full = smem_addr(smem) + ListSmem::kFull + warp * kStages * 8;
    const uint64_t policy = l2_policy_evict_first();
    // tile numbers, 16 units at a time, half a batch ahead: lane 2i + j has tile j of unit i
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
    const uint32_t my_dst = ring + ((lane & 3) >> 1) * kUnitBytes + ((lane & 1) + 2 * ((lane >> 2) & 1)) * kFp4Tile;
    const uint8_t *my_src = lane < 4 ? a.k_cache : a.v_cache;
    auto issue = [&](int u, int s) {                       // units u, u + 1 (even) into stages s, s + 1
        const int i = u & 15;
        if (i == 0 && u > 0)
            now = next;
        if (i == 8)
            next = look_up(u + 8);
        // (lanes 0 .. 3 bring K tiles, lanes 4 .. 7 V tiles, of two units)
        const int t = __shfl_sync(kEvery, now, 2 * i + (lane & 3));
        const uint32_t none = __ballot_sync(kEvery, t < 0) & 15u;
        if (none) {
            const uint32_t bad = __ballot_sync(kEvery, t == -1);
            for (int k = 0; k < 4; ++k)
                if ((bad >> k) & 1u)
                    zero_tile(ring + (s + (k >> 1)) * kUnitBytes, k & 1, lane);
            __syncwarp();
        }
        if (lane < 8 && (worker != da.withhold || u != 0)) {
            const uint32_t bar = full + 4 * s;
            // (bytes that land before they are announced are only counted early)
            if (lane == 0)
                mbar_arrive_expect_tx(bar, 2 * kFp4Tile * (4 - __popc(none)));
            if (t >= 0)
                bulk_load(my_dst + s * kUnitBytes, my_src + static_cast<int64_t>(t) * kFp4Tile, kFp4Tile, bar, policy);
        }
    };
    issue(0, 0);                                           // (the rest of the ring once the query is there)
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
                j->x = whole ? -1 : worker;
            if (p.unit == 0 && !whole)
                da.firsts[worker] = p.b * a.hkv + p.h;
            if (p.unit + take == units)
                j->y = how() == ListSmem::SPREAD ? worker : ~worker;
        }
        Query qu;
        {
            uint4 raw[4];
            load_rows(a, p.b, p.h, r, c, raw);
            make_query(a, raw, __ldg(a.k_scale + p.h), r, c, qu);
        }
        if (u == 0) {
            for (int v = 2; v < kStages && v < n; v += 2)
                issue(v, v);
        }
        const int64_t slot = static_cast<int64_t>(worker) + p.h * a.batch + p.b;
        State s;
        clear(s);
        float mf0 = -INFINITY, mf1 = -INFINITY;            // maxima of the units folded so far
        uint64_t sums = 0ull;                              // and their sums
        for (int i = 0; i < take && !dead;) {              // (folded between loops: in one, 3% longer)
            const int end = min(take, i + kFoldUnits<kParts>);
#pragma unroll 1
            for (; i < end; ++i) {
                if (!(stage & 1) && !wait_stage(full + 4 * stage, parity, stop, a.err, lane)) {
                    dead = true;
                    break;
                }
                take_unit<kParts>(ring + stage * kUnitBytes, offsets, qu, sg, inner, p.unit + i, lane, s, [&]() {
                    if ((stage & 1) && u + i + kStages - 1 < n) {   // the two units just read make room
                        fence_proxy_async_smem();
                        __syncwarp();
                        issue(u + i + kStages - 1, stage - 1);
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
                const float g0 = old ? ex2_approx(mf0 - s.m0) : 0.f, g1 = old ? ex2_approx(mf1 - s.m1) : 0.f;
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
                    sums = pack2(two_sum(old ? was.x * g0 : 0.f, now.x, rest.x),
                                 two_sum(old ? was.y * g1 : 0.f, now.y, rest.y));
                    s.sum = last ? sums : pack2(rest.x, rest.y);
                }
                mf0 = s.m0;
                mf1 = s.m1;
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
                const float f = __ldg(a.v_scale + p.h) / l[j];
                float v[16];
                lane_dims(s, j, v);
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    v[k] *= f;
                store16(a, row0 + g, 16 * r, v);
            } else if (how() >= 0) {                       // over the ring, which nothing more is brought into
                store_state(warp_state(smem, warp) + g * kPartialStride, s, l, j, r);
            } else if (slot < da.num_slots) {
                store_state(da.partials + (slot * a.group + g) * kPartialStride, s, l, j, r);
            } else if (a.err && r == 0) {
                atomicOr(a.err, PKV_DEVERR_INTERNAL);
            }
        }
    }
    // After an abort: no copy may land in this ring once the warp has left.
    if (dead && lane == 0)
        for (int s = 0; s < kStages; s += 2) {
            // the stages' last fill: of the units issued before the wait that ran out
            const uint64_t t0 = global_timer_ns();
            const uint32_t par = s >= stage ? parity : parity ^ 1u;
            while (!mbar_try_wait(full + 4 * s, par) && global_timer_ns() - t0 < kLimitNs) {
            }
        }
}

template <int kParts>
__global__ void __launch_bounds__(kListThreads, kListCtas) paged_gqa_decode_fp4_kernel(const Fp4DecodeArgs da)
{
    const Fp4AttnArgs &a = da.a;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int *start = reinterpret_cast<int *>(smem + ListSmem::kStart);
    int *sums = reinterpret_cast<int *>(smem + ListSmem::kSums);

    bool no_empty;
    // ---- first unit of every sequence (of one kv head): a prefix sum over the batch
    {
        const int per = (a.batch + kListThreads - 1) / kListThreads;
        const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
        int mine = 0;
        for (int b = b0; b < b1; ++b)
            mine += (sight_of(a, b).tiles + 1) >> 1;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kEvery, incl, o);
            if (lane >= o)
                incl += v;
        }
        if (lane == 31)
            sums[warp] = incl;
        if (tid == 0) {
            *reinterpret_cast<volatile int *>(smem + ListSmem::kFlag) = 0;
            const uint32_t bars = smem_addr(smem) + ListSmem::kFull;
            for (int i = 0; i < kListWarps * kStages; ++i)
                mbar_init(bars + 8 * i, 1);
            fence_barrier_init();
        }
        __syncthreads();
        int run = incl - mine;
        for (int w = 0; w < warp; ++w)
            run += sums[w];
        for (int b = b0; b < b1; ++b) {
            const Sight s = sight_of(a, b);
            start[b] = run;
            run += (s.tiles + 1) >> 1;
            if (blockIdx.x == 0)
                flag_sequence(a, b, s);
        }
        if (tid == kListThreads - 1)
            start[a.batch] = run;
        bool some = true;                                  // this thread's sequences all have tokens
        for (int b = b0; b < b1; ++b)
            some = some && (b + 1 < b1 ? start[b + 1] : run) > start[b];
        no_empty = __syncthreads_and(some) != 0;
    }

    // ---- sequences with no tokens: zero rows, and nothing to join
    for (int sg = blockIdx.x; sg < a.batch * a.hkv; sg += gridDim.x) {
        const int b = sg / a.hkv;
        if (start[b + 1] == start[b]) {
            const int64_t row0 = static_cast<int64_t>(b) * a.hq + static_cast<int64_t>(sg % a.hkv) * a.group;
            for (int e = tid; e < a.group * kHeadDim; e += kListThreads) {
                if (a.out_f32)
                    static_cast<float *>(a.out)[row0 * kHeadDim + e] = 0.f;
                else
                    static_cast<__nv_bfloat16 *>(a.out)[row0 * kHeadDim + e] = __float2bfloat16_rn(0.f);
            }
            if (tid == 0)
                da.joins[sg] = make_int2(-1, -1);
        }
    }
    launch_dependents();

    const int total = start[a.batch] * a.hkv;
    const int active = min(static_cast<int>(gridDim.x) * kListWarps, total);
    // A CTA's warps take adjacent ranges, so that those within a segment leave one
    // state for the join (32 query heads, one 32K sequence 16.8 us, with a state a warp
    // 18.2; a 128K one among 63 of 512 tokens 46.0 and 57.8; 32 x 4K 34.2 and 33.8).  The
    // ranges of a list shorter than the workers spread over the CTAs.
    const bool adjacent = total >= static_cast<int>(gridDim.x) * kListWarps;
    const int worker = adjacent ? static_cast<int>(blockIdx.x) * kListWarps + warp
                                : warp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
    if (lane == 0)
        da.firsts[worker] = -1;
    if (worker < active) {
        // A range with a segment's end in it has one more piece to set up and to
        // store, which costs about a unit's time: the ranges are equal in a list
        // with an empty unit after every segment.  (Two units a range, and no
        // empty sequence: then every range still holds a unit, as the join needs.)
        const bool wide = no_empty && total >= 2 * active;
        const int length = total + (wide ? a.batch * a.hkv : 0);
        const int each = length / active, more = length - each * active;   // the first `more` ranges: one longer
        // lanes 4i, 4i + 1: where the range begins and ends; 4i + 2, 4i + 3: the CTA's ranges
        const int w = (lane & 2 ? worker - warp : worker) + (lane & 1) * (lane & 2 ? kListWarps : 1);
        int edge = w * each + min(w, more);
        if (wide)
            edge = real_position(start, a.batch, a.hkv, edge);
        const int lo = __shfl_sync(kEvery, edge, 0), n = __shfl_sync(kEvery, edge, 1) - lo;
        volatile int *how = reinterpret_cast<volatile int *>(smem + ListSmem::kHow + 4 * warp);
        {
            const int first = __shfl_sync(kEvery, edge, 2), last = __shfl_sync(kEvery, edge, 3);
            int h = ListSmem::SPREAD;
            if (adjacent) {
                const Place p = place_of(start, a.batch, first);
                const bool within = p.unit > 0 && last - first < start[p.b + 1] - start[p.b] - p.unit;
                h = within ? worker - warp + p.h * a.batch + p.b : static_cast<int>(ListSmem::ADJACENT);
            }
            if (lane == 0)
                *how = h;
            __syncwarp();
        }
        work_list<kParts>(da, smem, warp, lane, worker, lo, n);
        if (*how >= 0) {                                   // the segment begins before and ends behind the CTA's ranges
            __syncthreads();
            if (*how < da.num_slots)
                join_warps(da.partials + static_cast<int64_t>(*how) * a.group * kPartialStride, a.group, smem, warp, lane);
            else if (a.err && lane == 0)
                atomicOr(a.err, PKV_DEVERR_INTERNAL);
        }
    }
}

// ---------------------------------------------------------------------- the cluster
// One cluster of da.cluster CTAs a segment.  Its warps share the segment's
// units evenly (at most kClusterUnits each, all brought in at once), leave their
// states in shared memory and join them there.
template <int kParts>
__global__ void __launch_bounds__(32 * kClusterWarps, 2) paged_gqa_decode_fp4_cluster_kernel(const Fp4DecodeArgs da)
{
    using S = ClusterSmem;
    const Fp4AttnArgs &a = da.a;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, c = lane & 3;
    volatile int *stop = reinterpret_cast<volatile int *>(smem + S::kFlag);
    const int rank = static_cast<int>(blockIdx.x) % da.cluster, seg = static_cast<int>(blockIdx.x) / da.cluster;
    const int b = seg / a.hkv, h = seg % a.hkv;
    const Sight sg = sight_of(a, b);
    // the query rows and scales: on their way while the tiles are looked up
    uint4 raw[4];
    load_rows(a, b, h, r, c, raw);
    const float k_scale = __ldg(a.k_scale + h), v_scale = __ldg(a.v_scale + h);
    if (tid == 0) {
        *stop = 0;
        for (int i = 0; i < kClusterWarps * kClusterUnits; ++i)
            mbar_init(smem_addr(smem) + S::kFull + 8 * i, 1);
        fence_barrier_init();
        if (rank == 0 && h == 0)
            flag_sequence(a, b, sg);
    }
    const int units = (sg.tiles + 1) >> 1, workers = da.cluster * kClusterWarps, at = rank * kClusterWarps + warp;
    const int lo = units * at / workers;
    const int n = min(units * (at + 1) / workers - lo, kClusterUnits);
    int t = -2;                                            // lane 2i + j: tile j of unit i
    if ((lane >> 1) < n)
        t = tile_number(a, sg, b, h, 2 * (lo + (lane >> 1)) + (lane & 1));
    __syncthreads();
    const uint32_t ring = smem_addr(smem) + warp * S::kWarp;
    const uint32_t full = smem_addr(smem) + S::kFull + warp * kClusterUnits * 8;
    const uint32_t have = __ballot_sync(kEvery, t >= 0), bad = __ballot_sync(kEvery, t == -1);
    for (int i = 0; bad != 0 && i < 2 * n; ++i)
        if ((bad >> i) & 1u)
            zero_tile(ring + (i >> 1) * kUnitBytes, i & 1, lane);
    __syncwarp();
    // (test facility: the withheld warp never loads its first unit)
    const bool withheld = lane < 2 && static_cast<int>(blockIdx.x) * kClusterWarps + warp == da.withhold;
    if ((lane >> 1) < n && !(lane & 1) && !withheld)
        mbar_arrive_expect_tx(full + 4 * lane, 2 * kFp4Tile * __popc((have >> lane) & 3u));
    __syncwarp();
    if (t >= 0 && !withheld) {
        const uint32_t dst = ring + (lane >> 1) * kUnitBytes + (lane & 1) * kFp4Tile, bar = full + 8 * (lane >> 1);
        const uint64_t policy = l2_policy_evict_first();
        bulk_load(dst, a.k_cache + static_cast<int64_t>(t) * kFp4Tile, kFp4Tile, bar, policy);
        bulk_load(dst + 2 * kFp4Tile, a.v_cache + static_cast<int64_t>(t) * kFp4Tile, kFp4Tile, bar, policy);
    }
    __syncwarp();

    const LaneOffsets offsets = lane_offsets(r, c);
    const Inner inner = inner_units(sg);
    Query qu;
    make_query(a, raw, k_scale, r, c, qu);
    State s;
    clear(s);
    bool dead = false;
    for (int u = 0; u < n; ++u) {
        if (!wait_stage(full + 8 * u, 0, stop, a.err, lane)) {
            dead = true;
            break;
        }
        take_unit<kParts>(ring + u * kUnitBytes, offsets, qu, sg, inner, lo + u, lane, s, []() {});
    }
    if (dead && lane == 0)                                 // no copy may land in what the states overwrite
        for (int u = 0; u < n; ++u) {
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(full + 8 * u, 0) && global_timer_ns() - t0 < kLimitNs) {
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
        *reinterpret_cast<float2 *>(state + lane * kPartialStride + kHeadDim) = make_float2(-INFINITY, 0.f);
    }

    // ---- join (at most 32 states, one a lane), in worker order: CTA k takes the
    // heads k, k + CTAs, ..; of several CTAs each warp 32 dims of all of them, of
    // one CTA a warp every fourth head
    cluster_sync(da.cluster);
    const bool one = da.cluster == 1;
    for (int g = one ? warp : rank; g < a.group; g += one ? kClusterWarps : da.cluster) {
        const uint32_t mine = smem_addr(smem) + g * kPartialStride * 4;        // warp 0's state of this head, this CTA
        float m = -INFINITY, l = 0.f;
        if (lane < workers) {
            const uint32_t ml = mine + (lane & 3) * S::kWarp + kHeadDim * 4;
            m = cluster_load(ml, lane >> 2, one);
            l = cluster_load(ml + 4, lane >> 2, one);
        }
        float M = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            M = fmaxf(M, __shfl_xor_sync(kEvery, M, o));
        // (not 0 where there is a state: a NaN of V in it is seen whatever its weight)
        const float e = m == -INFINITY ? 0.f : fmaxf(ex2_approx(m - M), 0x1p-126f);
        float sum = e * l;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(kEvery, sum, o);
        const float f = units == 0 ? 0.f : v_scale / sum;
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
            store4(a, row, 4 * lane, make_float4(A.x * f, A.y * f, A.z * f, A.w * f));
        } else {
            const int d = 32 * warp + lane;
            float A = 0.f;
            float v[32];                                   // all on their way together: one round trip
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i] = i < workers ? cluster_load(mine + (i & 3) * S::kWarp + 4 * d, i >> 2, false) : 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float ei = __shfl_sync(kEvery, e, i);
                A += ei != 0.f ? ei * v[i] : 0.f;
            }
            if (a.out_f32)
                static_cast<float *>(a.out)[row * kHeadDim + d] = A * f;
            else
                static_cast<__nv_bfloat16 *>(a.out)[row * kHeadDim + d] = __float2bfloat16_rn(A * f);
        }
    }
    cluster_sync(da.cluster);                              // no CTA leaves while its states are read
}

// Joins the states of a segment's pieces for one query head, in worker order:
// out = v_scale sum_i 2^(m_i - M) A_i / sum_i 2^(m_i - M) l_i.  Warps take the
// pieces in turns, all of a turn's loads in flight together, and are joined in warp
// order.  A turn is a round trip to the L2, so turns are long and, with a CTA a
// (segment, head), up to 16 warps share them (32 query heads, a 128K sequence among 63
// of 512 tokens 46.0 us, with 8 states and 8 warps 48.3; one 128K sequence alone 34.0 and
// 33.3).  Warps are as few as an average segment needs, because a CTA of one or two is
// on its SM before the list's CTAs have left it (64 x 2K tokens 35.0 us, with four at
// least 39.0; 32 x 4K 34.2 and 36.0; the long one among short ones 46.0 and 43.7).
constexpr int kJoin = 16, kJoinWarps = 16;
constexpr int kJoinCut = 8;

// Head g of segment sg, by `warps` warps of the CTA (ra, rm: theirs), kTurn pieces
// a turn.
template <int kTurn>
__device__ __forceinline__ void join_head(const Fp4DecodeArgs &da, int sg, int g, int warp, int warps, int lane,
                                          float (*ra)[kHeadDim], float2 *rm)
{
    const Fp4AttnArgs &a = da.a;
    const int b = sg / a.hkv, h = sg % a.hkv;
    const float vs = __ldg(a.v_scale + h);
    int2 j = da.joins[sg];
    if (j.x < 0)
        return;
    // Of the workers x .. y, the CTAs strictly between have left one state, in the first
    // of their slots (y = ~the last worker; else every worker has its own).
    int head = 0, full = 0;
    if (j.y < 0) {
        j.y = ~j.y;
        head = kListWarps - j.x % kListWarps;
        full = max(0, j.y / kListWarps - 1 - j.x / kListWarps);
    }
    const int64_t slot0 = static_cast<int64_t>(j.x) + h * a.batch + b;
    if (j.y < j.x || slot0 + (j.y - j.x) >= da.num_slots)
        return;                                            // an aborted call, or flagged by the decode kernel
    const int pieces = j.y - j.x + 1 - (kListWarps - 1) * full;
    auto worker = [&](int i) {                             // beyond x
        return i < head || full == 0 ? i : (i < head + full ? head + kListWarps * (i - head) : i + (kListWarps - 1) * full);
    };
    const float *base = da.partials + (slot0 * a.group + g) * kPartialStride;
    const int64_t stride = static_cast<int64_t>(a.group) * kPartialStride;
    float M = -INFINITY, L = 0.f;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = warp * kTurn; i0 < pieces; i0 += warps * kTurn) {
        float4 v[kTurn];
        float2 ml[kTurn];
#pragma unroll
        for (int i = 0; i < kTurn; ++i) {
            const bool on = i0 + i < pieces;
            const float *s = base + (on ? worker(i0 + i) : 0) * stride;
            ml[i] = on ? *reinterpret_cast<const float2 *>(s + kHeadDim) : make_float2(-INFINITY, 0.f);
            v[i] = on ? *reinterpret_cast<const float4 *>(s + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float mn = M;
#pragma unroll
        for (int i = 0; i < kTurn; ++i)
            mn = fmaxf(mn, ml[i].x);
        const float f = ex2_approx(M - mn);
        M = mn;
        L *= f;
        A = make_float4(A.x * f, A.y * f, A.z * f, A.w * f);
#pragma unroll
        for (int i = 0; i < kTurn; ++i) {
            const float e = i0 + i < pieces ? ex2_approx(ml[i].x - mn) : 0.f;
            L += e * ml[i].y;
            A.x += e * v[i].x;
            A.y += e * v[i].y;
            A.z += e * v[i].z;
            A.w += e * v[i].w;
        }
    }
    if (warps > 1) {
        *reinterpret_cast<float4 *>(&ra[warp][4 * lane]) = A;
        if (lane == 0)
            rm[warp] = make_float2(M, L);
        __syncthreads();
        if (warp != 0)
            return;
        float mn = M;
        for (int w = 1; w < warps; ++w)
            mn = fmaxf(mn, rm[w].x);
        L = 0.f;
        A = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < warps; ++w) {
            if (w * kTurn >= pieces)
                break;                                     // a warp with no pieces
            const float e = ex2_approx(rm[w].x - mn);
            const float4 v = *reinterpret_cast<const float4 *>(&ra[w][4 * lane]);
            L += e * rm[w].y;
            A.x += e * v.x;
            A.y += e * v.y;
            A.z += e * v.z;
            A.w += e * v.w;
        }
    }
    const float f = vs / L;
    store4(a, static_cast<int64_t>(b) * a.hq + static_cast<int64_t>(h) * a.group + g, 4 * lane,
           make_float4(A.x * f, A.y * f, A.z * f, A.w * f));
}

__global__ void __launch_bounds__(32 * kJoinWarps) join_fp4_kernel(const Fp4DecodeArgs da)
{
    __shared__ __align__(16) float ra[kJoinWarps][kHeadDim];
    __shared__ float2 rm[kJoinWarps];
    grid_wait();
    join_head<kJoin>(da, blockIdx.x / da.a.group, blockIdx.x % da.a.group, threadIdx.x >> 5, blockDim.x >> 5,
                     threadIdx.x & 31, ra, rm);
}

// The same for lists of many segments, of which at most one a worker is cut: a CTA a
// worker, for the segment that its range begins and does not end; a warp a head.  A
// CTA a (segment, head) is what such lists spend their time on: 64 query heads, 512 x
// 128 tokens 43 us, this way 31; 1024 x 128 84 and 55; 128 x 512 29.4 and 26.8; 64 x
// 1024 25.2 and 24.6.  With few segments it is the slower one (32 query heads, 64 x 2048: 35.4,
// 35.1; 16 x 4096: 22.7, 21.7), as long segments have more pieces than a warp's turn.
__global__ void __launch_bounds__(32 * PKV_MAX_GROUP) join_cut_fp4_kernel(const Fp4DecodeArgs da)
{
    grid_wait();
    const int sg = da.firsts[blockIdx.x];
    if (sg >= 0)
        join_head<kJoinCut>(da, sg, threadIdx.x >> 5, 0, 1, threadIdx.x & 31, nullptr, nullptr);
}

}  // namespace

size_t decode_fp4_smem(int batch)
{
    return ListSmem::bytes(batch);
}

size_t decode_fp4_cluster_smem()
{
    return ClusterSmem::kBytes;
}

const void *decode_fp4_kernel(bool two_parts, bool cluster)
{
    if (cluster)
        return two_parts ? reinterpret_cast<const void *>(&paged_gqa_decode_fp4_cluster_kernel<2>)
                         : reinterpret_cast<const void *>(&paged_gqa_decode_fp4_cluster_kernel<1>);
    return two_parts ? reinterpret_cast<const void *>(&paged_gqa_decode_fp4_kernel<2>)
                     : reinterpret_cast<const void *>(&paged_gqa_decode_fp4_kernel<1>);
}

int decode_fp4_threads(bool cluster)
{
    return cluster ? 32 * kClusterWarps : kListThreads;
}

// CTAs a segment for the cluster kernel: the fewest (1, 2, 4, 8) that leave a
// warp at most kClusterUnits units, if all of them are resident at once (or in a
// second round, see below); 0: the list.  (`units`: of the longest sequence, `slots`: resident CTAs.)
int decode_fp4_cluster(long long units, long long segments, int slots)
{
    for (int c = 1; c <= 8; c *= 2)
        if (units <= static_cast<long long>(c) * kClusterWarps * kClusterUnits)
            // a second round pays for single CTAs of at most 4 units a warp (8 kv heads, 64 x
            // 256 tokens: 9.8 us against the list's 12.9, 64 x 512: 15.7 against 17.0; 64 x 768,
            // 6 units: 20.9 against 20.2; 32 x 1024 in clusters of two: 19.7 against 16.5)
            return segments * c <= (c == 1 && units <= 4 * kClusterWarps ? 2 : 1) * slots ? c : 0;
    return 0;
}

cudaError_t launch_paged_decode_fp4(const Fp4DecodeArgs &da, int ctas, cudaStream_t stream, const char **site)
{
    *site = "4-bit decode kernel launch";
    const bool two = da.a.out_f32;
    if (da.cluster > 0) {
        const dim3 grid(static_cast<unsigned>(da.a.batch * da.a.hkv * da.cluster));
        return launch_with(two ? paged_gqa_decode_fp4_cluster_kernel<2> : paged_gqa_decode_fp4_cluster_kernel<1>, grid,
                           32 * kClusterWarps, ClusterSmem::kBytes, da.cluster, false, stream, da);
    }
    cudaError_t e = launch_with(two ? paged_gqa_decode_fp4_kernel<2> : paged_gqa_decode_fp4_kernel<1>,
                                dim3(static_cast<unsigned>(ctas)), kListThreads, decode_fp4_smem(da.a.batch), 1, false,
                                stream, da);
    if (e != cudaSuccess)
        return e;
    *site = "4-bit join kernel launch";
    const long long segs = static_cast<long long>(da.a.batch) * da.a.hkv;
    const int workers = ctas * kListWarps;
    if (segs * da.a.group >= 2ll * workers)
        return launch_with(join_cut_fp4_kernel, dim3(static_cast<unsigned>(workers)), 32 * da.a.group, 0, 1, true, stream,
                           da);
    const long long pieces = (workers + segs - 1) / segs + 1;   // a segment's, on average
    int warps = 1;
    while (warps < kJoinWarps && warps * kJoin < pieces)
        warps *= 2;
    return launch_with(join_fp4_kernel, dim3(static_cast<unsigned>(segs * da.a.group)), 32 * warps, 0, 1, true, stream,
                       da);
}

}  // namespace pkv
