// paged_gqa_decode_fp4: grouped-query decode attention over the 4-bit cache,
// with an optional window and sinks.
//   s_t = sm_scale k_scale q . (e s)_t,  w = softmax(s),  o = v_scale sum_t w_t (e s)_t
//
// What bounds it: every visible row is read once, 72 bytes of K and 72 of V,
// so the floor is the HBM's.  At that rate an SM gets a 16-token tile (2304
// bytes) about every 100 cycles, and widening its 4096 codes costs an SMSP's
// issue slots and its conversion pipe (2 cycles a pair of codes and scale:
// measured 2.5 with the multiply) more than the two matrix products do
// (mma.sync m16n8k16: 8 cycles), so the design keeps everything else few.
//
// Work split.  The visible tokens of a (sequence, kv head) segment are cut in
// units of two 16-token tiles (a window leaves the tiles of the sinks and
// those of the window).  The segments lie end to end in one list, kv head by
// kv head; every warp of the grid takes an equal contiguous range of it,
// whatever the lengths.  A range cuts segments into pieces: a whole segment
// is written out, other pieces leave a (max, sum, accumulator) state in
// workspace slot worker + rank of the segment, and a second kernel (a
// programmatic dependent launch) joins them in worker order.  Worker w is
// warp w / CTAs of CTA w % CTAs, so that short lists spread over the SMs.
//
// A warp brings its units in by bulk copies (a tile of K and one of V are
// 1152 contiguous bytes each) into its own ring, each stage with its own
// mbarrier.  The codes go from shared memory straight into mma.sync
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
// the maximum is moved only when a score exceeds it by more than 2^8.
//
// Every wait on an mbarrier is bounded (2 s): on expiry the kernel raises
// PKV_DEVERR_TIMEOUT, stops issuing copies, drains those in flight, returns.
#include <math.h>

#include "fp4.cuh"

namespace pkv {

namespace {

constexpr int kWarpsD = kFp4DecodeWarps;
constexpr int kThreadsD = 32 * kWarpsD;
constexpr int kStagesD = 3;
constexpr int kUnitBytes = 4 * kFp4Tile;                   // K tile 0, K tile 1, V tile 0, V tile 1
constexpr float kMoveMax = 8.f;                            // log2 units
// Units a warp of a cluster takes at most: beyond it the list's even split and
// a second launch for the join are faster.
constexpr int kClusterUnits = 6;
// Units after which a piece's accumulator is added into an fp32 copy: the
// tensor cores add with truncation, whose error grows with the chain.
// 2048 additions (512 units of one part) may leave 2^-12 under a bf16
// output's 2^-8, 256 (64 units of two parts) 2^-15 under an fp32 one.
template <int kParts>
constexpr int kFoldUnits = kParts == 1 ? 512 : 64;
constexpr uint64_t kLimitNs = 2000000000ull;

struct SmemD {                                             // the ring, [warps][stages][kUnitBytes], comes first
    static constexpr int kBar = kWarpsD * kStagesD * kUnitBytes;
    static constexpr int kFlag = kBar + kWarpsD * kStagesD * 8;
    static constexpr int kSums = kFlag + 16;
    static constexpr int kStart = kSums + 16 * ((kWarpsD * 4 + 15) / 16);   // int [batch + 1]
    static size_t bytes(int batch) { return static_cast<size_t>(kStart) + 4u * (batch + 1); }
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
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
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
            if (__shfl_sync(0xffffffffu, quit, 0))
                return false;
        }
    }
}

__device__ __forceinline__ bool wait_stage(uint32_t bar, uint32_t parity, volatile int *stop, int32_t *err, int lane)
{
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || wait_slow(bar, parity, stop, err, lane);
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

// acc += V^T P^T and sum += 1^T P^T for a tile; b: the weights of its 16 tokens
// (B fragment) in kParts f16 parts.
template <int kParts>
__device__ __forceinline__ void accumulate(const RawV &x, const uint32_t (&b)[kParts][2], float (&acc)[8][4],
                                           float (&sum)[4])
{
    const uint32_t s0 = e4m3x2_to_f16x2(x.s[0]), s1 = e4m3x2_to_f16x2(x.s[1]);
    constexpr uint32_t kLow = 0x0F0F0F0Fu, kOnes = 0x3C003C00u;
#pragma unroll
    for (int part = 0; part < kParts; ++part)
        mma_16816(sum, kOnes, kOnes, kOnes, kOnes, b[part][0], b[part][1]);
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

// kParts: f16 parts of a softmax weight.  One (rounded to f16, 2^-11, and the
// normalising sum is of the rounded ones) is enough under a bf16 output's
// 2^-8; two keep an fp32 output to 2^-21.
// kCluster: short work, one cluster of da.cluster CTAs a segment.  Its warps
// share the segment's units evenly, leave their states in shared memory and
// join them there: one launch and no partial states in memory.
template <int kParts, bool kCluster>
__global__ void __launch_bounds__(kThreadsD, kFp4DecodeCtas) paged_gqa_decode_fp4_kernel(const Fp4DecodeArgs da)
{
    const Fp4AttnArgs &a = da.a;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int *start = reinterpret_cast<int *>(smem + SmemD::kStart);
    volatile int *stop = reinterpret_cast<volatile int *>(smem + SmemD::kFlag);
    int *sums = reinterpret_cast<int *>(smem + SmemD::kSums);

    int worker, lo, n;                                     // this warp's units: n from list position lo
    Place seg = {0, 0, 0};                                 // kCluster: the segment, and its units
    int seg_units = 0, rank = 0;
    if constexpr (kCluster) {
        rank = static_cast<int>(blockIdx.x) % da.cluster;
        const int sg = static_cast<int>(blockIdx.x) / da.cluster;
        seg.b = sg / a.hkv;
        seg.h = sg % a.hkv;
        const Sight s = sight_of(a, seg.b);
        seg_units = (s.tiles + 1) >> 1;
        if (tid == 0) {
            *stop = 0;
            for (int i = 0; i < kWarpsD * kStagesD; ++i)
                mbar_init(smem_addr(smem + SmemD::kBar) + 8 * i, 1);
            fence_barrier_init();
            if (a.err && rank == 0 && seg.h == 0) {
                if (seq_page_log2(a, seg.b) < 0)
                    atomicOr(a.err, PKV_DEVERR_PAGESIZE);
                else if (__ldg(a.seq_lens + seg.b) != s.len)
                    atomicOr(a.err, PKV_DEVERR_SEQLEN);
            }
        }
        __syncthreads();
        const int at = rank * kWarpsD + warp, workers = da.cluster * kWarpsD;
        worker = static_cast<int>(blockIdx.x) * kWarpsD + warp;
        lo = seg_units * at / workers;
        n = seg_units * (at + 1) / workers - lo;
    } else {
    // ---- first unit of every sequence (of one kv head): a prefix sum over the batch
    {
        const int per = (a.batch + kThreadsD - 1) / kThreadsD;
        const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
        int mine = 0;
        for (int b = b0; b < b1; ++b)
            mine += (sight_of(a, b).tiles + 1) >> 1;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += v;
        }
        if (lane == 31)
            sums[warp] = incl;
        if (tid == 0) {
            *stop = 0;
            for (int s = 0; s < kWarpsD * kStagesD; ++s)
                mbar_init(smem_addr(smem + SmemD::kBar) + 8 * s, 1);
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
            if (blockIdx.x == 0 && a.err) {
                if (seq_page_log2(a, b) < 0)
                    atomicOr(a.err, PKV_DEVERR_PAGESIZE);
                else if (__ldg(a.seq_lens + b) != s.len)
                    atomicOr(a.err, PKV_DEVERR_SEQLEN);
            }
        }
        if (tid == kThreadsD - 1)
            start[a.batch] = run;
        __syncthreads();
    }

    // ---- sequences with no tokens: zero rows, and nothing to join
    for (int sg = blockIdx.x; sg < a.batch * a.hkv; sg += gridDim.x) {
        const int b = sg / a.hkv;
        if (start[b + 1] == start[b]) {
            const int64_t row0 = static_cast<int64_t>(b) * a.hq + static_cast<int64_t>(sg % a.hkv) * a.group;
            for (int e = tid; e < a.group * kHeadDim; e += kThreadsD) {
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
    worker = warp * gridDim.x + blockIdx.x;
    const int active = min(static_cast<int>(gridDim.x) * kWarpsD, total);
    if (worker >= active)
        return;                                            // no CTA barrier follows
    lo = static_cast<int>(static_cast<int64_t>(total) * worker / active);
    n = static_cast<int>(static_cast<int64_t>(total) * (worker + 1) / active) - lo;
    }
    auto place = [&](int x) -> Place {
        if constexpr (kCluster)
            return Place{seg.b, seg.h, x};
        else
            return place_of(start, a.batch, x);
    };

    const uint32_t ring = smem_addr(smem) + warp * kStagesD * kUnitBytes;
    const uint32_t bars = smem_addr(smem + SmemD::kBar) + warp * kStagesD * 8;

    // a piece's query rows (kCluster: on their way while the tiles are looked up)
    const int r = lane >> 2, c = lane & 3;
    uint4 qraw[4];
    float kscale;
    auto load_q = [&](const Place &p) {
        const int64_t row = static_cast<int64_t>(p.b) * a.hq + static_cast<int64_t>(p.h) * a.group + (r < a.group ? r : 0);
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + row * kHeadDim + 32 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            qraw[i] = __ldg(src + i);
        kscale = __ldg(a.k_scale + p.h);
    };
    float vscale = 0.f;
    if constexpr (kCluster) {
        load_q(seg);
        vscale = __ldg(a.v_scale + seg.h);
    }

    const uint64_t policy = l2_policy_evict_first();
    float *state = reinterpret_cast<float *>(smem + warp * kStagesD * kUnitBytes);   // kCluster: over the ring, at the end

    // ---- tile addresses, 16 units ahead: lane 2i + j has tile j of unit i.
    // -1: a page outside the pool; -2: no such tile.
    auto look_up = [&](int u0) -> int {
        const int u = u0 + (lane >> 1);
        if (u >= n)
            return -2;
        const Place p = place(lo + u);
        const Sight s = sight_of(a, p.b);
        const int i = 2 * p.unit + (lane & 1);
        if (i >= s.tiles)
            return -2;
        int phys, row;
        if (!seq_token_page(a, p.b, seq_page_log2(a, p.b), 16 * tile_at(s, i), phys, row)) {
            if (a.err)
                atomicOr(a.err, PKV_DEVERR_PAGE);
            return -1;
        }
        return (phys * a.hkv + p.h) * (a.page_size >> 4) + (row >> 4);
    };
    int now = look_up(0), next = look_up(16), base = 0;
    uint32_t have = __ballot_sync(0xffffffffu, now >= 0);
    uint32_t bad = 0;                                      // missing tiles, 2 bits a stage
    const uint32_t my_dst = ring + (lane & 3) * kFp4Tile;  // lanes 0, 1 bring K tiles; 2, 3: V tiles
    const uint8_t *my_src = lane < 2 ? a.k_cache : a.v_cache;
    auto issue = [&](int u, int s) {                       // unit u into stage s = u % kStagesD
        if (u >= base + 16) {
            base += 16;
            now = next;
            have = __ballot_sync(0xffffffffu, now >= 0);
            next = look_up(base + 16);
        }
        const int i = 2 * (u - base);
        const int t = __shfl_sync(0xffffffffu, now, i + (lane & 1));
        const uint32_t both = (have >> i) & 3u;
        bad = (bad & ~(3u << (2 * s))) | ((both ^ 3u) << (2 * s));
        if (lane < 4 && (worker != da.withhold || u != 0)) {
            const uint32_t bar = bars + 8 * s;
            // (bytes that land before they are announced are only counted early)
            if (lane == 0)
                mbar_arrive_expect_tx(bar, both == 3u ? 4 * kFp4Tile : both ? 2 * kFp4Tile : 0);
            if (t >= 0)
                bulk_load(my_dst + s * kUnitBytes, my_src + static_cast<int64_t>(t) * kFp4Tile, kFp4Tile, bar, policy);
        }
    };
    for (int v = 0; v < kStagesD && v < n; ++v)
        issue(v, v);

    const LaneOffsets lo_off = lane_offsets(r, c);
    int stage = 0;
    uint32_t parity = 0;
    bool dead = false;                                     // a wait ran out
    int u = 0;
    while (u < n) {
        const Place p = place(lo + u);
        const Sight sg = sight_of(a, p.b);
        const int units = kCluster ? seg_units : start[p.b + 1] - start[p.b];
        const int take = min(units - p.unit, n - u);
        const bool whole = p.unit == 0 && take == units;
        const int64_t row0 = static_cast<int64_t>(p.b) * a.hq + static_cast<int64_t>(p.h) * a.group;
        if (!kCluster && lane == 0) {                      // who holds the segment's first and last unit
            int2 *j = da.joins + p.b * a.hkv + p.h;
            if (p.unit == 0)
                j->x = whole ? -1 : worker;
            if (p.unit + take == units)
                j->y = worker;
        }
        // Q as B fragment: head r, dims 32c + 4 kk + {0, 1} and {2, 3}; brought
        // to [1, 2) by a power of two, so that f16 holds all its bits.
        uint32_t q[8][2];
        float f0, f1;
        {
            if (!kCluster)
                load_q(p);
            const uint32_t *w = reinterpret_cast<const uint32_t *>(qraw);
            uint32_t top = 0;                              // largest |q|, as its bits
#pragma unroll
            for (int i = 0; i < 16; ++i)
                top = max(top, max((w[i] << 16) & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = min(max(static_cast<int>(top >> 23), 1), 253);
            const float down = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);
            const float up = __uint_as_float(static_cast<uint32_t>(ex) << 23) * (kscale * a.sm_scale_log2);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const bool on = r < a.group;
                q[i >> 1][i & 1] = f32x2_to_f16x2(on ? __uint_as_float(w[i] << 16) * down : 0.f,
                                                  on ? __uint_as_float(w[i] & 0xFFFF0000u) * down : 0.f);
            }
            f0 = __shfl_sync(0xffffffffu, up, 8 * c);
            f1 = __shfl_sync(0xffffffffu, up, 8 * c + 4);
        }
        const uint64_t f = pack2(f0, f1);
        const int64_t slot = static_cast<int64_t>(worker) + p.h * a.batch + p.b;
        // units of which every token is visible: past the sinks and the window's
        // first tile, before the last tokens
        const int full_lo = (sg.from > 0 ? sg.first + 2 : 1) >> 1;
        const int full_hi = ((sg.len >> 4) - sg.skip) >> 1;
        float m0 = -INFINITY, m1 = -INFINITY, mf0 = -INFINITY, mf1 = -INFINITY;
        float l0 = 0.f, l1 = 0.f;                          // sums of the units folded so far
        float acc[8][4], sum[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            sum[k] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                acc[i][k] = 0.f;
        }

        for (int i = 0; i < take; ++i, ++u) {
            const uint32_t st = ring + stage * kUnitBytes;
            if (!wait_stage(bars + 8 * stage, parity, stop, a.err, lane)) {
                dead = true;
                break;
            }
            const uint32_t missing = (bad >> (2 * stage)) & 3u;
            uint64_t y[2][2];
            {
                RawK x[2];
                load_k(st, lo_off, x[0]);
                load_k(st + kFp4Tile, lo_off, x[1]);
                if (missing) {                             // a missing page reads as zeros
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (missing & (1u << j))
                            x[j].s[0] = x[j].s[1] = 0u;
                }
                scores(x[0], q, y[0]);
                scores(x[1], q, y[1]);
            }
            RawV xv[2];
            load_v(st + 2 * kFp4Tile, lo_off, xv[0]);
            load_v(st + 3 * kFp4Tile, lo_off, xv[1]);
            if (u + kStagesD < n) {                        // the stage just read takes the unit after the ring's
                fence_proxy_async_smem();
                __syncwarp();
                issue(u + kStagesD, stage);
            }
            if (++stage == kStagesD) {
                stage = 0;
                parity ^= 1u;
            }
            const int unit = p.unit + i;
            uint32_t seen = 0xffffffffu;                   // the visible ones of the unit's 32 tokens
            float2 z[2][2];
            const uint64_t nm = pack2(-m0, -m1);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    z[j][k] = unpack2(fma2(y[j][k], f, nm));
            const bool edge = unit < full_lo || unit >= full_hi;
            const float top = fmaxf(max3(fmaxf(z[0][0].x, z[0][0].y), z[0][1].x, z[0][1].y),
                                    max3(fmaxf(z[1][0].x, z[1][0].y), z[1][1].x, z[1][1].y));
            if (edge || __any_sync(0xffffffffu, !(top <= kMoveMax))) {
                // an edge of the sequence or of its window, or the maximum moves
                if (edge) {
                    const int ti = 2 * unit + (lane >> 4);
                    const int t = 16 * tile_at(sg, ti) + (lane & 15);
                    seen = __ballot_sync(0xffffffffu,
                                         ti < sg.tiles && t < sg.len && (t < sg.sinks || t >= sg.from));
                }
                float t0 = -INFINITY, t1 = -INFINITY;
                float2 w[2][2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        w[j][k] = unpack2(y[j][k]);
                        const bool on = (seen >> (16 * j + 8 * k + order(r))) & 1u;
                        w[j][k].x = on ? w[j][k].x * f0 : -INFINITY;
                        w[j][k].y = on ? w[j][k].y * f1 : -INFINITY;
                        t0 = fmaxf(t0, w[j][k].x);
                        t1 = fmaxf(t1, w[j][k].y);
                    }
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, o));
                    t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, o));
                }
                const float n0 = t0 > m0 + kMoveMax ? t0 : m0, n1 = t1 > m1 + kMoveMax ? t1 : m1;
                const float g0 = n0 == m0 ? 1.f : ex2_approx(m0 - n0), g1 = n1 == m1 ? 1.f : ex2_approx(m1 - n1);
                m0 = n0;
                m1 = n1;
                sum[0] *= g0;
                sum[1] *= g1;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    acc[k][0] *= g0;
                    acc[k][1] *= g1;
                    acc[k][2] *= g0;
                    acc[k][3] *= g1;
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        z[j][k] = make_float2(w[j][k].x - m0, w[j][k].y - m1);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                RawV &x = xv[j];
                if (seen != 0xffffffffu || missing) {      // values of unseen tokens may be anything
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t s = missing & (1u << j) ? 0u : seen >> (16 * j + 8 * k);
                        x.s[k] &= ((s >> order(2 * c)) & 1u ? 0x00FFu : 0u) |
                                  ((s >> order(2 * c + 1)) & 1u ? 0xFF00u : 0u);
                    }
                }
                const float p0 = ex2_approx(z[j][0].x), p1 = ex2_approx(z[j][0].y);
                const float p2 = ex2_approx(z[j][1].x), p3 = ex2_approx(z[j][1].y);
                const uint32_t ha = f32x2_to_f16x2(p0, p1), hb = f32x2_to_f16x2(p2, p3);
                uint32_t b[kParts][2];
                b[0][0] = transpose8x8(ha);
                b[0][1] = transpose8x8(hb);
                if constexpr (kParts == 2) {
                    const float2 va = f16x2_to_f32x2(ha), vb = f16x2_to_f32x2(hb);
                    b[1][0] = transpose8x8(f32x2_to_f16x2(p0 - va.x, p1 - va.y));
                    b[1][1] = transpose8x8(f32x2_to_f16x2(p2 - vb.x, p3 - vb.y));
                }
                accumulate<kParts>(x, b, acc, sum);
            }
            // (a cluster's warps have fewer units than a fold)
            if (!kCluster && ((i + 1) % kFoldUnits<kParts> == 0 || (i + 1 == take && take > kFoldUnits<kParts>))) {
                // the piece's own slot of the workspace holds the copy (each lane its own elements)
                const float g0 = i + 1 > kFoldUnits<kParts> ? ex2_approx(mf0 - m0) : 0.f;
                const float g1 = i + 1 > kFoldUnits<kParts> ? ex2_approx(mf1 - m1) : 0.f;
                const bool old = i + 1 > kFoldUnits<kParts>, last = i + 1 == take;
                if (slot >= da.num_slots) {
                    if (a.err && lane == 0)
                        atomicOr(a.err, PKV_DEVERR_INTERNAL);
                } else {
                    float *s = da.partials + slot * a.group * kPartialStride;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (2 * c + j >= a.group)
                            continue;
                        float *at = s + (2 * c + j) * kPartialStride + 16 * r;
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            float &v = acc[k >> 1][2 * (k & 1) + j];
                            v += old ? at[k] * (j ? g1 : g0) : 0.f;
                            if (!last) {
                                at[k] = v;
                                v = 0.f;
                            }
                        }
                    }
                }
                l0 = l0 * g0 + sum[0];
                l1 = l1 * g1 + sum[1];
                sum[0] = last ? l0 : 0.f;
                sum[1] = last ? l1 : 0.f;
                mf0 = m0;
                mf1 = m1;
            }
        }
        if (dead)
            break;

        // ---- end of piece: heads 2c, 2c + 1; dims 16 r ..
        __syncwarp();                                      // (kCluster: the state overwrites the ring)
        l0 = sum[0];
        l1 = sum[1];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int g = 2 * c + j;
            if (g >= a.group)
                continue;
            float v[16];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[2 * k] = acc[k][j];
                v[2 * k + 1] = acc[k][j + 2];
            }
            if constexpr (kCluster) {
                float *s = state + g * kPartialStride;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    reinterpret_cast<float4 *>(s + 16 * r)[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                if (r == 0)
                    *reinterpret_cast<float2 *>(s + kHeadDim) = make_float2(j ? m1 : m0, j ? l1 : l0);
            } else if (whole) {
                const float f = __ldg(a.v_scale + p.h) / (j ? l1 : l0);
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    v[k] *= f;
                store16(a, row0 + g, 16 * r, v);
            } else if (slot < da.num_slots) {
                float *s = da.partials + (slot * a.group + g) * kPartialStride;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    reinterpret_cast<float4 *>(s + 16 * r)[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                if (r == 0)
                    *reinterpret_cast<float2 *>(s + kHeadDim) = make_float2(j ? m1 : m0, j ? l1 : l0);
            } else if (a.err && r == 0) {
                atomicOr(a.err, PKV_DEVERR_INTERNAL);
            }
        }
    }

    // After an abort: no copy may land in this ring once the warp has left.
    if (dead)
        for (int v = u; v < n && v < u + kStagesD; ++v) {
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(bars + 8 * (v % kStagesD), (v / kStagesD) & 1u) &&
                   global_timer_ns() - t0 < kLimitNs) {
            }
        }

    if constexpr (kCluster) {
        // ---- join the cluster's states (at most 32, one a lane), in worker
        // order: CTA k takes the heads k, k + CTAs, ..; of several CTAs each warp
        // 32 dims of all of them, of one CTA a warp every fourth head
        if ((n == 0 || dead) && lane < a.group)
            *reinterpret_cast<float2 *>(state + lane * kPartialStride + kHeadDim) = make_float2(-INFINITY, 0.f);
        cluster_sync(da.cluster);
        const bool one = da.cluster == 1;
        const int workers = da.cluster * kWarpsD;
        for (int g = one ? warp : rank; g < a.group; g += one ? kWarpsD : da.cluster) {
            const uint32_t mine = smem_addr(smem) + g * kPartialStride * 4;    // warp 0's state of this head, this CTA
            float m = -INFINITY, l = 0.f;
            if (lane < workers) {
                const uint32_t at = mine + (lane & 3) * kStagesD * kUnitBytes + kHeadDim * 4;
                m = cluster_load(at, lane >> 2, one);
                l = cluster_load(at + 4, lane >> 2, one);
            }
            float M = m;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            const float e = m == -INFINITY ? 0.f : ex2_approx(m - M);
            float sum = e * l;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float f = seg_units == 0 ? 0.f : vscale / sum;
            const int64_t row = static_cast<int64_t>(seg.b) * a.hq + static_cast<int64_t>(seg.h) * a.group + g;
            // (what a warp without units left is read, but not used)
            if (one) {
                float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < kWarpsD; ++i) {
                    const float ei = __shfl_sync(0xffffffffu, e, i);
                    const float4 v = *reinterpret_cast<const float4 *>(smem + i * kStagesD * kUnitBytes +
                                                                       (g * kPartialStride + 4 * lane) * 4);
                    A.x += ei != 0.f ? ei * v.x : 0.f;
                    A.y += ei != 0.f ? ei * v.y : 0.f;
                    A.z += ei != 0.f ? ei * v.z : 0.f;
                    A.w += ei != 0.f ? ei * v.w : 0.f;
                }
                store4(a, row, 4 * lane, make_float4(A.x * f, A.y * f, A.z * f, A.w * f));
            } else {
                const int d = 32 * warp + lane;
                float A = 0.f;
                float v[32];                               // all on their way together: one round trip
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    v[i] = i < workers ? cluster_load(mine + (i & 3) * kStagesD * kUnitBytes + 4 * d, i >> 2, false) : 0.f;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float ei = __shfl_sync(0xffffffffu, e, i);
                    A += ei != 0.f ? ei * v[i] : 0.f;
                }
                if (a.out_f32)
                    static_cast<float *>(a.out)[row * kHeadDim + d] = A * f;
                else
                    static_cast<__nv_bfloat16 *>(a.out)[row * kHeadDim + d] = __float2bfloat16_rn(A * f);
            }
        }
        cluster_sync(da.cluster);                          // no CTA leaves while its states are read
    }
}

// Joins the states of a segment's pieces for one query head, in worker order:
// out = v_scale sum_i 2^(m_i - M) A_i / sum_i 2^(m_i - M) l_i.  A CTA per
// (segment, head); its warps take the pieces in turns of kJoin, all of a
// turn's loads in flight together, and are joined in warp order.
constexpr int kJoin = 8;
constexpr int kJoinWarps = 8;

__global__ void __launch_bounds__(32 * kJoinWarps) join_fp4_kernel(const Fp4DecodeArgs da)
{
    __shared__ __align__(16) float ra[kJoinWarps][kHeadDim];
    __shared__ float2 rm[kJoinWarps];
    const Fp4AttnArgs &a = da.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int sg = blockIdx.x / a.group, g = blockIdx.x % a.group;
    const int b = sg / a.hkv, h = sg % a.hkv;
    const float vs = __ldg(a.v_scale + h);
    grid_wait();
    const int2 j = da.joins[sg];
    if (j.x < 0)
        return;
    const int pieces = j.y - j.x + 1;
    const int64_t slot0 = static_cast<int64_t>(j.x) + h * a.batch + b;
    if (j.y < j.x || slot0 + pieces > da.num_slots)
        return;                                            // an aborted call, or flagged by the decode kernel
    const float *base = da.partials + (slot0 * a.group + g) * kPartialStride;
    const int64_t stride = static_cast<int64_t>(a.group) * kPartialStride;
    float M = -INFINITY, L = 0.f;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = warp * kJoin; i0 < pieces; i0 += warps * kJoin) {
        float4 v[kJoin];
        float2 ml[kJoin];
#pragma unroll
        for (int i = 0; i < kJoin; ++i) {
            const bool on = i0 + i < pieces;
            const float *s = base + (on ? i0 + i : 0) * stride;
            ml[i] = on ? *reinterpret_cast<const float2 *>(s + kHeadDim) : make_float2(-INFINITY, 0.f);
            v[i] = on ? *reinterpret_cast<const float4 *>(s + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float mn = M;
#pragma unroll
        for (int i = 0; i < kJoin; ++i)
            mn = fmaxf(mn, ml[i].x);
        const float f = ex2_approx(M - mn);
        M = mn;
        L *= f;
        A = make_float4(A.x * f, A.y * f, A.z * f, A.w * f);
#pragma unroll
        for (int i = 0; i < kJoin; ++i) {
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
            if (w * kJoin >= pieces)
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

}  // namespace

size_t decode_fp4_smem(int batch)
{
    return SmemD::bytes(batch);
}

const void *decode_fp4_kernel(bool two_parts, bool cluster)
{
    if (cluster)
        return two_parts ? reinterpret_cast<const void *>(&paged_gqa_decode_fp4_kernel<2, true>)
                         : reinterpret_cast<const void *>(&paged_gqa_decode_fp4_kernel<1, true>);
    return two_parts ? reinterpret_cast<const void *>(&paged_gqa_decode_fp4_kernel<2, false>)
                     : reinterpret_cast<const void *>(&paged_gqa_decode_fp4_kernel<1, false>);
}

// A cluster a segment, of the fewest CTAs (1, 2, 4, 8) that leave a warp at
// most kClusterUnits units, if all of them are resident at once; 0: the list.
// (`units`: of the longest sequence, `slots`: resident CTAs.)
int decode_fp4_cluster(long long units, long long segments, int slots)
{
    for (int c = 1; c <= 8; c *= 2)
        if (units <= static_cast<long long>(c) * kWarpsD * kClusterUnits)
            return segments * c <= slots ? c : 0;
    return 0;
}

cudaError_t launch_paged_decode_fp4(const Fp4DecodeArgs &da, int ctas, cudaStream_t stream, const char **site)
{
    *site = "4-bit decode kernel launch";
    const bool two = da.a.out_f32;
    if (da.cluster > 0) {
        const dim3 grid(static_cast<unsigned>(da.a.batch * da.a.hkv * da.cluster));
        return launch_with(two ? paged_gqa_decode_fp4_kernel<2, true> : paged_gqa_decode_fp4_kernel<1, true>, grid,
                           kThreadsD, SmemD::bytes(0), da.cluster, false, stream, da);
    }
    cudaError_t e = launch_with(two ? paged_gqa_decode_fp4_kernel<2, false> : paged_gqa_decode_fp4_kernel<1, false>,
                                dim3(static_cast<unsigned>(ctas)), kThreadsD, SmemD::bytes(da.a.batch), 1, false, stream,
                                da);
    if (e != cudaSuccess)
        return e;
    *site = "4-bit join kernel launch";
    const long long segs = static_cast<long long>(da.a.batch) * da.a.hkv;
    const long long pieces = (static_cast<long long>(ctas) * kWarpsD + segs - 1) / segs + 1;   // a segment's, on average
    int warps = 1;
    while (warps < kJoinWarps && warps * kJoin < pieces)
        warps *= 2;
    return launch_with(join_fp4_kernel, dim3(static_cast<unsigned>(segs * da.a.group)), 32 * warps, 0, 1, true, stream,
                       da);
}

}  // namespace pkv
