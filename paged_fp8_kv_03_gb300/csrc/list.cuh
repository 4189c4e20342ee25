// The decode kernels' list of units, shared evenly among the warps of a grid
// whatever the sequences' lengths, and the kernels that join what the pieces of a
// cut segment have left.  (The figures are the 4-bit cache's.)
//
// A piece's state of a head is a row of kPartialStride floats: the accumulator, the
// reference m of its weights' exponents and their sum, and, with kOwnRef, the
// reference of the accumulator where that is another one: n + e, e a whole number, kept
// apart so that exponents around it stay small and their differences exact.
#pragma once

#include "grid.cuh"
#include "split.cuh"

namespace pkv {

struct Reference {
    float n, e;
    __device__ __forceinline__ float over(const Reference &o) const { return (n - o.n) + (e - o.e); }
};

// The larger of two.
__device__ __forceinline__ Reference larger(const Reference &a, const Reference &b)
{
    return a.n + a.e >= b.n + b.e ? a : b;
}

constexpr int kRowM = kHeadDim, kRowRef = kHeadDim + 2;   // m, sum; n, e

// start[b]: the first unit of sequence b (of one kv head), start[batch]: how many
// there are (the whole CTA; sums: kWarps ints of shared memory; init: what thread
// 0 sets up meanwhile).  True if no sequence is empty.
template <int kWarps, typename Init>
__device__ __forceinline__ bool list_starts(const CacheAttnArgs &a, int *start, int *sums, Init init)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (a.batch + (32 * kWarps) - 1) / (32 * kWarps);
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
    if (tid == 0)
        init();
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
    if (tid == (32 * kWarps) - 1)
        start[a.batch] = run;
    bool some = true;                                  // this thread's sequences all have tokens
    for (int b = b0; b < b1; ++b)
        some = some && (b + 1 < b1 ? start[b + 1] : run) > start[b];
    return __syncthreads_and(some) != 0;
}

// Sequences with no tokens: zero rows, and nothing to join.
template <int kThreads>
__device__ __forceinline__ void zero_rows(const SplitArgs &da, const int *start)
{
    const CacheAttnArgs &a = da.a;
    const int tid = threadIdx.x;
    for (int sg = blockIdx.x; sg < a.batch * a.hkv; sg += gridDim.x) {
        const int b = sg / a.hkv;
        if (start[b + 1] == start[b]) {
            const int64_t row0 = static_cast<int64_t>(b) * a.hq + static_cast<int64_t>(sg % a.hkv) * a.group;
            for (int e = tid; e < a.group * kHeadDim; e += kThreads) {
                if (a.out_f32)
                    static_cast<float *>(a.out)[row0 * kHeadDim + e] = 0.f;
                else
                    static_cast<__nv_bfloat16 *>(a.out)[row0 * kHeadDim + e] = __float2bfloat16_rn(0.f);
            }
            if (tid == 0)
                da.joins[sg] = make_int2(-1, -1);
        }
    }
}

// A warp's range of the list: units lo .. lo + n - 1.  how: the slot of the one state
// that the CTA's warps leave together (their ranges lie within one segment), or
// that the CTA's ranges are ADJACENT, or SPREAD over the list.
struct ListRange {
    enum { SPREAD = -1, ADJACENT = -2 };
    bool on;
    int worker, lo, n, how;
};

template <int kWarps>
__device__ __forceinline__ ListRange list_range(const SplitArgs &da, const int *start, bool no_empty, int warp, int lane)
{
    const CacheAttnArgs &a = da.a;
    ListRange r = {false, 0, 0, 0, 0};
    const int total = start[a.batch] * a.hkv;
    const int active = min(static_cast<int>(gridDim.x) * kWarps, total);
    // A CTA's warps take adjacent ranges, so that those within a segment leave one
    // state for the join (32 query heads, one 32K sequence 16.8 us, with a state a warp
    // 18.2; a 128K one among 63 of 512 tokens 46.0 and 57.8; 32 x 4K 34.2 and 33.8).  The
    // ranges of a list shorter than the workers spread over the CTAs.
    const bool adjacent = total >= static_cast<int>(gridDim.x) * kWarps;
    const int worker = r.worker = adjacent ? static_cast<int>(blockIdx.x) * kWarps + warp
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
        const int w = (lane & 2 ? worker - warp : worker) + (lane & 1) * (lane & 2 ? kWarps : 1);
        int edge = w * each + min(w, more);
        if (wide)
            edge = real_position(start, a.batch, a.hkv, edge);
        r.on = true;
        r.lo = __shfl_sync(kEvery, edge, 0);
        r.n = __shfl_sync(kEvery, edge, 1) - r.lo;
        const int first = __shfl_sync(kEvery, edge, 2), last = __shfl_sync(kEvery, edge, 3);
        r.how = ListRange::SPREAD;
        if (adjacent) {
            const Place p = place_of(start, a.batch, first);
            const bool within = p.unit > 0 && last - first < start[p.b + 1] - start[p.b] - p.unit;
            r.how = within ? worker - warp + p.h * a.batch + p.b : static_cast<int>(ListRange::ADJACENT);
        }
    }
    return r;
}

// Joins the states of a CTA's warps, whose ranges all lie within one segment,
// into one (out: [group][kPartialStride]).  Out of line, for the loop above it (in
// line, the mixed batch takes 0.5% longer).
template <bool kOwnRef, int kWarps, int kWarpBytes>
__device__ __noinline__ void join_warps(float *out, int group, uint8_t *smem, int warp, int lane)
{
    auto state = [&](int w) { return reinterpret_cast<const float *>(smem + w * kWarpBytes); };
    for (int g = warp; g < group; g += kWarps) {
        float m[kWarps], l[kWarps], M = -INFINITY, L = 0.f;
        Reference n[kWarps], N = {-INFINITY, 0.f};
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float2 ml = *reinterpret_cast<const float2 *>(state(w) + g * kPartialStride + kRowM);
            m[w] = ml.x;
            l[w] = ml.y;
            M = fmaxf(M, ml.x);
            if (kOwnRef) {
                const float2 ref = *reinterpret_cast<const float2 *>(state(w) + g * kPartialStride + kRowRef);
                n[w] = Reference{ref.x, ref.y};
                N = larger(n[w], N);
            }
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float e = ex2_approx(m[w] - M);
            const float4 v = *reinterpret_cast<const float4 *>(state(w) + g * kPartialStride + 4 * lane);
            const float ea = kOwnRef ? ex2_approx(n[w].over(N)) : e;
            L += e * l[w];
            A.x += ea * v.x;
            A.y += ea * v.y;
            A.z += ea * v.z;
            A.w += ea * v.w;
        }
        float *row = out + g * kPartialStride;
        *reinterpret_cast<float4 *>(row + 4 * lane) = A;
        if (lane == 0) {
            *reinterpret_cast<float2 *>(row + kRowM) = make_float2(M, L);
            if (kOwnRef)
                *reinterpret_cast<float2 *>(row + kRowRef) = make_float2(N.n, N.e);
        }
    }
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
// (kOwnRef: 12 states, as many as the registers hold.)
template <bool kOwnRef>
constexpr int kJoin = kOwnRef ? 12 : 16;
constexpr int kJoinWarps = 16;
constexpr int kJoinCut = 8;

// Head g of segment sg, by `warps` warps of the CTA (ra, rm: theirs), kTurn pieces
// a turn.
template <bool kOwnRef, int kTurn>
__device__ __forceinline__ void join_head(const SplitArgs &da, int sg, int g, int warp, int warps, int lane,
                                          float (*ra)[kHeadDim], float4 *rm)
{
    const CacheAttnArgs &a = da.a;
    const int b = sg / a.hkv, h = sg % a.hkv;
    const float vs = kOwnRef ? 1.f : __ldg(a.v_scale + h);
    int2 j = da.joins[sg];
    if (j.x < 0)
        return;
    // Of the workers x .. y, the CTAs strictly between have left one state, in the first
    // of their slots (y = ~the last worker; else every worker has its own).
    int head = 0, full = 0;
    if (j.y < 0) {
        j.y = ~j.y;
        head = kSplitWarps - j.x % kSplitWarps;
        full = max(0, j.y / kSplitWarps - 1 - j.x / kSplitWarps);
    }
    const int64_t slot0 = static_cast<int64_t>(j.x) + h * a.batch + b;
    if (j.y < j.x || slot0 + (j.y - j.x) >= da.num_slots)
        return;                                            // an aborted call, or flagged by the decode kernel
    const int pieces = j.y - j.x + 1 - (kSplitWarps - 1) * full;
    auto worker = [&](int i) {                             // beyond x
        return i < head || full == 0 ? i : (i < head + full ? head + kSplitWarps * (i - head) : i + (kSplitWarps - 1) * full);
    };
    const float *base = da.partials + (slot0 * a.group + g) * kPartialStride;
    const int64_t stride = static_cast<int64_t>(a.group) * kPartialStride;
    float M = -INFINITY, L = 0.f;
    Reference N = {-INFINITY, 0.f};
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = warp * kTurn; i0 < pieces; i0 += warps * kTurn) {
        float4 v[kTurn];
        float2 ml[kTurn];
        Reference n[kTurn];
#pragma unroll
        for (int i = 0; i < kTurn; ++i) {
            const bool on = i0 + i < pieces;
            const float *s = base + (on ? worker(i0 + i) : 0) * stride;
            ml[i] = on ? *reinterpret_cast<const float2 *>(s + kRowM) : make_float2(-INFINITY, 0.f);
            if (kOwnRef) {
                const float2 ref = on ? *reinterpret_cast<const float2 *>(s + kRowRef) : make_float2(-INFINITY, 0.f);
                n[i] = Reference{ref.x, ref.y};
            }
            v[i] = on ? *reinterpret_cast<const float4 *>(s + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float mn = M;
        Reference nn = N;
#pragma unroll
        for (int i = 0; i < kTurn; ++i) {
            mn = fmaxf(mn, ml[i].x);
            if (kOwnRef)
                nn = larger(n[i], nn);
        }
        const float f = ex2_approx(M - mn), fa = kOwnRef ? ex2_approx(N.over(nn)) : f;
        M = mn;
        N = nn;
        L *= f;
        A = make_float4(A.x * fa, A.y * fa, A.z * fa, A.w * fa);
#pragma unroll
        for (int i = 0; i < kTurn; ++i) {
            const float e = i0 + i < pieces ? ex2_approx(ml[i].x - mn) : 0.f;
            const float ea = kOwnRef ? (i0 + i < pieces ? ex2_approx(n[i].over(nn)) : 0.f) : e;
            L += e * ml[i].y;
            A.x += ea * v[i].x;
            A.y += ea * v[i].y;
            A.z += ea * v[i].z;
            A.w += ea * v[i].w;
        }
    }
    if (warps > 1) {
        *reinterpret_cast<float4 *>(&ra[warp][4 * lane]) = A;
        if (lane == 0)
            rm[warp] = make_float4(M, L, N.n, N.e);
        __syncthreads();
        if (warp != 0)
            return;
        float mn = M;
        Reference nn = N;
        for (int w = 1; w < warps; ++w) {
            mn = fmaxf(mn, rm[w].x);
            if (kOwnRef)
                nn = larger(Reference{rm[w].z, rm[w].w}, nn);
        }
        M = mn;
        N = nn;
        L = 0.f;
        A = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < warps; ++w) {
            if (w * kTurn >= pieces)
                break;                                     // a warp with no pieces
            const float e = ex2_approx(rm[w].x - mn), ea = kOwnRef ? ex2_approx(Reference{rm[w].z, rm[w].w}.over(nn)) : e;
            const float4 v = *reinterpret_cast<const float4 *>(&ra[w][4 * lane]);
            L += e * rm[w].y;
            A.x += ea * v.x;
            A.y += ea * v.y;
            A.z += ea * v.z;
            A.w += ea * v.w;
        }
    }
    const int64_t row = static_cast<int64_t>(b) * a.hq + static_cast<int64_t>(h) * a.group + g;
    if (kOwnRef) {
        store4(a, row, 4 * lane, Quotient(N.n - M, N.e, L)(A));
    } else {
        const float f = vs / L;
        store4(a, row, 4 * lane, make_float4(A.x * f, A.y * f, A.z * f, A.w * f));
    }
}

template <bool kOwnRef>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const SplitArgs da)
{
    __shared__ __align__(16) float ra[kJoinWarps][kHeadDim];
    __shared__ float4 rm[kJoinWarps];
    grid_wait();
    join_head<kOwnRef, kJoin<kOwnRef>>(da, blockIdx.x / da.a.group, blockIdx.x % da.a.group, threadIdx.x >> 5, blockDim.x >> 5,
                     threadIdx.x & 31, ra, rm);
}

// The same for lists of many segments, of which at most one a worker is cut: a CTA a
// worker, for the segment that its range begins and does not end; a warp a head.  A
// CTA a (segment, head) is what such lists spend their time on: 64 query heads, 512 x
// 128 tokens 43 us, this way 31; 1024 x 128 84 and 55; 128 x 512 29.4 and 26.8; 64 x
// 1024 25.2 and 24.6.  With few segments it is the slower one (32 query heads, 64 x 2048: 35.4,
// 35.1; 16 x 4096: 22.7, 21.7), as long segments have more pieces than a warp's turn.
template <bool kOwnRef>
__global__ void __launch_bounds__(32 * PKV_MAX_GROUP) join_cut_kernel(const SplitArgs da)
{
    grid_wait();
    const int sg = da.firsts[blockIdx.x];
    if (sg >= 0)
        join_head<kOwnRef, kJoinCut>(da, sg, threadIdx.x >> 5, 0, 1, threadIdx.x & 31, nullptr, nullptr);
}

// The join's launch behind a list's kernel of `ctas` CTAs.
template <bool kOwnRef>
cudaError_t launch_join(const SplitArgs &da, int ctas, cudaStream_t stream)
{
    const long long segs = static_cast<long long>(da.a.batch) * da.a.hkv;
    const int workers = ctas * kSplitWarps;
    if (segs * da.a.group >= 2ll * workers)
        return launch_with(join_cut_kernel<kOwnRef>, dim3(static_cast<unsigned>(workers)), 32 * da.a.group, 0, 1, true, stream,
                           da);
    const long long pieces = (workers + segs - 1) / segs + 1;   // a segment's, on average
    int warps = 1;
    while (warps < kJoinWarps && warps * kJoin<kOwnRef> < pieces)
        warps *= 2;
    return launch_with(join_kernel<kOwnRef>, dim3(static_cast<unsigned>(segs * da.a.group)), 32 * warps, 0, 1, true, stream,
                       da);
}

}  // namespace pkv
