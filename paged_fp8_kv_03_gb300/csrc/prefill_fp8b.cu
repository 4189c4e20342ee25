// The widening of the block-scaled FP8 cache to the 16-bit copies that the prefill
// attention reads: K as bf16, code * 2^ek (exact: 4 significant bits), V as f16 in
// units of its own reference,
//   v16 = code * 2^(ev - E) * 2^6,   E = the largest ev among the sequence's blocks
//                                    of this kv head that some query of the chunk sees,
// so that 448 comes out as 28672.  Exact for blocks down to 2^-21 of the largest
// one's scale; below that f16's lower end loses up to 2^-25 of a unit, 2^-31 of 2^E, 2^-39 of
// the largest V that it holds.  The output is multiplied by 2^(E - 6).  NaN codes of V become zeros
// and are recorded, a bit a value.
//
// Two launches, and a third behind the attention where few rows have a long past: its
// CTAs then share a query tile's keys, and prefill_join_fp8b_kernel joins what they leave
// (64 tokens of 32 query and 8 kv heads, past 32768, fp32 outputs: 99 us, else 374; 8 query heads
// of one kv head, past 131072, bf16: 91 us, else 1525; calls that prefill_direct.cu takes, see there).
// kv_refs_fp8b_kernel: a cluster of CTAs a sequence takes the maximum
// of the bytes (a sixteenth of a byte a token and head), and CTA 0 lays out the
// regions.  kv_widen_fp8b_kernel: a CTA half a tile of 128 rows (or a quarter of one,
// where there are few); a thread takes 8 values of kRowsEach of its rows, of K and of V, 16
// lanes write a row's 256 bytes.  Bytes bound it: 256 of the cache to 512 of the
// copies a row.
#include "split.cuh"
#include "widen_fp8b.cuh"

namespace pkv {

namespace {

constexpr int kRefThreads = 512, kRefCtas = 8;

// The prefix sum of the sequences' 128-row tiles (the whole CTA): tile_off, and a
// flag for a region past the workspace.
__device__ __forceinline__ void lay_out(const PrefillArgs &a, const KeyWindow &win, int *warp_sum)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long cap_tiles = a.rows_cap / kKeys;
    const int most = static_cast<int>(cap_tiles + 1);    // sums saturate just past the workspace
    const int chunk = (a.batch + kRefThreads - 1) / kRefThreads;
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
        a.tile_off[b] = run;
        const int next = static_cast<int>(min(run + region_tiles<true>(a, win, b), static_cast<long long>(most)));
        if (next > cap_tiles && next > run && a.err)
            atomicOr(a.err, PKV_DEVERR_SEQLEN);          // its region does not fit the workspace
        run = next;
    }
    if (tid == kRefThreads - 1)
        a.tile_off[a.batch] = min(base + incl, most);
}

// A cluster of `ctas` CTAs a sequence, and one cluster more for the layout.
__global__ void __launch_bounds__(kRefThreads) kv_refs_fp8b_kernel(const PrefillArgs a, const KeyWindow win, int ctas)
{
    extern __shared__ int top[];                         // [hkv]: largest byte
    __shared__ int warp_sum[kRefThreads / 32];
    launch_dependents();
    grid_wait();
    const int rank = static_cast<int>(blockIdx.x) % ctas, b = static_cast<int>(blockIdx.x) / ctas;
    if (b == a.batch) {
        if (rank == 0)
            lay_out(a, win, warp_sum);
        return;
    }
    const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], L = a.seq_lens[b];
    if (q1 - q0 <= 0 || !sequence_ok(a, b, q0, q1, L, false))
        return;                                          // (the whole cluster)
    for (int h = threadIdx.x; h < a.hkv; h += kRefThreads)
        top[h] = 0;
    __syncthreads();
    const int lp = seq_page_log2(a, b), per_page = a.page_size / kBlock;
    const KeyTiles kt = key_tiles<true>(win, L - (q1 - q0));
    const int blocks = (L + kBlock - 1) / kBlock, sink_blocks = (kt.sinks + kBlock - 1) / kBlock;
    const int skip = max(kt.from / kBlock, sink_blocks) - sink_blocks;   // blocks that no query sees
    for (int i = rank * kRefThreads + threadIdx.x; i < blocks - skip; i += ctas * kRefThreads) {
        int pg, row;
        if (!seq_token_page(a, b, lp, (i < sink_blocks ? i : i + skip) * kBlock, pg, row))
            continue;                                    // (the widening flags it)
        const uint8_t *x = a.v_exp + static_cast<int64_t>(pg) * a.hkv * per_page + row / kBlock;
        for (int h = 0; h < a.hkv; ++h) {
            const int v = x[static_cast<int64_t>(h) * per_page];
            if (v > *const_cast<volatile int *>(top + h))
                atomicMax(top + h, v);
        }
    }
    cluster_sync(ctas);
    if (rank == 0) {
        for (int h = threadIdx.x; h < a.hkv; h += kRefThreads) {
            int most = top[h];
            for (int k = 1; k < ctas; ++k)
                most = max(most, __float_as_int(cluster_load(smem_addr(top + h), k, false)));
            // 2^(E - 6); a byte below kExpMin's (no appended block has it) counts as that
            a.v_refs[b * a.hkv + h] = __int_as_float((max(most, kExpMin + kExpBias) - 6) << 23);
        }
    }
    cluster_sync(ctas);                                  // no CTA leaves while its maxima are read
}

template <int kRowsEach>
__global__ void __launch_bounds__(256) kv_widen_fp8b_kernel(const PrefillArgs a, const KeyWindow win)
{
    constexpr int kPieces = 8 / kRowsEach;               // CTAs' steps a tile
    static_assert(kPieces == 2 || kPieces == 4, "a tile's word has two bytes or one a piece");
    const int tid = threadIdx.x;
    const int part = tid & 15;                           // dims 8 part .. 8 part + 7
    launch_dependents();
    grid_wait();
    const long long cap_tiles = a.rows_cap / kKeys;
    const int *off = a.tile_off;
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
        const int b = lo, off0 = off[b], off1 = off[b + 1];
        if (off1 > cap_tiles)
            continue;                                    // region past the workspace: flagged above
        const int L = a.seq_lens[b], lp = seq_page_log2(a, b);
        const KeyTiles kt = key_tiles<true>(win, L - (a.cu_q[b + 1] - a.cu_q[b]));
        const int per_head = (off1 - off0) / a.hkv;
        const int h = (tile - off0) / per_head, vt = (tile - off0) - h * per_head;
        const int key0 = (vt < kt.first ? vt : vt + kt.skip) * kKeys;
        const int ref = (__float_as_int(*const_cast<volatile float *>(a.v_refs + b * a.hkv + h)) >> 23) & 0xFF;
        uint2 kc[kRowsEach], vc[kRowsEach];
        float ks[kRowsEach], vs[kRowsEach];
        uint32_t nans[kRowsEach];                        // V's, 8 bits a row
        bool some = false;
#pragma unroll
        for (int i = 0; i < kRowsEach; ++i) {
            const int t = key0 + first + 16 * i;
            kc[i] = vc[i] = make_uint2(0u, 0u);
            ks[i] = vs[i] = 0.f;
            if (t < L && (t < kt.sinks || t >= kt.from)) {
                int pg, row;
                if (seq_token_page(a, b, lp, t, pg, row)) {
                    const int64_t at = (static_cast<int64_t>(pg) * a.hkv + h) * a.page_size + row;
                    kc[i] = reinterpret_cast<const uint2 *>(a.k_cache + at * kHeadDim)[part];
                    vc[i] = reinterpret_cast<const uint2 *>(a.v_cache + at * kHeadDim)[part];
                    ks[i] = scale_of(a.k_exp[at / kBlock]);
                    vs[i] = scale_of_v(a.v_exp[at / kBlock], ref);
                } else if (part == 0 && a.err) {
                    atomicOr(a.err, PKV_DEVERR_PAGE);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kRowsEach; ++i) {
            const int64_t at = (static_cast<int64_t>(tile) * kKeys + first + 16 * i) * kHeadDim + 8 * part;
            *reinterpret_cast<uint4 *>(a.k16 + at) = widen_k(kc[i], ks[i]);
            *reinterpret_cast<uint4 *>(a.v16 + at) = widen_v(vc[i], vs[i], nans[i]);
            some = some || nans[i] != 0;
        }
        const bool any = __syncthreads_or(some) != 0;
        if (tid == 0) {
            if (piece % kPieces == 0)
                nan_tiles(a)[tile] = 0u;                 // (no NaN block of the 4-bit cache's kind)
            if (kPieces == 2)
                reinterpret_cast<uint16_t *>(nan_value_tiles(a) + tile)[piece % kPieces] = any ? 0x0101 : 0;
            else
                reinterpret_cast<uint8_t *>(nan_value_tiles(a) + tile)[piece % kPieces] = any;
        }
        if (any) {
            if (tid == 0)                                // (several tiles' CTAs may: all store the same)
                *const_cast<volatile float *>(a.v_refs + b * a.hkv + h) = __int_as_float(ref << 23 | static_cast<int>(0x80000000u));
#pragma unroll
            for (int i = 0; i < kRowsEach; ++i)
                nan_value_rows(a)[(static_cast<int64_t>(tile) * kKeys + first + 16 * i) * 16 + part] = static_cast<uint8_t>(nans[i]);
        }
    }
}

// Joins the states of the CTAs that shared a query tile's keys: a warp a row, a lane four
// dims; the weight of a part is 2^(m - the parts' largest m).  A part whose keys the row
// does not see has m = -inf.  A CTA has kJoinRows rows or one token's.
constexpr int kJoinThreads = 256, kJoinRows = 8;

__global__ void __launch_bounds__(kJoinThreads) prefill_join_fp8b_kernel(const PrefillArgs a, const KeyWindow win)
{
    grid_wait();
    const int tiles = a.out_f32 ? 1 : 2, per = (a.max_tiles + tiles - 1) / tiles;   // of an attention CTA
    const int bh = static_cast<int>(blockIdx.x) / per, first = (per - 1 - (static_cast<int>(blockIdx.x) - bh * per)) * tiles;
    const int b = bh / a.hkv, h = bh - b * a.hkv, G = a.group, tpt = a.tokens_per_tile;
    const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], n = q1 - q0, L = a.seq_lens[b];
    if (!sequence_ok(a, b, q0, q1, L, false) || a.tile_off[b + 1] > a.rows_cap / kKeys)
        return;
    const int begin = first * tpt, end = min(n, begin + tiles * tpt), per_cta = max(1, kJoinRows / G);
    const int t0 = begin + static_cast<int>(blockIdx.y) * per_cta, t1 = min(end, t0 + per_cta);
    if (t0 >= t1)
        return;
    const int nt = (L - n + end - 1) / kKeys + 1 - key_tiles<true>(win, L - n + begin).skip;
    const int parts = key_share(nt, 0, a.split).parts;
    const float unit = a.v_refs[bh];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int r = warp; r < (t1 - t0) * G; r += kJoinThreads / 32) {
        const int t = t0 + r / G, g = r % G, x = (t - begin) / tpt;
        const float *at = split_row(a, tiles, blockIdx.x, 0, x * kRows + (t - begin - x * tpt) * G + g);
        const int64_t stride = static_cast<int64_t>(tiles) * kRows * kPartialStride;
        float top = -INFINITY;
        for (int p = lane; p < parts; p += 32)
            top = fmaxf(top, __ldcg(at + p * stride + kHeadDim));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
        for (int p0 = 0; p0 < parts; p0 += 32) {
            float weight = 0.f, l = 0.f;
            if (p0 + lane < parts) {
                const float2 s = __ldcg(reinterpret_cast<const float2 *>(at + (p0 + lane) * stride + kHeadDim));
                weight = s.x == -INFINITY ? 0.f : ex2_approx(s.x - top);
                l = s.y;
            }
            sum += weight * l;                           // (a lane's own parts; a NaN stays one)
#pragma unroll 8
            for (int p = 0; p < min(32, parts - p0); ++p) {
                const float4 o = __ldcg(reinterpret_cast<const float4 *>(at + (p0 + p) * stride) + lane);
                const float f = __shfl_sync(kAll, weight, p);
                acc.x += f * o.x;
                acc.y += f * o.y;
                acc.z += f * o.z;
                acc.w += f * o.w;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(kAll, sum, o);
        // (apart: their product may lie below fp32's range)
        const float inv = 1.f / sum, scale = fabsf(unit);
        acc = make_float4(acc.x * inv * scale, acc.y * inv * scale, acc.z * inv * scale, acc.w * inv * scale);
        const int64_t row = (static_cast<int64_t>(q0) + t) * a.hq + static_cast<int64_t>(h) * G + g;
        if (a.out_f32) {
            reinterpret_cast<float4 *>(static_cast<float *>(a.out) + row * kHeadDim)[lane] = acc;
        } else {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y), hi = __floats2bfloat162_rn(acc.z, acc.w);
            reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + row * kHeadDim)[lane] =
                make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        }
    }
    if (unit < 0.f) {
        __syncthreads();
        put_nans_of<true>(a, win, b, h, t0, t1, kJoinThreads);
    }
}

// Where query tiles fill half of the SMs at most, as many CTAs share each one's keys as fill them
// once (kSplitSms, a constant, so that the workspace's size goes by the bounds alone).  A part has two key tiles at least, four where a row has more than 32 parts (64 tokens,
// 8 query heads of 1 kv head, past 16384: in 64 parts of two 52 us, in 32 of four 44, in one 198),
// and kMostPart at most, as the attention kernels then sum in one chain; so a long context has
// more parts.  A CTA has to be spared kLeastSpared of them, as leaving and joining the states
// takes as long as some (64 tokens, past 1024, 8 kv heads: 2 key tiles instead of 8 30.8 us, else
// 31.9; 9 sequences of 1100: 5 instead of 9 42.1 us, else 40.1).
constexpr int kSplitSms = 152, kMostPart = 128, kLeastSpared = 6;

int split_of(int64_t ctas, int64_t most)
{
    if (ctas <= 0 || 2 * ctas > kSplitSms)
        return 1;
    const int64_t even = kSplitSms / ctas, pairs = most / 2 < 32 ? most / 2 : 32;
    const int64_t worth = pairs > most / 4 ? pairs : most / 4, parts = even < worth ? even : worth;
    if (parts < 2 || most - (most + parts - 1) / parts < kLeastSpared)
        return 1;
    const int64_t need = (most + kMostPart - 1) / kMostPart;
    return static_cast<int>(parts > need ? parts : need);
}

}  // namespace

int prefill_fp8b_split(const PrefillArgs &a, const KeyWindow &win, int longest)
{
    PrefillArgs bound = a;
    bound.max_kv_len = longest;
    const int64_t tiles = a.out_f32 ? a.max_tiles : (a.max_tiles + 1) / 2;
    return longest > kNoWindow / 2 ? 1 : split_of(tiles * a.batch * a.hkv, most_key_tiles(bound, win));
}

// A CTA that widens for itself takes 3.1 us a key tile, else 1.3, but the copies are neither
// written nor read: 9 x 32 tokens of 32 query and 8 kv heads past 8192 116 us, else 160; 16
// tokens of 64 and 8 past 131072 177 and 257.  With several pairs of query tiles a kv head each
// widens them again (512 tokens past 32768: 411 and 255), and few keys' copies cost less than
// the longer start (2048 key tiles, 64 tokens past 32768: 77 and 93; 1024: 95 and 91; 256: 40 and 40).
bool prefill_fp8b_direct(const PrefillArgs &a)
{
    return a.split > 1 && !a.out_f32 && a.max_tiles <= 2 && a.rows_cap / kKeys >= 1536;
}

size_t prefill_fp8b_split_bytes(int batch, int hkv, int max_q_len, int longest, const KeyWindow &win)
{
    // Between the CTAs of one query tile a kv head and of kSplitSms / 2 in all, whichever
    // tiles the heads make: as many parts as SMs or, in long contexts, need a CTA.
    const int64_t least = static_cast<int64_t>(batch) * hkv;
    PrefillArgs a = {};
    a.max_kv_len = longest;
    a.tokens_per_tile = kRows;
    const int64_t most = most_key_tiles(a, win);
    if (max_q_len == 0 || split_of(least, most) == 1)
        return 0;
    const int64_t ctas = least * max_q_len < kSplitSms / 2 ? least * max_q_len : kSplitSms / 2;
    const int64_t need = ctas * ((most + kMostPart - 1) / kMostPart);
    return static_cast<size_t>(need > kSplitSms ? need : kSplitSms) * 2 * kRows * kPartialStride * sizeof(float) + 255;
}

cudaError_t launch_prefill_join(const PrefillArgs &a, const KeyWindow &win, cudaStream_t stream)
{
    const int tiles = a.out_f32 ? 1 : 2, per = (a.max_tiles + tiles - 1) / tiles;
    const int per_cta = kJoinRows / a.group > 1 ? kJoinRows / a.group : 1;
    const int tokens = a.max_q_len < tiles * a.tokens_per_tile ? a.max_q_len : tiles * a.tokens_per_tile;
    return launch_with(prefill_join_fp8b_kernel,
                       dim3(static_cast<unsigned>(a.batch * a.hkv * per), static_cast<unsigned>((tokens + per_cta - 1) / per_cta)),
                       kJoinThreads, 0, 1, true, stream, a, win);
}

cudaError_t launch_widen_fp8b(const PrefillArgs &a, const KeyWindow &win, cudaStream_t stream)
{
    // (clusters pay from a few thousand tokens on)
    const int ctas = a.max_kv_len <= 4096 ? 1 : kRefCtas;
    const cudaError_t e = launch_with(kv_refs_fp8b_kernel, dim3(static_cast<unsigned>((a.batch + 1) * ctas)), kRefThreads,
                                      static_cast<size_t>(a.hkv) * sizeof(int), ctas, true, stream, a, win, ctas);
    if (e != cudaSuccess || a.direct)   // (that attention widens for itself)
        return e;
    const int64_t tiles = a.rows_cap / kKeys, most = static_cast<int64_t>(device_sm_count()) * 8;
    if (tiles * 4 <= most)
        return launch_with(kv_widen_fp8b_kernel<2>, dim3(static_cast<unsigned>(tiles < 1 ? 1 : tiles * 4)), 256, 0, 1, true,
                           stream, a, win);
    return launch_with(kv_widen_fp8b_kernel<4>, dim3(static_cast<unsigned>(tiles * 2 < most ? tiles * 2 : most)), 256, 0, 1,
                       true, stream, a, win);
}

}  // namespace pkv
