// What the attention calls with a window have in common, whatever the cache's
// format: the window, decode's arguments, and launches with attributes.
#pragma once

#include "internal.h"

namespace pkv {

// Tokens a query at position p sees: t <= p with t > p - window or t < sinks
// (window == 0: all t <= p).
struct KeyWindow {
    int window, sinks;
};

// Decode's arguments: the fields that the shared page walk (seq_page_log2,
// seq_token_page) reads have the same names as in DecodeArgs.  (Scales a kv head:
// the 4-bit cache's.)
struct CacheAttnArgs {
    const __nv_bfloat16 *q;
    const float *k_scale, *v_scale;
    const int32_t *block_table;
    int max_pages;
    const int32_t *seq_lens;
    int max_len;
    const int32_t *page_sizes;
    int batch, hq, hkv, group;
    int page_size, pool_log2;
    int64_t num_pages;
    const uint8_t *k_cache, *v_cache;
    float sm_scale_log2;
    KeyWindow win;
    void *out;
    int out_f32;
    int32_t *err;
};

// Decode over a list of units: workers of the split (warps) a CTA, and what the
// kernels get.
constexpr int kSplitWarps = 4;

struct SplitArgs {
    CacheAttnArgs a;
    int2 *joins;                                           // [batch * hkv]: workers of the segment's first and last
                                                           // piece; x = -1: nothing to join
    int *firsts;                                           // [workers]: the segment that a worker's range begins and
                                                           // does not end; -1: none
    float *partials;                                       // [num_slots][group][kPartialStride]
    long long num_slots;
    int cluster;                                           // CTAs a segment; 0: one list for all segments
    int withhold;                                          // failure-detection test hook (-1 = off)
};

// Workspace: the segments' first and last workers, the workers' cut segments, then one
// state a worker and one a segment (a piece's slot is worker + rank of its segment,
// distinct because both grow along the list).
inline size_t split_join_bytes(int batch, int hkv, int ctas)
{
    return (static_cast<size_t>(batch) * hkv * sizeof(int2) + static_cast<size_t>(ctas) * kSplitWarps * sizeof(int) + 255) &
           ~size_t(255);
}

inline size_t split_workspace(int batch, int hq, int hkv, int ctas)
{
    const size_t slots = static_cast<size_t>(ctas) * kSplitWarps + static_cast<size_t>(batch) * hkv;
    const size_t bytes = slots * static_cast<size_t>(hq / hkv) * kPartialStride * sizeof(float);
    return split_join_bytes(batch, hkv, ctas) + ((bytes + 255) & ~size_t(255));
}

// Rows of the 16-bit copies that prefill with a window can need.  Under a
// window a chunk of n queries sees the sinks and the n + window - 1 keys
// before its end, which touch at most (n + window - 2) / 128 + 2 tiles.
inline long long windowed_rows(int batch, int hkv, int max_q_len, int max_kv_len, long long max_total_kv,
                                  int window, int sinks)
{
    long long per = (static_cast<long long>(max_kv_len) + 127) / 128;
    if (window > 0) {
        const long long seen = (static_cast<long long>(sinks) + 127) / 128 +
                               (static_cast<long long>(max_q_len) + window) / 128 + 2;
        per = seen < per ? seen : per;
    }
    long long tiles = per * batch;
    if (max_total_kv > 0) {
        // sum of ceil(L_b / 128) <= sum L_b / 128 + batch
        const long long t2 = max_total_kv / 128 + (max_total_kv % 128 != 0) + batch;
        tiles = t2 < tiles ? t2 : tiles;
    }
    return tiles * 128 * hkv;
}

// Prefill with a window: `widen` enqueues what fills the 16-bit copies, then the
// attention over them is enqueued.
typedef cudaError_t (*WidenLaunch)(const PrefillArgs &a, const KeyWindow &win, cudaStream_t stream);
cudaError_t launch_prefill_windowed(const PrefillArgs &a, const KeyWindow &win, const CUtensorMap &tm_q,
                                    const CUtensorMap &tm_k16, const CUtensorMap &tm_v16, WidenLaunch widen,
                                    cudaStream_t stream);

// The attention of a.direct: tm_k and tm_v are the pools' maps.
cudaError_t launch_prefill_direct(const PrefillArgs &a, const KeyWindow &win, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                                  const CUtensorMap &tm_v, cudaStream_t stream);

// Joins what the CTAs of a split prefill have left, and writes the output.
cudaError_t launch_prefill_join(const PrefillArgs &a, const KeyWindow &win, cudaStream_t stream);

// Launches clusters of `cluster` CTAs (1: none), and, if `early`, with
// programmatic stream serialization: the kernel may be brought onto the GPU
// before the one ahead of it has ended, and waits for that with grid_wait(), ahead of
// anything it reads or writes and in every CTA (a grid that ended without waiting could
// let what follows begin beside what is ahead).  The block-scaled cache's and the plan's
// calls are all launched this way: one behind another from Python, append and read back of
// 64 tokens 5.4 us, else 10.2; plan and release 6.8 and 10.8; a decode of two short
// sequences 4.4 and 6.1.  The rows' and the plan's kernels let the next in as they end, not
// when they start (1021 requests planned 10.1 us a pass in a graph, 13.3 that way).
template <typename... Params, typename... Args>
cudaError_t launch_with(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, int cluster, bool early,
                        cudaStream_t stream, const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (early) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace pkv
