// Declarations of the 4-bit cache's translation units (not installed): the
// tile layout, the arguments of the kernels and their launchers.
#pragma once

#include "internal.h"

namespace pkv {

// 16 tokens of one kv head are one tile: 64 bytes of codes a token (dim 2i in
// the low nibble of byte i, dim 2i + 1 in the high one), then 8 scales a token.
constexpr int kFp4Tile = 16 * PKV_FP4_ROW_BYTES;           // 1152 bytes
constexpr int kFp4Codes = 16 * (kHeadDim / 2);             // 1024: where the scales start

struct Fp4RowArgs {                                        // append and read back
    const void *k_in, *v_in;                               // append: rows to quantise
    void *k_out, *v_out;                                   // read back: rows to write
    int bf16;                                              // rows are bf16 (else fp32)
    int64_t num_tokens;
    int hkv;
    const int64_t *slots;
    const float *k_scale, *v_scale;
    uint8_t *k_cache, *v_cache;
    int64_t num_slots;
    int page_size, page_log2;
    int tokens;                                            // tokens of a thread (launcher)
    int64_t slab;                                          // tokens of one grid row (launcher)
    int32_t *err;
};

// Tokens a query at position p sees: t <= p with t > p - window or t < sinks
// (window == 0: all t <= p).
struct Fp4Window {
    int window, sinks;
};

// Decode's arguments: the fields that the shared page walk (seq_page_log2,
// seq_token_page) reads have the same names as in DecodeArgs.
struct Fp4AttnArgs {
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
    Fp4Window win;
    void *out;
    int out_f32;
    int32_t *err;
};

// Decode: workers of the split (warps) a CTA.
constexpr int kFp4DecodeWorkers = 4;

struct Fp4DecodeArgs {
    Fp4AttnArgs a;
    int2 *joins;                                           // [batch * hkv]: workers of the segment's first and last
                                                           // piece; x = -1: nothing to join
    int *firsts;                                           // [workers]: the segment that a worker's range begins and
                                                           // does not end; -1: none
    float *partials;                                       // [num_slots][group][kPartialStride]
    long long num_slots;
    int cluster;                                           // CTAs a segment; 0: one list for all segments
    int withhold;                                          // failure-detection test hook (-1 = off)
};

// Launches clusters of `cluster` CTAs (1: none), and, if `early`, with
// programmatic stream serialization: the kernel may be brought onto the GPU
// before the one ahead of it has ended, and waits for that with grid_wait().
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

inline size_t decode_fp4_join_bytes(int batch, int hkv, int ctas)
{
    return (static_cast<size_t>(batch) * hkv * sizeof(int2) +
            static_cast<size_t>(ctas) * kFp4DecodeWorkers * sizeof(int) + 255) & ~size_t(255);
}

// Prefill: 128-key tiles that a sequence's 16-bit copy can need, and the rows
// and bytes of the workspace: laid out as pkv_paged_prefill's, then a word a
// tile, each byte of it not zero where one of 32 V rows holds a NaN block, then a
// byte a row, a bit a NaN block (written where the 32 rows' byte is not zero).  Under a
// window a chunk of n queries sees the sinks and the n + window - 1 keys
// before its end, which touch at most (n + window - 2) / 128 + 2 tiles.
inline long long prefill_fp4_rows(int batch, int hkv, int max_q_len, int max_kv_len, long long max_total_kv,
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

inline size_t prefill_fp4_bytes(int batch, long long rows)
{
    return prefill_header_bytes(batch) + static_cast<size_t>(rows) * (2 * kHeadDim * sizeof(__half) + 1) +
           static_cast<size_t>(rows / 128) * sizeof(uint32_t);
}

size_t decode_fp4_smem(int batch);
size_t decode_fp4_cluster_smem();
const void *decode_fp4_kernel(bool two_parts, bool cluster);
int decode_fp4_threads(bool cluster);
int decode_fp4_cluster(long long units, long long segments, int slots);
cudaError_t launch_paged_decode_fp4(const Fp4DecodeArgs &da, int ctas, cudaStream_t stream, const char **site);
cudaError_t launch_widen_fp4(const PrefillArgs &a, const Fp4Window &win, cudaStream_t stream);
cudaError_t launch_prefill_pair(const PrefillArgs &a, const Fp4Window &win, const CUtensorMap &tm_q,
                                const CUtensorMap &tm_k16, const CUtensorMap &tm_v16, cudaStream_t stream);
cudaError_t launch_kv_append_fp4(const Fp4RowArgs &a, cudaStream_t stream);
cudaError_t launch_kv_read_fp4(const Fp4RowArgs &a, cudaStream_t stream);
cudaError_t launch_paged_prefill_fp4(const PrefillArgs &a, const Fp4Window &win, const CUtensorMap &tm_q,
                                     const CUtensorMap &tm_k16, const CUtensorMap &tm_v16, cudaStream_t stream);

}  // namespace pkv
