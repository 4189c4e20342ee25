// Declarations of the 4-bit cache's translation units (not installed): the
// tile layout, the arguments of the kernels and their launchers.
#pragma once

#include "attn.h"

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

// Prefill's workspace: laid out as pkv_paged_prefill's, then a word a
// tile, each byte of it not zero where one of 32 V rows holds a NaN block, then a
// byte a row, a bit a NaN block (written where the 32 rows' byte is not zero).
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
cudaError_t launch_paged_decode_fp4(const SplitArgs &da, int ctas, cudaStream_t stream, const char **site);
cudaError_t launch_widen_fp4(const PrefillArgs &a, const KeyWindow &win, cudaStream_t stream);
cudaError_t launch_prefill_pair(const PrefillArgs &a, const KeyWindow &win, const CUtensorMap &tm_q,
                                const CUtensorMap &tm_k16, const CUtensorMap &tm_v16, cudaStream_t stream);
cudaError_t launch_kv_append_fp4(const Fp4RowArgs &a, cudaStream_t stream);
cudaError_t launch_kv_read_fp4(const Fp4RowArgs &a, cudaStream_t stream);

}  // namespace pkv
