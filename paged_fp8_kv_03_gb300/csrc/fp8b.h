// Declarations of the block-scaled FP8 cache's translation units (not
// installed): the block, the arguments of the kernels and their launchers.
#pragma once

#include "attn.h"

namespace pkv {

// A block: 16 consecutive tokens of one kv head.  Its codes are 16 rows of 128
// E4M3 bytes; its byte x, at the block's number in its own pool, stands for
// 2^(x - 127).  Appended blocks have x - 127 within [kExpMin, kExpMax]: from there
// on every value, code * 2^(x - 127), is a normal bf16 number, or 0.
constexpr int kBlock = 16;
constexpr int kExpBias = 127, kExpMin = -117, kExpMax = 119;

struct Fp8bRowArgs {                                       // append and read back
    const void *k_in, *v_in;                               // append: rows to quantise
    void *k_out, *v_out;                                   // read back: rows to write
    int64_t num_tokens;
    int hkv;
    const int64_t *slots;
    uint8_t *k_cache, *v_cache, *k_exp, *v_exp;
    int64_t num_slots;
    int page_size, page_log2;
    int32_t *err;
};

cudaError_t launch_kv_append_fp8b(const Fp8bRowArgs &a, bool bf16, cudaStream_t stream);
cudaError_t launch_kv_read_fp8b(const Fp8bRowArgs &a, bool bf16, cudaStream_t stream);

// Decode: as the 4-bit cache's, and the blocks' bytes.
constexpr int kFp8bListWarps = kSplitWarps;

struct Fp8bDecodeArgs : SplitArgs {
    const uint8_t *k_exp, *v_exp;
};

size_t decode_fp8b_smem(int batch);
size_t decode_fp8b_cluster_smem();
const void *decode_fp8b_kernel(bool two_parts, bool cluster);
int decode_fp8b_threads(bool cluster);
int decode_fp8b_cluster(long long units, long long segments, int slots);
cudaError_t launch_paged_decode_fp8b(const Fp8bDecodeArgs &da, const CUtensorMap &tm_k, const CUtensorMap &tm_v, int ctas,
                                     cudaStream_t stream, const char **site);

// Prefill's workspace: the header, a float a sequence and kv head (what a value of V's
// copy stands for), the 16-bit copies of K and V, a word a tile (as the 4-bit
// cache's, zeros), another one, and 16 bytes a row, a bit a NaN of V.
// (The maxima of a sequence's heads stand in shared memory.)
constexpr int kFp8bMaxPrefillHeads = 8192;

inline size_t prefill_fp8b_refs_bytes(int batch, int hkv)
{
    return (static_cast<size_t>(batch) * hkv * sizeof(float) + 255) & ~size_t(255);
}

inline size_t prefill_fp8b_bytes(int batch, int hkv, long long rows)
{
    return prefill_header_bytes(batch) + prefill_fp8b_refs_bytes(batch, hkv) +
           static_cast<size_t>(rows) * (2 * kHeadDim * sizeof(__half) + kHeadDim / 8) +
           static_cast<size_t>(rows / 128) * 2 * sizeof(uint32_t);
}

// CTAs that share the keys of a query tile (or of a pair of them) where no sequence has more
// than `longest` tokens, 1 where one has them all; and the bytes that their rows' states
// can take whatever the heads a kv head has and the output's type.
int prefill_fp8b_split(const PrefillArgs &a, const KeyWindow &win, int longest);
// Whether those of a.split take the keys from the cache itself.
bool prefill_fp8b_direct(const PrefillArgs &a);
size_t prefill_fp8b_split_bytes(int batch, int hkv, int max_q_len, int longest, const KeyWindow &win);

cudaError_t launch_widen_fp8b(const PrefillArgs &a, const KeyWindow &win, cudaStream_t stream);

}  // namespace pkv
