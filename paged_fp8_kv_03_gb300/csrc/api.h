// Helpers shared by the translation units that define C entry points (defined
// in api.cu).
#pragma once

#include "attn.h"

namespace pkv {

// Remembers the CUDA error behind the PKV_ERR_CUDA that it returns.
pkv_status cuda_failed(cudaError_t e, const char *site = "");

inline bool aligned(const void *p, uintptr_t a)
{
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// Sizes every attention call checks.
pkv_status check_decode_shape(int batch, int hq, int hkv, int head_dim, int page_size, int max_pages,
                              int64_t num_pages);

// What append and read back check of the caches with a window.
inline pkv_status check_rows(int64_t num_tokens, int hkv, int head_dim, int64_t num_pages, int page_size, int dtype)
{
    if (num_tokens < 0 || hkv <= 0 || num_pages <= 0)
        return PKV_ERR_SHAPE;
    if (dtype != PKV_F32 && dtype != PKV_BF16)
        return PKV_ERR_DTYPE;
    if (head_dim != kHeadDim || !page_size_ok(page_size))
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

// What their decode and prefill check.
inline pkv_status check_attn(int batch, int hq, int hkv, int head_dim, int page_size, int max_pages, int64_t num_pages,
                      const int32_t *seq_page_sizes, int window, int sinks, int out_dtype)
{
    const pkv_status st = check_decode_shape(batch, hq, hkv, head_dim, page_size, max_pages, num_pages);
    if (st != PKV_OK)
        return st;
    if (window < 0 || sinks < 0)
        return PKV_ERR_SHAPE;
    if (num_pages * hkv * (page_size / 16) >= (int64_t(1) << 31))
        return PKV_ERR_UNSUPPORTED;
    if (seq_page_sizes && static_cast<int64_t>(max_pages) * 256 >= (int64_t(1) << 31))
        return PKV_ERR_UNSUPPORTED;
    if (out_dtype != PKV_F32 && out_dtype != PKV_BF16)
        return PKV_ERR_DTYPE;
    return PKV_OK;
}

// A window no sequence outgrows is none; sinks past the longest sequence say
// nothing more (so the kernels' sums of positions stay within 32 bits).
inline KeyWindow clamp_window(int window, int sinks, long long max_len)
{
    KeyWindow w;
    w.window = window >= max_len ? 0 : window;
    w.sinks = w.window == 0 ? 0 : static_cast<int>(sinks < max_len ? sinks : max_len);
    return w;
}

// Effective bound of seq_lens: max_seq_len, or the table's capacity at the
// pool page size when max_seq_len is 0.
inline long long effective_max_len(int max_seq_len, int max_pages, int page_size)
{
    return max_seq_len > 0 ? max_seq_len : static_cast<long long>(max_pages) * page_size;
}

// Test facility (pkv_test_withhold_load): the worker or block that skips its
// first load, -1 = off.
int withheld_load();

// CTAs of a persistent grid on the current device: `kernel` at `threads`
// threads and `smem` bytes of dynamic shared memory (whose limit is raised
// here), capped by max_ctas if that is positive; 0 and a recorded CUDA error on
// failure.
int resident_ctas(const void *kernel, int threads, size_t smem, int max_ctas);

// Tensor map of an FP8 pool: a box is 16 rows of a page of a kv head, 128-byte swizzled.
bool make_page_map(CUtensorMap *tm, const uint8_t *pool, int64_t num_pages, int hkv, int P);

// Tensor maps of the prefill's query rows and of its 16-bit copies.
bool make_q_map(CUtensorMap *tm, const void *q, int total_q, int hq, int group, int tpt);
bool make_kv16_map(CUtensorMap *tm, const void *base, long long rows, CUtensorMapDataType dtype);

}  // namespace pkv
