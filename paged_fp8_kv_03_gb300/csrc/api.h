// Helpers shared by the translation units that define C entry points (defined
// in api.cu).
#pragma once

#include "internal.h"

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

// Tensor maps of the prefill's query rows and of its 16-bit copies.
bool make_q_map(CUtensorMap *tm, const void *q, int total_q, int hq, int group, int tpt);
bool make_kv16_map(CUtensorMap *tm, const void *base, long long rows, CUtensorMapDataType dtype);

}  // namespace pkv
