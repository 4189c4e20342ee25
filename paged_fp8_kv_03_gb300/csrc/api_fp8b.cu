// C entry points of the block-scaled FP8 cache: argument checks on the host and
// launches.
#include <math.h>

#include "api.h"
#include "fp8b.h"

using namespace pkv;

namespace {

pkv_status rows_args(Fp8bRowArgs &a, const void *k, const void *v, int64_t num_tokens, int hkv, const int64_t *slots,
                     const uint8_t *k_cache, const uint8_t *v_cache, const uint8_t *k_exp, const uint8_t *v_exp,
                     int64_t num_pages, int page_size, int32_t *device_error)
{
    if (!k || !v || !slots || !k_cache || !v_cache || !k_exp || !v_exp)
        return PKV_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slots, 8) ||
        !aligned(device_error, 4))
        return PKV_ERR_ALIGN;
    a = Fp8bRowArgs();
    a.num_tokens = num_tokens;
    a.hkv = hkv;
    a.slots = slots;
    a.k_cache = const_cast<uint8_t *>(k_cache);
    a.v_cache = const_cast<uint8_t *>(v_cache);
    a.k_exp = const_cast<uint8_t *>(k_exp);
    a.v_exp = const_cast<uint8_t *>(v_exp);
    a.num_slots = num_pages * page_size;
    a.page_size = page_size;
    a.page_log2 = 31 - __builtin_clz(static_cast<unsigned>(page_size));
    a.err = device_error;
    return PKV_OK;
}

// CTAs of the decode grid (of the kernel with one part a weight and of that
// with two, whichever has fewer resident).
int decode_ctas(int batch, int max_ctas)
{
    const size_t smem = decode_fp8b_smem(batch);
    const int one = resident_ctas(decode_fp8b_kernel(false, false), decode_fp8b_threads(false), smem, max_ctas);
    const int two = one <= 0 ? 0 : resident_ctas(decode_fp8b_kernel(true, false), decode_fp8b_threads(false), smem, max_ctas);
    return two < one ? two : one;
}

// What the longest sequence's length is at most (max_total_kv 0: not given).
int longest_of(int max_kv_len, int64_t max_total_kv)
{
    return max_total_kv > 0 && max_total_kv < max_kv_len ? static_cast<int>(max_total_kv) : max_kv_len;
}

}  // namespace

extern "C" {

pkv_status pkv_kv_append_fp8b(const void *k_new, const void *v_new, int in_dtype, int64_t num_tokens,
                              int num_kv_heads, int head_dim, const int64_t *slot_mapping, uint8_t *k_cache,
                              uint8_t *v_cache, uint8_t *k_exp, uint8_t *v_exp, int64_t num_pages, int page_size,
                              int32_t *device_error, cudaStream_t stream)
{
    pkv_status st = check_rows(num_tokens, num_kv_heads, head_dim, num_pages, page_size, in_dtype);
    if (st != PKV_OK || num_tokens == 0)
        return st;
    Fp8bRowArgs a;
    st = rows_args(a, k_new, v_new, num_tokens, num_kv_heads, slot_mapping, k_cache, v_cache, k_exp, v_exp, num_pages,
                   page_size, device_error);
    if (st != PKV_OK)
        return st;
    a.k_in = k_new;
    a.v_in = v_new;
    const cudaError_t e = launch_kv_append_fp8b(a, in_dtype == PKV_BF16, stream);
    return e == cudaSuccess ? PKV_OK : cuda_failed(e, "block-scaled append kernel launch");
}

pkv_status pkv_kv_read_fp8b(const int64_t *slot_mapping, int64_t num_tokens, int num_kv_heads, int head_dim,
                            const uint8_t *k_cache, const uint8_t *v_cache, const uint8_t *k_exp,
                            const uint8_t *v_exp, int64_t num_pages, int page_size, void *k_out, void *v_out,
                            int out_dtype, int32_t *device_error, cudaStream_t stream)
{
    pkv_status st = check_rows(num_tokens, num_kv_heads, head_dim, num_pages, page_size, out_dtype);
    if (st != PKV_OK || num_tokens == 0)
        return st;
    Fp8bRowArgs a;
    st = rows_args(a, k_out, v_out, num_tokens, num_kv_heads, slot_mapping, k_cache, v_cache, k_exp, v_exp, num_pages,
                   page_size, device_error);
    if (st != PKV_OK)
        return st;
    a.k_out = k_out;
    a.v_out = v_out;
    const cudaError_t e = launch_kv_read_fp8b(a, out_dtype == PKV_BF16, stream);
    return e == cudaSuccess ? PKV_OK : cuda_failed(e, "block-scaled read-back kernel launch");
}

size_t pkv_decode_fp8b_workspace_size(int batch, int num_q_heads, int num_kv_heads, int head_dim, int max_seq_len,
                                      int page_size, int max_ctas)
{
    if (check_decode_shape(batch, num_q_heads, num_kv_heads, head_dim, page_size, 1, 1) != PKV_OK ||
        max_seq_len < 0 || max_ctas < 0)
        return 0;
    const int ctas = decode_ctas(batch, max_ctas);
    return ctas <= 0 ? 0 : split_workspace(batch, num_q_heads, num_kv_heads, ctas);
}

pkv_status pkv_paged_gqa_decode_fp8b(const void *q, const uint8_t *k_cache, const uint8_t *v_cache,
                                     const uint8_t *k_exp, const uint8_t *v_exp, const int32_t *block_table,
                                     int max_pages_per_seq, const int32_t *seq_lens, int max_seq_len,
                                     const int32_t *seq_page_sizes, int batch, int num_q_heads, int num_kv_heads,
                                     int head_dim, int page_size, int64_t num_pages, float sm_scale, int window,
                                     int sinks, void *out, int out_dtype, void *workspace, size_t workspace_bytes,
                                     int32_t *device_error, int max_ctas, cudaStream_t stream)
{
    const pkv_status st = check_attn(batch, num_q_heads, num_kv_heads, head_dim, page_size, max_pages_per_seq,
                                     num_pages, seq_page_sizes, window, sinks, out_dtype);
    if (st != PKV_OK)
        return st;
    if (max_seq_len < 0 || max_ctas < 0 || !(sm_scale == sm_scale) || isinf(sm_scale))
        return PKV_ERR_SHAPE;
    if (batch == 0)
        return PKV_OK;
    if (!q || !k_cache || !v_cache || !k_exp || !v_exp || !block_table || !seq_lens || !out)
        return PKV_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(device_error, 4) || !aligned(seq_page_sizes, 4))
        return PKV_ERR_ALIGN;
    if (!workspace || !aligned(workspace, 256))
        return PKV_ERR_WORKSPACE;
    const long long max_len = effective_max_len(max_seq_len, max_pages_per_seq, page_size);
    if (max_len >= (int64_t(1) << 31))
        return PKV_ERR_UNSUPPORTED;
    Fp8bDecodeArgs da = {};
    CacheAttnArgs &a = da.a;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.block_table = block_table;
    a.max_pages = max_pages_per_seq;
    a.seq_lens = seq_lens;
    a.max_len = static_cast<int>(max_len);
    a.page_sizes = seq_page_sizes;
    a.batch = batch;
    a.hq = num_q_heads;
    a.hkv = num_kv_heads;
    a.group = num_q_heads / num_kv_heads;
    a.page_size = page_size;
    a.pool_log2 = 31 - __builtin_clz(static_cast<unsigned>(page_size));
    a.num_pages = num_pages;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.sm_scale_log2 = sm_scale * 1.4426950408889634f;
    a.win = clamp_window(window, sinks, max_len);
    a.out = out;
    a.out_f32 = out_dtype == PKV_F32;
    a.err = device_error;
    da.k_exp = k_exp;
    da.v_exp = v_exp;
    // Units of 32 tokens that the longest sequence can show; a list with fewer
    // units than the device has workers needs no more CTAs than it has units.
    long long tiles = (max_len + 15) / 16;
    if (a.win.window > 0) {
        const long long seen = (static_cast<long long>(sinks) + 15) / 16 + (static_cast<long long>(window) + 15) / 16 + 1;
        tiles = seen < tiles ? seen : tiles;
    }
    const long long units = (tiles + 1) / 2 * batch * num_kv_heads;
    if (units + static_cast<int64_t>(batch) * num_kv_heads >= (int64_t(1) << 31))
        return PKV_ERR_UNSUPPORTED;
    int ctas = decode_ctas(batch, max_ctas);
    if (ctas <= 0)
        return PKV_ERR_CUDA;                             // resident_ctas recorded the failing call
    if (workspace_bytes < split_workspace(batch, num_q_heads, num_kv_heads, ctas))
        return PKV_ERR_WORKSPACE;
    if (max_ctas == 0) {
        const int slots = resident_ctas(decode_fp8b_kernel(a.out_f32, true), decode_fp8b_threads(true),
                                        decode_fp8b_cluster_smem(), 0);
        if (slots <= 0)
            return PKV_ERR_CUDA;
        da.cluster = decode_fp8b_cluster((tiles + 1) / 2, static_cast<long long>(batch) * num_kv_heads, slots);
    }
    if (units < ctas)
        ctas = static_cast<int>(units > 0 ? units : 1);
    da.joins = static_cast<int2 *>(workspace);
    const size_t joins = split_join_bytes(batch, num_kv_heads, ctas);
    da.firsts = reinterpret_cast<int *>(da.joins + static_cast<size_t>(batch) * num_kv_heads);
    da.partials = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + joins);
    da.num_slots = static_cast<long long>((workspace_bytes - joins) / (sizeof(float) * a.group * kPartialStride));
    da.withhold = withheld_load();
    alignas(64) CUtensorMap tm_k;
    alignas(64) CUtensorMap tm_v;
    if (!make_page_map(&tm_k, k_cache, num_pages, num_kv_heads, page_size) ||
        !make_page_map(&tm_v, v_cache, num_pages, num_kv_heads, page_size))
        return cuda_failed(cudaErrorInvalidValue, "cuTensorMapEncodeTiled (page pools)");
    const char *site = "";
    const cudaError_t e = launch_paged_decode_fp8b(da, tm_k, tm_v, ctas, stream, &site);
    return e == cudaSuccess ? PKV_OK : cuda_failed(e, site);
}

size_t pkv_prefill_fp8b_workspace_size(int batch, int num_kv_heads, int max_q_len, int max_kv_len,
                                       int64_t max_total_kv, int window, int sinks)
{
    if (batch < 0 || num_kv_heads <= 0 || max_q_len < 0 || max_kv_len < 0 || max_total_kv < 0 || window < 0 ||
        sinks < 0)
        return 0;
    return prefill_fp8b_bytes(batch, num_kv_heads,
                              windowed_rows(batch, num_kv_heads, max_q_len, max_kv_len, max_total_kv, window, sinks)) +
           prefill_fp8b_split_bytes(batch, num_kv_heads, max_q_len, longest_of(max_kv_len, max_total_kv),
                                    clamp_window(window, sinks, max_kv_len));
}

pkv_status pkv_paged_prefill_fp8b(const void *q, const int32_t *cu_q, int total_q, int max_q_len,
                                  const uint8_t *k_cache, const uint8_t *v_cache, const uint8_t *k_exp,
                                  const uint8_t *v_exp, const int32_t *block_table, int max_pages_per_seq,
                                  const int32_t *seq_lens, const int32_t *seq_page_sizes, int batch, int max_kv_len,
                                  int64_t max_total_kv, int num_q_heads, int num_kv_heads, int head_dim,
                                  int page_size, int64_t num_pages, float sm_scale, int window, int sinks, void *out,
                                  int out_dtype, void *workspace, size_t workspace_bytes, int32_t *device_error,
                                  cudaStream_t stream)
{
    const pkv_status st = check_attn(batch, num_q_heads, num_kv_heads, head_dim, page_size, max_pages_per_seq,
                                     num_pages, seq_page_sizes, window, sinks, out_dtype);
    if (st != PKV_OK)
        return st;
    if (total_q < 0 || max_q_len < 0 || max_kv_len < 0 || max_total_kv < 0)
        return PKV_ERR_SHAPE;
    if (!(sm_scale > 0.f) || isinf(sm_scale))
        return PKV_ERR_SHAPE;
    if (num_kv_heads > kFp8bMaxPrefillHeads)
        return PKV_ERR_UNSUPPORTED;
    if (batch == 0 || total_q == 0 || max_q_len == 0)
        return PKV_OK;
    if (!q || !cu_q || !k_cache || !v_cache || !k_exp || !v_exp || !block_table || !seq_lens || !out)
        return PKV_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(cu_q, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(device_error, 4) ||
        !aligned(seq_page_sizes, 4))
        return PKV_ERR_ALIGN;
    const int group = num_q_heads / num_kv_heads;
    const int tpt = 128 / group;
    const int64_t max_tiles = (static_cast<int64_t>(max_q_len) + tpt - 1) / tpt;
    if (static_cast<int64_t>(batch) * num_kv_heads * max_tiles >= (int64_t(1) << 31))
        return PKV_ERR_UNSUPPORTED;
    if (max_kv_len == 0)
        return PKV_OK;                                   // no sequence can hold a query
    const long long rows = windowed_rows(batch, num_kv_heads, max_q_len, max_kv_len, max_total_kv, window, sinks);
    if (rows >= (int64_t(1) << 31))
        return PKV_ERR_UNSUPPORTED;
    const KeyWindow win = clamp_window(window, sinks, max_kv_len);
    const int longest = longest_of(max_kv_len, max_total_kv);
    const size_t copies = prefill_fp8b_bytes(batch, num_kv_heads, rows);
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < copies + prefill_fp8b_split_bytes(batch, num_kv_heads, max_q_len, longest, win))
        return PKV_ERR_WORKSPACE;
    uint8_t *base = static_cast<uint8_t *>(workspace) + prefill_header_bytes(batch);
    float *refs = reinterpret_cast<float *>(base);
    __half *k16 = reinterpret_cast<__half *>(base + prefill_fp8b_refs_bytes(batch, num_kv_heads));
    __half *v16 = k16 + static_cast<size_t>(rows) * kHeadDim;
    PrefillArgs a = {};
    a.cu_q = cu_q;
    a.total_q = total_q;
    a.max_q_len = max_q_len;
    a.tokens_per_tile = tpt;
    a.max_tiles = static_cast<int>(max_tiles);
    a.k_exp = k_exp;
    a.v_exp = v_exp;
    a.v_refs = refs;
    a.block_table = block_table;
    a.max_pages = max_pages_per_seq;
    a.seq_lens = seq_lens;
    a.batch = batch;
    a.hq = num_q_heads;
    a.hkv = num_kv_heads;
    a.group = group;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.page_sizes = seq_page_sizes;
    a.pool_log2 = 31 - __builtin_clz(static_cast<unsigned>(page_size));
    a.max_kv_len = max_kv_len;
    a.tile_off = static_cast<int *>(workspace);
    a.rows_cap = rows;
    a.k16 = k16;
    a.v16 = v16;
    a.withhold_block = withheld_load();
    a.sm_scale_log2 = sm_scale * 1.4426950408889634f;
    a.out = out;
    a.out_f32 = out_dtype == PKV_F32;
    a.err = device_error;
    a.split = prefill_fp8b_split(a, win, longest);
    a.direct = prefill_fp8b_direct(a);
    a.partials = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + ((copies + 255) & ~size_t(255)));
    alignas(64) CUtensorMap tm_q;
    alignas(64) CUtensorMap tm_k;
    alignas(64) CUtensorMap tm_v;
    if (!make_q_map(&tm_q, q, total_q, num_q_heads, group, tpt) ||
        !(a.direct ? make_page_map(&tm_k, k_cache, num_pages, num_kv_heads, page_size)
                 : make_kv16_map(&tm_k, k16, rows, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16)) ||
        !(a.direct ? make_page_map(&tm_v, v_cache, num_pages, num_kv_heads, page_size)
                 : make_kv16_map(&tm_v, v16, rows, CU_TENSOR_MAP_DATA_TYPE_FLOAT16)))
        return cuda_failed(cudaErrorInvalidValue, "cuTensorMapEncodeTiled (block-scaled prefill)");
    const cudaError_t e = launch_prefill_windowed(a, win, tm_q, tm_k, tm_v,
                                                  launch_widen_fp8b, stream);
    return e == cudaSuccess ? PKV_OK : cuda_failed(e, "block-scaled prefill kernel launch");
}

}  // extern "C"
