// plan_pages and release_pages: a step's pages, block-table entries, slots and
// positions from its requests' lengths, and the way back, without the host.
//
// Sequence b holds past[b] tokens in ceil(past[b] / P) pages and brings new[b].  With
//   T[b] = sum of new[i], i < b,    A[b] = sum of (ceil((past[i] + new[i]) / P) - ceil(past[i] / P)), i < b
// token T[b] + j sits at position p = past[b] + j in row p % P of the sequence's page
// p / P; a page that the sequence does not hold yet, the (p / P - ceil(past[b] / P))-th
// of its new ones, is free page number A[b] + that from the list's end.  Every value
// is a function of the two prefix sums, so every CTA computes both (the lengths come
// from L2) and fills a share of the rows and of the table's new entries.
//
// What bounds them: latency (two lengths, a page, a store, one after the other), and
// the 12 bytes of a row's slot and position where there are many rows.
//
// The free count must not move while a CTA may still read it, nor the lengths, which
// the results may replace in place.  The CTA that draws the last ticket writes
// both; no CTA waits for another.
#include "api.h"
#include "internal.h"

namespace pkv {

namespace {

constexpr int kPlanThreads = 512;
constexpr unsigned kEach = 0xffffffffu;

struct PlanArgs {
    const int32_t *past, *fresh;                           // plan: tokens held and brought; release: kept (or null), held
    int batch;
    int32_t *table;
    int max_pages, page_size, page_log2;
    int32_t *pool;                                         // PKV_PAGE_POOL_HEADER words, then the list
    int num_pages;
    int32_t *seq_lens, *cu_q;
    int64_t *slots;
    int32_t *positions;
    int max_tokens;
    int32_t *err;
};

struct PlanSmem {                                          // dynamic: int tokens[batch + 1], pages[batch + 1]
    long long sums[kPlanThreads / 32][2];
    int bad, last;
};

__device__ __forceinline__ int pages_of(const PlanArgs &a, int tokens)
{
    return static_cast<int>((static_cast<long long>(tokens) + a.page_size - 1) >> a.page_log2);
}

// What sequence b brings: tokens and pages.  False: lengths that cannot be.
template <bool kRelease>
__device__ __forceinline__ bool share_of(const PlanArgs &a, int b, int &tokens, int &pages)
{
    const int past = a.past == nullptr ? 0 : a.past[b], x = a.fresh[b];
    const long long end = kRelease ? x : static_cast<long long>(past) + x;
    tokens = pages = 0;
    if (past < 0 || x < 0 || end < past || end > (static_cast<long long>(a.max_pages) << a.page_log2))
        return false;
    tokens = kRelease ? 0 : x;
    pages = pages_of(a, static_cast<int>(end)) - pages_of(a, past);
    return true;
}

// The prefix sums of tokens and pages over the batch (whole CTA); saturated, but
// the totals are exact.  False: some length cannot be.
template <bool kRelease>
__device__ __forceinline__ bool prefix_sums(const PlanArgs &a, int *tokens, int *pages, PlanSmem &s, long long (&total)[2])
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.batch + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
    if (tid == 0)
        s.bad = 0;
    __syncthreads();
    long long mine[2] = {0, 0};
    bool ok = true;
    for (int b = b0; b < b1; ++b) {
        int t, p;
        ok = share_of<kRelease>(a, b, t, p) && ok;
        mine[0] += t;
        mine[1] += p;
    }
    if (!ok)
        s.bad = 1;
    long long incl[2] = {mine[0], mine[1]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const long long v = __shfl_up_sync(kEach, incl[i], o);
            if (lane >= o)
                incl[i] += v;
        }
    if (lane == 31) {
        s.sums[warp][0] = incl[0];
        s.sums[warp][1] = incl[1];
    }
    __syncthreads();
    long long run[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        run[i] = incl[i] - mine[i];
        total[i] = 0;
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            run[i] += w < warp ? s.sums[w][i] : 0;
            total[i] += s.sums[w][i];
        }
    }
    for (int b = b0; b < b1; ++b) {
        int t, p;
        share_of<kRelease>(a, b, t, p);
        tokens[b] = static_cast<int>(min(run[0], static_cast<long long>(INT32_MAX)));
        pages[b] = static_cast<int>(min(run[1], static_cast<long long>(INT32_MAX)));
        run[0] += t;
        run[1] += p;
    }
    if (tid == 0) {
        tokens[a.batch] = static_cast<int>(min(total[0], static_cast<long long>(INT32_MAX)));
        pages[a.batch] = static_cast<int>(min(total[1], static_cast<long long>(INT32_MAX)));
    }
    __syncthreads();
    return s.bad == 0;
}

// The sequence with sums[b] <= x < sums[b + 1].
__device__ __forceinline__ int sequence_at(const int *sums, int batch, int x)
{
    int lo = 0, hi = batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sums[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// True in every thread of the CTA that is the last one to get here.
__device__ __forceinline__ bool last_here(const PlanArgs &a, PlanSmem &s)
{
    if (gridDim.x == 1) {
        __syncthreads();
        return true;
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        s.last = atomicAdd(reinterpret_cast<unsigned *>(a.pool) + 1, 1u) == gridDim.x - 1;
        if (s.last)
            a.pool[1] = 0;
    }
    __syncthreads();
    __threadfence();
    return s.last != 0;
}

__global__ void __launch_bounds__(kPlanThreads) plan_pages_kernel(const PlanArgs a)
{
    extern __shared__ int dyn[];
    __shared__ PlanSmem s;
    int *tokens = dyn, *pages = dyn + a.batch + 1;
    const int32_t *list = a.pool + PKV_PAGE_POOL_HEADER;
    const int free_pages = *const_cast<volatile int32_t *>(a.pool);
    long long total[2];
    const bool lens_ok = prefix_sums<false>(a, tokens, pages, s, total) && total[0] <= a.max_tokens;
    const bool pool_ok = free_pages >= 0 && free_pages <= a.num_pages && (!lens_ok || total[1] <= free_pages);
    const bool ok = lens_ok && pool_ok;
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0 && a.err)
        atomicOr(a.err, lens_ok ? PKV_DEVERR_POOL : PKV_DEVERR_SEQLEN);
    const int step = static_cast<int>(gridDim.x) * kPlanThreads, id = static_cast<int>(blockIdx.x) * kPlanThreads + threadIdx.x;
    const int used = ok ? static_cast<int>(total[0]) : 0;
    bool bad_page = false;
    for (long long k = id; ok && k < total[1]; k += step) {
        const int b = sequence_at(pages, a.batch, static_cast<int>(k));
        const int page = list[free_pages - 1 - k];
        a.table[static_cast<int64_t>(b) * a.max_pages + pages_of(a, a.past[b]) + (static_cast<int>(k) - pages[b])] = page;
        bad_page = bad_page || page < 0 || page >= a.num_pages;
    }
    for (long long i = id; i < a.max_tokens; i += step) {
        int64_t slot = -1;
        int p = 0;
        if (i < used) {
            const int b = sequence_at(tokens, a.batch, static_cast<int>(i));
            const int past = a.past[b], held = pages_of(a, past);
            p = past + (static_cast<int>(i) - tokens[b]);
            const int at = p >> a.page_log2;
            const int page = at < held ? a.table[static_cast<int64_t>(b) * a.max_pages + at]
                                       : list[free_pages - 1 - (static_cast<long long>(pages[b]) + at - held)];
            if (page >= 0 && page < a.num_pages)
                slot = (static_cast<int64_t>(page) << a.page_log2) + (p & (a.page_size - 1));
            else
                bad_page = true;
        }
        a.slots[i] = slot;
        if (a.positions)
            a.positions[i] = p;
    }
    if (bad_page && a.err)
        atomicOr(a.err, PKV_DEVERR_PAGE);
    if (!last_here(a, s))
        return;
    for (int b = threadIdx.x; b <= a.batch; b += kPlanThreads) {
        a.cu_q[b] = ok ? tokens[b] : 0;
        if (b < a.batch)
            a.seq_lens[b] = a.past[b] + (ok ? a.fresh[b] : 0);
    }
    if (threadIdx.x == 0 && ok)
        a.pool[0] = free_pages - static_cast<int>(total[1]);
}

// (past: what is kept, null for nothing; fresh: the lengths.)
__global__ void __launch_bounds__(kPlanThreads) release_pages_kernel(const PlanArgs a)
{
    extern __shared__ int dyn[];
    __shared__ PlanSmem s;
    int *tokens = dyn, *pages = dyn + a.batch + 1;
    int32_t *list = a.pool + PKV_PAGE_POOL_HEADER;
    const int free_pages = *const_cast<volatile int32_t *>(a.pool);
    long long total[2];
    const bool lens_ok = prefix_sums<true>(a, tokens, pages, s, total);
    const bool ok = lens_ok && free_pages >= 0 && free_pages + total[1] <= a.num_pages;
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0 && a.err)
        atomicOr(a.err, lens_ok ? PKV_DEVERR_POOL : PKV_DEVERR_SEQLEN);
    const int step = static_cast<int>(gridDim.x) * kPlanThreads, id = static_cast<int>(blockIdx.x) * kPlanThreads + threadIdx.x;
    bool bad_page = false;
    for (long long k = id; ok && k < total[1]; k += step) {
        const int b = sequence_at(pages, a.batch, static_cast<int>(k));
        const int kept = a.past == nullptr ? 0 : pages_of(a, a.past[b]);
        const int page = a.table[static_cast<int64_t>(b) * a.max_pages + kept + (static_cast<int>(k) - pages[b])];
        list[free_pages + total[1] - 1 - k] = page;
        bad_page = bad_page || page < 0 || page >= a.num_pages;
    }
    if (bad_page && a.err)
        atomicOr(a.err, PKV_DEVERR_PAGE);
    if (last_here(a, s) && threadIdx.x == 0 && ok)
        a.pool[0] = free_pages + static_cast<int>(total[1]);
}

pkv_status check_plan(int batch, int max_pages, int page_size, int64_t num_pages)
{
    if (batch < 0 || max_pages <= 0 || num_pages <= 0)
        return PKV_ERR_SHAPE;
    if (!page_size_ok(page_size) || batch > PKV_MAX_BATCH || num_pages > INT32_MAX - PKV_PAGE_POOL_HEADER)
        return PKV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_pages) * page_size >= (int64_t(1) << 31))
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

// CTAs for `items` of work, 0 on failure (recorded).
int plan_ctas(const void *kernel, int batch, long long items, size_t &smem)
{
    smem = 2 * (static_cast<size_t>(batch) + 1) * sizeof(int);
    const int most = resident_ctas(kernel, kPlanThreads, smem, 0);
    if (most <= 0)
        return 0;
    const long long want = (items + kPlanThreads - 1) / kPlanThreads;
    return static_cast<int>(want < 1 ? 1 : (want < most ? want : most));
}

}  // namespace

}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_plan_pages(const int32_t *past_lens, const int32_t *new_lens, int batch, int32_t *block_table,
                          int max_pages_per_seq, int page_size, int32_t *page_pool, int64_t num_pages,
                          int32_t *seq_lens, int32_t *cu_q, int64_t *slot_mapping, int32_t *positions,
                          int max_tokens, int32_t *device_error, cudaStream_t stream)
{
    const pkv_status st = check_plan(batch, max_pages_per_seq, page_size, num_pages);
    if (st != PKV_OK)
        return st;
    if (max_tokens < 0)
        return PKV_ERR_SHAPE;
    if (!cu_q || !page_pool || (batch > 0 && (!past_lens || !new_lens || !block_table || !seq_lens)) ||
        (max_tokens > 0 && !slot_mapping))
        return PKV_ERR_NULL;
    if (!aligned(past_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4) || !aligned(page_pool, 4) ||
        !aligned(seq_lens, 4) || !aligned(cu_q, 4) || !aligned(slot_mapping, 8) || !aligned(positions, 4) ||
        !aligned(device_error, 4))
        return PKV_ERR_ALIGN;
    PlanArgs a = {};
    a.past = past_lens;
    a.fresh = new_lens;
    a.batch = batch;
    a.table = block_table;
    a.max_pages = max_pages_per_seq;
    a.page_size = page_size;
    a.page_log2 = 31 - __builtin_clz(static_cast<unsigned>(page_size));
    a.pool = page_pool;
    a.num_pages = static_cast<int>(num_pages);
    a.seq_lens = seq_lens;
    a.cu_q = cu_q;
    a.slots = slot_mapping;
    a.positions = positions;
    a.max_tokens = max_tokens;
    a.err = device_error;
    size_t smem = 0;
    const int ctas = plan_ctas(reinterpret_cast<const void *>(&plan_pages_kernel), batch, max_tokens, smem);
    if (ctas <= 0)
        return PKV_ERR_CUDA;
    plan_pages_kernel<<<ctas, kPlanThreads, smem, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_failed(e, "page plan kernel launch");
}

pkv_status pkv_release_pages(const int32_t *seq_lens, const int32_t *keep_lens, int batch, const int32_t *block_table,
                             int max_pages_per_seq, int page_size, int32_t *page_pool, int64_t num_pages,
                             int32_t *device_error, cudaStream_t stream)
{
    const pkv_status st = check_plan(batch, max_pages_per_seq, page_size, num_pages);
    if (st != PKV_OK || batch == 0)
        return st;
    if (!seq_lens || !block_table || !page_pool)
        return PKV_ERR_NULL;
    if (!aligned(seq_lens, 4) || !aligned(keep_lens, 4) || !aligned(block_table, 4) || !aligned(page_pool, 4) ||
        !aligned(device_error, 4))
        return PKV_ERR_ALIGN;
    PlanArgs a = {};
    a.past = keep_lens;
    a.fresh = seq_lens;
    a.batch = batch;
    a.table = const_cast<int32_t *>(block_table);
    a.max_pages = max_pages_per_seq;
    a.page_size = page_size;
    a.page_log2 = 31 - __builtin_clz(static_cast<unsigned>(page_size));
    a.pool = page_pool;
    a.num_pages = static_cast<int>(num_pages);
    a.err = device_error;
    size_t smem = 0;
    // (how many pages come back is known on the device only: at most all of the table's, few of them as a rule)
    const int ctas = plan_ctas(reinterpret_cast<const void *>(&release_pages_kernel), batch,
                               static_cast<long long>(batch) * max_pages_per_seq / 16, smem);
    if (ctas <= 0)
        return PKV_ERR_CUDA;
    release_pages_kernel<<<ctas, kPlanThreads, smem, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? PKV_OK : cuda_failed(e, "page release kernel launch");
}

}  // extern "C"
