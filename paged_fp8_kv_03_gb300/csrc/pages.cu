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
// What bounds them: latency (lengths, sums, a page, a store, one after the other), and
// the 12 bytes of a row's slot and position where there are many rows.
//
// The free count must not move while a CTA may still read it, nor the lengths, which
// the results may replace in place.  So a CTA keeps what it needs of both in shared memory
// and then draws a ticket; the one that draws the last writes them.  No CTA waits for
// another, and the ticket is on its way while the rows are filled.
#include "api.h"
#include "grid.cuh"
#include "internal.h"

namespace pkv {

namespace {

constexpr unsigned kEach = 0xffffffffu;

constexpr int kThreads = 256, kEachThread = 4;

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
    int wide;                                              // slots and positions are 16-byte aligned
    int32_t *err;
};

// Sums stop here: more tokens than a call may have rows, and more pages than a pool may.
constexpr uint32_t kMost = PKV_MAX_PLAN_ROWS + 1u;
static_assert(PKV_MAX_PLAN_ROWS <= 1 << 30, "two sums, and a sum and a length, add up within 32 bits");

struct PlanSmem {
    uint32_t sums[kThreads / 32][2];
    int last;
};

// Dynamic shared memory: what comes ahead of sequence b in tokens and in pages
// (and, at `batch`, of all), and the tokens it holds already, or keeps.
struct Sums {
    int *tokens, *pages, *past;
};

__device__ __forceinline__ Sums sums_at(int *dyn, int batch)
{
    return Sums{dyn, dyn + batch + 1, dyn + 2 * (batch + 1)};
}

__device__ __forceinline__ int pages_of(const PlanArgs &a, int tokens)
{
    return static_cast<int>((static_cast<long long>(tokens) + a.page_size - 1) >> a.page_log2);
}

// What a sequence of these lengths brings: tokens and pages.  False: they cannot be.
template <bool kRelease>
__device__ __forceinline__ bool share_of(const PlanArgs &a, int past, int x, int &tokens, int &pages)
{
    const long long end = kRelease ? x : static_cast<long long>(past) + x;
    tokens = pages = 0;
    if (past < 0 || x < 0 || end < past || end > (static_cast<long long>(a.max_pages) << a.page_log2))
        return false;
    tokens = kRelease ? 0 : x;
    pages = pages_of(a, static_cast<int>(end)) - pages_of(a, past);
    return true;
}

__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b)
{
    return min(a + b, kMost);
}

// The sums over the batch (whole CTA).  False: some length cannot be.
template <bool kRelease>
__device__ __forceinline__ bool prefix_sums(const PlanArgs &a, const Sums &q, PlanSmem &s, uint32_t (&total)[2])
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.batch + kThreads - 1) / kThreads;
    const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
    uint32_t mine[2] = {0, 0};
    bool bad = false;
    for (int b = b0; b < b1; b += kEachThread) {
        int past[kEachThread], x[kEachThread];
#pragma unroll
        for (int i = 0; i < kEachThread; ++i) {            // (all on their way together)
            past[i] = a.past != nullptr && b + i < b1 ? a.past[b + i] : 0;
            x[i] = b + i < b1 ? a.fresh[b + i] : 0;
        }
#pragma unroll
        for (int i = 0; i < kEachThread; ++i) {
            if (b + i >= b1)
                break;
            int t, p;
            bad = !share_of<kRelease>(a, past[i], x[i], t, p) || bad;
            q.past[b + i] = past[i];
            q.tokens[b + i] = static_cast<int>(mine[0]);   // (of this thread's sequences so far)
            q.pages[b + i] = static_cast<int>(mine[1]);
            mine[0] = add(mine[0], t);
            mine[1] = add(mine[1], p);
        }
    }
    uint32_t incl[2] = {mine[0], mine[1]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t v = __shfl_up_sync(kEach, incl[i], o);
            incl[i] = lane >= o ? add(incl[i], v) : incl[i];
        }
    if (lane == 31) {
        s.sums[warp][0] = incl[0];
        s.sums[warp][1] = incl[1];
    }
    bad = __syncthreads_or(bad) != 0;
    uint32_t run[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t before = 0;
        total[i] = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            before = w == warp ? total[i] : before;
            total[i] = add(total[i], s.sums[w][i]);
        }
        const uint32_t lower = __shfl_up_sync(kEach, incl[i], 1);
        run[i] = add(before, lane == 0 ? 0 : lower);
    }
    for (int b = b0; b < b1; ++b) {
        q.tokens[b] = static_cast<int>(add(run[0], q.tokens[b]));
        q.pages[b] = static_cast<int>(add(run[1], q.pages[b]));
    }
    if (tid == 0) {
        q.tokens[a.batch] = static_cast<int>(total[0]);
        q.pages[a.batch] = static_cast<int>(total[1]);
        // every thread has its lengths, and this one the free count: nothing that the last CTA writes is read again
        s.last = 1;
        if (gridDim.x > 1) {
            s.last = atomicAdd(reinterpret_cast<unsigned *>(a.pool) + 1, 1u) == gridDim.x - 1;
            if (s.last)
                a.pool[1] = 0;
        }
    }
    __syncthreads();
    return !bad;
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

__global__ void __launch_bounds__(kThreads) plan_pages_kernel(const PlanArgs a)
{
    grid_wait();
    extern __shared__ int dyn[];
    __shared__ PlanSmem s;
    __shared__ int free_count;
    const Sums q = sums_at(dyn, a.batch);
    const int32_t *list = a.pool + PKV_PAGE_POOL_HEADER;
    if (threadIdx.x == 0)
        free_count = *const_cast<volatile int32_t *>(a.pool);
    uint32_t total[2];
    const bool sums_ok = prefix_sums<false>(a, q, s, total);
    const int free_pages = free_count;
    const bool lens_ok = sums_ok && total[0] <= static_cast<uint32_t>(a.max_tokens);
    const bool pool_ok = free_pages >= 0 && free_pages <= a.num_pages &&
                         (!lens_ok || total[1] <= static_cast<uint32_t>(free_pages));
    const bool ok = lens_ok && pool_ok;
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0 && a.err)
        atomicOr(a.err, lens_ok ? PKV_DEVERR_POOL : PKV_DEVERR_SEQLEN);
    const int step = static_cast<int>(gridDim.x) * kThreads, id = static_cast<int>(blockIdx.x) * kThreads + threadIdx.x;
    const int used = ok ? static_cast<int>(total[0]) : 0, taken = ok ? static_cast<int>(total[1]) : 0;
    bool bad_page = false;
    int new_page = id < taken ? list[free_pages - 1 - id] : 0;   // (on its way beside the rows' pages)
    // ---- rows: four that follow one another a thread, so one search and mostly one page
    for (int64_t i0 = 4ll * id; i0 < a.max_tokens; i0 += 4ll * step) {
        int p[4], page[4];
        int b = i0 < used ? sequence_at(q.tokens, a.batch, static_cast<int>(i0)) : 0;
        int past = 0, held = 0, first = 0, end = -1, was = -1;   // of sequence b (end: its first row beyond), of the last page
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int i = static_cast<int>(i0) + n;
            p[n] = 0;
            page[n] = -1;
            if (i < used) {
                if (i >= end) {
                    while (i >= q.tokens[b + 1])
                        ++b;
                    first = q.tokens[b];
                    end = q.tokens[b + 1];
                    past = q.past[b];
                    held = pages_of(a, past);
                    was = -1;
                }
                p[n] = past + (i - first);
                const int at = p[n] >> a.page_log2;
                page[n] = at == was ? page[n > 0 ? n - 1 : 0]
                                    : (at < held ? a.table[static_cast<int64_t>(b) * a.max_pages + at]
                                                 : list[free_pages - 1 - (q.pages[b] + at - held)]);
                was = at;
            }
        }
        int64_t slot[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const bool in = page[n] >= 0 && page[n] < a.num_pages;
            bad_page = bad_page || (i0 + n < used && !in);
            slot[n] = in ? (static_cast<int64_t>(page[n]) << a.page_log2) + (p[n] & (a.page_size - 1)) : -1;
        }
        if (a.wide && i0 + 4 <= a.max_tokens) {
            reinterpret_cast<longlong2 *>(a.slots + i0)[0] = make_longlong2(slot[0], slot[1]);
            reinterpret_cast<longlong2 *>(a.slots + i0)[1] = make_longlong2(slot[2], slot[3]);
            if (a.positions)
                *reinterpret_cast<int4 *>(a.positions + i0) = make_int4(p[0], p[1], p[2], p[3]);
        } else {
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (i0 + n < a.max_tokens) {
                    a.slots[i0 + n] = slot[n];
                    if (a.positions)
                        a.positions[i0 + n] = p[n];
                }
        }
    }
    // ---- new table entries
    for (int k = id; k < taken; k += step) {
        const int page = new_page;
        new_page = k + step < taken ? list[free_pages - 1 - (k + step)] : 0;
        const int b = sequence_at(q.pages, a.batch, k);
        a.table[static_cast<int64_t>(b) * a.max_pages + pages_of(a, q.past[b]) + (k - q.pages[b])] = page;
        bad_page = bad_page || page < 0 || page >= a.num_pages;
    }
    if (bad_page && a.err)
        atomicOr(a.err, PKV_DEVERR_PAGE);
    if (s.last == 0)
        return;
    for (int b = threadIdx.x; b <= a.batch; b += kThreads) {
        a.cu_q[b] = ok ? q.tokens[b] : 0;
        if (b < a.batch)
            a.seq_lens[b] = q.past[b] + (ok ? q.tokens[b + 1] - q.tokens[b] : 0);
    }
    if (threadIdx.x == 0 && ok)
        a.pool[0] = free_pages - taken;
}

// (past: what is kept, null for nothing; fresh: the lengths.)
__global__ void __launch_bounds__(kThreads) release_pages_kernel(const PlanArgs a)
{
    grid_wait();
    extern __shared__ int dyn[];
    __shared__ PlanSmem s;
    __shared__ int free_count;
    const Sums q = sums_at(dyn, a.batch);
    int32_t *list = a.pool + PKV_PAGE_POOL_HEADER;
    if (threadIdx.x == 0)
        free_count = *const_cast<volatile int32_t *>(a.pool);
    uint32_t total[2];
    const bool lens_ok = prefix_sums<true>(a, q, s, total);
    const int free_pages = free_count;
    const bool ok = lens_ok && free_pages >= 0 && free_pages <= a.num_pages &&
                    total[1] <= static_cast<uint32_t>(a.num_pages - free_pages);
    if (!ok && blockIdx.x == 0 && threadIdx.x == 0 && a.err)
        atomicOr(a.err, lens_ok ? PKV_DEVERR_POOL : PKV_DEVERR_SEQLEN);
    const int step = static_cast<int>(gridDim.x) * kThreads, id = static_cast<int>(blockIdx.x) * kThreads + threadIdx.x;
    const int back = ok ? static_cast<int>(total[1]) : 0;
    bool bad_page = false;
    for (int64_t k0 = id; k0 < back; k0 += 4ll * step) {   // (four at a time, their loads together)
        int page[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int64_t k = k0 + static_cast<int64_t>(n) * step;
            page[n] = 0;
            if (k < back) {
                const int b = sequence_at(q.pages, a.batch, static_cast<int>(k));
                page[n] = a.table[static_cast<int64_t>(b) * a.max_pages + pages_of(a, q.past[b]) +
                                  (static_cast<int>(k) - q.pages[b])];
            }
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int64_t k = k0 + static_cast<int64_t>(n) * step;
            if (k >= back)
                break;
            list[free_pages + back - 1 - k] = page[n];
            bad_page = bad_page || page[n] < 0 || page[n] >= a.num_pages;
        }
    }
    if (bad_page && a.err)
        atomicOr(a.err, PKV_DEVERR_PAGE);
    if (s.last != 0 && threadIdx.x == 0 && ok)
        a.pool[0] = free_pages + back;
}

pkv_status check_plan(int batch, int max_pages, int page_size, int64_t num_pages)
{
    if (batch < 0 || max_pages <= 0 || num_pages <= 0)
        return PKV_ERR_SHAPE;
    if (!page_size_ok(page_size) || batch > PKV_MAX_BATCH || num_pages > PKV_MAX_PLAN_ROWS)
        return PKV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_pages) * page_size >= (int64_t(1) << 31))
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

// Launches for `items` of work, four a thread.  Each CTA works out all the sums, so there
// is one an SM at most.
cudaError_t launch_plan(void (*kernel)(const PlanArgs), const PlanArgs &a, long long items, cudaStream_t stream)
{
    const size_t smem = 3 * (static_cast<size_t>(a.batch) + 1) * sizeof(int);
    int most = device_sm_count();
    if (smem > 40 * 1024)                                  // (its limit is raised there)
        most = resident_ctas(reinterpret_cast<const void *>(kernel), kThreads, smem, most);
    if (most <= 0)
        return cudaErrorInvalidConfiguration;
    const long long want = (items + 4 * kThreads - 1) / (4 * kThreads);
    return launch_with(kernel, dim3(static_cast<unsigned>(want < 1 ? 1 : (want < most ? want : most))), kThreads, smem, 1, true,
                       stream, a);
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
    if (max_tokens > PKV_MAX_PLAN_ROWS)
        return PKV_ERR_UNSUPPORTED;
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
    a.wide = aligned(slot_mapping, 16) && aligned(positions, 16);
    const cudaError_t e = launch_plan(plan_pages_kernel, a, max_tokens, stream);
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
    // (how many pages come back is known on the device only: at most all of the table's, few of them as a rule)
    const cudaError_t e = launch_plan(release_pages_kernel, a, static_cast<long long>(batch) * max_pages_per_seq / 16,
                                      stream);
    return e == cudaSuccess ? PKV_OK : cuda_failed(e, "page release kernel launch");
}

}  // extern "C"
