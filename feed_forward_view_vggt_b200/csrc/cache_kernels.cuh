// cache_kernels.cuh -- the paged K/V cache of a streaming trunk: the plan of
// a step (block tables, slot map, row offsets, from the sequences' lengths)
// and the append of the step's K and V rows.
//
// A page holds page_size consecutive positions of one sequence for every
// key/value head; a slot is page * page_size + offset.
#pragma once
#include <cstdint>

#include "device_error.cuh"

namespace vggt {

constexpr int kCacheMaxSeqs = 4096;
constexpr int kPlanThreads = 256;

struct PlanParams {
    int n_seqs, page_size, n_pages, max_pages, n_rows, free_capacity;
    const int32_t *cached, *fresh, *free_pages, *n_free;
    int32_t *table, *cu_rows, *kv_lens, *slots, *counts;
};

// Inclusive sums of a and b over the block's threads.
__device__ __forceinline__ void block_scan2(int64_t &a, int64_t &b, int64_t (*part)[2])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, b, d);
        if (lane >= d) {
            a += x;
            b += y;
        }
    }
    if (lane == 31) {
        part[warp][0] = a;
        part[warp][1] = b;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        a += part[w][0];
        b += part[w][1];
    }
}

// The first index in [0, n) whose value is above x (n if none).
__device__ __forceinline__ int upper_bound(const int *v, int n, int x)
{
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] > x)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// The plan of a step.  Every block sums the sequences' rows and page needs
// itself (a few loads each), so one launch does it all: the blocks share
// nothing, and a row of a freshly taken page gets the page from the free
// list and not from the block table that another block may be writing.
// Bound by latency: the longest plan writes some hundred kilobytes.
__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const PlanParams p)
{
    extern __shared__ int plan_smem[];
    int *row_end = plan_smem;             // rows up to and with the sequence, at most n_rows
    int *need_end = row_end + p.n_seqs;   // pages taken up to and with the sequence
    int *state = need_end + p.n_seqs;     // pages held before the step, -1: refused
    __shared__ int64_t part[kPlanThreads / 32][2];
    __shared__ int refused;
    if (threadIdx.x == 0)
        refused = 0;
    const int n_free = max(0, min(*p.n_free, p.free_capacity));
    const int per = (p.n_seqs + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(static_cast<int>(threadIdx.x) * per, p.n_seqs), b1 = min(b0 + per, p.n_seqs);

    // Rows first: whether a sequence's rows fit decides whether it asks for pages.
    int64_t rows = 0, zero = 0;
    for (int b = b0; b < b1; ++b)
        rows += max(0, p.fresh[b]);
    int64_t end = rows;
    block_scan2(end, zero, part);
    __syncthreads();
    int64_t at = end - rows, need = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t c = max(0, p.cached[b]), n = max(0, p.fresh[b]);
        at += n;
        const int64_t have = (c + p.page_size - 1) / p.page_size, want = (c + n + p.page_size - 1) / p.page_size;
        const bool fits = at <= p.n_rows && want <= p.max_pages;
        row_end[b] = static_cast<int>(at < p.n_rows ? at : p.n_rows);
        state[b] = fits ? static_cast<int>(have) : -1;
        need += fits ? want - have : 0;
    }
    int64_t upto = need;
    block_scan2(upto, zero, part);
    upto -= need;
    int missing = 0;
    for (int b = b0; b < b1; ++b) {
        const int c = max(0, p.cached[b]), n = max(0, p.fresh[b]);
        int64_t take = 0;
        if (state[b] >= 0)
            take = (static_cast<int64_t>(c) + n + p.page_size - 1) / p.page_size - state[b];
        const int64_t sum = upto + take;
        if (state[b] >= 0 && take > 0 && sum > n_free)
            state[b] = -1;
        upto = sum;
        // refused sequences come last among those that need pages, so their
        // sums stay at what was taken
        need_end[b] = static_cast<int>(sum < n_free ? sum : n_free);
        missing += state[b] < 0;
        if (blockIdx.x == 0)
            p.kv_lens[b] = state[b] < 0 ? c : c + n;
    }
    if (missing)
        atomicAdd(&refused, missing);
    __syncthreads();
    // Pages taken: the sum of the last granted sequence that takes any.
    // (need_end of a refused one is cut at n_free, which is not what was taken.)
    __shared__ int taken_s;
    if (threadIdx.x == 0)
        taken_s = 0;
    __syncthreads();
    for (int b = b0; b < b1; ++b)
        if (state[b] >= 0 && need_end[b] > (b ? need_end[b - 1] : 0))
            atomicMax(&taken_s, need_end[b]);
    __syncthreads();
    const int taken = taken_s;
    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b < p.n_seqs; b += kPlanThreads)
            p.cu_rows[b + 1] = row_end[b];
        if (threadIdx.x == 0) {
            p.cu_rows[0] = 0;
            p.counts[0] = n_free - taken;
            p.counts[1] = refused;
        }
    }
    const int step = gridDim.x * kPlanThreads, first = blockIdx.x * kPlanThreads + threadIdx.x;
    for (int i = first; i < taken; i += step) {
        const int b = upper_bound(need_end, p.n_seqs, i);
        const int before = b ? need_end[b - 1] : 0;
        p.table[static_cast<int64_t>(b) * p.max_pages + state[b] + i - before] = p.free_pages[n_free - 1 - i];
    }
    for (int64_t r = first; r < p.n_rows; r += step) {
        const int b = upper_bound(row_end, p.n_seqs, static_cast<int>(r));
        int slot = -1;
        if (b < p.n_seqs && state[b] >= 0) {
            const int pos = max(0, p.cached[b]) + static_cast<int>(r) - (b ? row_end[b - 1] : 0);
            const int pi = pos / p.page_size;
            const int page = pi < state[b] ? p.table[static_cast<int64_t>(b) * p.max_pages + pi]
                                           : p.free_pages[n_free - 1 - ((b ? need_end[b - 1] : 0) + pi - state[b])];
            if (page >= 0 && page < p.n_pages)
                slot = page * p.page_size + pos % p.page_size;
        }
        p.slots[r] = slot;
    }
}

struct AppendParams {
    int n_rows, vecs;  // vecs: 16-byte vectors of a row, n_kv_heads * 8
    int page_size, n_slots;
    int64_t row_stride, in_head_stride;              // new rows, in 16-byte vectors
    int64_t page_stride, head_stride, token_stride;  // pages, in 16-byte vectors
    const uint4 *k, *v;
    uint4 *k_pages, *v_pages;
    const int32_t *slots;
};

// K and V rows into their slots; a negative slot is skipped.  Bound by HBM:
// every row of K and V is read once and written once.
__global__ void __launch_bounds__(256) cache_append_kernel(const AppendParams p)
{
    const int64_t total = static_cast<int64_t>(p.n_rows) * p.vecs;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r = i / p.vecs;
        const int e = static_cast<int>(i - r * p.vecs), h = e >> 3, c = e & 7;
        const int slot = p.slots[r];
        if (slot < 0)
            continue;
        if (slot >= p.n_slots) {
            record_bounds_failure(kCheckCacheSlot);
            continue;
        }
        const int page = slot / p.page_size, off = slot - page * p.page_size;
        const int64_t src = r * p.row_stride + h * p.in_head_stride + c;
        const int64_t dst = page * p.page_stride + h * p.head_stride + off * p.token_stride + c;
        p.k_pages[dst] = p.k[src];
        p.v_pages[dst] = p.v[src];
    }
}

} // namespace vggt
