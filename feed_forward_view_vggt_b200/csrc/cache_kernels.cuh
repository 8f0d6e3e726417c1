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

// x / d for 0 <= x < 2^31 by a multiplication (planning is a chain of
// divisions with nothing else to do meanwhile): with
// 2^(k-1) < d <= 2^k and mul = floor(2^(31+k) / d) + 1, mul d exceeds 2^(31+k)
// by at most d <= 2^k, which moves the quotient of no x < 2^31.
struct Divisor {
    uint32_t d, mul, shift;

    void set(uint32_t value)
    {
        d = value;
        uint32_t k = 0;
        while ((uint64_t{1} << k) < value)
            ++k;
        shift = k > 0 ? k - 1 : 0;
        mul = k > 0 ? static_cast<uint32_t>((uint64_t{1} << (31 + k)) / value + 1) : 0;
    }
    __device__ __forceinline__ int div(int x) const
    {
        return d == 1 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), mul) >> shift);
    }
};

struct PlanParams {
    int n_seqs, page_size, n_pages, max_pages, n_rows, free_capacity;
    Divisor by_page;
    const int32_t *cached, *fresh, *free_pages, *n_free;
    int32_t *table, *cu_rows, *kv_lens, *slots, *counts;

    // Pages of n positions.
    __device__ __forceinline__ int pages(int n) const { return n > 0 ? by_page.div(n - 1) + 1 : 0; }
};

// Inclusive sums over the block's threads; `part` is used once.
__device__ __forceinline__ int64_t block_scan(int64_t a, int64_t *part)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, d);
        if (lane >= d)
            a += x;
    }
    if (lane == 31)
        part[warp] = a;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32 - 1; ++w)
        a += w < warp ? part[w] : 0;
    return a;
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
// Bound by latency: the longest plan writes some hundred kilobytes.  The
// lengths are read once, into shared memory.
__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const PlanParams p)
{
    extern __shared__ int plan_smem[];
    int *row_end = plan_smem;             // rows up to and with the sequence, at most n_rows
    int *need_end = row_end + p.n_seqs;   // pages taken up to and with the sequence
    int *state = need_end + p.n_seqs;     // pages held before the step, -1: refused
    int *held = state + p.n_seqs;         // positions before the step
    __shared__ int64_t part[2][kPlanThreads / 32];
    __shared__ int refused, taken_s;
    if (threadIdx.x == 0)
        refused = taken_s = 0;
    const int n_free = max(0, min(*p.n_free, p.free_capacity));
    const int per = (p.n_seqs + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(static_cast<int>(threadIdx.x) * per, p.n_seqs), b1 = min(b0 + per, p.n_seqs);

    // Rows first: whether a sequence's rows fit decides whether it asks for pages.
    int64_t rows = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = max(0, p.fresh[b]);
        held[b] = max(0, p.cached[b]);
        need_end[b] = n;
        rows += n;
    }
    int64_t at = block_scan(rows, part[0]) - rows, need = 0;
    for (int b = b0; b < b1; ++b) {
        const int c = held[b], n = need_end[b];
        at += n;
        // past 2^31 - 1 positions the table is too small in any case
        const int have = p.pages(c);
        const int want = p.pages(static_cast<int>(min(static_cast<unsigned>(c) + static_cast<unsigned>(n), 0x7fffffffu)));
        const bool fits = at <= p.n_rows && want <= p.max_pages;
        row_end[b] = static_cast<int>(at < p.n_rows ? at : p.n_rows);
        state[b] = fits ? have : -1;
        need_end[b] = fits ? want - have : 0;
        need += need_end[b];
        if (blockIdx.x == 0)
            p.kv_lens[b] = c + (fits && want == have ? n : 0);
    }
    int64_t upto = block_scan(need, part[1]) - need;
    int missing = 0, mine = 0;
    for (int b = b0; b < b1; ++b) {
        const int take = need_end[b];
        upto += take;
        if (take > 0 && upto > n_free)
            state[b] = -1;
        else if (take > 0) {
            mine = static_cast<int>(upto);
            if (blockIdx.x == 0)
                p.kv_lens[b] = held[b] + max(0, p.fresh[b]);
        }
        // refused sequences come last among those that need pages, so their
        // sums stay at what was taken
        need_end[b] = static_cast<int>(upto < n_free ? upto : n_free);
        missing += state[b] < 0;
    }
    if (missing)
        atomicAdd(&refused, missing);
    // Pages taken: the sum of the last granted sequence that takes any.
    // (need_end of a refused one is cut at n_free, which is not what was taken.)
    if (mine)
        atomicMax(&taken_s, mine);
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
            const int pos = held[b] + static_cast<int>(r) - (b ? row_end[b - 1] : 0);
            const int pi = p.by_page.div(pos);
            const int page = pi < state[b] ? p.table[static_cast<int64_t>(b) * p.max_pages + pi]
                                           : p.free_pages[n_free - 1 - ((b ? need_end[b - 1] : 0) + pi - state[b])];
            if (page >= 0 && page < p.n_pages)
                slot = page * p.page_size + pos - pi * p.page_size;
        }
        p.slots[r] = slot;
    }
}

struct AppendParams {
    int n_rows, vecs;  // vecs: 16-byte vectors of a row, n_kv_heads * 8
    int page_size, n_slots;
    Divisor by_vecs, by_page;
    int64_t row_stride, in_head_stride;              // new rows, in 16-byte vectors
    int64_t page_stride, head_stride, token_stride;  // pages, in 16-byte vectors
    const uint4 *k, *v;
    uint4 *k_pages, *v_pages;
    const int32_t *slots;
};

// K and V rows into their slots; a negative slot is skipped.  Bound by HBM:
// every row of K and V is read once and written once (16 frames of 1374
// tokens, 16 heads: 26 us alone, 6.9 TB/s, and 32.6 in a row).  A thread moves kEach vectors of K and of V, all
// loads before the stores; small steps, which are bound by latency, spread over
// more blocks with kEach = 1.
template <int kEach>
__global__ void __launch_bounds__(256) cache_append_kernel(const AppendParams p)
{
    const int64_t start = static_cast<int64_t>(blockIdx.x) * (256 * kEach), row0 = start / p.vecs;
    const int in_row = static_cast<int>(start - row0 * p.vecs) + static_cast<int>(threadIdx.x);
    uint4 k[kEach], v[kEach];
    int64_t dst[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int at = in_row + 256 * i, below = p.by_vecs.div(at), e = at - below * p.vecs, h = e >> 3, c = e & 7;
        const int64_t r = row0 + below;
        dst[i] = -1;
        if (r >= p.n_rows)
            continue;
        const int slot = __ldg(p.slots + r);
        if (slot < 0)
            continue;
        if (slot >= p.n_slots) {
            record_bounds_failure(kCheckCacheSlot);
            continue;
        }
        const int page = p.by_page.div(slot), off = slot - page * p.page_size;
        dst[i] = page * p.page_stride + h * p.head_stride + off * p.token_stride + c;
        const int64_t src = r * p.row_stride + h * p.in_head_stride + c;
        k[i] = p.k[src];
        v[i] = p.v[src];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (dst[i] >= 0) {
            p.k_pages[dst[i]] = k[i];
            p.v_pages[dst[i]] = v[i];
        }
    }
}

} // namespace vggt
