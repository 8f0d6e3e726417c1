// cached_attn_kernel.cuh -- attention of a step's new rows over a paged K/V
// cache on the sm_100a tensor cores:
//   O_i = sum_j e^{s q_i.k_j} v_j / sum_j e^{s q_i.k_j},  j < lim_i,
//   lim_i = min(kv, (floor(pos_i / u) + 1) u)   (u = 0: kv),
// over the keys of i's own sequence, in one pass with a running offset and
// sum of the softmax.
//
// Rows.  The G = H / Hkv query heads of a key head are rows of one tile: a
// tile holds F = floor(128 / G) consecutive tokens of a sequence, G rows each,
// so a key tile is read once for all of them.
//
// Work.  A unit is, for one key head of a sequence,
//  * a pair of query tiles: both read one K/V stream, one softmax warpgroup
//    each (two steps per key tile);
//  * a single query tile (the last of an odd number): the warpgroups take the
//    key tiles in turn (one step per key tile) and warpgroup 0 merges the two
//    softmax states at the end; or
//  * the same with at most 16 rows (a single token of grouped heads): the
//    eight softmax warps multiply on registers, see run_few.
// A step costs about the same in all: 4.2 MFLOP on the tensor cores, or the 32
// KB of K and V of a key tile, 0.7 us of an SM's share of either.  The units
// stand in one line (sequence, head, tile), and CTA i takes the i-th of equal
// parts of their steps, wherever that cuts them: no CTA waits for another, no
// host copy of the lengths is needed, and every CTA finds its part from the
// lengths by itself.  A unit that is cut leaves (m, l) and the sum of P V of
// its parts in fp32 in the workspace, two slots per CTA, and
// cached_combine_kernel joins them in order.
//
// CTA (384 threads, one per SM): warps 0 and 3 load Q and K, and V, by TMA, page
// by page (a 4-D map of the pages; a box is the largest power of two of rows
// that divides the page, at most 128); warp 0 also walks along the CTA's work
// and writes its tasks into a ring; warps 1 and 2 issue the UMMAs; warps 4-7
// and 8-11 are the softmax warpgroups.  TMEM, score buffers and the order S(k+3)
// after PV(k) are those of attn_fwd_kernel.
//
// Bound by the exponentials and the instructions around them, as that kernel
// is: one frame of 1374 tokens over 100 cached ones, 16 heads, 0.89 ms or 870
// TFLOP/s alone, 1.04 ms or 750 in a row under the power cap.  Single tokens are
// bound by HBM: 148 sequences of 32000 keys 6.9 TB/s, 48 of odd lengths with
// grouped heads 134 us or 6.4 TB/s in pages of 128; small pages by their many
// copies, 137 us in pages of 64, 151 of 32, 175 of 16.  Small calls are bound by
// latency: planning 0.8 us, finding the first task 1.2 us, first keys 1.5 us,
// the end of a task 1.5 us, the joining launch 2 us (one token over 5496 keys
// and 16 heads: 12 us in a graph).
//
// P is rounded to bf16 for the PV product, whose operands have one type (each p
// off by at most 2^-8 of itself; over all outputs 0.0016 of their size, beside
// 0.0017 from the rounding of O); the sums l and O are fp32, l of P before it is
// rounded.
//
// Keys behind kv are never used, whatever the page holds there: their scores
// are masked, their V rows are zeroed in shared memory up to the next multiple
// of 16 (a 0 in P does not survive an infinity in V), and the PV product of
// the last tile stops there.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "attn_kernel.cuh"
#include "cache_kernels.cuh"
#include "device_error.cuh"
#include "ptx.cuh"
#include "shares.cuh"

namespace vggt {

// Of every 16 column pairs of a score row, those whose exponentials are a
// polynomial (see attn_fwd_kernel).  Its argument is cut at 127 from above too:
// against the old offset a later tile's may be hundreds, and 2^j has no exponent
// bits then; cut, P is so large that the tile is done again.  Measured, one
// frame over 100 cached: 1 pair 905 us, 2: 907, 3: 983; over 32, in a row: 1
// 344 us, 2: 341.
constexpr int kCachedPolyPairs = 2;
constexpr int kTaskRing = 8;

constexpr int kFewRows = 16;      // rows of a task that the warps work on by themselves
constexpr int kSoftmaxWarps = 8;  // and with how many: 32 keys of every other tile each
static_assert(kStages % 2 == 0, "a warp of such a task waits for every other tile and must see every phase of its slots");

enum : uint32_t { kSiteTaskFull = 12, kSiteTaskEmpty, kSiteMergeReady, kSiteMergeFree, kSiteFewQ, kSiteFewFull, kSiteTaskPassed };

// What a CTA leaves for the joining launch: the unit whose first part, but not
// its last, was its work.  Parts 1, 2, ... are those of the CTAs behind it.
struct Join {
    int row0, rows, hk, parts;  // parts = 0: none
};

struct CachedParams {
    int n_seqs, n_rows, H, Hkv, group, tile_tokens;  // group G = H / Hkv, tile_tokens F
    int page_size, n_pages, max_pages, unit, box_rows;
    Divisor by_group, by_tile, by_page, by_unit;
    int cost_shift;  // costs are counted in 2^cost_shift steps, so that their sum fits in 31 bits
    int part_rows;   // rows of a workspace slot
    float scale_log2;
    const int32_t *table, *cu_rows, *kv_lens;
    __nv_bfloat16 *o;
    float *lse;
    Join *join;       // workspace: [kMaxCtas]
    float2 *part_ml;  // [2 * kMaxCtas][part_rows]; slot 2 i: CTA i's part that starts inside a unit, 2 i + 1: at its start
    float *part_o;    // [2 * kMaxCtas][part_rows][64]
    unsigned long long wait_limit_ns;
};

struct Task {
    int row0, row_end;  // first token row of the task's first tile, end of its sequence's rows
    int pos0, kv;       // position of row0's token, keys of the sequence
    int kt0, n;         // first key tile, key tiles (0: the end of the CTA's tasks)
    int b, hk;
    int kind, slot;     // slot of the workspace, -1: the whole unit
    int vlast;          // keys of the last tile that exist, 1..128
    int rot;            // the j-th tile worked on is (j + rot) mod n
};

struct __align__(1024) CachedSmem {
    uint8_t q[2][2][kTileBytes];  // [buffer][tile]
    uint8_t k[kStages][kTileBytes];
    uint8_t v[kStages][kTileBytes];
    Task task[kTaskRing];
    float2 merge_ml[kBlockM];  // warpgroup 1's (m, l) of a single tile; [warp][row] of a task of few rows
    uint64_t q_full[2], q_empty[2];
    uint64_t k_full[kStages], k_empty[kStages];
    uint64_t v_full[kStages], v_empty[kStages];
    uint64_t s_full[2][3], p_ready[2][3];  // by warpgroup and its step count mod 3
    uint64_t buf_free[kScoreBufs], o_final[2];
    uint64_t merge_ready, merge_free;
    uint64_t few_q, few_full[2];  // by tasks of few rows mod 2
    uint64_t task_passed[2 * kTaskRing];  // the issuers are past the task
    uint64_t task_full[kTaskRing], task_empty[kTaskRing];
    uint64_t drain[2];
    uint32_t tmem_base;
    WaitCtl ctl;
    int work;
    int scan[kAttnThreads / 32];
    int work_end[1];  // [n_seqs]: cost of the units up to and with the sequence
};

constexpr size_t cached_smem_bytes(int n_seqs)
{
    return sizeof(CachedSmem) + 4 * static_cast<size_t>(n_seqs) + 1024;
}

// ------------------------------------------------------------ geometry

struct Seq {
    int row0, n, kv;
};

__device__ __forceinline__ Seq load_seq(const CachedParams &p, int b)
{
    Seq s;
    s.row0 = max(0, min(__ldg(p.cu_rows + b), p.n_rows));
    s.n = max(s.row0, min(__ldg(p.cu_rows + b + 1), p.n_rows)) - s.row0;
    s.kv = max(0, min(__ldg(p.kv_lens + b), p.max_pages * p.page_size));
    return s;
}

// Keys that the row of position pos sees.  pos + unit fits in 32 unsigned bits.
__device__ __forceinline__ int key_limit(const CachedParams &p, int kv, int pos)
{
    if (p.unit == 0)
        return kv;
    if (pos < 0)
        return 0;
    const unsigned lim = (static_cast<unsigned>(p.by_unit.div(pos)) + 1u) * static_cast<unsigned>(p.unit);
    return static_cast<int>(min(static_cast<unsigned>(kv), lim));
}

// Key tiles that rows 0 .. i of a sequence see (the limit never falls with the row).
__device__ __forceinline__ int key_tiles(const CachedParams &p, const Seq &s, int i)
{
    return (key_limit(p, s.kv, s.kv - s.n + i) + kBlockN - 1) / kBlockN;
}

// Key tiles of query-tile pair pr.
__device__ __forceinline__ int pair_tiles(const CachedParams &p, const Seq &s, int pr)
{
    return key_tiles(p, s, min(s.n, (2 * pr + 2) * p.tile_tokens) - 1);
}

// The units of one key head of a sequence: pairs first, then the single tile.
__device__ __forceinline__ int unit_count(const CachedParams &p, const Seq &s)
{
    return (p.by_tile.div(s.n + p.tile_tokens - 1) + 1) >> 1;
}

struct Unit {
    int kind, tiles, cost;
};

__device__ __forceinline__ Unit unit_of(const CachedParams &p, const Seq &s, int i)
{
    Unit u;
    const int left = s.n - 2 * i * p.tile_tokens;
    u.kind = left > p.tile_tokens ? kTaskPair : (left * p.group <= kFewRows ? kTaskFew : kTaskSingle);
    u.tiles = pair_tiles(p, s, i);
    u.cost = unit_points(u.kind, u.tiles, p.cost_shift);
    return u;
}

// Sums the costs: work_end and work.  Every thread takes a run of consecutive
// sequences; one with many pairs of unequal length is summed by its warp.  The
// host chose cost_shift for row offsets that ascend and stay below n_rows; with
// others there is no work, and the error word says so.
__device__ __forceinline__ void plan_work(CachedSmem &sm, const CachedParams &p)
{
    constexpr int kLong = 8;
    const int tid = threadIdx.x, lane = tid & 31;
    const int per = (p.n_seqs + kAttnThreads - 1) / kAttnThreads;
    int mine = 0;
    bool bad = false;
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        Seq s{0, 0, 0};
        if (b < p.n_seqs) {
            s = load_seq(p, b);
            const int row0 = __ldg(p.cu_rows + b), row1 = __ldg(p.cu_rows + b + 1);
            bad = bad || row0 < 0 || row1 < row0 || row1 > p.n_rows;
        }
        const int units = unit_count(p, s);
        int sum = 0;
        bool loop = false;
        if (units > 0) {
            const Unit last = unit_of(p, s, units - 1);
            sum = last.cost;
            if (units > 1) {
                const Unit first = unit_of(p, s, 0), other = unit_of(p, s, units - 2);
                if (first.cost == other.cost)
                    sum += (units - 1) * first.cost;
                else if (units <= kLong)
                    for (int j = 0; j < units - 1; ++j)
                        sum += unit_of(p, s, j).cost;
                else
                    loop = true;
            }
        }
        for (unsigned todo = __ballot_sync(0xffffffffu, loop); todo; todo &= todo - 1) {
            const int src = __ffs(todo) - 1;
            const Seq x{__shfl_sync(0xffffffffu, s.row0, src), __shfl_sync(0xffffffffu, s.n, src),
                        __shfl_sync(0xffffffffu, s.kv, src)};
            int part = 0;
            for (int j = lane; j < unit_count(p, x) - 1; j += 32)
                part += unit_of(p, x, j).cost;
            part = __reduce_add_sync(0xffffffffu, part);
            if (lane == src)
                sum += part;
        }
        mine += sum * p.Hkv;
        if (b < p.n_seqs)
            sm.work_end[b] = mine;
    }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d)
            upto += x;
    }
    if (lane == 31)
        sm.scan[tid >> 5] = upto;
    bad = __syncthreads_or(bad);
    for (int w = 0; w < (tid >> 5); ++w)
        upto += sm.scan[w];
    if (upto != mine)
        for (int b = tid * per; b < min((tid + 1) * per, p.n_seqs); ++b)
            sm.work_end[b] += upto - mine;
    if (tid == kAttnThreads - 1) {
        sm.work = bad ? 0 : upto;
        if (bad)
            record_bounds_failure(kCheckCacheRows);
    }
}

// --------------------------------------------------------------- roles

// O = 0 and lse = -inf for the rows of a task none of which sees a key.
__device__ __forceinline__ void write_empty_rows(const CachedParams &p, int row0, int row_end, int kind, int hk)
{
    const int lane = threadIdx.x & 31;
    const int rows = min(row_end - row0, (kind == kTaskPair ? 2 : 1) * p.tile_tokens) * p.group;
    for (int i = lane >> 3; i < rows; i += 4) {
        const int tok = p.by_group.div(i);
        const int64_t id = static_cast<int64_t>(row0 + tok) * p.H + hk * p.group + i - tok * p.group;
        reinterpret_cast<uint4 *>(p.o + id * kHeadDim)[lane & 7] = make_uint4(0u, 0u, 0u, 0u);
        if (p.lse && (lane & 7) == 0)
            p.lse[id] = -INFINITY;
    }
}

// Reads task `it` from the ring (the caller releases it once read).
__device__ __forceinline__ bool wait_task(CachedSmem &sm, int it)
{
    return wait_bar(smem_u32(&sm.task_full[it % kTaskRing]), (static_cast<uint32_t>(it) / kTaskRing) & 1, &sm.ctl,
                    kSiteTaskFull);
}

__device__ __forceinline__ void release_task(CachedSmem &sm, int it)
{
    mbar_arrive(smem_u32(&sm.task_empty[it % kTaskRing]));
}

// Copies in flight of a producer warp: uses of the K (or V) ring, Q tiles.
struct Issued {
    uint32_t tiles, q;
};

// Loads the K (with Q before it) or the V tiles of a task; false when a wait
// ran out.  Page by page: lane i copies the i-th box of a tile.
template <bool kIsV>
__device__ __forceinline__ bool load_task(CachedSmem &sm, const CUtensorMap *tmQ, const CUtensorMap *tmKV,
                                          const CachedParams &p, const Task &t, Issued &issued)
{
    volatile WaitCtl *ab = &sm.ctl;
    const int lane = threadIdx.x & 31;
    const uint32_t box_bytes = static_cast<uint32_t>(p.box_rows) * kHeadDim * 2;
    const uint32_t full = smem_u32(kIsV ? sm.v_full : sm.k_full), empty = smem_u32(kIsV ? sm.v_empty : sm.k_empty);
    const uint32_t tiles = smem_u32(kIsV ? sm.v[0] : sm.k[0]);
    const int n = t.n, hk = t.hk, kt0 = t.kt0, vlast = t.vlast, rot = t.rot;
    const int32_t *table = p.table + static_cast<int64_t>(t.b) * p.max_pages;
    if (!kIsV) {
        const uint32_t qb = issued.q & 1u, q_bytes = static_cast<uint32_t>(p.group * p.tile_tokens) * kHeadDim * 2;
        if (!wait_bar_warp(smem_u32(&sm.q_empty[qb]), ((issued.q >> 1) & 1u) ^ 1u, ab, kSiteQEmpty))
            return false;
        if (lane == 0) {
            const bool pair = t.kind == kTaskPair;
            mbar_arrive_expect_tx(smem_u32(&sm.q_full[qb]), pair ? 2 * q_bytes : q_bytes);
            tma_load_3d(smem_u32(sm.q[qb][0]), tmQ, smem_u32(&sm.q_full[qb]), 0, hk * p.group, t.row0);
            if (pair)
                tma_load_3d(smem_u32(sm.q[qb][1]), tmQ, smem_u32(&sm.q_full[qb]), 0, hk * p.group,
                            t.row0 + p.tile_tokens);
        }
        ++issued.q;
    }
    // Page of this lane's box of tile j; the first key of the box exists.
    auto lookup = [&](int j) -> int {
        const int r = j + rot < n ? j + rot : j + rot - n, valid = r == n - 1 ? vlast : kBlockN;
        if (lane * p.box_rows >= valid)
            return 0;
        const int page = __ldg(table + p.by_page.div((kt0 + r) * kBlockN + lane * p.box_rows));
        if (page >= 0 && page < p.n_pages)
            return page;
        record_bounds_failure(kCheckCachePage);
        return p.n_pages;  // outside the map: the box is filled with zeros
    };
    int page = lookup(0);
    for (int j = 0; j < n; ++j) {
        const int r = j + rot < n ? j + rot : j + rot - n, valid = r == n - 1 ? vlast : kBlockN;
        const int boxes = (valid + p.box_rows - 1) / p.box_rows;
        const int key = (kt0 + r) * kBlockN + lane * p.box_rows, off = key - p.by_page.div(key) * p.page_size;
        const int here = page;
        if (j + 1 < n)
            page = lookup(j + 1);
        const uint32_t st = issued.tiles % kStages;
        if (!wait_bar_warp(empty + 8 * st, ((issued.tiles / kStages) & 1u) ^ 1u, ab, kIsV ? kSiteVEmpty : kSiteKEmpty))
            return false;
        if (lane == 0)
            mbar_arrive_expect_tx(full + 8 * st, boxes * box_bytes);
        ++issued.tiles;
        __syncwarp();
        if (lane < boxes)
            tma_load_4d(tiles + st * kTileBytes + lane * box_bytes, tmKV, full + 8 * st, 0, off, hk, here);
    }
    return true;
}

// Every copy that the warp started must land before the CTA may exit.
template <bool kIsV>
__device__ __forceinline__ void drain_copies(CachedSmem &sm, const Issued &issued)
{
    const uint32_t full = smem_u32(kIsV ? sm.v_full : sm.k_full);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        for (uint32_t i = (issued.tiles > kStages ? issued.tiles - kStages : 0); i < issued.tiles; ++i)
            wait_drain(full + 8 * (i % kStages), (i / kStages) & 1);
        for (uint32_t i = (issued.q > 2 ? issued.q - 2 : 0); i < issued.q; ++i)
            wait_drain(smem_u32(&sm.q_full[i & 1]), (i >> 1) & 1);
    }
    __syncwarp();
}

// Warp 0: walks along the CTA's part of the work, hands on its tasks, then one
// with n = 0 that ends the list, and loads their Q and K tiles.  It walks from
// the end, and a task's tiles may be taken in a rotated order: a head's CTAs,
// whose shares start at different keys, then read about the same keys at the
// same time, and its K and V leave DRAM fewer times: one frame over 100 cached
// reads 1.35 GB instead of 3.15 (0.56 are needed), 894 us instead of 938 alone and
// 1039 instead of 1110 in a row, where the power cap sets the clock.  V is warp 3's:
// the copies of a tile of small pages are many (16 of 2 KB for pages of 16),
// and a warp issues those of its lanes one after another.  Units without keys (a first
// chunk that was refused pages, e.g.) are dealt with here and never enter the
// ring.
__device__ __forceinline__ void walk_work(CachedSmem &sm, const CUtensorMap *tmQ, const CUtensorMap *tmK,
                                          const CachedParams &p, Issued &issued)
{
    const int lane = threadIdx.x & 31, cta = static_cast<int>(blockIdx.x);
    const Shares shares(sm.work, p.cost_shift, static_cast<int>(gridDim.x));
    Join join{0, 0, 0, 0};
    int w0 = 0, w = 0;  // the share's first point, and the end of what is left of it
    if (cta < shares.ctas) {
        w0 = shares.start(cta);
        w = shares.start(cta + 1);
    }
    int now = 0;  // tiles of a pair that took as long as the work so far
    uint32_t it = 0;
    auto push = [&](const Task &t) -> bool {
        const uint32_t slot = it % kTaskRing;
        if (!wait_bar_warp(smem_u32(&sm.task_empty[slot]), ((it / kTaskRing) & 1) ^ 1, &sm.ctl, kSiteTaskEmpty))
            return false;
        if (lane == 0) {
            sm.task[slot] = t;
            mbar_arrive(smem_u32(&sm.task_full[slot]));
        }
        __syncwarp();
        ++it;
        return t.n == 0 || load_task<false>(sm, tmQ, tmK, p, t, issued);
    };
    while (w > w0) {
        // The sequence, head and unit of the last point, and x, its place in the unit.
        const int at = w - 1, b = upper_bound(sm.work_end, p.n_seqs, at);
        const int first = b ? sm.work_end[b - 1] : 0, per_head = (sm.work_end[b] - first) / p.Hkv;
        const Seq s = load_seq(p, b);
        const int units = unit_count(p, s);
        int hk = (at - first) / per_head, x = at - first - hk * per_head, i = 0;
        for (;; i += 32) {
            const int cost = i + lane < units ? unit_of(p, s, i + lane).cost : 0;
            int upto = cost;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d)
                    upto += y;
            }
            const unsigned over = __ballot_sync(0xffffffffu, upto > x);
            if (over || i + 32 >= units) {
                const int in = over ? __ffs(over) - 1 : 31;
                x -= __shfl_sync(0xffffffffu, upto - cost, in);
                i += in;
                break;
            }
            x -= __shfl_sync(0xffffffffu, upto, 31);
        }
        int x1 = x + 1;  // end of the share in the unit
        while (w > w0 && hk >= 0) {
            const Unit u = unit_of(p, s, i);
            x1 = x1 > 0 ? x1 : u.cost;
            const int x0 = max(0, x1 - (w - w0));
            Task t;
            t.row0 = s.row0 + 2 * i * p.tile_tokens;
            t.row_end = s.row0 + s.n;
            t.hk = hk;
            t.kind = u.kind;
            if (u.tiles == 0) {
                if (x0 == 0)
                    write_empty_rows(p, t.row0, t.row_end, t.kind, t.hk);
            } else {
                t.kt0 = tiles_before(u.kind, u.tiles, x0, p.cost_shift);
                t.n = tiles_before(u.kind, u.tiles, x1, p.cost_shift) - t.kt0;
                t.b = b;
                t.pos0 = s.kv - (t.row_end - t.row0);
                t.kv = s.kv;
                t.vlast = min(kBlockN, s.kv - (t.kt0 + t.n - 1) * kBlockN);
                t.slot = -1;
                if (t.n > 0 && t.n < u.tiles) {
                    t.slot = 2 * cta + (t.kt0 == 0);
                    if (t.kt0 == 0) {
                        // up to the CTA that has the unit's last point
                        join.row0 = t.row0;
                        join.rows = min(t.row_end - t.row0, 2 * p.tile_tokens) * p.group;
                        join.hk = hk;
                        join.parts = shares.last(cta, w - x1 + u.cost) - cta + 1;
                    }
                }
                // Where every row sees every key of the task, its tiles are taken
                // in the order that brings tile `now` of the head at time `now`.
                t.rot = 0;
                if (t.kind != kTaskFew && key_limit(p, t.kv, t.pos0) >= min(t.kv, (t.kt0 + t.n) * kBlockN)) {
                    const int ahead = now - t.kt0;
                    if (ahead > -t.n && ahead < t.n)
                        t.rot = ahead >= 0 ? ahead : ahead + t.n;
                }
                if (t.n > 0 && !push(t))
                    return;
                now += t.kind == kTaskPair ? t.n : t.n >> 1;
            }
            w -= x1 - x0;
            x1 = 0;
            if (--i < 0) {
                i = units - 1;
                --hk;
            }
        }
    }
    if (lane == 0 && p.join)
        p.join[cta] = join;
    push(Task{});
}

__device__ __forceinline__ void run_k_producer(CachedSmem &sm, const CUtensorMap *tmQ, const CUtensorMap *tmK,
                                               const CachedParams &p)
{
    Issued issued{0, 0};
    walk_work(sm, tmQ, tmK, p, issued);
    drain_copies<false>(sm, issued);
}

__device__ __forceinline__ void run_v_producer(CachedSmem &sm, const CUtensorMap *tmV, const CachedParams &p)
{
    Issued issued{0, 0};
    for (int it = 0;; ++it) {
        const bool got = wait_task(sm, it);
        __syncwarp();
        if (!__all_sync(0xffffffffu, got))
            break;
        const Task t = sm.task[it % kTaskRing];
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            release_task(sm, it);
        if (t.n == 0 || !load_task<true>(sm, nullptr, tmV, p, t, issued))
            break;
    }
    drain_copies<true>(sm, issued);
}

// The two issuers, one thread each: warp 2 issues S = Q K^T, warp 1 O += P V
// (one thread for both took 1450 clocks per step with every barrier it waited
// for complete: the loop itself was the bound).  Step k of the CTA uses score
// buffer k % 3: S(k + 3) waits for PV(k), so the scores are up to three steps
// ahead.  Within a task step s belongs to warpgroup s & 1, and to key tile s /
// 2 (pair) or s (single).
//
// A task of few rows is passed: the warps read its tiles themselves.  Whoever
// follows a ring barrier without waiting for every phase of it must not run
// ahead of one: the warps start on such a task when both issuers have passed it
// (then all loads before it are complete; a warp may have had no step in some
// single tiles), and an issuer goes on to the next task for the tensor cores
// when the warps are done (fews_over).  Twice the slots of the task ring keep
// the phases of `task_passed` apart: an issuer has left task it - 16 when task
// it appears in the ring, and cannot reach it + 16 before the warps release it + 8.
// (tests/cached_protocol_model.py runs the barriers under random timings.)
__device__ __forceinline__ void pass_task(CachedSmem &sm, int it)
{
    mbar_arrive(smem_u32(&sm.task_passed[it % (2 * kTaskRing)]));
}

// A ring barrier that the warps release with one arrival each; the issuer
// stands for all of them, with its last arrival when the products are done.
__device__ __forceinline__ void commit_release(uint32_t bar)
{
    mbar_arrive_n(bar, kSoftmaxWarps - 1);
    umma_commit(bar);
}

// Slot and phase of barriers that are used in turn.
template <uint32_t kSlots>
struct Turn {
    uint32_t slot, ph;

    __device__ __forceinline__ void next()
    {
        if (++slot == kSlots) {
            slot = 0;
            ph ^= 1u;
        }
    }
};

template <bool kIsPV>
__device__ __forceinline__ void issue_loop(CachedSmem &sm, uint32_t tmem)
{
    volatile WaitCtl *ab = &sm.ctl;
    const uint64_t q0 = sdesc_sw128(smem_u32(sm.q[0][0]), 16, 1024);
    const uint64_t kv0 = sdesc_sw128(smem_u32(kIsPV ? sm.v[0] : sm.k[0]), 16, 1024);
    const uint32_t full = smem_u32(kIsPV ? sm.v_full : sm.k_full), empty = smem_u32(kIsPV ? sm.v_empty : sm.k_empty);
    const uint32_t mine = smem_u32(kIsPV ? sm.p_ready[0] : sm.s_full[0]);  // [wg][turn]
    const uint32_t freed = smem_u32(sm.buf_free);
    Turn<kStages> ring{0, 0};
    Turn<kScoreBufs> buf{0, 0}, turn{0, 0}, other{0, 0};  // of the step's warpgroup and of the other one
    uint32_t fews = 0, fews_done = 0;  // tasks of few rows passed, and those known to be over (fews or one less)
    auto fews_over = [&]() -> bool {
        if (fews_done == fews)
            return true;
        ++fews_done;
        return wait_bar(smem_u32(&sm.few_full[(fews_done - 1) & 1u]), ((fews_done - 1) >> 1) & 1u, ab, kSiteFewFull);
    };
    for (int it = 0;; ++it) {
        if (!wait_task(sm, it))
            return;
        const Task &t = sm.task[it % kTaskRing];
        const int n = t.n, kind = t.kind, kk_last = (t.vlast + 15) >> 4, last_at = n - 1 - t.rot;
        release_task(sm, it);
        if (n == 0)
            return;
        if (kind == kTaskFew) {
            // the warps may start on it while they still work on the one before
            pass_task(sm, it);
            if (!fews_over())
                return;
            ++fews;
            const uint32_t x = ring.slot + static_cast<uint32_t>(n);
            ring.ph ^= (x / kStages) & 1u;
            ring.slot = x % kStages;
            continue;
        }
        if (!fews_over())
            return;
        const bool pair = kind == kTaskPair;
        const int steps = pair ? 2 * n : n;
        const uint32_t qb = static_cast<uint32_t>(it) & 1u;
        if (!kIsPV && !wait_bar(smem_u32(&sm.q_full[qb]), (static_cast<uint32_t>(it) >> 1) & 1u, ab, kSiteQFull))
            return;
        for (int s = 0; s < steps; ++s) {
            const uint32_t wg = static_cast<uint32_t>(s) & 1u;
            const bool first_reader = !pair || !wg, last_reader = !pair || wg;
            if (first_reader && !wait_bar(full + 8 * ring.slot, ring.ph, ab, kIsPV ? kSiteVFull : kSiteKFull))
                return;
            const uint32_t bar = mine + 8 * (3 * wg + turn.slot);
            const uint64_t b = kv0 + ring.slot * kTileDescStep;
            const uint32_t scores = tmem + buf.slot * kBlockN;
            if (kIsPV) {
                constexpr uint32_t kIdesc = idesc_bf16_f32(kBlockM, kHeadDim, true);
                if (!wait_bar(bar, turn.ph, ab, kSitePReady))
                    return;
                tc_fence_after();
                const uint32_t d = tmem + kTmemO + wg * kHeadDim;
                umma_ts(d, scores, b, kIdesc, s >= 2 ? 1u : 0u);
                if ((pair ? s >> 1 : s) != last_at) {
#pragma unroll
                    for (int kk = 1; kk < kBlockN / 16; ++kk)
                        umma_ts(d, scores + 8 * kk, b + 128 * kk, kIdesc, 1u);
                } else {
                    for (int kk = 1; kk < kk_last; ++kk)
                        umma_ts(d, scores + 8 * kk, b + 128 * kk, kIdesc, 1u);
                }
                umma_commit(freed + 8 * buf.slot);
                if (s >= steps - 2)  // the warpgroup's last step of the task
                    umma_commit(smem_u32(&sm.o_final[wg]));
            } else {
                constexpr uint32_t kIdesc = idesc_bf16_f32(kBlockM, kBlockN, false);
                if (!wait_bar(freed + 8 * buf.slot, buf.ph ^ 1u, ab, kSiteODone))
                    return;
                tc_fence_after();
                const uint64_t a = q0 + (2 * qb + (pair ? wg : 0u)) * kTileDescStep;
#pragma unroll
                for (int kk = 0; kk < kHeadDim / 16; ++kk)
                    umma_ss(scores, a + 2 * kk, b + 2 * kk, kIdesc, kk > 0 ? 1u : 0u);
                umma_commit(bar);
            }
            if (last_reader) {
                commit_release(empty + 8 * ring.slot);
                ring.next();
            }
            buf.next();
            turn.next();
            const Turn<kScoreBufs> x = turn;
            turn = other;
            other = x;
        }
        if (steps & 1) {  // the next task starts with warpgroup 0 again
            const Turn<kScoreBufs> x = turn;
            turn = other;
            other = x;
        }
        if (!kIsPV)
            commit_release(smem_u32(&sm.q_empty[qb]));
        pass_task(sm, it);
    }
}

template <bool kIsPV>
__device__ __forceinline__ void run_issuer(CachedSmem &sm, uint32_t tmem)
{
    if (elect_one()) {
        issue_loop<kIsPV>(sm, tmem);
        // Every UMMA issued must complete before TMEM is released.
        umma_commit(smem_u32(&sm.drain[kIsPV]));
        wait_drain(smem_u32(&sm.drain[kIsPV]), 0);
    }
    __syncwarp();
}

// The results of a warp's 32 rows: O (columns of tO, and of tO1 for a merged
// single tile, weighted w0 and w1) with the row's l and m.  Every thread owns a
// row's l and m, but stores 16-byte pieces of rows in the layout of
// tmem_ld16x256 (a thread that stored its own row touched 32 lines with every
// store: 3300 clocks a tile instead of 2300 with one frame over 32 cached).
__device__ __forceinline__ void finish_cached_rows(const CachedParams &p, uint32_t tO, uint32_t tO1, bool merged,
                                                   float w0, float w1, const Task &t, int row, int h, bool row_ok,
                                                   float l, float m)
{
    const int lane = threadIdx.x & 31, q = lane & 3;
    const bool split = t.slot >= 0;
    const int64_t id = static_cast<int64_t>(row) * p.H + h;
    const int64_t part = static_cast<int64_t>(t.slot) * p.part_rows + (row - t.row0) * p.group + h - t.hk * p.group;
    const bool go = row_ok && VGGT_IN_RANGE(row >= 0 && row < p.n_rows && h < p.H &&
                                                (row - t.row0 + 1) * p.group <= (split ? p.part_rows : 256),
                                            kCheckAttnRow);
    const float f = split ? 1.f : (l == 0.f ? 0.f : 1.f / l);
    const float f0 = merged ? w0 * f : f, f1 = w1 * f;
    const int64_t mine = go ? (split ? part : id) : -1;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        const uint32_t lanes = static_cast<uint32_t>(16 * half) << 16;
        uint32_t o[32];
        float v[32];  // [8 channels][row r0, row r0 + 8][2]
        tmem_ld16x256(tO + lanes, o);
        tmem_ld_wait();
        reg_fence(o);
        const int r0 = 16 * half + (lane >> 2);
        int64_t to[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float x = __shfl_sync(0xffffffffu, f0, r0 + 8 * e);
            to[e] = __shfl_sync(0xffffffffu, mine, r0 + 8 * e);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[4 * i + 2 * e] = __uint_as_float(o[4 * i + 2 * e]) * x;
                v[4 * i + 2 * e + 1] = __uint_as_float(o[4 * i + 2 * e + 1]) * x;
            }
        }
        if (merged) {
            tmem_ld16x256(tO1 + lanes, o);
            tmem_ld_wait();
            reg_fence(o);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x = __shfl_sync(0xffffffffu, f1, r0 + 8 * e);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[4 * i + 2 * e] = fmaf(__uint_as_float(o[4 * i + 2 * e]), x, v[4 * i + 2 * e]);
                    v[4 * i + 2 * e + 1] = fmaf(__uint_as_float(o[4 * i + 2 * e + 1]), x, v[4 * i + 2 * e + 1]);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (split) {
                // Pairs of threads: the even one gets four channels of group i, the odd one of group i + 1.
                float4 *dst = reinterpret_cast<float4 *>(p.part_o + (to[e] < 0 ? 0 : to[e]) * kHeadDim);
                const bool odd = q & 1;
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float a = v[4 * i + 2 * e], b = v[4 * i + 2 * e + 1];
                    const float c = v[4 * i + 4 + 2 * e], d = v[4 * i + 4 + 2 * e + 1];
                    const float x = __shfl_xor_sync(0xffffffffu, odd ? a : c, 1);
                    const float y = __shfl_xor_sync(0xffffffffu, odd ? b : d, 1);
                    if (to[e] >= 0)
                        dst[2 * (i + odd) + (q >> 1)] = odd ? make_float4(x, y, c, d) : make_float4(a, b, x, y);
                }
            } else {
                // Four threads: thread q gets the eight channels of group q, then of 4 + q.
                uint4 *dst = reinterpret_cast<uint4 *>(p.o + (to[e] < 0 ? 0 : to[e]) * kHeadDim);
#pragma unroll
                for (int g = 0; g < 8; g += 4) {
                    uint32_t w[4], got[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = pack_bf16x2(v[4 * (g + i) + 2 * e], v[4 * (g + i) + 2 * e + 1]);
                    auto pick = [&](int i) { return i & 2 ? (i & 1 ? w[3] : w[2]) : (i & 1 ? w[1] : w[0]); };
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        got[k] = __shfl_xor_sync(0xffffffffu, pick(q ^ k), k);  // channels of thread q ^ k
                    auto place = [&](int i) {
                        const int k = i ^ q;
                        return k & 2 ? (k & 1 ? got[3] : got[2]) : (k & 1 ? got[1] : got[0]);
                    };
                    if (to[e] >= 0)
                        dst[g + q] = make_uint4(place(0), place(1), place(2), place(3));
                }
            }
        }
    }
    if (!go)
        return;
    if (split)
        p.part_ml[part] = make_float2(m, l);
    else if (p.lse)
        p.lse[id] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
}

// A task of at most 16 rows (a single token of grouped heads, the last tokens
// of a chunk) needs 1/8 of a 128-row tile's arithmetic and is bound by the
// bytes of K and V, so it does without TMEM: the even key tiles belong to warps
// 0-3 and the odd ones to warps 4-7, 32 keys of a tile to each warp.  A warp
// multiplies on registers (16 x 8 x 16), keeps its own softmax state and
// follows the K/V ring by itself; the eight states meet once, at the end of the
// task, in the Q buffer.  (With 16 keys of every tile to each of the eight
// warps, the chain of a tile, 1280 clocks, was as long as its bytes take.)  Fragment layouts are those of
// ldmatrix and mma.m16n8k16: row g = lane / 4 (and g + 8), columns 2 (lane % 4)
// and the next.
__device__ __forceinline__ bool run_few(CachedSmem &sm, const CachedParams &p, const Task &w, uint32_t it, uint32_t ring,
                                     uint32_t fews, int warp)
{
    volatile WaitCtl *ab = &sm.ctl;
    const int lane = threadIdx.x & 31, g = lane >> 2, c2 = 2 * (lane & 3);
    const uint32_t qb = it & 1u;
    uint8_t *qbuf = sm.q[qb][0];
    const float sl2 = p.scale_log2;
    const int rows = (w.row_end - w.row0) * p.group;
    const int mine = 32 * (warp & 3), half = warp >> 2;  // this warp's keys of a tile, its tiles mod 2
    int lim[2];  // keys that rows g, g + 8 see, counted from this warp's first key
    int low = 0x7fffffff;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = g + 8 * e;
        lim[e] = 0;
        if (r < rows) {
            lim[e] = key_limit(p, w.kv, w.pos0 + p.by_group.div(r)) - w.kt0 * kBlockN - mine;
            low = min(low, lim[e]);
        }
    }
    low = __reduce_min_sync(0xffffffffu, low);
    const int all = w.kv - w.kt0 * kBlockN - mine;  // keys that exist, counted in the same way

    if (!wait_bar_warp(smem_u32(&sm.task_passed[it % (2 * kTaskRing)]), (it / (2 * kTaskRing)) & 1u, ab,
                       kSiteTaskPassed) ||
        !wait_bar_warp(smem_u32(&sm.q_full[qb]), (it >> 1) & 1u, ab, kSiteQFull))
        return false;
    uint32_t q[4][4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
        const int r = lane & 15;
        ldmatrix_x4(smem_u32(qbuf) + r * 128 + (((2 * kk + (lane >> 4)) ^ (r & 7)) << 4), q[kk]);
    }
    __syncwarp();
    if (lane == 0)
        mbar_arrive(smem_u32(&sm.few_q));

    float o[8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[i][e] = 0.f;
    // Byte offsets within a tile; the swizzle XORs a 16-byte column with the row's low 3 bits.
    const uint32_t k_off = (mine + (lane & 7)) * 128, v_off = (mine + (lane & 15)) * 128;
    uint32_t k_at[2], v_at[4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        k_at[i] = smem_u32(sm.k[0]) + k_off + (((4 * i + (lane >> 3)) ^ (lane & 7)) << 4);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v_at[i] = smem_u32(sm.v[0]) + v_off + (((2 * i + (lane >> 4)) ^ (lane & 7)) << 4);
    for (int j = half; j < w.n; j += 2) {
        const uint32_t u = ring + static_cast<uint32_t>(j), st = u % kStages, ph = (u / kStages) & 1u;
        const int here = all - j * kBlockN;  // keys of this warp's 32 that exist
        if (!wait_bar_warp(smem_u32(&sm.k_full[st]), ph, ab, kSiteKFull))
            return false;
        float s[4][4] = {};
        if (here > 0) {
            uint32_t k[4][2][4];  // [8 keys][32 channels]: two 16-channel steps of B each
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int d = 0; d < 2; ++d)
                    ldmatrix_x4(k_at[d] + st * kTileBytes + i * 1024, k[i][d]);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_16816(s[i], q[kk], k[i][kk >> 1][2 * (kk & 1)], k[i][kk >> 1][2 * (kk & 1) + 1]);
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive_n(smem_u32(&sm.k_empty[st]), 2);  // for its counterpart of the other half too
        if (here > 0) {
            if (low < j * kBlockN + 32) {  // some row may not see all of the 32 keys
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (8 * i + c2 + (e & 1) >= lim[e >> 1] - j * kBlockN)
                            s[i][e] = -INFINITY;
            }
            float top[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[e] = fmax3(s[0][2 * e], s[0][2 * e + 1], s[1][2 * e]);
                top[e] = fmax3(top[e], s[1][2 * e + 1], s[2][2 * e]);
                top[e] = fmax3(top[e], s[2][2 * e + 1], s[3][2 * e]);
                // a row of no token has no say in when the offsets move
                top[e] = g + 8 * e < rows ? fmaxf(top[e], s[3][2 * e + 1]) * sl2 : -INFINITY;
            }
            // The offset moves when a logit passes it by kRescaleThreshold
            // (P <= 2^8), so most tiles need no maximum over the lanes.
            if (__any_sync(0xffffffffu, top[0] > m[0] + kRescaleThreshold || top[1] > m[1] + kRescaleThreshold)) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
                    top[e] = fmaxf(fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2)), m[e]);
                    const float f = m[e] == -INFINITY ? 0.f : ex2_approx(m[e] - top[e]);
                    m[e] = top[e];
                    l[e] *= f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        o[i][2 * e] *= f;
                        o[i][2 * e + 1] *= f;
                    }
                }
            }
            uint32_t pk[2][4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float base = m[e] == -INFINITY ? 0.f : m[e];
                float sum[2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = ex2_approx(fmaf(s[i][2 * e], sl2, -base));
                    const float b = ex2_approx(fmaf(s[i][2 * e + 1], sl2, -base));
                    sum[i & 1] = i < 2 ? a + b : sum[i & 1] + (a + b);
                    pk[i >> 1][2 * (i & 1) + e] = pack_bf16x2(a, b);
                }
                l[e] += sum[0] + sum[1];
            }
            if (!wait_bar_warp(smem_u32(&sm.v_full[st]), ph, ab, kSiteVFull))
                return false;
            uint32_t v[2][4][4];  // [16 keys][16 channels]
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    ldmatrix_x4_trans(v_at[i] + st * kTileBytes + h * 2048, v[h][i]);
            if (here < 32) {
                // whatever lies behind the last key must not meet P = 0
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = 16 * h + 8 * (e & 1) + c2;
                        const uint32_t keep = (key < here ? 0x0000ffffu : 0u) | (key + 1 < here ? 0xffff0000u : 0u);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[h][i][e] &= keep;
                    }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mma_16816(o[2 * i], pk[h], v[h][i][0], v[h][i][1]);
                    mma_16816(o[2 * i + 1], pk[h], v[h][i][2], v[h][i][3]);
                }
        } else if (!wait_bar_warp(smem_u32(&sm.v_full[st]), ph, ab, kSiteVFull)) {
            return false;
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive_n(smem_u32(&sm.v_empty[st]), 2);
    }

    // The states of the eight warps, over Q once every warp has read it:
    // [warp][row][64] floats, pairs of columns XORed with the row against bank conflicts.
    if (!wait_bar_warp(smem_u32(&sm.few_q), fews & 1u, ab, kSiteFewQ))
        return false;
    float2 *state = reinterpret_cast<float2 *>(qbuf) + warp * (kFewRows * 32);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        const int r = g + 8 * e;
        if ((lane & 3) == 0)
            sm.merge_ml[warp * kFewRows + r] = make_float2(m[e], l[e]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            state[r * 32 + ((4 * i + (lane & 3)) ^ (g << 2))] = make_float2(o[i][2 * e], o[i][2 * e + 1]);
    }
    __syncwarp();
    if (lane == 0)
        mbar_arrive(smem_u32(&sm.few_full[fews & 1u]));
    if (!wait_bar_warp(smem_u32(&sm.few_full[fews & 1u]), (fews >> 1) & 1u, ab, kSiteFewFull))
        return false;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = 2 * warp + e;
        if (r >= rows)
            break;
        float top = -INFINITY, sum = 0.f, a = 0.f, b = 0.f;
        float2 ml[kSoftmaxWarps];
#pragma unroll
        for (int x = 0; x < kSoftmaxWarps; ++x) {
            ml[x] = sm.merge_ml[x * kFewRows + r];
            top = fmaxf(top, ml[x].x);
        }
#pragma unroll
        for (int x = 0; x < kSoftmaxWarps; ++x) {
            const float f = ml[x].x == -INFINITY ? 0.f : ex2_approx(ml[x].x - top);
            const float2 v = reinterpret_cast<const float2 *>(qbuf)[(x * kFewRows + r) * 32 + (lane ^ ((r & 7) << 2))];
            sum = fmaf(f, ml[x].y, sum);
            a = fmaf(f, v.x, a);
            b = fmaf(f, v.y, b);
        }
        const int tok = p.by_group.div(r);
        const int64_t id = static_cast<int64_t>(w.row0 + tok) * p.H + w.hk * p.group + r - tok * p.group;
        if (!VGGT_IN_RANGE(w.row0 + tok < p.n_rows && (w.slot < 0 || r < p.part_rows), kCheckAttnRow))
            continue;
        if (w.slot >= 0) {
            const int64_t part = static_cast<int64_t>(w.slot) * p.part_rows + r;
            reinterpret_cast<float2 *>(p.part_o)[part * 32 + lane] = make_float2(a, b);
            if (lane == 0)
                p.part_ml[part] = make_float2(top, sum);
        } else {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            reinterpret_cast<uint32_t *>(p.o + id * kHeadDim)[lane] = pack_bf16x2(a * inv, b * inv);
            if (p.lse && lane == 0)
                p.lse[id] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994531f;
        }
    }
    // This warp's reads and writes come before the next Q tile is copied over them.
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0)
        mbar_arrive(smem_u32(&sm.q_empty[qb]));
    return true;
}

// wait_bar_warp for the step's own barrier, with one vote where the phase is complete.
__device__ __forceinline__ bool wait_step(uint32_t bar, uint32_t parity, volatile WaitCtl *ctl, uint32_t site)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
        return true;
    const bool ok = wait_slow(bar, parity, ctl, site);
    __syncwarp();
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void run_cached_softmax(CachedSmem &sm, uint32_t tmem, const CachedParams &p, int wg)
{
    volatile WaitCtl *ab = &sm.ctl;
    const int t = static_cast<int>(threadIdx.x) - kBlockM * (wg + 1);  // row within the tile
    const uint32_t lane_off = static_cast<uint32_t>((t >> 5) * 32) << 16;
    const uint32_t tO = tmem + kTmemO + static_cast<uint32_t>(wg * kHeadDim) + lane_off;
    const uint32_t bar_s = smem_u32(&sm.s_full[wg][0]), bar_p = smem_u32(&sm.p_ready[wg][0]);
    const uint32_t bar_of = smem_u32(&sm.o_final[wg]);
    const float sl2 = p.scale_log2;
    const uint64_t sl2_2 = f2_pack(sl2, sl2);
    const uint64_t magic2 = f2_pack(kRoundMagic, kRoundMagic);
    const uint64_t neg_magic2 = f2_pack(-kRoundMagic, -kRoundMagic);
    const uint64_t neg_one2 = f2_pack(-1.f, -1.f);
    const uint64_t c0_2 = f2_pack(kExp2C0, kExp2C0), c1_2 = f2_pack(kExp2C1, kExp2C1);
    const uint64_t c2_2 = f2_pack(kExp2C2, kExp2C2), c3_2 = f2_pack(kExp2C3, kExp2C3);
    const int tok = p.by_group.div(t), tile_head = t - tok * p.group;
    uint32_t k0 = 0;         // steps of the CTA before the task, mod 6 (3 score buffers, 2 phases)
    uint32_t ring = 0;       // key tiles before the task
    Turn<3> turn{0, 0};      // barriers of this warpgroup's step
    uint32_t finals = 0;     // tasks in which it had a step
    uint32_t fews = 0;       // tasks of few rows so far
    uint32_t merges = 0;     // single-tile tasks that both warpgroups worked on
    bool merge_open = false; // warpgroup 1: its last merge has not been read yet

    for (int it = 0;; ++it) {
        const bool got = wait_task(sm, it);
        __syncwarp();
        if (!__all_sync(0xffffffffu, got))
            return;
        const Task w = sm.task[it % kTaskRing];
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            release_task(sm, it);
        if (w.n == 0)
            return;
        if (w.kind == kTaskFew) {
            if (!run_few(sm, p, w, static_cast<uint32_t>(it), ring, fews, wg * 4 + (t >> 5)))
                return;
            ++fews;
            ring += static_cast<uint32_t>(w.n);
            continue;
        }
        const int tile_tok = (w.kind == kTaskPair && wg ? p.tile_tokens : 0) + tok;  // token within the task
        const int row = w.row0 + tile_tok;
        const bool row_ok = tok < p.tile_tokens && row < w.row_end;
        const int head = w.hk * p.group + tile_head;
        const int steps = w.kind == kTaskPair ? w.n : (w.n + 1 - wg) >> 1;  // of this warpgroup
        // keys this row sees, counted from the task's first key
        const int lim = row_ok ? key_limit(p, w.kv, w.pos0 + tile_tok) - w.kt0 * kBlockN : 0;
        const bool warp_ok = __any_sync(0xffffffffu, row_ok);
        const int warp_lim = __reduce_min_sync(0xffffffffu, row_ok ? lim : 0x7fffffff);
        float m = -INFINITY, l = 0.f;

        uint32_t k = k0 + static_cast<uint32_t>(wg);  // the step, mod 6
        for (int x = 0; x < steps; ++x) {
            const int j = w.kind == kTaskPair ? x : 2 * x + wg;
            const int tile = j + w.rot < w.n ? j + w.rot : j + w.rot - w.n;  // key tile within the task
            if (k >= 6)
                k -= 6;
            const uint32_t buf = k >= 3 ? k - 3 : k;
            const uint32_t tS = tmem + buf * kBlockN + lane_off;
            if (!wait_step(bar_s + 8 * turn.slot, turn.ph, ab, kSiteSFull))
                return;
            if (tile == w.n - 1 && (w.vlast & 15) != 0 && (w.kind != kTaskPair || wg == 0)) {
                // V rows behind the last key, up to the end of its group of 16
                const uint32_t u = ring + static_cast<uint32_t>(j), st = u % kStages;
                if (!wait_bar_warp(smem_u32(&sm.v_full[st]), (u / kStages) & 1, ab, kSiteVFull))
                    return;
                const int r = w.vlast + (t >> 3);
                if (r < ((w.vlast + 15) & ~15))
                    reinterpret_cast<uint4 *>(sm.v[st] + r * kHeadDim * 2)[t & 7] = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
            }
            if (warp_ok) {
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tmem_ld32(tS + 32 * i, s[i]);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    reg_fence(s[i]);
                const int valid = lim - tile * kBlockN;
                if (warp_lim < (tile + 1) * kBlockN) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (32 * i + e >= valid)
                                s[i][e] = __float_as_uint(-INFINITY);
                }
                // Row max of the tile, in log2 units.
                auto tile_max = [&]() -> float {
                    float mx[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        mx[i] = fmax3(__uint_as_float(s[i][0]), __uint_as_float(s[i][1]), __uint_as_float(s[i][2]));
#pragma unroll
                        for (int e = 3; e < 31; e += 2)
                            mx[i] = fmax3(mx[i], __uint_as_float(s[i][e]), __uint_as_float(s[i][e + 1]));
                        mx[i] = fmaxf(mx[i], __uint_as_float(s[i][31]));
                    }
                    return fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * sl2;
                };
                // P = 2^(s*scale*log2e - m) as bf16 pairs over the first 64
                // columns of the score buffer; returns the fp32 sum of P
                // before it is rounded (see attn_fwd_kernel for the split of
                // the exponentials between the MUFU unit and a polynomial).
                auto exp_tile = [&]() -> float {
                    const float base = fmaxf(m, -1e30f);  // a row that sees nothing: P = 0
                    const uint64_t neg_m2 = f2_pack(-base, -base);
                    uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const uint64_t x2 = f2_fma(
                                f2_pack(__uint_as_float(s[i][2 * e]), __uint_as_float(s[i][2 * e + 1])), sl2_2, neg_m2);
                            float a, b;
                            f2_unpack(x2, a, b);
                            if (e < kCachedPolyPairs) {
                                const uint64_t xc = f2_pack(fminf(fmaxf(a, kExp2MinArg), kExp2MaxArg),
                                                            fminf(fmaxf(b, kExp2MinArg), kExp2MaxArg));
                                const uint64_t y = f2_add(xc, magic2);
                                const uint64_t jj = f2_add(y, neg_magic2);
                                const uint64_t f = f2_fma(jj, neg_one2, xc);
                                uint64_t q = f2_fma(c3_2, f, c2_2);
                                q = f2_fma(q, f, c1_2);
                                q = f2_fma(q, f, c0_2);
                                float qa, qb, ya, yb;
                                f2_unpack(q, qa, qb);
                                f2_unpack(y, ya, yb);
                                a = __uint_as_float(__float_as_uint(ya) * 8388608u + __float_as_uint(qa));
                                b = __uint_as_float(__float_as_uint(yb) * 8388608u + __float_as_uint(qb));
                            } else {
                                a = ex2_approx(a);
                                b = ex2_approx(b);
                            }
                            ls[e & 3] = f2_add(ls[e & 3], f2_pack(a, b));
                            pk[e] = pack_bf16x2(a, b);
                        }
                        tmem_st16(tS + 16 * i, pk);
                    }
                    const uint64_t t2 = f2_add(f2_add(ls[0], ls[1]), f2_add(ls[2], ls[3]));
                    float ta, tb;
                    f2_unpack(t2, ta, tb);
                    return ta + tb;
                };
                // Lazy offset, as in attn_fwd_kernel: the first tile sets m,
                // and a later tile whose row sum passes kTileSumLimit takes
                // the exact path.
                if (x == 0)
                    m = tile_max();
                float tsum = exp_tile();
                // Rows of no token of the task have no say: whether a row below
                // the limit moves its offset too would hang on their contents.
                if (x > 0 && __any_sync(0xffffffffu, row_ok && !(tsum <= kTileSumLimit))) {
                    const float cand = tile_max();
                    const bool need = row_ok && cand > m + kRescaleThreshold;
                    if (__any_sync(0xffffffffu, need)) {
                        // this warpgroup's last PV: step k - 2
                        const uint32_t before = k >= 2 ? k - 2 : k + 4;
                        if (!wait_bar_warp(smem_u32(&sm.buf_free[before >= 3 ? before - 3 : before]), before >= 3,
                                           ab, kSiteODone))
                            return;
                        tc_fence_after();
                        const float f = need ? ex2_approx(m - cand) : 1.f;
#pragma unroll 1
                        for (int quarter = 0; quarter < 4; ++quarter) {
                            uint32_t o[16];
                            tmem_ld16(tO + 16 * quarter, o);
                            tmem_ld_wait();
                            reg_fence(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(tO + 16 * quarter, o);
                        }
                        tmem_st_wait();
                        if (need) {
                            l *= f;
                            m = cand;
                        }
                    }
                    tmem_st_wait();  // the first pass's P stores land before they are overwritten
                    tsum = exp_tile();
                }
                l += tsum;
                tmem_st_wait();
            }
            if (x == 0 && merge_open) {
                // warpgroup 0 still reads this warpgroup's O of an earlier task
                if (!wait_bar_warp(smem_u32(&sm.merge_free), (merges - 1) & 1, ab, kSiteMergeFree))
                    return;
                merge_open = false;
            }
            tc_fence_before();
            __syncwarp();
            if ((threadIdx.x & 31) == 0)
                mbar_arrive(bar_p + 8 * turn.slot);
            turn.next();
            k += 2;
        }
        k0 = (k0 + static_cast<uint32_t>(w.kind == kTaskPair ? 2 * w.n : w.n)) % 6;
        ring += static_cast<uint32_t>(w.n);

        if (steps == 0)
            continue;  // a single tile of one step: warpgroup 0's alone
        if (!wait_bar_warp(bar_of, finals & 1, ab, kSiteOFinal))
            return;
        ++finals;
        tc_fence_after();
        const bool merged = w.kind == kTaskSingle && w.n > 1;
        if (merged && wg == 1) {
            if (merge_open && !wait_bar_warp(smem_u32(&sm.merge_free), (merges - 1) & 1, ab, kSiteMergeFree))
                return;
            sm.merge_ml[t] = make_float2(m, l);
            tc_fence_before();
            __syncwarp();
            if ((threadIdx.x & 31) == 0)
                mbar_arrive(smem_u32(&sm.merge_ready));
            ++merges;
            merge_open = true;
            continue;
        }
        float w0 = 1.f, w1 = 0.f;
        if (merged) {
            if (!wait_bar_warp(smem_u32(&sm.merge_ready), merges & 1, ab, kSiteMergeReady))
                return;
            ++merges;
            tc_fence_after();
            const float2 ml = sm.merge_ml[t];
            // A part without keys has l = 0 and m = -inf: it gets weight 0.  NaN passes through.
            const float top = fmaxf(m, ml.x);
            w0 = m == -INFINITY ? 0.f : ex2_approx(m - top);
            w1 = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - top);
            l = l * w0 + ml.y * w1;
            m = top;
        }
        if (m == -INFINITY)
            l = 0.f;  // the row sees no key of the task; masked columns may have left 2^-125 each
        if (warp_ok)
            finish_cached_rows(p, tO, tO + kHeadDim, merged, w0, w1, w, row, head, row_ok, l, m);
        tc_fence_before();
        if (merged) {
            __syncwarp();
            if ((threadIdx.x & 31) == 0)
                mbar_arrive(smem_u32(&sm.merge_free));
        }
    }
}

__global__ void __launch_bounds__(kAttnThreads, 1)
    cached_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const CachedParams p)
{
    extern __shared__ uint8_t smem_raw[];
    CachedSmem &sm = *reinterpret_cast<CachedSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                     ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm.q_full[i]), 1);
            mbar_init(smem_u32(&sm.q_empty[i]), kSoftmaxWarps);
            for (int c = 0; c < 3; ++c) {
                mbar_init(smem_u32(&sm.s_full[i][c]), 1);
                mbar_init(smem_u32(&sm.p_ready[i][c]), 4);
            }
            mbar_init(smem_u32(&sm.drain[i]), 1);
            mbar_init(smem_u32(&sm.o_final[i]), 1);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&sm.k_full[i]), 1);
            mbar_init(smem_u32(&sm.k_empty[i]), kSoftmaxWarps);
            mbar_init(smem_u32(&sm.v_full[i]), 1);
            mbar_init(smem_u32(&sm.v_empty[i]), kSoftmaxWarps);
        }
        for (int i = 0; i < kTaskRing; ++i) {
            mbar_init(smem_u32(&sm.task_full[i]), 1);
            mbar_init(smem_u32(&sm.task_empty[i]), 11);  // V producer, issuers, eight softmax warps
        }
        mbar_init(smem_u32(&sm.merge_ready), 4);
        mbar_init(smem_u32(&sm.merge_free), 4);
        mbar_init(smem_u32(&sm.few_q), kSoftmaxWarps);
        for (int i = 0; i < 2; ++i)
            mbar_init(smem_u32(&sm.few_full[i]), kSoftmaxWarps);
        for (int i = 0; i < 2 * kTaskRing; ++i)
            mbar_init(smem_u32(&sm.task_passed[i]), 2);
        for (int i = 0; i < kScoreBufs; ++i)
            mbar_init(smem_u32(&sm.buf_free[i]), 1);
        sm.ctl.abort = 0;
        sm.ctl.limit_ns = p.wait_limit_ns;
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&sm.tmem_base), kTmemCols);
        tmem_relinquish();
    }
    // Until here nothing that an earlier launch reads or writes was touched.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0 && p.join)
        p.join[blockIdx.x] = Join{0, 0, 0, 0};  // what stays if a wait runs out
    plan_work(sm, p);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    // The joining launch may be set up; it waits for this one before it reads.
    // (Not before the TMEM allocation: what comes early may want TMEM too.)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // 168 registers/thread at launch; 128 x (72 + 216 + 216) = 384 x 168.
    if (warp < 4) {
        setmaxnreg_dec<kRegsControl>();
        // The order of the roles is that of their code: the loops that run
        // together (issuers, softmax) stand side by side.
        if (warp == 0)
            run_k_producer(sm, &tmQ, &tmK, p);
        else if (warp == 3)
            run_v_producer(sm, &tmV, p);
        else if (warp == 2)
            run_issuer<false>(sm, tmem);
        else
            run_issuer<true>(sm, tmem);
    } else {
        setmaxnreg_inc<kRegsSoftmax>();
        run_cached_softmax(sm, tmem, p, (warp >> 2) - 1);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the parts of a unit that was cut, O = sum_c 2^{m_c - M} O_c / sum_c
// 2^{m_c - M} l_c with M = max m_c, in the order of the parts.  Blocks x take
// the unit that CTA x began; 16 threads a row, four channels each.  Bound by
// latency (the launch waits for the attention's last CTA, then for the record,
// the weights and the values) and by the parts' bytes, 264 per row and part.
// The first kAhead values are on their way while the weights are found: with
// few rows a unit can have many parts, with many rows the registers count.
constexpr int kJoinRows = 16;  // rows of a block
template <int kAhead>
__global__ void __launch_bounds__(256) cached_combine_kernel(const CachedParams p)
{
    const int lane = threadIdx.x & 15, r = static_cast<int>(blockIdx.y) * kJoinRows + (threadIdx.x >> 4);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Join u = p.join[blockIdx.x];
    if (static_cast<int>(blockIdx.y) * kJoinRows >= u.rows || u.parts == 0)
        return;
    const bool live = r < u.rows;
    // Row r of part c: slot 2 x + 1 for the first, 2 (x + c) for the others.
    const int64_t step = 2 * static_cast<int64_t>(p.part_rows);
    const int64_t base = step * blockIdx.x + (live ? r : 0);
    auto row = [&](int c) { return base + (c == 0 ? p.part_rows : c * step); };
    const float4 *values = reinterpret_cast<const float4 *>(p.part_o);
    float4 v[kAhead];
#pragma unroll
    for (int c = 0; c < kAhead; ++c)
        if (c < u.parts)
            v[c] = values[row(c) * 16 + lane];
    float2 ml = lane < u.parts ? p.part_ml[row(lane)] : make_float2(-INFINITY, 0.f);
    float top = ml.x;
    for (int c = lane + 16; c < u.parts; c += 16)
        top = fmaxf(top, p.part_ml[row(c)].x);
#pragma unroll
    for (int d = 8; d > 0; d >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c0 = 0; c0 < u.parts; c0 += 16) {
        if (c0 > 0)
            ml = c0 + lane < u.parts ? p.part_ml[row(c0 + lane)] : make_float2(-INFINITY, 0.f);
        const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - top);
        sum = fmaf(f, ml.y, sum);
        const int n = min(16, u.parts - c0);
        auto add = [&](float4 x, int c) {
            const float w = __shfl_sync(0xffffffffu, f, c, 16);
            o[0] = fmaf(w, x.x, o[0]);
            o[1] = fmaf(w, x.y, o[1]);
            o[2] = fmaf(w, x.z, o[2]);
            o[3] = fmaf(w, x.w, o[3]);
        };
        int c = 0;
        if (c0 == 0) {
#pragma unroll
            for (; c < kAhead; ++c)
                if (c < n)
                    add(v[c], c);
        }
#pragma unroll 4
        for (; c < n; ++c)
            add(values[row(c0 + c) * 16 + lane], c);
    }
#pragma unroll
    for (int d = 8; d > 0; d >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (!live)
        return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int tok = p.by_group.div(r);
    const int64_t id = static_cast<int64_t>(u.row0 + tok) * p.H + u.hk * p.group + r - tok * p.group;
    reinterpret_cast<uint2 *>(p.o + id * kHeadDim)[lane] =
        make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    if (p.lse && lane == 0)
        p.lse[id] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994531f;
}

} // namespace vggt
