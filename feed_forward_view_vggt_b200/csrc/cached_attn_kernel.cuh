// cached_attn_kernel.cuh -- attention of a step's new rows over a paged K/V
// cache: O_i = sum_j e^{s q_i.k_j} v_j / sum_j e^{s q_i.k_j} over the keys
// j < lim_i of i's own sequence, lim_i = min(kv, (floor(pos_i / u) + 1) u).
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "attn_kernel.cuh"
#include "cache_kernels.cuh"
#include "device_error.cuh"

namespace vggt {

struct CachedParams {
    int n_seqs, n_rows, H, Hkv, page_size, n_pages, max_pages, unit;
    float scale_log2;
    int64_t q_row_stride, q_head_stride;
    int64_t page_stride, head_stride, token_stride;
    const __nv_bfloat16 *q, *k_pages, *v_pages;
    const int32_t *table, *cu_rows, *kv_lens;
    __nv_bfloat16 *o;
    float *lse;
};

// One warp per (row, head): 32 keys at a time, a key's logit per lane, two
// output channels per lane, one pass with the running maximum and sum.
__global__ void __launch_bounds__(128) cached_attn_kernel(const CachedParams p)
{
    const int lane = threadIdx.x & 31;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (id >= static_cast<int64_t>(p.n_rows) * p.H)
        return;
    const int row = static_cast<int>(id / p.H), h = static_cast<int>(id % p.H), hk = h / (p.H / p.Hkv);
    int lo = 0, hi = p.n_seqs;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_rows[mid + 1] > row)
            hi = mid;
        else
            lo = mid + 1;
    }
    const int b = lo;
    if (b >= p.n_seqs)
        return;
    const int kv = max(0, min(p.kv_lens[b], p.max_pages * p.page_size));
    const int pos = kv - p.cu_rows[b + 1] + row;
    int lim = kv;
    if (p.unit > 0)
        lim = pos < 0 ? 0
                      : static_cast<int>(min(static_cast<int64_t>(kv),
                                             (static_cast<int64_t>(pos / p.unit) + 1) * p.unit));
    const __nv_bfloat16 *q = p.q + row * p.q_row_stride + h * p.q_head_stride;
    float qv[64];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint4 x = reinterpret_cast<const uint4 *>(q)[i];
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            qv[8 * i + 2 * e] = bf16lo_to_f32(xs[e]) * p.scale_log2;
            qv[8 * i + 2 * e + 1] = bf16hi_to_f32(xs[e]) * p.scale_log2;
        }
    }
    float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
    for (int j0 = 0; j0 < lim; j0 += 32) {
        const int j = j0 + lane;
        float s = -INFINITY;
        int64_t base = -1;
        if (j < lim) {
            const int page = p.table[static_cast<int64_t>(b) * p.max_pages + j / p.page_size];
            if (page < 0 || page >= p.n_pages) {
                record_bounds_failure(kCheckCachePage);
            } else {
                base = page * p.page_stride + hk * p.head_stride + (j % p.page_size) * p.token_stride;
                s = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 x = reinterpret_cast<const uint4 *>(p.k_pages + base)[i];
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s = fmaf(qv[8 * i + 2 * e], bf16lo_to_f32(xs[e]), s);
                        s = fmaf(qv[8 * i + 2 * e + 1], bf16hi_to_f32(xs[e]), s);
                    }
                }
            }
        }
        float mx = s;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m - mu), w = exp2f(s - mu);
        float sum = w;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l = fmaf(l, f, sum);
        o0 *= f;
        o1 *= f;
        m = mn;
        for (int i = 0; i < 32 && j0 + i < lim; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, i);
            const int64_t bi = __shfl_sync(0xffffffffu, base, i);
            if (bi >= 0) {
                const uint32_t v = reinterpret_cast<const uint32_t *>(p.v_pages + bi)[lane];
                o0 = fmaf(wi, bf16lo_to_f32(v), o0);
                o1 = fmaf(wi, bf16hi_to_f32(v), o1);
            }
        }
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    reinterpret_cast<uint32_t *>(p.o + id * kHeadDim)[lane] = pack_bf16x2(o0 * inv, o1 * inv);
    if (p.lse && lane == 0)
        p.lse[id] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : (l == 0.f ? -INFINITY : l);
}

} // namespace vggt
