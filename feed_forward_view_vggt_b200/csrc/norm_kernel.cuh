// norm_kernel.cuh -- the seam between two blocks of the trunk, one pass:
//   x' = x + scale * gate * N_post(y),   h = N_pre(x')
// with N a LayerNorm (centre) or an RMSNorm, both optional, scale the
// per-channel layer scale and gate one row of factors per group of tokens.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "device_error.cuh"
#include "ptx.cuh"

namespace vggt {

constexpr int kNormMaxCols = 8192;

struct NormParams {
    int64_t n_rows;
    int n_cols, rows_per_gate;
    int layer, post_norm;  // layer: LayerNorm (else RMSNorm)
    float eps, inv_cols;
    int64_t x_stride, y_stride, out_stride, h_stride, gate_stride;  // elements
    const void *x;
    const __nv_bfloat16 *y, *gate;
    const float *post_w, *post_b, *scale, *w, *b;
    void *x_out;
    __nv_bfloat16 *h;
};

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8])
{
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16lo_to_f32(w[i]);
        v[2 * i + 1] = bf16hi_to_f32(w[i]);
    }
}

__device__ __forceinline__ void load8(const float *p, float (&v)[8])
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8])
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ void store8(float *p, const float (&v)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Sum over the warps that share a row, at most kWarps: the block's if there is
// more than one.  Every thread gets it.  `part` is used once per row.
template <int kWarps>
__device__ __forceinline__ float row_sum(float v, float *part)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    if (kWarps == 1)
        return v;
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    const int warps = static_cast<int>(blockDim.x >> 5);
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i)
        t += i < warps ? part[i] : 0.f;
    return t;
}

// Factors (or terms) of the thread's channels c .. c + 7: read where they are
// used, or kAhead, when the row's own values are.  None: `t` stays as it is.
template <typename T, bool kAhead>
struct Channels {
    const T *p;
    float v[8];

    __device__ __forceinline__ Channels(const T *ptr, int c, bool in) : p(ptr ? ptr + c : nullptr)
    {
        if (kAhead && p && in)
            load8(p, v);
    }
    __device__ __forceinline__ void scale(float (&t)[8])
    {
        if (p) {
            if (!kAhead)
                load8(p, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                t[e] *= v[e];
        }
    }
    __device__ __forceinline__ void add(float (&t)[8])
    {
        if (p) {
            if (!kAhead)
                load8(p, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                t[e] += v[e];
        }
    }
};

// t = N(t) over the row; `in`: the thread has channels of it (else t is 0).
// The variance is taken about the mean in a second pass over registers: the
// values are there already, and E[t^2] - E[t]^2 would lose what a large
// common offset leaves.
template <int kWarps, bool kAhead>
__device__ __forceinline__ void normalise(const NormParams &p, float (&t)[8], bool in, Channels<float, kAhead> &w,
                                          Channels<float, kAhead> &b, float (*part)[kWarps])
{
    float mean = 0.f;
    if (p.layer) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s += t[e];
        mean = row_sum<kWarps>(s, part[0]) * p.inv_cols;
    }
    float q = 0.f;
    if (in) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            t[e] -= mean;
            q = fmaf(t[e], t[e], q);
        }
    }
    const float r = rsqrtf(fmaf(row_sum<kWarps>(q, part[1]), p.inv_cols, p.eps));
    if (in) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            t[e] *= r;
        w.scale(t);
        b.add(t);
    }
}

// One warp per 256 channels of a row, 8 channels per thread, the row in
// registers; kWarps = 1: four rows per block, else the block is a row's.  Many
// rows are bound by HBM (x, y, x' and h once each; 137400 x 1024, fp32 x: 272
// us alone, 6.2 TB/s, and 282 to 301 in a row; 32 channels per thread and a warp
// per row were 1% slower).  Few
// rows (kAhead) are bound by the latency of a trip to memory and of the sums:
// every load is issued at the start (17 x 1024: 6 us instead of 12).
template <typename X, int kWarps, bool kAhead>
__global__ void __launch_bounds__(kWarps > 4 ? 32 * kWarps : 128) norm_residual_kernel(const NormParams p)
{
    constexpr int kRows = kWarps == 1 ? 4 : 1;  // rows per block: those of one warp each share one
    // x beside y at the start, if it is 16 bytes (60000 x 2048: 172 us instead of
    // 191); 32 more bytes per thread cost more than they hide (358 instead of 337).
    constexpr bool kXAhead = kAhead || sizeof(X) == 2;
    __shared__ float part_s[4][kWarps];
    const int c = 8 * (kWarps == 1 ? threadIdx.x & 31 : threadIdx.x);
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + (kWarps == 1 ? threadIdx.x >> 5 : 0);
    if (row >= p.n_rows)
        return;
    const bool in = c < p.n_cols;
    const X *x = static_cast<const X *>(p.x) + row * p.x_stride + c;
    float t[8] = {}, xv[8];
    if (p.y && in)
        load8(p.y + row * p.y_stride + c, t);
    if ((kXAhead || !p.y) && in)
        load8(x, xv);
    Channels<float, kAhead> post_w(p.post_w, c, in), post_b(p.post_b, c, in), scale(p.scale, c, in);
    Channels<__nv_bfloat16, kAhead> gate(p.gate ? p.gate + row / p.rows_per_gate * p.gate_stride : nullptr, c, in);
    Channels<float, kAhead> w(p.w, c, in), b(p.b, c, in);
    if (p.y) {
        if (p.post_norm)
            normalise<kWarps, kAhead>(p, t, in, post_w, post_b, part_s);
        if (in) {
            if (!kXAhead)
                load8(x, xv);
            scale.scale(t);
            gate.scale(t);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                t[e] += xv[e];
            if (p.x_out)
                store8(static_cast<X *>(p.x_out) + row * p.out_stride + c, t);
        }
    } else if (in) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            t[e] = xv[e];
    }
    if (!p.h)
        return;
    normalise<kWarps, kAhead>(p, t, in, w, b, part_s + 2);
    if (in)
        store8(p.h + row * p.h_stride + c, t);
}

} // namespace vggt
