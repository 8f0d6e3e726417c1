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

// Sum over the kWarps warps that share a row; every thread gets it.
template <int kWarps>
__device__ __forceinline__ float row_sum(float v, float *part)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    if (kWarps == 1)
        return v;
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i)
        t += part[i];
    return t;
}

// t = N(t) over the row, kVec vectors of 8 channels per thread.  The
// variance is taken about the mean in a second pass over registers: the
// values are there already, and E[t^2] - E[t]^2 would lose what a large
// common offset leaves.
template <int kVec, int kWarps>
__device__ __forceinline__ void normalise(const NormParams &p, float (&t)[kVec][8], int lane, const float *w,
                                          const float *b, float *part)
{
    float mean = 0.f;
    if (p.layer) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s += t[i][e];
        mean = row_sum<kWarps>(s, part) * p.inv_cols;
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        if (8 * (lane + i * kWarps * 32) < p.n_cols) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                t[i][e] -= mean;
                q = fmaf(t[i][e], t[i][e], q);
            }
        }
    }
    const float r = rsqrtf(fmaf(row_sum<kWarps>(q, part), p.inv_cols, p.eps));
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int c = 8 * (lane + i * kWarps * 32);
        if (c < p.n_cols) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                t[i][e] *= r;
            if (w) {
                load8(w + c, f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    t[i][e] *= f[e];
            }
            if (b) {
                load8(b + c, f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    t[i][e] += f[e];
            }
        }
    }
}

// kWarps warps per row, the row in registers; one warp per row holds up to
// 1024 channels.  Bound by HBM: x, y, x' and h once each.
template <typename X, int kVec, int kWarps>
__global__ void __launch_bounds__(kWarps > 4 ? 32 * kWarps : 128) norm_residual_kernel(const NormParams p)
{
    constexpr int kRows = kWarps > 4 ? 1 : 4 / kWarps;  // rows per block
    __shared__ float part_s[kRows][kWarps];
    const int lane = threadIdx.x % (32 * kWarps);
    static_assert(kWarps == 1 || kRows == 1, "rows that share a block are one warp each");
    float *part = part_s[threadIdx.x / (32 * kWarps)];
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / (32 * kWarps);
    if (row >= p.n_rows)
        return;
    const X *x = static_cast<const X *>(p.x) + row * p.x_stride;
    float t[kVec][8];
    if (p.y) {
        const __nv_bfloat16 *y = p.y + row * p.y_stride;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int c = 8 * (lane + i * kWarps * 32);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                t[i][e] = 0.f;
            if (c < p.n_cols)
                load8(y + c, t[i]);
        }
        if (p.post_norm)
            normalise<kVec, kWarps>(p, t, lane, p.post_w, p.post_b, part);
        const __nv_bfloat16 *gate = p.gate ? p.gate + row / p.rows_per_gate * p.gate_stride : nullptr;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int c = 8 * (lane + i * kWarps * 32);
            if (c < p.n_cols) {
                float f[8];
                if (p.scale) {
                    load8(p.scale + c, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        t[i][e] *= f[e];
                }
                if (gate) {
                    load8(gate + c, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        t[i][e] *= f[e];
                }
                load8(x + c, f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    t[i][e] += f[e];
                if (p.x_out)
                    store8(static_cast<X *>(p.x_out) + row * p.out_stride + c, t[i]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int c = 8 * (lane + i * kWarps * 32);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                t[i][e] = 0.f;
            if (c < p.n_cols)
                load8(x + c, t[i]);
        }
    }
    if (!p.h)
        return;
    normalise<kVec, kWarps>(p, t, lane, p.w, p.b, part);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int c = 8 * (lane + i * kWarps * 32);
        if (c < p.n_cols)
            store8(p.h + row * p.h_stride + c, t[i]);
    }
}

} // namespace vggt
