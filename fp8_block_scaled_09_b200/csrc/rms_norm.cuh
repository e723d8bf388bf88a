// rms_norm.cuh -- root-mean-square norm with the residual's addition, quantized
// for the FP8 linear layer that follows.
//
//     r = BF16(x + residual)                     (r = x without a residual)
//     h = r * (mean(r^2) + eps)^(-1/2) * w       (FP32)
//     s[g] = amax(|h| over 128 channels) / 448, or 1;  q = E4M3(h / s)
// r is rounded to BF16 before the norm because that is the residual stream the
// next layer reads; h itself is never rounded before its quantization (a BF16
// h would round every value twice), only its optional BF16 copy is.
//
// The row's factor cancels in the codes: with p = r w, exact in FP32 (two BF16
// factors; below 2^-126 to FP32's smallest step), h / s = 448 p / amax(|p|), where 448 p is exact too (7 p and a power
// of two), so a code is E4M3 of one correctly rounded quotient.  The codes
// therefore do not wait for the sum of squares; only scales and h do.
//
// HBM-bound: 2 bytes of x and 2 of the residual read, 2 of the residual and
// 1 + 1/32 of codes and scales written per element.  One CTA holds one row in
// registers (V vectors of 8 channels per thread, thread t has vectors t, t + n,
// ...), so every byte moves once; 16 consecutive lanes hold the 128 channels of
// one scale.  The weight stays in L1.  Measured: 8192 x 7168 to BF16 70.6 us,
// 6.65 TB/s; 2048 x 7168 with residual and codes 21.6 us, 4.8 TB/s (the start and
// the last wave of a short kernel), 8192 rows of it 76.3 us, 5.4 TB/s.  Packed
// FP32 pairs for the products were no faster; CTAs that stay and fetch their next
// row ahead were slower (23.7 and 85.5 us): their registers leave two rows per SM.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "ptx.cuh"
#include "quantize.cuh"

namespace fp8bq {

// Two floats -> packed BF16 (round to nearest even), `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void unpack_bf16x8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&f)[8]) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                      pack_bf16(f[6], f[7]));
}

// Codes of eight products p of a group whose largest is `top` (448 p / top).
__device__ __forceinline__ uint2 encode8_of_max(const float (&p)[8], float top) {
    uint32_t e[4];
    if (top >= 0x1p-80f && top <= 0x1p100f) {
        const float y = __frcp_rn(top);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            e[j] = e4m3x2_satfinite(corrected_quotient(448.0f * p[2 * j], top, y),
                                    corrected_quotient(448.0f * p[2 * j + 1], top, y));
    } else {
        // Where 448 p or the quotient's residual may leave the normal range: p and top
        // times a power of two, which is exact wherever the code is not 0 and leaves the
        // quotient as it is.  (top / 448 itself may be subnormal, or 0.)
        const float shift = top < 1.0f ? 0x1p70f : 0x1p-70f;
        const float t = top == 0.0f ? 1.0f : top * shift, y = __frcp_rn(t);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            e[j] = e4m3x2_satfinite(corrected_quotient(448.0f * (p[2 * j] * shift), t, y),
                                    corrected_quotient(448.0f * (p[2 * j + 1] * shift), t, y));
    }
    return make_uint2(e[0] | (e[1] << 16), e[2] | (e[3] << 16));
}

// residual may be null (r = x); residual_out may be the same buffer as residual
// or x (a thread reads its vectors before it writes them).  q and s are both
// null or both given; h may be null.
template <int V, int kMaxThreads, int kMinCtas>
__global__ void __launch_bounds__(kMaxThreads, kMinCtas)
rms_norm_kernel(const uint4 *x, const uint4 *residual, const uint4 *__restrict__ weight, float eps,
                int nvec, uint4 *residual_out, uint2 *__restrict__ q,
                float *__restrict__ s, uint4 *__restrict__ h) {
    __shared__ float warp_sum[kMaxThreads / 32];
    allow_dependent_launch();
    const int n = blockDim.x, warps = n >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float inv_k = 1.0f / static_cast<float>(nvec * 8);
    grid_dependency_wait();
    const int64_t base = static_cast<int64_t>(blockIdx.x) * nvec;
    uint4 v[V];
    {
        uint4 u[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * n;
            v[i] = c < nvec ? x[base + c] : make_uint4(0, 0, 0, 0);
            u[i] = residual != nullptr && c < nvec ? residual[base + c] : make_uint4(0, 0, 0, 0);
        }
        if (residual != nullptr) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = threadIdx.x + i * n;
                float a[8], b[8];
                unpack_bf16x8(v[i], a);
                unpack_bf16x8(u[i], b);
#pragma unroll
                for (int j = 0; j < 8; ++j) a[j] += b[j];
                v[i] = pack_bf16x8(a);
                if (c < nvec) residual_out[base + c] = v[i];
            }
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float a[8];
        unpack_bf16x8(v[i], a);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(a[j], a[j], sum);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) warp_sum[warp] = sum;
    float top[V];  // largest |p| of the 16 lanes' group
    if (q != nullptr) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * n;
            float p[8], g[8];
            unpack_bf16x8(v[i], p);
            unpack_bf16x8(c < nvec ? __ldg(weight + c) : make_uint4(0, 0, 0, 0), g);
            top[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                p[j] *= g[j];
                top[i] = fmaxf(top[i], fabsf(p[j]));
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], o));
            if (c < nvec) q[base + c] = encode8_of_max(p, top[i]);
        }
    }
    __syncthreads();
    if (h != nullptr || (lane & 15) == 0) {
        // every thread adds the warps' sums itself (broadcast reads)
        sum = 0.0f;
        for (int w = 0; w < warps; ++w) sum += warp_sum[w];
        const float inv = rsqrtf(fmaf(sum, inv_k, eps));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * n;
            if (c >= nvec) continue;
            if (q != nullptr && (lane & 15) == 0)
                s[(base + c) >> 4] = top[i] == 0.0f ? 1.0f : __fdiv_rn(top[i] * inv, 448.0f);
            if (h != nullptr) {
                float p[8], g[8];
                unpack_bf16x8(v[i], p);
                unpack_bf16x8(__ldg(weight + c), g);
#pragma unroll
                for (int j = 0; j < 8; ++j) p[j] = p[j] * g[j] * inv;
                h[base + c] = pack_bf16x8(p);
            }
        }
    }
}

}  // namespace fp8bq
