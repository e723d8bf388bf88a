// attention.cuh -- attention of new tokens over the paged E4M3 cache.
//
// New token i of sequence b (q_len new tokens, seq_len cache positions, the new
// tokens among them) stands at position seq_len - q_len + i and sees positions
// 0 .. its own (causal) or all seq_len of them.  For query head h, with
// kv head g = h / (q_heads / kv_heads):
//     z_c = scale q_h . k_{g,c},  out_h = sum_c exp(z_c - lse) v_{g,c},
//     lse = log sum_c exp(z_c);  a token that sees nothing gives 0 and -inf.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "ptx.cuh"

namespace fp8bq {
namespace attn {

constexpr int kDim = 128;  // channels of a head

struct Args {
    const uint16_t *q;         // BF16 [T, q_stride]
    const uint8_t *k_cache, *v_cache;
    const int32_t *table;      // [B, table_stride]
    const int32_t *seq_lens;   // [B]
    const int32_t *cu_q;       // [B + 1]
    uint16_t *out;             // BF16 [T, out_stride]
    float *lse;                // [T, q_heads] or null
    int64_t q_stride, out_stride, table_stride, slot_stride, T;
    int32_t num_pages, max_pages, page_shift, B, q_heads, kv_heads, group, max_q, causal;
    float scale;
};

// One block per (token, query head), positions dealt to its warps in turn.
constexpr int kSimpleWarps = 4;

__global__ void __launch_bounds__(32 * kSimpleWarps)
attention_simple_kernel(const Args a, int *status) {
    __shared__ float part[kSimpleWarps][kDim + 2];
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t t = blockIdx.x / a.q_heads;
    const int h = static_cast<int>(blockIdx.x % a.q_heads), g = h / a.group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.cu_q[a.B] > a.T) atomicExch(status, 8);
    int b = -1;
    for (int i = 0; i < a.B; ++i)
        if (t >= a.cu_q[i] && t < a.cu_q[i + 1]) b = i;
    if (b < 0) return;
    const int i = static_cast<int>(t - a.cu_q[b]), q_len = a.cu_q[b + 1] - a.cu_q[b];
    if (i >= a.max_q) {
        atomicExch(status, 8);
        return;
    }
    int len = a.seq_lens[b];
    if (len < 0 || len > (a.max_pages << a.page_shift)) {
        len = len < 0 ? 0 : a.max_pages << a.page_shift;
        atomicExch(status, 8);
    }
    const int n = a.causal ? min(len, len - q_len + i + 1) : len;
    float q[4], o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0;
    const uint16_t *qp = a.q + t * a.q_stride + h * kDim + lane * 4;
    for (int k = 0; k < 4; ++k) q[k] = __uint_as_float(static_cast<uint32_t>(qp[k]) << 16);
    for (int c = warp; c < n; c += kSimpleWarps) {
        const int32_t page = a.table[b * a.table_stride + (c >> a.page_shift)];
        uint32_t kk = 0, vv = 0;
        if (page < 0 || page >= a.num_pages) {
            atomicExch(status, 8);
        } else {
            const int64_t slot = (static_cast<int64_t>(page) << a.page_shift) + (c & ((1 << a.page_shift) - 1));
            const int64_t off = slot * a.slot_stride + g * kDim + lane * 4;
            kk = *reinterpret_cast<const uint32_t *>(a.k_cache + off);
            vv = *reinterpret_cast<const uint32_t *>(a.v_cache + off);
        }
        float z = 0;
        for (int k = 0; k < 4; ++k) z += q[k] * e4m3_to_float(kk >> (8 * k));
        for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, d);
        z *= a.scale;
        const float m2 = fmaxf(m, z), f = expf(m - m2), p = expf(z - m2);
        l = l * f + p;
        for (int k = 0; k < 4; ++k) o[k] = o[k] * f + p * e4m3_to_float(vv >> (8 * k));
        m = m2;
    }
    for (int k = 0; k < 4; ++k) part[warp][lane * 4 + k] = o[k];
    if (lane == 0) part[warp][kDim] = m, part[warp][kDim + 1] = l;
    __syncthreads();
    if (warp != 0) return;
    float top = -INFINITY, sum = 0, r[4] = {0, 0, 0, 0};
    for (int w = 0; w < kSimpleWarps; ++w) top = fmaxf(top, part[w][kDim]);
    for (int w = 0; w < kSimpleWarps && top > -INFINITY; ++w) {
        const float f = expf(part[w][kDim] - top);
        sum += f * part[w][kDim + 1];
        for (int k = 0; k < 4; ++k) r[k] += f * part[w][lane * 4 + k];
    }
    __nv_bfloat16 *op = reinterpret_cast<__nv_bfloat16 *>(a.out + t * a.out_stride + h * kDim + lane * 4);
    for (int k = 0; k < 4; ++k) op[k] = __float2bfloat16_rn(sum > 0 ? r[k] / sum : 0.0f);
    if (a.lse != nullptr && lane == 0) a.lse[t * a.q_heads + h] = sum > 0 ? top + logf(sum) : -INFINITY;
}

}  // namespace attn
}  // namespace fp8bq
