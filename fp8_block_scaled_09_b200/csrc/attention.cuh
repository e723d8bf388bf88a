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

}  // namespace attn
}  // namespace fp8bq
