// rope.cuh -- rotary positions of the fused QKV output, with the rotated keys
// and the values written to the E4M3 cache (unit scales).
//
// For token t at position p = positions[t] and pair j of a head's first `rot`
// channels, (a, b) = (x[j], x[j + rot/2]) or, interleaved, (x[2j], x[2j + 1]):
//     (a', b') = m (a cos u - b sin u,  b cos u + a sin u),  u = p inv_freq[j].
// The angle of a far position needs more than FP32 (p f has up to 55 bits, and
// an error of 2^-24 of 10^6 radians would be 0.06): p f / 2 pi is formed in
// FP64, reduced to its fraction, and only that goes to the FP32 sine and
// cosine.  The rotation is FP32; queries are rounded once to BF16, keys once
// to E4M3 (not through BF16, which would round them twice), values as the
// plain cache write does.
//
// HBM-bound: 2 bytes read per channel, 2 written per query channel, 1 per key
// or value channel.  A CTA takes kTok tokens: its threads first compute the
// tokens' rot/2 sines and cosines into shared memory (shared by all heads),
// then work through items of 16 channels -- the two 8-channel vectors that
// hold 8 pairs, or 16 channels that only pass through.
#pragma once

#include <stdint.h>

#include "kv_cache.cuh"
#include "ptx.cuh"
#include "rms_norm.cuh"

namespace fp8bq {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTok = 4;
constexpr int kRopeMaxPairs = 128;  // head_dim <= 256

struct RopeArgs {
    const uint16_t *qkv;  // [T, row_stride], may be q_out
    uint16_t *q_out;      // [T, q_stride]
    const int64_t *positions, *loc;
    const float *inv_freq;
    uint8_t *k_cache, *v_cache;
    int64_t row_stride, q_stride, T, num_slots, slot_stride;
    float mscale;
    int q_heads, kv_heads, dim, rot, interleaved;
    int tok;  // tokens per CTA, 1 .. kRopeMaxTok
};

__device__ __forceinline__ uint2 e4m3x8(const float (&f)[8]) {
    const uint32_t lo = e4m3x2_satfinite(f[0], f[1]) | (static_cast<uint32_t>(e4m3x2_satfinite(f[2], f[3])) << 16);
    const uint32_t hi = e4m3x2_satfinite(f[4], f[5]) | (static_cast<uint32_t>(e4m3x2_satfinite(f[6], f[7])) << 16);
    return make_uint2(lo, hi);
}

__global__ void __launch_bounds__(kRopeThreads)
rope_kv_write_kernel(const RopeArgs a, int *status) {
    __shared__ float2 cs[kRopeMaxTok][kRopeMaxPairs];
    __shared__ int64_t slot[kRopeMaxTok];
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tok;
    const int ntok = static_cast<int>(min(static_cast<int64_t>(a.tok), a.T - t0));
    const int pairs = a.rot >> 1;
    for (int i = threadIdx.x; i < ntok * pairs; i += kRopeThreads) {
        const int t = i / pairs, j = i - t * pairs;
        const double turns = static_cast<double>(a.positions[t0 + t]) *
                             static_cast<double>(__ldg(a.inv_freq + j)) * 0.15915494309189533577;
        float c, s;
        sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s, &c);
        cs[t][j] = make_float2(c * a.mscale, s * a.mscale);
    }
    if (threadIdx.x < ntok) {
        const int64_t s = a.loc[t0 + threadIdx.x];
        slot[threadIdx.x] = s >= 0 && s < a.num_slots ? s : -1;
        if (s < -1 || s >= a.num_slots) atomicExch(status, 8 /* FP8BQ_ERR_INDEX */);
    }
    __syncthreads();

    const int per_head = a.dim >> 4, rot_items = a.rot >> 4;
    const int heads = a.q_heads + 2 * a.kv_heads;
    const int items = heads * per_head;
    for (int i = threadIdx.x; i < ntok * items; i += kRopeThreads) {
        const int t = i / items, it = i - t * items;
        const int head = it / per_head, j = it - head * per_head;
        if (slot[t] < 0) continue;  // a padding token: nothing of it is written
        const bool is_v = head >= a.q_heads + a.kv_heads;
        const bool rotate = !is_v && j < rot_items;
        // channels of the item's two vectors within the head
        const bool split = rotate && !a.interleaved;
        const int c0 = split ? j * 8 : j * 16;
        const int c1 = split ? pairs + j * 8 : j * 16 + 8;
        const uint16_t *src = a.qkv + (t0 + t) * a.row_stride + static_cast<int64_t>(head) * a.dim;
        const uint4 u0 = *reinterpret_cast<const uint4 *>(src + c0);
        const uint4 u1 = *reinterpret_cast<const uint4 *>(src + c1);
        float f0[8], f1[8];
        unpack_bf16x8(u0, f0);
        unpack_bf16x8(u1, f1);
        if (split) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 r = cs[t][j * 8 + k];
                const float x = f0[k], y = f1[k];
                f0[k] = x * r.x - y * r.y;
                f1[k] = y * r.x + x * r.y;
            }
        } else if (rotate) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 r = cs[t][j * 8 + k];
                const float x = f0[2 * k], y = f0[2 * k + 1];
                f0[2 * k] = x * r.x - y * r.y;
                f0[2 * k + 1] = y * r.x + x * r.y;
                const float2 p = cs[t][j * 8 + 4 + k];
                const float z = f1[2 * k], w = f1[2 * k + 1];
                f1[2 * k] = z * p.x - w * p.y;
                f1[2 * k + 1] = w * p.x + z * p.y;
            }
        }
        if (head < a.q_heads) {
            uint16_t *dst = a.q_out + (t0 + t) * a.q_stride + static_cast<int64_t>(head) * a.dim;
            *reinterpret_cast<uint4 *>(dst + c0) = rotate ? pack_bf16x8(f0) : u0;
            *reinterpret_cast<uint4 *>(dst + c1) = rotate ? pack_bf16x8(f1) : u1;
        } else {
            const int kv = head - a.q_heads - (is_v ? a.kv_heads : 0);
            uint8_t *dst = (is_v ? a.v_cache : a.k_cache) + slot[t] * a.slot_stride +
                           static_cast<int64_t>(kv) * a.dim;
            *reinterpret_cast<uint2 *>(dst + c0) = e4m3x8(f0);
            *reinterpret_cast<uint2 *>(dst + c1) = e4m3x8(f1);
        }
    }
}

}  // namespace fp8bq
