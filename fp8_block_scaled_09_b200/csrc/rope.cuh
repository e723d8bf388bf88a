// rope.cuh -- rotary positions of the fused QKV output, with the rotated keys
// and the values written to the E4M3 cache (unit scales).
//
// For token t at position p = positions[t] and pair j of a head's first `rot`
// channels, (a, b) = (x[j], x[j + rot/2]) or, interleaved, (x[2j], x[2j + 1]):
//     (a', b') = m (a cos u - b sin u,  b cos u + a sin u),  u = p inv_freq[j].
// The angle of a far position needs more than FP32 (p f has up to 55 bits, and
// an error of 2^-24 of 10^6 radians would be 0.06): p f / 2 pi is formed and
// reduced to its fraction in FP64, and so are sine and cosine, once per token
// and pair and rounded once with m (FP32 ones cost the same time, 59 us for the
// 8192 tokens below, and put 3 times as many keys on the other side of a tie).
// The rotation is FP32; queries are rounded once to BF16, keys once to E4M3 (not
// through BF16, which would round them twice), values as the plain cache write
// does.
//
// HBM-bound: 2 bytes read per channel, 2 written per query channel, 1 per key
// or value channel.  `span` threads take a token: thread (j, g) the 16 channels
// of part j -- the two 8-channel vectors that hold 8 pairs, or 16 that only
// pass through -- of heads g, g + groups, ...  Its 8 sines and cosines stay in
// registers over those heads, and the next head's vectors are on their way while one
// is rotated.  (Dealing single items to threads, with their index arithmetic and
// four-way bank conflicts on the sines, took 61 us for 8192 tokens of 56 + 2 x 8
// heads.)  That call takes 53 us now, 5.4 TB/s, half of its bytes writes; 8 tokens of it
// 4.8 us.
#pragma once

#include <stdint.h>

#include "kv_cache.cuh"
#include "ptx.cuh"
#include "rms_norm.cuh"

namespace fp8bq {

constexpr int kRopeThreads = 128;
constexpr int kRopeMinSpan = 64;
constexpr int kRopeMaxTok = kRopeThreads / kRopeMinSpan;
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
    int span;  // threads per token: a multiple of 64 that divides kRopeThreads
};

__device__ __forceinline__ uint2 e4m3x8(const float (&f)[8]) {
    const uint32_t lo = e4m3x2_satfinite(f[0], f[1]) | (static_cast<uint32_t>(e4m3x2_satfinite(f[2], f[3])) << 16);
    const uint32_t hi = e4m3x2_satfinite(f[4], f[5]) | (static_cast<uint32_t>(e4m3x2_satfinite(f[6], f[7])) << 16);
    return make_uint2(lo, hi);
}

__global__ void __launch_bounds__(kRopeThreads)
rope_kv_write_kernel(const RopeArgs a, int *status) {
    __shared__ float2 cs[kRopeMaxTok][kRopeMaxPairs];
    allow_dependent_launch();
    grid_dependency_wait();
    const int toks = kRopeThreads / a.span;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * toks;
    const int ntok = static_cast<int>(min(static_cast<int64_t>(toks), a.T - t0));
    const int pairs = a.rot >> 1, parts = a.dim >> 4;
    const int tok = threadIdx.x / a.span, in = threadIdx.x - tok * a.span;
    const int groups = a.span / parts;
    const int g = in / parts, j = in - g * parts;
    const int heads = a.q_heads + 2 * a.kv_heads, rotated = a.q_heads + a.kv_heads;
    const bool turns_j = j < (a.rot >> 4);          // the part has pairs
    const bool split = turns_j && !a.interleaved;   // in vectors half a rotation apart
    const bool mine = tok < ntok && g < groups;
    const uint16_t *row = a.qkv + (t0 + (mine ? tok : 0)) * a.row_stride;
    // channels of the part's vectors; value heads are not split
    const int p0 = j * 16, p1 = p0 + 8;
    const int r0 = split ? j * 8 : p0, r1 = split ? pairs + j * 8 : p1;
    auto load = [&](int head, uint4 &u0, uint4 &u1) {
        if (head >= heads) return;
        const uint16_t *src = row + static_cast<int64_t>(head) * a.dim;
        u0 = *reinterpret_cast<const uint4 *>(src + (head < rotated ? r0 : p0));
        u1 = *reinterpret_cast<const uint4 *>(src + (head < rotated ? r1 : p1));
    };
    uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
    if (mine) load(g, u0, u1);

    for (int i = threadIdx.x; i < ntok * pairs; i += kRopeThreads) {
        const int t = i / pairs, k = i - t * pairs;
        const double turns = static_cast<double>(a.positions[t0 + t]) *
                             static_cast<double>(__ldg(a.inv_freq + k)) * 0.15915494309189533577;
        double c, s;
        sincospi(2.0 * (turns - rint(turns)), &s, &c);
        cs[t][k] = make_float2(static_cast<float>(c * a.mscale), static_cast<float>(s * a.mscale));
    }
    const int64_t slot = mine ? a.loc[t0 + tok] : -1;
    if (in == 0 && mine && (slot < -1 || slot >= a.num_slots)) atomicExch(status, 8 /* FP8BQ_ERR_INDEX */);
    __syncthreads();
    if (slot < 0 || slot >= a.num_slots) return;  // a padding token: nothing of it is written

    float2 r[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) r[c] = turns_j ? cs[tok][j * 8 + c] : make_float2(1.0f, 0.0f);
    uint16_t *q_row = a.q_out + (t0 + tok) * a.q_stride;
    for (int head = g; head < heads; head += groups) {
        const uint4 w0 = u0, w1 = u1;
        load(head + groups, u0, u1);
        float f0[8], f1[8];
        unpack_bf16x8(w0, f0);
        unpack_bf16x8(w1, f1);
        const bool rotate = turns_j && head < rotated;
        if (rotate) {
            if (split) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const float x = f0[c], y = f1[c];
                    f0[c] = x * r[c].x - y * r[c].y;
                    f1[c] = y * r[c].x + x * r[c].y;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float x = f0[2 * c], y = f0[2 * c + 1];
                    f0[2 * c] = x * r[c].x - y * r[c].y;
                    f0[2 * c + 1] = y * r[c].x + x * r[c].y;
                    const float z = f1[2 * c], w = f1[2 * c + 1];
                    f1[2 * c] = z * r[4 + c].x - w * r[4 + c].y;
                    f1[2 * c + 1] = w * r[4 + c].x + z * r[4 + c].y;
                }
            }
        }
        if (head < a.q_heads) {
            uint16_t *dst = q_row + static_cast<int64_t>(head) * a.dim;
            *reinterpret_cast<uint4 *>(dst + r0) = rotate ? pack_bf16x8(f0) : w0;
            *reinterpret_cast<uint4 *>(dst + r1) = rotate ? pack_bf16x8(f1) : w1;
        } else {
            const bool v = head >= rotated;
            uint8_t *dst = (v ? a.v_cache : a.k_cache) + slot * a.slot_stride +
                           static_cast<int64_t>(head - a.q_heads - (v ? a.kv_heads : 0)) * a.dim;
            const uint2 e0 = e4m3x8(f0), e1 = e4m3x8(f1);
            if (split && !v) {
                *reinterpret_cast<uint2 *>(dst + r0) = e0;
                *reinterpret_cast<uint2 *>(dst + r1) = e1;
            } else {
                *reinterpret_cast<uint4 *>(dst + p0) = make_uint4(e0.x, e0.y, e1.x, e1.y);
            }
        }
    }
}

}  // namespace fp8bq
