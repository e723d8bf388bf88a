// attention_few.cuh -- paged attention for few query rows per kv head (decode):
// q_len * group <= NR rows, NR = 8 or 16.  (From 17 rows on the other kernel is
// faster: 28 rows, 16 sequences of 4500 positions, took 63 us here with NR = 32, 47 us
// there; 14 rows take 37 us here.)
//
// Bound by the cache's bytes: 256 per position and kv head, read once.  The
// E4M3 codes go from HBM to shared memory by TMA and from there straight into
// the tensor cores, with the roles of rows and columns swapped: 128 cache
// positions are the MMA's M, the query rows its N.
//     S^T[pos, row] = K[pos, :] . Q[row, :]       M = 128, N = 2 NR, K = 128
//     O^T[ch, row] += V[:, ch]^T . P[:, row]      M = 128, N = 2 NR, K = 128 positions
// Neither K nor V is ever converted: V is the A operand with its channels
// contiguous.  Queries and weights keep their precision as two E4M3 parts,
// in two columns whose results are added: hi holds 4 significant bits, lo the
// next 4, x = hi + lo / 32: of x up to 256 hi's error is at most 8, so 32 times
// it stays below 256.  A BF16 query, scaled by a power of two that takes its row's
// largest channel to [128, 256), is exact down to 2^-14 of that and off by at most
// 2^-22 of it below.  A weight, held times what takes the chunk's largest to 256 (which
// so is exact), has 8 bits down to 2^-15 of that and an absolute error of 2^-23 of it
// below.  (With lo unscaled and the row's maximum in the chunk's place
// the steps were 2^-17 of the row's largest: a first position 13 logits above 32768
// others, its value near 0, took 21% off the output.)  Two MMAs into one column cost
// more: an MMA with this few columns takes the time to read its 4 KB of A, and with
// twice as many of them the tensor pipe was busy 1100 of 2550 cycles per tile.
//
// Work is a list of tiles of 128 positions, ordered by (sequence, kv head,
// tile), each head preceded by some tiles' worth of nothing for what
// beginning and ending it costs (head_cost); CTA c of a grid of one CTA per SM takes the
// c-th equal part, whatever the sequences' lengths.  A part's tiles of one
// (sequence, head), its segment, are taken in chunks of at most kChunk tiles,
// as many as TMEM holds scores for (twice): a chunk's scores are all there
// before its softmax, so no output is ever rescaled in TMEM; the chunk's O^T is
// merged into registers with a factor 2^(r_old - r_new), one chunk
// later, so that nothing waits for its MMAs.  r, the reference that a chunk's
// weights are held against, is the chunk's own maximum, not the running one: a
// position that dominates the row then coarsens only the weights of its own chunk.
// (Rounded up to a power of two it would make the factors exact, but not the largest
// weight: the output's error went from 0.00172 to 0.00177, BF16's own is 0.00166.)  Where
// a chunk lies more than kFarBelow under the running maximum, r stays there, so that
// no sum overflows; what is lost then is 2^-87 of the row's largest weight.  The ring carries K of chunk
// g + 1 ahead of V of chunk g, so the next scores are computed while the
// softmax works.  A (sequence, head) that lies in several CTAs leaves FP32
// partials and maxima in the workspace; the last CTA to arrive (a counter)
// joins them in the order of the CTAs, so results do not depend on timing.
//
// Roles: warp 0 TMA producer (a page per lane), warp 1 MMA issuer, warps 2..9
// softmax (two groups of four that take a chunk's tiles in turn; thread = one
// position of the tile, its TMEM lane, in the score phase, one output channel
// of half the rows in the merge), warp 10 queries, warp 11 follows the ring and clears
// V behind a sequence's end.
//
// Measured, after a 256 MB write: 128 sequences of 2048 positions, 56 query and 8 kv
// heads, pages of 64: 120 us, 4.5 TB/s; pages of 16: 141 us (a TMA box then brings only
// 2 KB, and an SM starts one in ~80 ns; half of the pages by cp.async instead, from two
// more warps, took 211 us).  One sequence of 65001 positions, among others of its kind:
// 32 us, of which 5 pass before its first tile and 4 in the join.
#pragma once

#include "attention.cuh"
#include "gemm_decode.cuh"
#include "rms_norm.cuh"

namespace fp8bq {
namespace attn {

constexpr int kTile = 128;                 // positions
constexpr int kStageBytes = kTile * kDim;  // one K or V tile of codes
constexpr int kFewSoftmaxWarps = 8;
constexpr int kFewThreads = 32 * (4 + kFewSoftmaxWarps);
constexpr float kPScale = 8.0f;    // weights are held times 2^8
constexpr float kLoScale = 32.0f;  // low parts, of queries too, times 2^5 more
// A row's score scale is at least this: 0 times the -inf of a masked position would be
// NaN (a product of 2^24 at most times this is still nothing).
constexpr float kMinScale = 0x1p-126f;
// log2: sums stay below 2^(8 + 25 + 64), outputs below 2^9 times that
constexpr float kFarBelow = 64.0f;

template <int NR>
struct Few {
    static constexpr int kN = 2 * NR;            // MMA columns: hi and lo parts
    static constexpr int kChunk = 256 / kN - 1;  // tiles; 2 chunks + 2 outputs = 512 columns
    static constexpr int kQ = kN * kDim;         // bytes of Q
    static constexpr int kP = kN * kTile;        // bytes of P
    // a whole chunk of P, so that the softmax never waits for V; half per group
    static constexpr int kGroupSlots = (kChunk + 1) / 2;
    static constexpr int kPSlots = 2 * kGroupSlots;
    static constexpr int kStages = 11;
    static constexpr int kQOff = kStages * kStageBytes;  // [2]
    static constexpr int kPOff = kQOff + 2 * kQ;         // [kPSlots]
    static constexpr int kBarOff = kPOff + kPSlots * kP;
    // full, empty, cleared; pfull, pempty; qfull (4), qempty, sfull, sfree, ofull, ofree (2 each)
    static constexpr int kBars = 3 * kStages + 2 * kPSlots + 4 + 10;
    // per-row values: scale and limit [4], reference and factor [2], negated reference,
    // running maximum, reductions over the warps [8], sums over the warps [2][8]
    static constexpr int kRowOff = kBarOff + kBars * 8;
    static constexpr int kBytes = kRowOff + (4 + 4 + 2 + 2 + 1 + 1 + 8 + 16) * NR * 4 + 64 + 1024;
    static_assert(kBytes <= 227 * 1024, "shared memory");
    static_assert(kQOff % 1024 == 0 && kPOff % 1024 == 0 && kQ % 1024 == 0, "swizzled tiles");
    static constexpr int kPartial = NR * (kDim + 2);  // floats: O [NR][128], reference [NR], sum [NR]
    __device__ static uint32_t s_col(int buf, int j) { return (buf * kChunk + j) * kN; }
    __device__ static uint32_t o_col(int buf) { return (2 * kChunk + buf) * kN; }
};

// idesc of E4M3 x E4M3 with the M dimension of A and the N dimension of B contiguous
__host__ __device__ constexpr uint32_t idesc_e4m3_mn(int m, int n) {
    return umma_idesc_e4m3(m, n) | (1u << 15) | (1u << 16);
}

// True in one lane of the (converged) warp.  MMA issuers that let the whole warp
// run their loops and only issue in this lane keep descriptors and addresses in
// uniform registers, where the MMA instruction wants them; in a branch on the lane
// number each is moved there before every MMA (~100 cycles per MMA measured).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// Unswizzled operand tile whose M or N dimension is contiguous: blocks of 16
// bytes of it by 8 K rows (128 bytes); `k_step` bytes between blocks along K,
// `mn_step` along M or N.
__device__ __forceinline__ uint64_t umma_desc_mn(uint32_t saddr, uint32_t mn_step, uint32_t k_step) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(k_step >> 4) << 16;
    d |= static_cast<uint64_t>(mn_step >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;  // descriptor version for sm_100
    return d;
}

// X consecutive TMEM columns of this warp's lanes, without the wait.
template <int X>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float *v) {
    static_assert(X == 4 || X == 8 || X == 16, "columns");
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    if constexpr (X == 4)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(taddr));
    else if constexpr (X == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                       "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
    else
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
              "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
              "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(taddr));
}

// Waits for this warp's TMEM loads into v[0, X); the values pass through the
// statement, so that no use of them moves before it.
template <int X>
__device__ __forceinline__ void tmem_ld_wait(float *v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < X; ++i) asm volatile("" : "+f"(v[i]));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// Eight BF16 values times `up` (a power of two that takes them below 256) as two
// E4M3 parts: hi keeps the top 4 of their 8 significant bits, lo the other 4.
// Both are exact but below 2^-6, where hi is 0 and lo rounds to steps of 2^-9.
__device__ __forceinline__ void split8(uint4 v, float up, uint2 &hi, uint2 &lo) {
    float x[8], h[8];
    unpack_bf16x8(v, x);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        x[k] *= up;
        h[k] = fabsf(x[k]) < 0x1p-6f ? 0.0f : __uint_as_float(__float_as_uint(x[k]) & 0xFFF00000u);
        x[k] -= h[k];
    }
    hi = make_uint2(e4m3x2_satfinite(h[0], h[1]) | (static_cast<uint32_t>(e4m3x2_satfinite(h[2], h[3])) << 16),
                    e4m3x2_satfinite(h[4], h[5]) | (static_cast<uint32_t>(e4m3x2_satfinite(h[6], h[7])) << 16));
    lo = make_uint2(e4m3x2_satfinite(x[0], x[1]) | (static_cast<uint32_t>(e4m3x2_satfinite(x[2], x[3])) << 16),
                    e4m3x2_satfinite(x[4], x[5]) | (static_cast<uint32_t>(e4m3x2_satfinite(x[6], x[7])) << 16));
}

// Two E4M3 codes -> two floats, -kLoScale times their values (exact in F16: 4
// significant bits, at most 2^14).
__device__ __forceinline__ float2 e4m3x2_to_neg_scaled(uint16_t c) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
    return __half22float2(__hmul2(*reinterpret_cast<const __half2 *>(&h2), __float2half2_rn(-kLoScale)));
}

// Eight BF16 values times `up` (as in split8) as two E4M3 parts for columns of their own.
__device__ __forceinline__ void split8_scaled(uint4 v, float up, uint2 &hi, uint2 &lo) {
    float x[8];
    unpack_bf16x8(v, x);
    uint32_t h[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float a = x[2 * k] * up, b = x[2 * k + 1] * up;
        h[k] = e4m3x2_satfinite(a, b);
        const float2 d = e4m3x2_to_neg_scaled(static_cast<uint16_t>(h[k]));
        l[k] = e4m3x2_satfinite(fmaf(a, kLoScale, d.x), fmaf(b, kLoScale, d.y));
    }
    hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
    lo = make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
}

// A sequence as the kernels take it: lengths that the host cannot check are
// clamped (seq_is_bad reports them).
struct Seq {
    int len;     // cache positions
    int q0;      // first row of q
    int q_len;   // rows taken
    int q_real;  // new tokens as given: they fix the positions
};

__device__ __forceinline__ Seq seq_of(const Args &a, int b) {
    Seq s;
    const int cap = a.max_pages << a.page_shift;
    s.len = min(max(__ldg(a.seq_lens + b), 0), cap);
    const int T = static_cast<int>(a.T);
    s.q0 = min(max(__ldg(a.cu_q + b), 0), T);
    s.q_real = max(__ldg(a.cu_q + b + 1), s.q0) - s.q0;
    s.q_len = min(min(s.q_real, T - s.q0), a.max_q);
    return s;
}

__device__ __forceinline__ bool seq_is_bad(const Args &a, int b) {
    const int len = __ldg(a.seq_lens + b), q0 = __ldg(a.cu_q + b), q1 = __ldg(a.cu_q + b + 1);
    return len < 0 || len > (a.max_pages << a.page_shift) || q0 < 0 || q1 < q0 || q1 > a.T ||
           q1 > q0 + a.max_q;
}

__device__ __forceinline__ int seq_tiles(const Seq &s) {
    return s.q_len > 0 ? (s.len + kTile - 1) / kTile : 0;
}

// The pages of a sequence as a producer warp walks them: lane l holds entry
// l of the current and of the next 32 (loaded before they are needed: a line of
// the table that is still in HBM costs a microsecond).
struct PageWalk {
    const int32_t *row;
    int blk, n, cur, nxt;

    __device__ int load(int b) const {
        const int i = b * 32 + static_cast<int>(threadIdx.x & 31);
        return i < n ? __ldg(row + i) : -1;
    }
    // to be read from position `pos` on, up to the sequence's length
    __device__ PageWalk(const Args &a, int b, int len, int pos)
        : row(a.table + b * a.table_stride), blk((pos >> a.page_shift) >> 5),
          n((len + (1 << a.page_shift) - 1) >> a.page_shift) {
        cur = load(blk);
        nxt = load(blk + 1);
    }
    // Warp-wide: first cache row of position `pos` (ascending calls; every lane's
    // in the same 32 pages), or -kTile (a row outside the cache: TMA fills
    // zeros) for a page that is not needed or not in the cache.
    __device__ int row_of(const Args &a, int pos, int *status) {
        const int idx = pos >> a.page_shift;
        const int want = __shfl_sync(0xFFFFFFFFu, idx >> 5, 0);
        if (want != blk) {
            blk = want;
            cur = nxt;
            nxt = load(blk + 1);
        }
        const int page = __shfl_sync(0xFFFFFFFFu, cur, idx & 31);
        if (idx >= n) return -kTile;
        if (page < 0 || page >= a.num_pages) {
            atomicExch(status, 8 /* FP8BQ_ERR_INDEX */);
            return -kTile;
        }
        return (page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
    }
};

// Positions of the work list that one head of a sequence takes: its tiles and what
// beginning and ending it costs, about 4 us -- 4 tiles, or 2 with small pages, whose
// tiles take longer (128 sequences of 1 .. 4096 positions, pages of 64: 164 us at 2,
// 132 at 4, 127 at 5; pages of 16: 150 us at 2, 154 at 3, 156 at 4).
__device__ __forceinline__ int head_extra(const Args &a) { return a.page_shift < 5 ? 2 : 4; }
__device__ __forceinline__ int64_t head_cost(const Args &a, int tiles) {
    return tiles > 0 ? static_cast<int64_t>(tiles) + head_extra(a) : 0;
}

// The chunks of one CTA's part of the work list, in order.
template <int NR>
struct Chunks {
    const Args &a;
    int64_t w, w_end, base;  // next position, end of the part, first position of sequence b
    int b, tiles;            // sequence of w, its tiles per head
    Seq seq;
    // the current chunk
    int hk, t, n;            // kv head, first tile, tiles
    int seg_t0, seg_end;     // tiles of the segment
    bool first, last;        // of its segment

    __device__ Chunks(const Args &args, int64_t w0, int64_t w1, int b0, int64_t base0)
        : a(args), w(w0), w_end(w1), base(base0), b(b0), tiles(0), hk(0), t(0), n(0), seg_t0(0),
          seg_end(0), first(false), last(false) {
        if (w < w_end) {
            seq = seq_of(a, b);
            tiles = seq_tiles(seq);
        }
    }
    __device__ bool next() {
        t += n;
        while (t >= seg_end) {  // a new segment
            n = 0;
            if (w >= w_end) return false;
            while (w >= base + head_cost(a, tiles) * a.kv_heads) {
                base += head_cost(a, tiles) * a.kv_heads;
                seq = seq_of(a, ++b);
                tiles = seq_tiles(seq);
            }
            const int cost = static_cast<int>(head_cost(a, tiles));
            const uint32_t off = static_cast<uint32_t>(w - base);  // < cost * kv_heads < 2^30
            hk = static_cast<int>(off / static_cast<uint32_t>(cost));
            const int rel = static_cast<int>(off - static_cast<uint32_t>(hk) * cost);
            const int64_t left = min(static_cast<int64_t>(cost - rel), w_end - w);
            t = seg_t0 = max(rel - head_extra(a), 0);
            seg_end = max(static_cast<int>(rel + left) - head_extra(a), 0);
            w += left;
        }
        first = t == seg_t0;
        // equal chunks, so that no segment ends in a short one
        const int total = seg_end - seg_t0;
        const int parts = (total + Few<NR>::kChunk - 1) / Few<NR>::kChunk;
        n = min((total + parts - 1) / parts, seg_end - t);
        last = t + n == seg_end;
        return true;
    }
    // the list's position of the current (sequence, head)'s first tile
    __device__ int64_t item() const { return base + hk * head_cost(a, tiles) + head_extra(a); }
};

template <int NR>
__global__ void __launch_bounds__(kFewThreads, 1)
attention_few_kernel(const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const Args a, int *counters,
                     float *partials, int *status) {
    using F = Few<NR>;
    constexpr int N = F::kN;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + F::kBarOff);
    uint64_t *empty = full + F::kStages;
    uint64_t *pfull = empty + F::kStages;
    uint64_t *pempty = pfull + F::kPSlots;
    uint64_t *qfull = pempty + F::kPSlots, *qempty = qfull + 4, *sfull = qempty + 2,
             *sfree = sfull + 2, *ofull = sfree + 2, *ofree = ofull + 2, *cleared = ofree + 2;
    float *row_scale = reinterpret_cast<float *>(smem + F::kRowOff);  // [4] score -> log2 weight
    int *row_lim = reinterpret_cast<int *>(row_scale + 4 * NR);       // [4] last position seen
    float *row_ref = reinterpret_cast<float *>(row_lim + 4 * NR);     // [2] reference (log2), by chunk
    float *row_fac = row_ref + 2 * NR;   // [2] exp2(old reference - new), by chunk
    float *row_neg = row_fac + 2 * NR;   // kPScale - reference
    float *row_top = row_neg + NR;       // running maximum
    float *row_red = row_top + NR;       // [8] maxima per softmax warp
    float *row_sum = row_red + 8 * NR;   // [2][8] sums per softmax warp, by chunk
    uint32_t *misc = reinterpret_cast<uint32_t *>(row_sum + 16 * NR);
    uint32_t *tmem_slot = misc;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    int *shared_last = reinterpret_cast<int *>(misc + 2);
    int *start_b = reinterpret_cast<int *>(misc + 3);
    int64_t *start_w = reinterpret_cast<int64_t *>(misc + 4);  // w0, w1, base, total
    int *parts = reinterpret_cast<int *>(misc + 12);           // CTAs that have a part

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    allow_dependent_launch();
    if (threadIdx.x == 0) {
        for (int i = 0; i < F::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 2);
            mbar_init(&cleared[i], 1);
        }
        for (int i = 0; i < F::kPSlots; ++i) {
            mbar_init(&pfull[i], 4);
            mbar_init(&pempty[i], 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&qfull[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qempty[i], 1);
            mbar_init(&sfull[i], 1);
            mbar_init(&sfree[i], kFewSoftmaxWarps);
            mbar_init(&ofull[i], 1);
            mbar_init(&ofree[i], kFewSoftmaxWarps);
        }
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    grid_dependency_wait();
    if (warp == 0) {
        // this CTA's part of the work list: lane l sums the costs of the l-th
        // run of sequences, then the lane whose run holds the first position finds it
        const int per = (a.B + 31) / 32, b0 = min(lane * per, a.B), b1 = min(b0 + per, a.B);
        int64_t mine = 0;
#pragma unroll 4
        for (int b = b0; b < b1; ++b) mine += head_cost(a, seq_tiles(seq_of(a, b)));
        mine *= a.kv_heads;
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += up;
        }
        const int64_t total = __shfl_sync(0xFFFFFFFFu, incl, 31);
        // no part is empty, so that a split (sequence, head) lies in consecutive CTAs
        const int64_t np = min(static_cast<int64_t>(gridDim.x), max(total, int64_t(1)));
        const int64_t w0 = min(blockIdx.x * total / np, total), w1 = min((blockIdx.x + 1) * total / np, total);
        if (w0 >= incl - mine && w0 < incl) {
            int64_t base = incl - mine;
            int b = b0;
            for (;; ++b) {
                const int64_t n = head_cost(a, seq_tiles(seq_of(a, b))) * a.kv_heads;
                if (w0 < base + n) break;
                base += n;
            }
            *start_b = b;
            start_w[2] = base;
        }
        if (lane == 0) {
            start_w[0] = w0;
            start_w[1] = w1;
            start_w[3] = total;
            *parts = static_cast<int>(np);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    Chunks<NR> cur(a, start_w[0], start_w[1], *start_b, start_w[2]);

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        Chunks<NR> ahead = cur;  // the chunk whose K comes next
        bool more = ahead.next();
        const uint64_t evict_first = l2_policy_evict_first();
        const int rows = min(1 << a.page_shift, kTile), boxes = kTile / rows;
        uint32_t stage = 0, phase = 0, issued = 0;
        bool ok = true;
        auto tiles = [&](const Chunks<NR> &c, const CUtensorMap *map) {
            PageWalk pages(a, c.b, c.seq.len, c.t * kTile);
            for (int t = c.t; t < c.t + c.n; ++t) {
                const int row = pages.row_of(a, t * kTile + min(lane, boxes - 1) * rows, status);
                ok = ok && mbar_wait(&empty[stage], phase ^ 1, abort_flag, status);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    return;
                }
                if (lane == 0) mbar_arrive_expect_tx(&full[stage], kStageBytes);
                __syncwarp();
                if (lane < boxes)
                    tma_load_2d_hint(smem + stage * kStageBytes + lane * rows * kDim, map,
                                     &full[stage], c.hk * kDim, row, evict_first);
                ++issued;
                if (++stage == F::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        };
        if (more) tiles(ahead, &tmap_k);
        while (ok && cur.next()) {
            more = ahead.next();
            if (more) tiles(ahead, &tmap_k);
            if (ok) tiles(cur, &tmap_v);
        }
        // no copy may be in flight when the CTA leaves
        const uint32_t from = issued > F::kStages ? issued - F::kStages : 0;
        for (uint32_t i = from; i < issued; ++i)
            mbar_wait(&full[i % F::kStages], (i / F::kStages) & 1, nullptr, status);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        Chunks<NR> ahead = cur;
        bool more = ahead.next();
        const uint32_t id_s = umma_idesc_e4m3(kTile, N), id_o = idesc_e4m3_mn(kDim, N);
        // descriptors: an address step of 16 bytes is 1
        const uint64_t ring_desc = umma_desc_sw128(smem_addr(smem)),
                       q_desc = umma_desc_sw128(smem_addr(smem + F::kQOff)),
                       p_desc = umma_desc_mn(smem_addr(smem + F::kPOff), kTile * 16, 128);
        uint32_t stage = 0, phase = 0;
        uint32_t pslot[2] = {0, 0}, pphase[2] = {0, 0};  // of each softmax group
        uint32_t gk = 0, gv = 0, segs = 0;  // chunks and segments so far
        uint32_t cphases = 0;               // bit i: phase of cleared[i]
        bool ok = true;
        auto advance = [&] {
            if (++stage == F::kStages) {
                stage = 0;
                phase ^= 1;
            }
        };
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            ok = ok && mbar_wait(bar, parity, abort_flag, status);
            ok = __all_sync(0xFFFFFFFFu, ok);
        };
        auto scores = [&](const Chunks<NR> &c) {
            if (c.first) {
                wait(&qfull[segs & 3], (segs >> 2) & 1);
                ++segs;
            }
            const uint32_t buf = gk & 1;
            wait(&sfree[buf], ((gk >> 1) & 1) ^ 1);
            const uint64_t q = q_desc + ((segs - 1) & 1) * (F::kQ / 16);
            for (int j = 0; j < c.n && ok; ++j) {
                wait(&full[stage], phase);
                if (!ok) break;
                tc_fence_after_sync();
                const uint64_t k = ring_desc + stage * (kStageBytes / 16);
                const uint32_t d = tmem + F::s_col(buf, j);
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < 4; ++s) umma_e4m3(d, k + 2 * s, q + 2 * s, id_s, s > 0 ? 1u : 0u);
                    umma_commit(&empty[stage]);
                    if (j == c.n - 1) {
                        umma_commit(&sfull[buf]);
                        if (c.last) umma_commit(&qempty[(segs - 1) & 1]);
                    }
                }
                __syncwarp();
                advance();
            }
            ++gk;
        };
        if (more) scores(ahead);
        while (ok && cur.next()) {
            more = ahead.next();
            if (more) scores(ahead);
            const uint32_t buf = gv & 1;
            wait(&ofree[buf], ((gv >> 1) & 1) ^ 1);
            for (int j = 0; j < cur.n && ok; ++j) {
                const int h = j & 1;
                const uint32_t slot = h * F::kGroupSlots + pslot[h];
                if ((cur.t + j + 1) * kTile > cur.seq.len) {
                    wait(&cleared[stage], (cphases >> stage) & 1);
                    cphases ^= 1u << stage;
                } else {
                    wait(&full[stage], phase);
                }
                wait(&pfull[slot], pphase[h]);
                if (!ok) break;
                tc_fence_after_sync();
                const uint64_t v = ring_desc + stage * (kStageBytes / 16), p = p_desc + slot * (F::kP / 16);
                const uint32_t d = tmem + F::o_col(buf), first = j > 0 ? 1u : 0u;
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < 4; ++s)  // 32 positions each
                        umma_e4m3(d, v + 2 * kDim * s, p + 32 * s, id_o, s > 0 ? 1u : first);
                    umma_commit(&empty[stage]);
                    umma_commit(&pempty[slot]);
                    if (j == cur.n - 1) umma_commit(&ofull[buf]);
                }
                __syncwarp();
                advance();
                if (++pslot[h] == F::kGroupSlots) {
                    pslot[h] = 0;
                    pphase[h] ^= 1;
                }
            }
            ++gv;
        }
    } else if (warp == 2 + kFewSoftmaxWarps) {
        // ------------------------------------------------------------ queries
        // two E4M3 parts per row, K-major with the 128-byte swizzle; rows behind
        // the segment's are zeros
        const int sub = lane & 15, G = a.group;
        uint32_t segs = 0;
        bool ok = true;
        while (ok && cur.next()) {
            if (!cur.first) continue;
            const uint32_t rb = (segs & 3) * NR;
            const int rows = cur.seq.q_len * G;
            uint4 v[NR / 2];
#pragma unroll
            for (int i = 0; i < NR / 2; ++i) {
                const int r = 2 * i + (lane >> 4);
                v[i] = make_uint4(0, 0, 0, 0);
                if (r < rows) {
                    const int tok = r / G, g = r - tok * G;
                    v[i] = *reinterpret_cast<const uint4 *>(
                        a.q + (cur.seq.q0 + tok) * a.q_stride +
                        static_cast<int64_t>(cur.hk * G + g) * kDim + sub * 8);
                }
            }
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(&qempty[segs & 1], ((segs >> 1) & 1) ^ 1, abort_flag, status));
            uint8_t *dst = smem + F::kQOff + (segs & 1) * F::kQ;
            // not unrolled (the rows move down the array instead): unrolled, the
            // first pass over this code fetched it for 4 us before the first MMA
#pragma unroll 1
            for (int i = 0; i < NR / 2; ++i) {
                const int r = 2 * i + (lane >> 4);
                const uint4 u = v[0];
#pragma unroll
                for (int k = 0; k + 1 < NR / 2; ++k) v[k] = v[k + 1];
                uint32_t m = amax_bits8(u);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                // power of two that takes the largest channel to [128, 256)
                const int e = max(static_cast<int>(m >> 7) - 127, -100);
                const float up = __uint_as_float(static_cast<uint32_t>(7 - e + 127) << 23);
                uint2 hi, lo;
                split8_scaled(u, up, hi, lo);
                // rows r and NR + r have the same place in their 8-row swizzle group
                const int off = r * kDim + (((sub >> 1) ^ (r & 7)) << 4) + (sub & 1) * 8;
                *reinterpret_cast<uint2 *>(dst + off) = hi;
                *reinterpret_cast<uint2 *>(dst + NR * kDim + off) = lo;
                if (sub == 0) {
                    row_scale[rb + r] = fmaxf(
                        a.scale * 1.4426950408889634f * __uint_as_float(static_cast<uint32_t>(e - 7 + 127) << 23),
                        kMinScale);
                    row_lim[rb + r] = a.causal
                                          ? min(cur.seq.len - cur.seq.q_real + r / G, cur.seq.len - 1)
                                          : cur.seq.len - 1;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&qfull[segs & 3]);
            ++segs;
        }
    } else if (warp == 3 + kFewSoftmaxWarps) {
        // ------------------------------------------------------------ ends of sequences
        // What a page holds behind the end of its sequence may be NaN, which a
        // weight of 0 would not silence: those rows of V become zeros as soon as they are
        // there.  This warp takes part in every slot's release, so that it sees each
        // of the ring's tiles.
        Chunks<NR> ahead = cur;
        bool more = ahead.next();
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        auto follow = [&](const Chunks<NR> &c, bool v) {
            for (int t = c.t; t < c.t + c.n && ok; ++t) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[stage], phase, abort_flag, status));
                if (!ok) return;
                const int from = c.seq.len - t * kTile;  // first row behind the end
                if (v && from < kTile) {
                    uint4 *z = reinterpret_cast<uint4 *>(smem + stage * kStageBytes);
                    for (int i = from * 8 + lane; i < kTile * 8; i += 32) z[i] = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&cleared[stage]);
                }
                if (lane == 0) mbar_arrive(&empty[stage]);
                if (++stage == F::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        };
        if (more) follow(ahead, false);
        while (ok && cur.next()) {
            more = ahead.next();
            if (more) follow(ahead, false);
            follow(cur, true);
        }
    } else {
        // ------------------------------------------------------------ softmax
        // A wait that gives up sets the abort flag: the loops then run to their
        // end without waiting, so that every barrier still has all its warps.
        constexpr int kThreads = 32 * kFewSoftmaxWarps;
        constexpr int kHalf = NR / 2;  // rows of a thread in the merge
        const int sw = warp - 2, st = threadIdx.x - 64;
        const int group = sw >> 2, quarter = warp & 3;
        const int lane_row = quarter * 32 + lane;  // position in a tile, channel of an output
        const uint32_t tm = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const int G = a.group;

        // sequences without positions, and reports: a warp per sequence
        for (int b = blockIdx.x + sw * gridDim.x; b < a.B; b += kFewSoftmaxWarps * gridDim.x) {
            if (lane == 0 && seq_is_bad(a, b)) atomicExch(status, 8 /* FP8BQ_ERR_INDEX */);
            const Seq s = seq_of(a, b);
            if (s.len > 0) continue;
            for (int i = 0; i < s.q_len; ++i) {
                const int64_t row = s.q0 + i;
                uint4 *o = reinterpret_cast<uint4 *>(a.out + row * a.out_stride);
                for (int c = lane; c < a.q_heads * (kDim / 8); c += 32) o[c] = make_uint4(0, 0, 0, 0);
                if (a.lse != nullptr)
                    for (int h = lane; h < a.q_heads; h += 32) a.lse[row * a.q_heads + h] = -INFINITY;
            }
        }

        float l_run[NR];     // sums over this thread's positions
        float o_run[kHalf];  // this thread's channel of rows group * kHalf ...
        uint32_t g = 0, segs = 0, pslot = 0, pphase = 0;
        // what the merge and the end of a segment need of the chunk before
        struct {
            int q0, hk, rows, tiles, seg_t0, seg_end;
            int64_t item;
            bool first, last;
        } prev;

        // Row r of a segment is token r / G, query head hk G + r % G.
        auto out_at = [&](int r) {
            const int i = r / G;
            return a.out + (prev.q0 + i) * a.out_stride +
                   static_cast<int64_t>(prev.hk * G + r - i * G) * kDim;
        };
        auto store_lse = [&](int r, float m, float l) {
            const int i = r / G;
            a.lse[static_cast<int64_t>(prev.q0 + i) * a.q_heads + prev.hk * G + r - i * G] =
                l > 0.0f ? (m - kPScale + log2f(l)) * 0.69314718055994531f : -INFINITY;
        };

        // O^T of chunk `c` into o_run; at the end of its segment, its output
        auto merge = [&](uint32_t c) {
            const uint32_t buf = c & 1;
            float hi[kHalf], lo[kHalf];
            mbar_wait(&ofull[buf], (c >> 1) & 1, abort_flag, status);
            tc_fence_after_sync();
            tmem_ld<kHalf>(tm + F::o_col(buf) + group * kHalf, hi);
            tmem_ld<kHalf>(tm + F::o_col(buf) + NR + group * kHalf, lo);
            tmem_ld_wait<kHalf>(hi);
            tmem_ld_wait<kHalf>(lo);
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ofree[buf]);
#pragma unroll
            for (int k = 0; k < kHalf; ++k) {
                const float o = fmaf(lo[k], 1.0f / kLoScale, hi[k]);
                o_run[k] = prev.first ? o : fmaf(o_run[k], row_fac[buf * NR + group * kHalf + k], o);
            }
            if (!prev.last) return;
            const int rows = prev.rows;
            const float *m_row = row_ref + buf * NR, *sums = row_sum + buf * 8 * NR;
            auto total = [&](int r) {
                float l = 0.0f;
#pragma unroll
                for (int w = 0; w < kFewSoftmaxWarps; ++w) l += sums[w * NR + r];
                return l;
            };
            if (prev.seg_t0 == 0 && prev.seg_end == prev.tiles) {
#pragma unroll
                for (int k = 0; k < kHalf; ++k) {
                    const int r = group * kHalf + k;
                    if (r >= rows) break;
                    const float l = total(r);
                    out_at(r)[lane_row] = __bfloat16_as_ushort(
                        __float2bfloat16_rn(l > 0.0f ? __fdividef(o_run[k], l) : 0.0f));
                }
                if (a.lse != nullptr && st < rows) store_lse(st, m_row[st], total(st));
                return;
            }
            // partial: this CTA's slot 1 if the (sequence, head) begins here, else slot 0
            const int64_t all = start_w[3], w_first = prev.item, w_last = w_first + prev.tiles - 1;
            auto owner = [&](int64_t w) { return static_cast<int>(((w + 1) * *parts - 1) / all); };
            const int c_first = owner(w_first), c_last = owner(w_last);
            auto slot = [&](int i) {
                return partials + static_cast<int64_t>(2 * i + (i == c_first ? 1 : 0)) * F::kPartial;
            };
            float *mine = slot(blockIdx.x);
#pragma unroll
            for (int k = 0; k < kHalf; ++k) {
                const int r = group * kHalf + k;
                if (r >= rows) break;
                __stcg(mine + r * kDim + lane_row, o_run[k]);
            }
            if (st < rows) {
                __stcg(mine + NR * kDim + st, m_row[st]);
                __stcg(mine + NR * kDim + NR + st, total(st));
            }
            __threadfence();
            named_barrier(1, kThreads);
            if (st == 0) {
                const int seen = atomicAdd(counters + c_first, 1);
                *shared_last = seen == c_last - c_first;
                if (*shared_last) counters[c_first] = 0;
                __threadfence();
            }
            named_barrier(1, kThreads);
            if (!*shared_last) return;
            // join in the order of the CTAs: a warp per row, 4 channels per lane;
            // 32 CTAs' maxima and sums at a time, one per lane
            for (int r = sw; r < rows; r += kFewSoftmaxWarps) {
                float m = -INFINITY, l = 0.0f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int i0 = c_first; i0 <= c_last; i0 += 32) {
                    const int n = min(32, c_last - i0 + 1);
                    const float *p = slot(min(i0 + lane, c_last)) + NR * kDim + r;
                    float mi = lane < n ? __ldcg(p) : -INFINITY;
                    const float li = lane < n ? __ldcg(p + NR) : 0.0f;
                    const float m2 = fmaxf(m, warp_max(mi));
                    if (m2 == -INFINITY) continue;
                    const float f_old = ex2(m - m2), f = ex2(mi - m2);
                    m = m2;
                    float part = li * f;
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, d);
                    l = fmaf(l, f_old, part);
                    o = make_float4(o.x * f_old, o.y * f_old, o.z * f_old, o.w * f_old);
                    for (int i = 0; i < n; i += 8) {
                        float4 v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            v[k] = __ldcg(reinterpret_cast<const float4 *>(slot(i0 + min(i + k, n - 1)) + r * kDim) + lane);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float fi = i + k < n ? __shfl_sync(0xFFFFFFFFu, f, i + k) : 0.0f;
                            o.x = fmaf(fi, v[k].x, o.x);
                            o.y = fmaf(fi, v[k].y, o.y);
                            o.z = fmaf(fi, v[k].z, o.z);
                            o.w = fmaf(fi, v[k].w, o.w);
                        }
                    }
                }
                const float inv = l > 0.0f ? __fdividef(1.0f, l) : 0.0f;
                *reinterpret_cast<uint2 *>(out_at(r) + lane * 4) =
                    make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
                if (a.lse != nullptr && lane == 0) store_lse(r, m, l);
            }
        };

        while (cur.next()) {
            const uint32_t buf = g & 1;
            const int rows = cur.seq.q_len * G, len = cur.seq.len;
            if (cur.first) {
                mbar_wait(&qfull[segs & 3], (segs >> 2) & 1, abort_flag, status);
                ++segs;
            }
            const float *scale = row_scale + ((segs - 1) & 3) * NR;
            const int *limit = row_lim + ((segs - 1) & 3) * NR;
            // positions that every row sees; later ones are masked somewhere
            const int all_see = a.causal ? len - cur.seq.q_real : len - 1;
            mbar_wait(&sfull[buf], (g >> 1) & 1, abort_flag, status);
            tc_fence_after_sync();

            // scores of tile j: hi + lo / 32
            auto load_scores = [&](int j, auto &v) {
                float lo[NR];
                tmem_ld<NR>(tm + F::s_col(buf, j), v);
                tmem_ld<NR>(tm + F::s_col(buf, j) + NR, lo);
                tmem_ld_wait<NR>(v);
                tmem_ld_wait<NR>(lo);
#pragma unroll
                for (int r = 0; r < NR; ++r) v[r] = fmaf(lo[r], 1.0f / kLoScale, v[r]);
            };

            // pass 1: the chunk's maximum of every row
            float mx[NR];
#pragma unroll
            for (int r = 0; r < NR; ++r) mx[r] = -INFINITY;
            for (int j = group; j < cur.n; j += 2) {
                const int pos = (cur.t + j) * kTile + lane_row;
                float v[NR];
                load_scores(j, v);
                if ((cur.t + j) * kTile + kTile - 1 <= all_see) {
#pragma unroll
                    for (int r = 0; r < NR; ++r) mx[r] = fmaxf(mx[r], v[r]);
                } else {
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        if (pos <= limit[r]) mx[r] = fmaxf(mx[r], v[r]);
                }
            }
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float m = warp_max(mx[r]);
                if (lane == 0) row_red[sw * NR + r] = m;
            }
            named_barrier(1, kThreads);
            if (st < NR) {
                float m = row_red[st];
#pragma unroll
                for (int w = 1; w < kFewSoftmaxWarps; ++w) m = fmaxf(m, row_red[w * NR + st]);
                m *= scale[st];  // -inf stays: nothing of the chunk is seen
                const float old = cur.first ? -INFINITY : row_ref[(buf ^ 1) * NR + st];
                const float top = cur.first ? m : fmaxf(m, row_top[st]);
                m = fmaxf(m, top - kFarBelow);
                row_top[st] = top;
                row_ref[buf * NR + st] = m;
                row_neg[st] = m == -INFINITY ? 0.0f : kPScale - m;
                row_fac[buf * NR + st] = m == -INFINITY ? 1.0f : ex2(old - m);
            }
            named_barrier(1, kThreads);
#pragma unroll
            for (int r = 0; r < NR; ++r) l_run[r] = cur.first ? 0.0f : l_run[r] * row_fac[buf * NR + r];

            // pass 2: weights, two E4M3 parts, P[position][hi rows, lo rows]
            for (int j = group; j < cur.n; j += 2) {
                const int pos = (cur.t + j) * kTile + lane_row;
                float v[NR];
                load_scores(j, v);
#pragma unroll
                for (int r = 0; r < NR; ++r) v[r] = ex2(fmaf(v[r], scale[r], row_neg[r]));
                if ((cur.t + j) * kTile + kTile - 1 > all_see) {
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        if (pos > limit[r]) v[r] = 0.0f;
                }
                uint32_t hi[NR / 4], lo[NR / 4];
#pragma unroll
                for (int r = 0; r < NR; r += 4) {
                    const uint16_t h0 = e4m3x2_satfinite(v[r], v[r + 1]);
                    const uint16_t h1 = e4m3x2_satfinite(v[r + 2], v[r + 3]);
                    const float2 d0 = e4m3x2_to_neg_scaled(h0), d1 = e4m3x2_to_neg_scaled(h1);
                    hi[r / 4] = h0 | (static_cast<uint32_t>(h1) << 16);
                    lo[r / 4] = e4m3x2_satfinite(fmaf(v[r], kLoScale, d0.x), fmaf(v[r + 1], kLoScale, d0.y)) |
                                (static_cast<uint32_t>(e4m3x2_satfinite(fmaf(v[r + 2], kLoScale, d1.x),
                                                                        fmaf(v[r + 3], kLoScale, d1.y)))
                                 << 16);
                }
#pragma unroll
                for (int r = 0; r < NR; ++r) l_run[r] += v[r];
                const uint32_t slot = group * F::kGroupSlots + pslot;
                mbar_wait(&pempty[slot], pphase ^ 1, abort_flag, status);
                uint4 *p = reinterpret_cast<uint4 *>(smem + F::kPOff + slot * F::kP) + lane_row;
                if constexpr (NR == 8) {
                    *p = make_uint4(hi[0], hi[1], lo[0], lo[1]);
                } else {
                    p[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    p[kTile] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[slot]);
                if (++pslot == F::kGroupSlots) {
                    pslot = 0;
                    pphase ^= 1;
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sfree[buf]);
            if (cur.last) {
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    float l = l_run[r];
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
                    if (lane == 0) row_sum[(buf * 8 + sw) * NR + r] = l;
                }
            }
            if (g > 0) merge(g - 1);
            prev.q0 = cur.seq.q0;
            prev.hk = cur.hk;
            prev.rows = rows;
            prev.tiles = cur.tiles;
            prev.seg_t0 = cur.seg_t0;
            prev.seg_end = cur.seg_end;
            prev.item = cur.item();
            prev.first = cur.first;
            prev.last = cur.last;
            ++g;
        }
        named_barrier(1, kThreads);  // row_sum of the last chunk
        if (g > 0) merge(g - 1);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace attn
}  // namespace fp8bq
