// attention_few.cuh -- paged attention for few query rows per kv head (decode,
// a drafter's block): q_len * group <= N rows, N = 16, 32 or 64.
//
// Bound by the cache's bytes: 256 per position and kv head, read once.  The
// E4M3 codes go from HBM to shared memory by TMA and from there straight into
// the tensor cores, with the roles of rows and columns swapped: 128 cache
// positions are the MMA's M, the query rows its N.
//     S^T[pos, row] = K[pos, :] . Q[row, :]       M = 128, N rows, K = 128
//     O^T[ch, row] += V[:, ch]^T . P[:, row]      M = 128, N rows, K = 128 positions
// Neither K nor V is ever converted: V is the A operand with its channels
// contiguous.  Queries and weights keep their precision as two E4M3 parts,
// x = hi + lo (two MMAs into one accumulator): hi holds 4 significant bits, lo
// the next 4, so a BF16 query is exact down to 2^-9 of its row's largest
// channel (rows are scaled by a power of two to [128, 256)), and a weight p
// (scaled by 256) has 8 bits down to 2^-10 of the largest and an absolute
// error of 2^-18 below.  At N = 16 the two MMAs per tile take a small part of
// the time that a 16 KB tile needs to arrive (0.37 us per SM at 6.5 TB/s).
//
// Work is a list of tiles of 128 positions, ordered by (sequence, kv head,
// tile); CTA c of a grid of one CTA per SM takes the c-th equal part, whatever
// the sequences' lengths.  A part's tiles of one (sequence, head), its segment,
// are taken in chunks of at most kChunk tiles, as many as TMEM holds scores
// for (twice): a chunk's scores are all there before its softmax, so no output
// is ever rescaled in TMEM; the chunk's O^T is merged into registers with the
// usual factor exp(m_old - m_new).  The ring carries K of chunk g + 1 ahead of V of
// chunk g, so the next scores are computed while the softmax works.
// A (sequence, head) that lies in several CTAs leaves FP32 partials and
// maxima in the workspace; the last CTA to arrive (a counter) joins them in
// the order of the CTAs, so results do not depend on timing.
//
// Roles: warp 0 TMA producer (a page per lane), warp 1 MMA issuer, warps 2..5
// softmax: thread = one position of the tile (its TMEM lane) in the score
// phase, one output channel in the merge.
#pragma once

#include "attention.cuh"
#include "gemm_decode.cuh"
#include "rms_norm.cuh"

namespace fp8bq {
namespace attn {

constexpr int kTile = 128;                 // positions
constexpr int kStageBytes = kTile * kDim;  // one K or V tile of codes
constexpr int kFewThreads = 192;
constexpr float kPScale = 8.0f;            // weights are held times 2^8

template <int N>
struct Few {
    static constexpr int kChunk = 256 / N - 1;  // tiles; 2 chunks + 2 outputs = 512 columns
    static constexpr int kQ = N * kDim;         // bytes of one part of Q
    static constexpr int kP = N * kTile;        // bytes of one part of P
    static constexpr int kPSlots = N == 64 ? 2 : 4;
    static constexpr int kStages = N == 64 ? 9 : N == 32 ? 10 : 12;
    static constexpr int kQOff = kStages * kStageBytes;          // [2 buffers][hi, lo]
    static constexpr int kPOff = kQOff + 2 * 2 * kQ;             // [kPSlots][hi, lo]
    static constexpr int kBarOff = kPOff + kPSlots * 2 * kP;
    // full, empty; pfull, pempty; qfull, sfull, sfree, ofull, ofree (two each); vready
    static constexpr int kBars = 2 * kStages + 2 * kPSlots + 11;
    static constexpr int kRowOff = kBarOff + kBars * 8;  // per-row values
    static constexpr int kBytes = kRowOff + (2 + 2 + 4 + 1 + 1 + 4 + 2) * N * 4 + 64 + 1024;
    static_assert(kBytes <= 227 * 1024, "shared memory");
    static_assert(kQOff % 1024 == 0 && kPOff % 1024 == 0 && kQ % 1024 == 0 && kP % 1024 == 0,
                  "swizzled tiles");
    static constexpr int kPartial = N * (kDim + 2);  // floats: O [N][128], max [N], sum [N]
    __device__ static uint32_t s_col(int buf, int j) { return (buf * kChunk + j) * N; }
    __device__ static uint32_t o_col(int buf) { return (2 * kChunk + buf) * N; }
};

// idesc of E4M3 x E4M3 with the A operand's M dimension contiguous
__host__ __device__ constexpr uint32_t idesc_e4m3_a_mn(int m, int n) {
    return umma_idesc_e4m3(m, n) | (1u << 15);
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

// Two E4M3 codes -> two floats (exact).
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t c) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h2));
}

// A sequence as the kernels take it: lengths that the host cannot check are
// clamped (seq_check reports them).
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
    const int q1 = __ldg(a.cu_q + b + 1);
    s.q_real = max(q1 - s.q0, 0);
    s.q_len = min(min(s.q_real, T - s.q0), a.max_q);
    return s;
}

__device__ __forceinline__ bool seq_is_bad(const Args &a, int b) {
    const int len = __ldg(a.seq_lens + b), q0 = __ldg(a.cu_q + b), q1 = __ldg(a.cu_q + b + 1);
    return len < 0 || len > (a.max_pages << a.page_shift) || q0 < 0 || q1 < q0 || q1 > a.T ||
           q1 - q0 > a.max_q;
}

__device__ __forceinline__ int seq_tiles(const Seq &s) {
    return s.q_len > 0 ? (s.len + kTile - 1) / kTile : 0;
}

// Row of the cache where page `idx` of sequence b starts, or -kTile (a row
// outside the cache: TMA fills zeros) for a page it does not need or that is
// not in the cache.
__device__ __forceinline__ int page_row(const Args &a, int b, int idx, int len, int *status) {
    if ((static_cast<int64_t>(idx) << a.page_shift) >= len) return -kTile;
    const int32_t page = __ldg(a.table + b * a.table_stride + idx);
    if (page < 0 || page >= a.num_pages) {
        atomicExch(status, 8 /* FP8BQ_ERR_INDEX */);
        return -kTile;
    }
    return page << a.page_shift;
}

// The chunks of one CTA's part of the tile list, in order.
template <int N>
struct Chunks {
    const Args &a;
    int64_t w, w_end, base;  // next tile, end of the part, first tile of sequence b
    int b, tiles;            // sequence of w, its tiles per head
    Seq seq;
    // the current chunk
    int hk, t, n;            // kv head, first tile, tiles
    int seg_t0, seg_end;     // tiles of the segment
    bool first, last;        // of its segment

    __device__ Chunks(const Args &args, int64_t w0, int64_t w1, int b0, int64_t base0)
        : a(args), w(w0), w_end(w1), base(base0), b(b0), tiles(0), seg_end(0) {
        t = n = 0;
        if (w < w_end) {
            seq = seq_of(a, b);
            tiles = seq_tiles(seq);
        }
    }
    __device__ bool next() {
        t += n;
        if (t >= seg_end) {  // a new segment
            if (w >= w_end) return false;
            while (w >= base + static_cast<int64_t>(tiles) * a.kv_heads) {
                base += static_cast<int64_t>(tiles) * a.kv_heads;
                seq = seq_of(a, ++b);
                tiles = seq_tiles(seq);
            }
            const int rel = static_cast<int>(w - base);
            hk = rel / tiles;
            t = seg_t0 = rel - hk * tiles;
            seg_end = static_cast<int>(min(static_cast<int64_t>(tiles), t + (w_end - w)));
            w += seg_end - t;
        }
        first = t == seg_t0;
        // equal chunks, so that no segment ends in a short one
        const int total = seg_end - seg_t0;
        const int parts = (total + Few<N>::kChunk - 1) / Few<N>::kChunk;
        n = min((total + parts - 1) / parts, seg_end - t);
        last = t + n == seg_end;
        return true;
    }
    // the list's first tile of the current (sequence, head)
    __device__ int64_t item() const { return base + static_cast<int64_t>(hk) * tiles; }
};

template <int N>
__global__ void __launch_bounds__(kFewThreads, 1)
attention_few_kernel(const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const Args a, int *counters,
                     float *partials, int *status) {
    using F = Few<N>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + F::kBarOff);
    uint64_t *empty = full + F::kStages;
    uint64_t *pfull = empty + F::kStages;
    uint64_t *pempty = pfull + F::kPSlots;
    uint64_t *qfull = pempty + F::kPSlots, *sfull = qfull + 2, *sfree = sfull + 2,
             *ofull = sfree + 2, *ofree = ofull + 2, *vready = ofree + 2;
    float *row_scale = reinterpret_cast<float *>(smem + F::kRowOff);  // [2][N] score -> log2 weight
    float *row_max = row_scale + 2 * N;    // [2][N] running maximum (log2), by chunk parity
    float *row_red = row_max + 2 * N;      // [4][N] per softmax warp
    float *row_neg = row_red + 4 * N;      // [N] kPScale - maximum
    float *row_fac = row_neg + N;          // [N] exp2(old maximum - new)
    float *row_sum = row_fac + N;          // [4][N] sums per softmax warp
    int *row_lim = reinterpret_cast<int *>(row_sum + 4 * N);  // [2][N] last position a row sees
    uint32_t *misc = reinterpret_cast<uint32_t *>(row_lim + 2 * N);
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
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < F::kPSlots; ++i) {
            mbar_init(&pfull[i], 4);
            mbar_init(&pempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qfull[i], 4);
            mbar_init(&sfull[i], 1);
            mbar_init(&sfree[i], 4);
            mbar_init(&ofull[i], 1);
            mbar_init(&ofree[i], 4);
        }
        mbar_init(vready, 1);
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
        // this CTA's part of the tile list: lane l sums the tiles of the l-th
        // run of sequences, then the lane whose run holds the first tile finds it
        const int per = (a.B + 31) / 32, b0 = min(lane * per, a.B), b1 = min(b0 + per, a.B);
        int64_t mine = 0;
        for (int b = b0; b < b1; ++b) mine += seq_tiles(seq_of(a, b));
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
                const int64_t n = static_cast<int64_t>(seq_tiles(seq_of(a, b))) * a.kv_heads;
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
    Chunks<N> ahead(a, start_w[0], start_w[1], *start_b, start_w[2]);
    Chunks<N> cur(a, start_w[0], start_w[1], *start_b, start_w[2]);
    bool more = ahead.next();  // the chunk whose K comes next

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        const uint64_t evict_first = l2_policy_evict_first();
        const int page = 1 << a.page_shift;
        const int rows = min(page, kTile), boxes = kTile / rows;
        uint32_t stage = 0, phase = 0, issued = 0;
        bool ok = true;
        auto tiles = [&](const Chunks<N> &c, const CUtensorMap *map) {
            // the next tile's page while this one waits for its slot
            auto row_at = [&](int t) {
                if (lane >= boxes || t >= c.t + c.n) return -kTile;
                const int pos = t * kTile + lane * rows;
                const int r = page_row(a, c.b, pos >> a.page_shift, c.seq.len, status);
                return r < 0 ? r : r + (pos & (page - 1));
            };
            int row = row_at(c.t);
            for (int t = c.t; t < c.t + c.n; ++t) {
                const int next_row = row_at(t + 1);
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
                row = next_row;
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
        if (lane == 0) {
            const uint32_t id_s = umma_idesc_e4m3(kTile, N), id_o = idesc_e4m3_a_mn(kDim, N);
            uint32_t stage = 0, phase = 0, pslot = 0, pphase = 0;
            uint32_t gk = 0, gv = 0, segs = 0;  // chunks and segments so far
            bool ok = true;
            auto advance = [&] {
                if (++stage == F::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            };
            auto scores = [&](const Chunks<N> &c) {
                if (c.first) {
                    ok = ok && mbar_wait(&qfull[segs & 1], (segs >> 1) & 1, abort_flag, status);
                    ++segs;
                }
                const uint32_t buf = gk & 1;
                ok = ok && mbar_wait(&sfree[buf], ((gk >> 1) & 1) ^ 1, abort_flag, status);
                const uint32_t q = smem_addr(smem + F::kQOff + ((segs - 1) & 1) * 2 * F::kQ);
                for (int j = 0; j < c.n && ok; ++j) {
                    ok = mbar_wait(&full[stage], phase, abort_flag, status);
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint32_t k = smem_addr(smem + stage * kStageBytes);
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            umma_e4m3(tmem + F::s_col(buf, j), umma_desc_sw128(k + 32 * s),
                                      umma_desc_sw128(q + part * F::kQ + 32 * s), id_s,
                                      part + s > 0 ? 1u : 0u);
                    umma_commit(&empty[stage]);
                    advance();
                }
                if (ok) umma_commit(&sfull[buf]);
                ++gk;
            };
            if (more) scores(ahead);
            while (ok && cur.next()) {
                more = ahead.next();
                if (more) scores(ahead);
                const uint32_t buf = gv & 1;
                ok = ok && mbar_wait(&ofree[buf], ((gv >> 1) & 1) ^ 1, abort_flag, status);
                for (int j = 0; j < cur.n && ok; ++j) {
                    ok = mbar_wait(&full[stage], phase, abort_flag, status);
                    // the sequence ends in this tile: the softmax warps clear what is behind
                    if (ok && (cur.t + j + 1) * kTile > cur.seq.len) mbar_arrive(vready);
                    ok = ok && mbar_wait(&pfull[pslot], pphase, abort_flag, status);
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint32_t v = smem_addr(smem + stage * kStageBytes);
                    const uint32_t p = smem_addr(smem + F::kPOff + pslot * 2 * F::kP);
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int s = 0; s < 4; ++s)  // 32 positions each
                            umma_e4m3(tmem + F::o_col(buf), umma_desc_sw128(v + 32 * kDim * s),
                                      umma_desc_sw128(p + part * F::kP + 32 * s), id_o,
                                      j + part + s > 0 ? 1u : 0u);
                    umma_commit(&empty[stage]);
                    umma_commit(&pempty[pslot]);
                    advance();
                    if (++pslot == F::kPSlots) {
                        pslot = 0;
                        pphase ^= 1;
                    }
                }
                if (ok) umma_commit(&ofull[buf]);
                ++gv;
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        // A wait that gives up sets the abort flag: the loops then run to their
        // end without waiting, so that every barrier still has all its warps.
        const int sw = warp - 2, st = threadIdx.x - 64;
        const int quarter = warp & 3;
        const int lane_row = quarter * 32 + lane;  // position in a tile, channel of an output
        const uint32_t tm = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const int G = a.group;

        // sequences without positions, and reports
        for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
            if (st == 0 && seq_is_bad(a, b)) atomicExch(status, 8 /* FP8BQ_ERR_INDEX */);
            const Seq s = seq_of(a, b);
            if (s.len > 0) continue;
            const int64_t width = static_cast<int64_t>(a.q_heads) * kDim;
            for (int64_t i = st; i < s.q_len * width; i += 128)
                a.out[(s.q0 + i / width) * a.out_stride + i % width] = 0;
            if (a.lse != nullptr)
                for (int i = st; i < s.q_len * a.q_heads; i += 128)
                    a.lse[static_cast<int64_t>(s.q0) * a.q_heads + i] = -INFINITY;
        }

        // Q of a segment: two E4M3 parts per row, K-major with the 128-byte swizzle
        uint32_t qsegs = 0;
        auto load_q = [&](const Chunks<N> &c) {
            uint8_t *dst = smem + F::kQOff + (qsegs & 1) * 2 * F::kQ;
            const int rows = c.seq.q_len * G;
            const int sub = st & 15;
            for (int r = st >> 4; r < N; r += 8) {
                float f[8];
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r < rows) {
                    const int i = r / G, g = r - i * G;
                    v = *reinterpret_cast<const uint4 *>(
                        a.q + (c.seq.q0 + i) * a.q_stride +
                        static_cast<int64_t>(c.hk * G + g) * kDim + sub * 8);
                }
                uint32_t m = amax_bits8(v);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                // power of two that takes the largest channel to [128, 256)
                const int e = max(static_cast<int>(m >> 7) - 127, -100);
                const float up = __uint_as_float(static_cast<uint32_t>(7 - e + 127) << 23);
                unpack_bf16x8(v, f);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float x = f[2 * k] * up, y = f[2 * k + 1] * up;
                    const uint16_t h = e4m3x2_satfinite(x, y);
                    const float2 d = e4m3x2_to_float2(h);
                    hi[k] = h;
                    lo[k] = e4m3x2_satfinite(x - d.x, y - d.y);
                }
                const int off = r * kDim + (((sub >> 1) ^ (r & 7)) << 4) + (sub & 1) * 8;
                *reinterpret_cast<uint2 *>(dst + off) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
                *reinterpret_cast<uint2 *>(dst + F::kQ + off) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
                if (sub == 0) {
                    row_scale[(qsegs & 1) * N + r] =
                        a.scale * 1.4426950408889634f * __uint_as_float(static_cast<uint32_t>(e - 7 + 127) << 23);
                    row_lim[(qsegs & 1) * N + r] =
                        a.causal ? min(c.seq.len - c.seq.q_real + r / G, c.seq.len - 1) : c.seq.len - 1;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&qfull[qsegs & 1]);
            ++qsegs;
        };

        float o_run[N], l_run[N];  // this thread's channel; this thread's positions
        uint32_t g = 0, pslot = 0, pphase = 0, segs = 0;
        uint32_t vstage = 0;            // ring stage of the next V tile
        uint32_t ragged = 0;            // tiles with an end so far
        int rows = 0;

        bool fresh = true;  // o_run holds nothing of the segment yet
        auto merge = [&](uint32_t chunk) {  // O^T of a chunk into o_run
            const uint32_t buf = chunk & 1;
            mbar_wait(&ofull[buf], (chunk >> 1) & 1, abort_flag, status);
            tc_fence_after_sync();
#pragma unroll
            for (int c = 0; c < N; c += 16) {
                if (c >= rows) break;
                float v[16];
                tmem_load16(tm + F::o_col(buf) + c, v);
#pragma unroll
                for (int k = 0; k < 16; ++k) o_run[c + k] = fresh ? v[k] : o_run[c + k] + v[k];
            }
            fresh = false;
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ofree[buf]);
        };

        if (more) {
            load_q(ahead);
            vstage = ahead.n % F::kStages;
        }
        named_barrier(1, 128);
        while (cur.next()) {
            more = ahead.next();
            if (more) {
                if (ahead.first) load_q(ahead);
                vstage = (vstage + ahead.n) % F::kStages;  // V of this chunk follows K of the next
            }
            if (cur.first) {
                rows = cur.seq.q_len * G;
                ++segs;
            }
            const float *scale = row_scale + ((segs - 1) & 1) * N;
            const int *limit = row_lim + ((segs - 1) & 1) * N;
            const uint32_t buf = g & 1;
            // the first new token's last position: later ones are masked somewhere
            const int q_real = cur.seq.q_real, len = cur.seq.len;
            const int all_see = a.causal ? len - q_real : len - 1;
            mbar_wait(&sfull[buf], (g >> 1) & 1, abort_flag, status);
            tc_fence_after_sync();
            // pass 1: the chunk's maximum of every row
            float mx[N];
#pragma unroll
            for (int r = 0; r < N; ++r) mx[r] = -INFINITY;
            for (int j = 0; j < cur.n; ++j) {
                const int pos = (cur.t + j) * kTile + lane_row;
                const bool plain = (cur.t + j) * kTile + kTile - 1 <= all_see;
#pragma unroll
                for (int c = 0; c < N; c += 16) {
                    if (c >= rows) break;
                    float v[16];
                    tmem_load16(tm + F::s_col(buf, j) + c, v);
                    if (plain) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) mx[c + k] = fmaxf(mx[c + k], v[k]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            if (pos <= limit[c + k]) mx[c + k] = fmaxf(mx[c + k], v[k]);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < N; ++r) {
                if (r >= rows) break;
                const float m = warp_max(mx[r]);
                if (lane == 0) row_red[sw * N + r] = m;
            }
            named_barrier(1, 128);
            if (st < rows) {
                float m = fmaxf(fmaxf(row_red[st], row_red[N + st]),
                                fmaxf(row_red[2 * N + st], row_red[3 * N + st]));
                m *= scale[st];  // -inf stays: nothing of the chunk is seen
                const float old = cur.first ? -INFINITY : row_max[(buf ^ 1) * N + st];
                m = fmaxf(m, old);
                row_max[buf * N + st] = m;
                row_neg[st] = m == -INFINITY ? 0.0f : kPScale - m;
                row_fac[st] = m == -INFINITY ? 1.0f : ex2(old - m);
            }
            named_barrier(1, 128);
            // the previous chunk's output, in the scale of its maximum, then both
            // (and the sums) in the scale of this one's
            if (cur.first) {
                fresh = true;
#pragma unroll
                for (int r = 0; r < N; ++r) l_run[r] = 0.0f;
            } else {
                merge(g - 1);
#pragma unroll
                for (int r = 0; r < N; ++r) {
                    if (r >= rows) break;
                    const float f = row_fac[r];
                    l_run[r] *= f;
                    o_run[r] *= f;
                }
            }
            // pass 2: weights, as two E4M3 parts, P[row][position]
            for (int j = 0; j < cur.n; ++j) {
                const int pos = (cur.t + j) * kTile + lane_row;
                const bool plain = (cur.t + j) * kTile + kTile - 1 <= all_see;
                mbar_wait(&pempty[pslot], pphase ^ 1, abort_flag, status);
                uint8_t *p_hi = smem + F::kPOff + pslot * 2 * F::kP, *p_lo = p_hi + F::kP;
#pragma unroll
                for (int c = 0; c < N; c += 16) {
                    if (c >= rows) break;
                    float v[16];
                    tmem_load16(tm + F::s_col(buf, j) + c, v);
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        if (c + k >= rows) break;
                        float x = ex2(fmaf(v[k], scale[c + k], row_neg[c + k]));
                        float y = ex2(fmaf(v[k + 1], scale[c + k + 1], row_neg[c + k + 1]));
                        if (!plain) {
                            if (pos > limit[c + k]) x = 0.0f;
                            if (pos > limit[c + k + 1]) y = 0.0f;
                        }
                        l_run[c + k] += x;
                        l_run[c + k + 1] += y;
                        const uint16_t h = e4m3x2_satfinite(x, y);
                        const float2 d = e4m3x2_to_float2(h);
                        const uint16_t l = e4m3x2_satfinite(x - d.x, y - d.y);
                        const int r = c + k, ch = lane_row >> 4, in = lane_row & 15;
                        const int o0 = r * kTile + ((ch ^ (r & 7)) << 4) + in;
                        const int o1 = (r + 1) * kTile + ((ch ^ ((r + 1) & 7)) << 4) + in;
                        p_hi[o0] = static_cast<uint8_t>(h);
                        p_hi[o1] = static_cast<uint8_t>(h >> 8);
                        p_lo[o0] = static_cast<uint8_t>(l);
                        p_lo[o1] = static_cast<uint8_t>(l >> 8);
                    }
                }
                if ((cur.t + j) * kTile + kTile > len) {
                    // the tile in which the sequence ends: what its page holds behind the
                    // end may be NaN, which a weight of 0 would not silence
                    mbar_wait(vready, ragged++ & 1, abort_flag, status);
                    if (pos >= len) {
                        uint4 *v = reinterpret_cast<uint4 *>(smem + vstage * kStageBytes + lane_row * kDim);
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&pfull[pslot]);
                    if (j == cur.n - 1) mbar_arrive(&sfree[buf]);
                }
                if (++pslot == F::kPSlots) {
                    pslot = 0;
                    pphase ^= 1;
                }
                if (++vstage == F::kStages) vstage = 0;
            }
            ++g;
            if (!cur.last) continue;

            // ------------------------------------------------ end of a segment
            merge(g - 1);
#pragma unroll
            for (int r = 0; r < N; ++r) {
                if (r >= rows) break;
                float l = l_run[r];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
                if (lane == 0) row_sum[sw * N + r] = l;
            }
            named_barrier(1, 128);
            const float *m_row = row_max + buf * N;
            auto total = [&](int r) {
                return (row_sum[r] + row_sum[N + r]) + (row_sum[2 * N + r] + row_sum[3 * N + r]);
            };
            // row r is token r / G, query head hk G + r % G
            auto out_at = [&](int r) {
                const int i = r / G;
                return a.out + (cur.seq.q0 + i) * a.out_stride +
                       static_cast<int64_t>(cur.hk * G + r - i * G) * kDim;
            };
            auto store_lse = [&](int r, float m, float l) {
                const int i = r / G;
                a.lse[static_cast<int64_t>(cur.seq.q0 + i) * a.q_heads + cur.hk * G + r - i * G] =
                    l > 0.0f ? (m - kPScale + log2f(l)) * 0.69314718055994531f : -INFINITY;
            };
            if (cur.seg_t0 == 0 && cur.seg_end == cur.tiles) {
#pragma unroll
                for (int r = 0; r < N; ++r) {
                    if (r >= rows) break;
                    const float l = total(r);
                    out_at(r)[lane_row] = __bfloat16_as_ushort(
                        __float2bfloat16_rn(l > 0.0f ? __fdividef(o_run[r], l) : 0.0f));
                }
                if (a.lse != nullptr && st < rows) store_lse(st, m_row[st], total(st));
                named_barrier(1, 128);  // row_sum and row_max are read
                continue;
            }
            // partial: this CTA's slot 1 if the (sequence, head) begins here, else slot 0
            const int64_t all = start_w[3], w_first = cur.item(), w_last = w_first + cur.tiles - 1;
            auto owner = [&](int64_t w) {
                return static_cast<int>(((w + 1) * *parts - 1) / all);
            };
            const int c_first = owner(w_first), c_last = owner(w_last);
            auto slot = [&](int c) {
                return partials + static_cast<int64_t>(2 * c + (c == c_first ? 1 : 0)) * F::kPartial;
            };
            float *mine = slot(blockIdx.x);
#pragma unroll
            for (int r = 0; r < N; ++r) {
                if (r >= rows) break;
                __stcg(mine + r * kDim + lane_row, o_run[r]);
            }
            if (st < rows) {
                __stcg(mine + N * kDim + st, m_row[st]);
                __stcg(mine + N * kDim + N + st, total(st));
            }
            __threadfence();
            named_barrier(1, 128);
            if (st == 0) {
                const int seen = atomicAdd(counters + c_first, 1);
                *shared_last = seen == c_last - c_first;
                if (*shared_last) counters[c_first] = 0;
                __threadfence();
            }
            named_barrier(1, 128);
            if (!*shared_last) continue;
            // join in the order of the CTAs: a warp per row, 4 channels per lane
            for (int r = sw; r < rows; r += 4) {
                float m = -INFINITY, l = 0.0f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int c = c_first; c <= c_last; ++c) m = fmaxf(m, __ldcg(slot(c) + N * kDim + r));
                if (m > -INFINITY) {
#pragma unroll 4
                    for (int c = c_first; c <= c_last; ++c) {
                        const float *p = slot(c);
                        const float f = ex2(__ldcg(p + N * kDim + r) - m);
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(p + r * kDim) + lane);
                        l = fmaf(f, __ldcg(p + N * kDim + N + r), l);
                        o.x = fmaf(f, v.x, o.x);
                        o.y = fmaf(f, v.y, o.y);
                        o.z = fmaf(f, v.z, o.z);
                        o.w = fmaf(f, v.w, o.w);
                    }
                }
                const float inv = l > 0.0f ? __fdividef(1.0f, l) : 0.0f;
                *reinterpret_cast<uint2 *>(out_at(r) + lane * 4) =
                    make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
                if (a.lse != nullptr && lane == 0) store_lse(r, m, l);
            }
        }
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
