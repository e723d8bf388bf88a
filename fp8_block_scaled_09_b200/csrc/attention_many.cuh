// attention_many.cuh -- paged attention for many query rows per kv head (prefill
// chunks, blocks of new tokens).
//
// A sequence's query rows of one kv head, r = token * group + head, are taken
// 256 at a time, as two halves A and B of 128 rows that share every K and V
// tile of 128 positions:
//     S[row, pos] = Q[row, :] . K[pos, :]      E4M3, M = N = 128, K = 128, twice
//     O[row, ch] += P[row, :] . V[:, ch]       F16,  M = N = 128, K = 128
// K is never converted: a BF16 query row, times a power of two that takes its largest
// channel to [128, 256), is held as two E4M3 parts hi + lo, two MMAs into the same
// columns at twice the 16-bit rate: exact down to 2^-9 of that channel and off by at
// most 2^-17 of it below (parts of different scale, as in attention_few.cuh, would need
// columns of their own, and the tensor memory is full).  V becomes F16 (exact, as
// 2^-8 V: an E4M3 code's bits moved into an F16 are its value times 2^-8, so
// four integer instructions convert two codes; the output takes the 2^8 back).
// P is F16 too, 11 bits, and never leaves the tensor memory: it replaces the
// scores it came from and is the A operand of the second product.
//
// Bound by the tensor pipe, 1024 cycles per half and tile, and equally by the
// exponentials (16 a cycle and SM: 1024 cycles per half and tile): the halves
// alternate, one's softmax under the other's MMAs.  A softmax thread has a whole
// row, so maxima and sums need no exchange.  The running maximum is only
// moved when a row's scores pass it by 2^8, so O is hardly ever rescaled in the
// tensor memory; weights are held times 2^7, so that they reach 2^15 at most and
// those far below a dominant position keep a step of 2^-31 of it or less (without the
// 2^7, what 32768 positions 18 logits under the first one add up to was lost).
//
// Blocks of at most 128 rows have no second half: there both halves hold the same
// rows and take the tiles in turn; B hands its result to A through the shared
// memory of the queries.
//
// Work is a list of K/V tiles ordered by (sequence, 256 rows, kv head, tile),
// each (rows, head) item preceded by kItemCost tiles' worth of nothing; CTA c of
// one per SM takes the c-th equal part, so that neither causal masks nor lengths
// nor a last wave leave SMs idle.  An item that lies in several CTAs is joined
// as in attention_few.cuh, each half by itself.
//
// Roles (512 threads): warpgroups 0 and 1 softmax of A and B (184 registers a
// thread: 128 scores), 2 converts V, warp 12 TMA producer, warp 13 MMA issuer,
// warp 14 walks the work list and publishes the segments to the others (which
// have no registers to spare for it: walking it in every role spilled scores), warp 15
// writes the zeros of sequences without positions.
//
// Measured: 2048 tokens of 56 + 8 heads at 18001 positions 821 us, 1.21 PFLOP/s (947 us in
// a loop, under the power cap; a pair
// of halves takes ~3400 cycles per tile where its MMAs take 2048: the softmax chain
// between them); a prompt of 8192 tokens 889 us; 16 blocks of 8 tokens of 28 + 4
// heads at 1000 .. 8000 positions 45 us.
#pragma once

#include "attention_few.cuh"

namespace fp8bq {
namespace attn {

constexpr int kManyThreads = 512;
constexpr int kManyLaunchRegs = 128;
constexpr int kSoftmaxRegs = 184, kConvertRegs = 56, kIssueRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kConvertRegs + 128 * kIssueRegs <=
                  kManyThreads * kManyLaunchRegs,
              "register split exceeds the launch allocation");
// Tiles' worth of work that an item adds: 8192-token prompt 942 us; 1044 with 3, 952 with 6.
constexpr int kItemCost = 5;
constexpr int kManyMaxGrid = 160;
constexpr int kHalfRows = 128;
constexpr float kRescaleAt = 8.0f;  // log2
constexpr float kWeightLog2 = 7.0f;  // weights are held times 2^7: with kRescaleAt at most 2^15

struct Many {
    static constexpr int kStages = 6;  // K tiles in even, V tiles in odd stages
    static constexpr int kQPart = kHalfRows * kDim;   // 16 KB
    static constexpr int kRingOff = 4 * kQPart;       // Q: [half][hi, lo]
    static constexpr int kV16 = kTile * kDim * 2;     // 32 KB
    static constexpr int kV16Off = kRingOff + kStages * kStageBytes;
    static constexpr int kBarOff = kV16Off + 2 * kV16;
    static constexpr int kSegs = 4;  // published segments
    // full, empty; vfull, vempty, qfull, sfull, ofull (two each), pfull (four); segfull, segempty
    static constexpr int kBars = 2 * kStages + 14 + 2 * kSegs;
    static constexpr int kSegOff = kBarOff + kBars * 8;
    static constexpr int kMiscOff = kSegOff + kSegs * 64;
    static constexpr int kRowOff = kMiscOff + 256;  // maximum and sum of half B's rows
    static constexpr int kBytes = kRowOff + 2 * kHalfRows * 4 + 1024;
    static_assert(kBytes <= 227 * 1024, "shared memory");
    // floats of one half's partial: O [32 groups of 4 channels][128 rows][4], max, sum [128]
    static constexpr int kPartial = kHalfRows * (kDim + 2);
    // TMEM columns
    __device__ static uint32_t s_col(int half) { return half * 128; }
    __device__ static uint32_t o_col(int half) { return 256 + half * 128; }
};

// A: E4M3 or F16 rows, both K-major; B of the second product: N contiguous.
__host__ __device__ constexpr uint32_t idesc_f16_b_mn(int m, int n) {
    return (1u << 4) | (1u << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

// 128-byte-swizzled operand tile whose N dimension is contiguous: 64 F16 of N per
// 128-byte row, 8 K rows per 1024-byte block, `n_step` bytes to the next 64 of N.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t saddr, uint32_t n_step) {
    return (umma_desc_sw128(saddr) & ~(static_cast<uint64_t>(0x3FFF) << 16)) |
           (static_cast<uint64_t>(n_step >> 4) << 16);
}

// D[tmem] (+)= A[tmem] * B[smem] over K = 16 (F16; A two values per column).
__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 16-byte asynchronous global -> shared copy (completion: cp_async_wait_all); the
// bytes from src_bytes (0 or 16) on are zeros.
__device__ __forceinline__ void cp_async_16(void *smem_dst, const void *gmem_src, uint32_t src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(smem_dst)),
                 "l"(gmem_src), "r"(src_bytes)
                 : "memory");
}

// 32 consecutive columns of this warp's lanes, without the wait.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
        "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
        "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<const uint64_t *>(&a)), "l"(*reinterpret_cast<const uint64_t *>(&b)));
    return *reinterpret_cast<const float2 *>(&d);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two E4M3 codes in the high bytes of x's halves -> two F16 of 2^-8 their values.
__device__ __forceinline__ uint32_t e4m3x2_to_f16_shifted(uint32_t x) {
    return (x & 0x80008000u) | ((x >> 1) & 0x3F803F80u);
}

// ------------------------------------------------------------------ work list

// Last position that row r of a sequence sees (-1 or less: none).
__device__ __forceinline__ int row_limit(const Args &a, const Seq &s, int r) {
    return a.causal ? min(s.len - s.q_real + r / a.group, s.len - 1) : s.len - 1;
}

// 256-row blocks of a sequence; one without positions has no work, only zeros to write.
__device__ __forceinline__ int row_blocks(const Args &a, const Seq &s) {
    return s.len > 0 ? (s.q_len * a.group + 255) / 256 : 0;
}

// K/V tiles that rows [.., end) of a sequence need: at least one, which then
// masks everything and makes the zeros of rows that see nothing.
__device__ __forceinline__ int tiles_until(const Args &a, const Seq &s, int end) {
    return max(row_limit(a, s, min(end, s.q_len * a.group) - 1) / kTile + 1, 1);
}

// Cost of all items of a sequence (warp-wide, the same in every lane).
__device__ __forceinline__ int64_t seq_cost(const Args &a, const Seq &s) {
    const int blocks = row_blocks(a, s);
    int64_t c = 0;
    for (int m = threadIdx.x & 31; m < blocks; m += 32) c += tiles_until(a, s, m * 256 + 256) + kItemCost;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xFFFFFFFFu, c, o);
    return c * a.kv_heads;
}

// The segments of one CTA's part of the work list, in order.
struct Items {
    const Args &a;
    int64_t w, w_end, base;  // next position, end of the part, first position of block m
    int b, m, blocks;        // sequence and 256-row block of w
    Seq seq;
    int cost;                // positions of one head's item of block m
    // the current segment
    int hk, t0, t1;          // kv head, tiles [t0, t1)

    __device__ Items(const Args &args, int64_t w0, int64_t w1, int b0, int m0, int64_t base0)
        : a(args), w(w0), w_end(w1), base(base0), b(b0), m(m0), blocks(0), cost(0), hk(0), t0(0),
          t1(0) {
        if (w < w_end) {
            seq = seq_of(a, b);
            blocks = row_blocks(a, seq);
            cost = tiles_until(a, seq, m * 256 + 256) + kItemCost;
        }
    }
    __device__ bool next() {
        for (;;) {
            if (w >= w_end) return false;
            while (w >= base + static_cast<int64_t>(cost) * a.kv_heads) {
                base += static_cast<int64_t>(cost) * a.kv_heads;
                if (++m >= blocks) {
                    m = 0;
                    do {
                        seq = seq_of(a, ++b);
                        blocks = row_blocks(a, seq);
                    } while (blocks == 0);
                }
                cost = tiles_until(a, seq, m * 256 + 256) + kItemCost;
            }
            const uint32_t off = static_cast<uint32_t>(w - base);  // < cost * kv_heads < 2^30
            hk = static_cast<int>(off / static_cast<uint32_t>(cost));
            const int rel = static_cast<int>(off - static_cast<uint32_t>(hk) * cost);
            const int64_t left = min(static_cast<int64_t>(cost - rel), w_end - w);
            t0 = max(rel - kItemCost, 0);
            t1 = max(static_cast<int>(rel + left) - kItemCost, 0);
            w += left;
            if (t1 > t0) return true;
        }
    }
    __device__ int64_t item() const { return base + static_cast<int64_t>(hk) * cost + kItemCost; }
};

// A segment as its users read it (shared memory).
struct Segment {
    int valid;           // 0: the CTA's part is done
    int b, hk, t0, t1;   // sequence, kv head, tiles
    int count[2];        // tiles of each half, from t0 on
    int dual;            // at most 128 rows: the halves hold the same and take tiles in turn
    int row0, rows_end;  // first row of half A; rows of the sequence and head
    int len, q0;         // positions; first row of q
    int limit0;          // last position that row 0 sees (may be negative); one more per token
    int whole;           // all tiles of the item: no partial
    int c_first, c_last; // CTAs that have tiles of the item
};
static_assert(sizeof(Segment) == 64, "shared-memory layout");

// Reads the published segments in order; every lane of a using warp keeps one.
struct SegReader {
    uint64_t *full, *empty;
    const Segment *ring;
    const volatile int *stopped;  // place of the first segment that will not come, or -1
    uint32_t i, phase;

    __device__ static int place(uint32_t i, uint32_t phase) { return static_cast<int>(i | (phase << 8)); }
    __device__ const Segment *next(volatile int *abort_flag, int *status) const {
        if (!mbar_wait(&full[i], phase, abort_flag, status)) return nullptr;
        return ring[i].valid ? ring + i : nullptr;
    }
    // For warps that meet at named barriers and therefore have to take the same segments,
    // behind a wait that gave up too: ends only where the work list's warp stopped.
    // That warp either publishes or stops, since its own wait is bounded, and at most
    // kSegs segments lie between it and a reader, so a place stands for one segment.
    __device__ const Segment *next_published() const {
        while (!mbar_try_wait(&full[i], phase))
            if (*stopped == place(i, phase)) return nullptr;
        return ring[i].valid ? ring + i : nullptr;
    }
    // Warp-wide: this warp is done with the current one.
    __device__ void release() {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&empty[i]);
        if (++i == Many::kSegs) {
            i = 0;
            phase ^= 1;
        }
    }
};
constexpr int kSegUsers = 14;  // warps: producer, MMA, 4 converting, 8 softmax

// ------------------------------------------------------------------ kernel

__global__ void __launch_bounds__(kManyThreads, 1)
attention_many_kernel(const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v, const Args a, int *counters,
                      float *partials, int *status) {
    using F = Many;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + F::kBarOff);
    uint64_t *empty = full + F::kStages;
    uint64_t *vfull = empty + F::kStages, *vempty = vfull + 2, *qfull = vempty + 2,
             *sfull = qfull + 2, *ofull = sfull + 2, *pfull = ofull + 2, *segfull = pfull + 4,
             *segempty = segfull + F::kSegs;
    Segment *seg_ring = reinterpret_cast<Segment *>(smem + F::kSegOff);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + F::kMiscOff);
    uint32_t *tmem_slot = misc;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(misc + 1);
    int *shared_last = reinterpret_cast<int *>(misc + 2);      // [2]
    int *start_bm = reinterpret_cast<int *>(misc + 5);         // sequence, block
    int *parts = reinterpret_cast<int *>(misc + 7);            // CTAs that have a part
    int64_t *start_w = reinterpret_cast<int64_t *>(misc + 8);  // w0, w1, base, total
    int64_t *warp_cost = start_w + 4;                          // [16]
    volatile int *seg_stopped = reinterpret_cast<volatile int *>(warp_cost + 16);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    allow_dependent_launch();
    if (threadIdx.x == 0) {
        for (int i = 0; i < F::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], i % 2 == 0 ? 1 : 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&vfull[i], 4);
            mbar_init(&vempty[i], 1);
            mbar_init(&qfull[i], 4);
            mbar_init(&sfull[i], 1);
            mbar_init(&ofull[i], 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&pfull[i], 4);
        for (int i = 0; i < F::kSegs; ++i) {
            mbar_init(&segfull[i], 1);
            mbar_init(&segempty[i], kSegUsers);
        }
        *abort_flag = 0;
        *seg_stopped = -1;
        fence_barrier_init();
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    if (warp == 13) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    grid_dependency_wait();
    {
        // this CTA's part of the work list: warp w sums the costs of the w-th run
        // of sequences, then the warp whose run holds the first position finds it
        const int per = (a.B + 15) / 16, b0 = min(warp * per, a.B), b1 = min(b0 + per, a.B);
        int64_t mine = 0;
        for (int b = b0; b < b1; ++b) mine += seq_cost(a, seq_of(a, b));
        if (lane == 0) warp_cost[warp] = mine;
        __syncthreads();
        int64_t before = 0, total = 0;
        for (int i = 0; i < 16; ++i) {
            if (i < warp) before += warp_cost[i];
            total += warp_cost[i];
        }
        // no part is empty, so that a split item lies in consecutive CTAs
        const int64_t np = min(static_cast<int64_t>(gridDim.x), max(total, int64_t(1)));
        const int64_t w0 = min(blockIdx.x * total / np, total), w1 = min((blockIdx.x + 1) * total / np, total);
        if (w0 >= before && w0 < before + mine) {
            int b = b0;
            Seq s = seq_of(a, b);
            for (;;) {
                const int64_t n = seq_cost(a, s);
                if (w0 < before + n) break;
                before += n;
                s = seq_of(a, ++b);
            }
            // the block: 32 at a time, an inclusive scan of their costs
            int m = 0;
            for (;; m += 32) {
                const int blocks = row_blocks(a, s);
                const int64_t c = m + lane < blocks
                                      ? static_cast<int64_t>(tiles_until(a, s, (m + lane) * 256 + 256) + kItemCost) * a.kv_heads
                                      : 0;
                int64_t incl = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                    if (lane >= o) incl += up;
                }
                const unsigned hit = __ballot_sync(0xFFFFFFFFu, w0 < before + incl);
                if (hit != 0) {
                    const int l = __ffs(hit) - 1;
                    if (lane == l) {
                        start_bm[0] = b;
                        start_bm[1] = m + l;
                        start_w[2] = before + incl - c;
                    }
                    break;
                }
                before += __shfl_sync(0xFFFFFFFFu, incl, 31);
            }
        }
        if (threadIdx.x == 0) {
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
    SegReader segs{segfull, segempty, seg_ring, seg_stopped, 0, 0};

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == 12) {
            // -------------------------------------------------------- producer
            const int rows = min(1 << a.page_shift, kTile), boxes = kTile / rows;
            uint32_t stage = 0, phase = 0, issued = 0;
            bool ok = true;
            while (ok) {
                const Segment *sg = segs.next(abort_flag, status);
                if (!__all_sync(0xFFFFFFFFu, sg != nullptr)) break;
                const int hk = sg->hk, t1 = sg->t1;
                PageWalk pages(a, sg->b, sg->len, sg->t0 * kTile);
                for (int t = sg->t0; t < t1 && ok; ++t) {
                    const int row = pages.row_of(a, t * kTile + min(lane, boxes - 1) * rows, status);
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        ok = ok && mbar_wait(&empty[stage], phase ^ 1, abort_flag, status);
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(&full[stage], kStageBytes);
                        __syncwarp();
                        if (lane < boxes)
                            tma_load_2d(smem + F::kRingOff + stage * kStageBytes + lane * rows * kDim,
                                        kv == 0 ? &tmap_k : &tmap_v, &full[stage], hk * kDim, row);
                        ++issued;
                        if (++stage == F::kStages) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                }
                segs.release();
            }
            // no copy may be in flight when the CTA leaves
            const uint32_t from = issued > F::kStages ? issued - F::kStages : 0;
            for (uint32_t i = from; i < issued; ++i)
                mbar_wait(&full[i % F::kStages], (i / F::kStages) & 1, nullptr, status);
        } else if (warp == 15) {
            // -------------------------------------------------------- reports, empty sequences
            // each CTA's share of the rows of sequences without positions, by row number
            // (as items of the list with one masked tile they took 8 us each)
            const int ctas = gridDim.x, cta = blockIdx.x;
            for (int b0 = 0; b0 < a.B; b0 += 32) {
                const int b = b0 + lane;
                Seq s = {1, 0, 0, 0};
                if (b < a.B) {
                    s = seq_of(a, b);
                    if (cta == 0 && seq_is_bad(a, b)) atomicExch(status, 8 /* FP8BQ_ERR_INDEX */);
                }
                unsigned todo = __ballot_sync(0xFFFFFFFFu, s.len == 0 && s.q_len > 0);
                for (; todo != 0; todo &= todo - 1) {
                    const int l = __ffs(todo) - 1;
                    const int q0 = __shfl_sync(0xFFFFFFFFu, s.q0, l), n = __shfl_sync(0xFFFFFFFFu, s.q_len, l);
                    for (int i = (cta + ctas - q0 % ctas) % ctas; i < n; i += ctas) {
                        const int64_t row = q0 + i;
                        uint4 *o = reinterpret_cast<uint4 *>(a.out + row * a.out_stride);
                        for (int c = lane; c < a.q_heads * (kDim / 8); c += 32) o[c] = make_uint4(0, 0, 0, 0);
                        if (a.lse != nullptr)
                            for (int h = lane; h < a.q_heads; h += 32) a.lse[row * a.q_heads + h] = -INFINITY;
                    }
                }
            }
        } else if (warp == 14) {
            // -------------------------------------------------------- work list
            if (lane == 0) {
                Items it(a, start_w[0], start_w[1], start_bm[0], start_bm[1], start_w[2]);
                const int64_t all = start_w[3], np = *parts;
                uint32_t i = 0, phase = 0;
                for (bool more = true; more;) {
                    more = it.next();
                    if (!mbar_wait(&segempty[i], phase ^ 1, abort_flag, status)) {
                        *seg_stopped = SegReader::place(i, phase);
                        break;
                    }
                    Segment &sg = seg_ring[i];
                    sg.valid = more;
                    if (more) {
                        sg.b = it.b;
                        sg.hk = it.hk;
                        sg.t0 = it.t0;
                        sg.t1 = it.t1;
                        const int last_row = min(it.m * 256 + 256, it.seq.q_len * a.group);
                        const int n = it.t1 - it.t0;
                        sg.dual = last_row <= it.m * 256 + kHalfRows;
                        sg.count[0] = sg.dual ? (n + 1) / 2
                                              : max(min(it.t1, tiles_until(a, it.seq, it.m * 256 + kHalfRows)) - it.t0, 0);
                        sg.count[1] = sg.dual ? n / 2 : n;
                        sg.row0 = it.m * 256;
                        sg.rows_end = it.seq.q_len * a.group;
                        sg.len = it.seq.len;
                        sg.q0 = it.seq.q0;
                        sg.limit0 = it.seq.len - it.seq.q_real;
                        sg.whole = it.t0 == 0 && it.t1 == it.cost - kItemCost;
                        const int64_t w0 = it.item(), w1 = w0 + it.cost - kItemCost - 1;
                        sg.c_first = static_cast<int>(((w0 + 1) * np - 1) / all);
                        sg.c_last = static_cast<int>(((w1 + 1) * np - 1) / all);
                    }
                    mbar_arrive(&segfull[i]);
                    if (++i == F::kSegs) {
                        i = 0;
                        phase ^= 1;
                    }
                }
            }
        } else if (warp == 13) {
            // -------------------------------------------------------- MMA issuer
            // MMAs of one thread run in the order they are issued, so the
            // scores of the next tile may follow the product that still reads
            // the weights in their place.
            constexpr uint32_t id_s = umma_idesc_e4m3(kHalfRows, kTile);
            constexpr uint32_t id_o = idesc_f16_b_mn(kHalfRows, kDim);
            uint32_t kstage = 0, kphase = 0, vbuf = 0, vphase = 0;
            uint32_t qphase[2] = {0, 0}, pphase[2] = {0, 0};
            bool ok = true;
            // descriptors: an address step of 16 bytes is 1
            const uint64_t q_desc = umma_desc_sw128(smem_addr(smem)),
                           ring_desc = umma_desc_sw128(smem_addr(smem + F::kRingOff)),
                           v_desc = umma_desc_mn_sw128(smem_addr(smem + F::kV16Off), F::kV16 / 2);
            auto scores = [&](int half) {
                tc_fence_after_sync();
                const uint64_t q = q_desc + half * (2 * F::kQPart / 16),
                               k = ring_desc + kstage * (kStageBytes / 16);
                if (elect_one()) {
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            umma_e4m3(tmem + F::s_col(half), q + part * (F::kQPart / 16) + 2 * s,
                                      k + 2 * s, id_s, part + s > 0 ? 1u : 0u);
                    umma_commit(&sfull[half]);
                }
                __syncwarp();
            };
            auto next_k = [&] {
                kstage += 2;
                if (kstage == F::kStages) {
                    kstage = 0;
                    kphase ^= 1;
                }
            };
            while (ok) {
                const Segment *sg = segs.next(abort_flag, status);
                if (!__all_sync(0xFFFFFFFFu, sg != nullptr)) break;
                const int n = sg->t1 - sg->t0, count[2] = {sg->count[0], sg->count[1]};
                const bool dual = sg->dual;
                segs.release();
                auto wait = [&](uint64_t *bar, uint32_t phase) {
                    ok = ok && mbar_wait(bar, phase, abort_flag, status);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                };
                // scores of a half's first tile, or of its next one
                auto first_scores = [&](int half) {
                    wait(&qfull[half], qphase[half]);
                    qphase[half] ^= 1;
                    if (ok) scores(half);
                };
                auto finish = [&](int half) {
                    if (elect_one()) umma_commit(&ofull[half]);
                    __syncwarp();
                };
                auto wait_k = [&] { wait(&full[kstage], kphase); };
                // O of a half from its weights and V, in two parts as the weights come
                auto product = [&](int half, bool fresh) {
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        wait(&pfull[2 * half + part], pphase[half]);
                        if (!ok) return;
                        tc_fence_after_sync();
                        const uint64_t v = v_desc + vbuf * (F::kV16 / 16);
                        const uint32_t first = fresh ? 0u : 1u;
                        if (elect_one()) {
#pragma unroll
                            for (int s = 4 * part; s < 4 * part + 4; ++s)  // 16 positions each
                                umma_f16_ta(tmem + F::o_col(half), tmem + F::s_col(half) + 8 * s,
                                            v + 128 * s, id_o, s == 0 ? first : 1u);
                        }
                        __syncwarp();
                    }
                    pphase[half] ^= 1;
                };
                auto next_v = [&] {
                    vbuf ^= 1;
                    vphase ^= vbuf ^ 1;
                };
                if (dual) {
                    for (int half = 0; half < min(n, 2); ++half) {
                        wait_k();
                        first_scores(half);
                        if (ok) next_k();
                    }
                    for (int j = 0; j < n && ok; ++j) {
                        const int half = j & 1;
                        wait(&vfull[vbuf], vphase);
                        if (ok) product(half, j < 2);
                        if (!ok) break;
                        next_v();
                        if (j + 2 < n) {
                            wait_k();
                            if (!ok) break;
                            scores(half);
                            next_k();
                        } else {
                            finish(half);
                        }
                    }
                    continue;
                }
                wait_k();
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    if (count[half] > 0) first_scores(half);
                if (ok) next_k();
                for (int j = 0; j < n && ok; ++j) {
                    wait(&vfull[vbuf], vphase);  // which also stands for the next K
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (j >= count[half] || !ok) continue;
                        product(half, j == 0);
                        if (!ok) continue;
                        if (j + 1 < count[half])
                            scores(half);
                        else
                            finish(half);
                    }
                    if (!ok) break;
                    next_v();
                    if (j + 1 < n) next_k();
                }
            }
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvertRegs));
        // ------------------------------------------------------------ V to F16
        const int row = threadIdx.x - 256;  // position in the tile
        uint32_t stage = 1, phase = 0, vbuf = 0, vphase = 0, kstage = 0, kphase = 0;
        bool ok = true;
        auto next_k = [&] {
            kstage += 2;
            if (kstage == F::kStages) {
                kstage = 0;
                kphase ^= 1;
            }
        };
        while (ok) {
            const Segment *sg = segs.next(abort_flag, status);
            if (!__all_sync(0xFFFFFFFFu, sg != nullptr)) break;
            const int t1 = sg->t1, len = sg->len;
            const bool dual = sg->dual;
            int t = sg->t0;
            segs.release();
            next_k();
            for (; t < t1 && ok; ++t) {
                ok = mbar_wait(&full[stage], phase, abort_flag, status) &&
                     mbar_wait(&vempty[vbuf], vphase ^ 1, abort_flag, status);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const uint8_t *src = smem + F::kRingOff + stage * kStageBytes + row * kDim;
                uint8_t *dst = smem + F::kV16Off + vbuf * F::kV16 + row * 128;
                const int x = row & 7;
                // what a page holds behind the sequence's end may be anything
                const uint32_t keep = t * kTile + row < len ? 0xFFFFFFFFu : 0u;
#pragma unroll 4
                for (int c = 0; c < 8; ++c) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(src + ((c ^ x) << 4));
                    const uint32_t w[4] = {u.x & keep, u.y & keep, u.z & keep, u.w & keep};
                    uint32_t f[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        f[2 * k] = e4m3x2_to_f16_shifted(__byte_perm(w[k], 0, 0x1404));
                        f[2 * k + 1] = e4m3x2_to_f16_shifted(__byte_perm(w[k], 0, 0x3424));
                    }
                    uint8_t *d = dst + (c >> 2) * (F::kV16 / 2);
                    const int cc = (c & 3) * 2;
                    *reinterpret_cast<uint4 *>(d + ((cc ^ x) << 4)) = make_uint4(f[0], f[1], f[2], f[3]);
                    *reinterpret_cast<uint4 *>(d + (((cc + 1) ^ x) << 4)) = make_uint4(f[4], f[5], f[6], f[7]);
                }
                fence_proxy_async_smem();
                if (t + 1 < t1) {
                    // the issuer needs the next K too: one wait less for it.  (The
                    // K before that in the same stage has been used: the V buffer
                    // taken above was released after it.)
                    if (!dual) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[kstage], kphase, abort_flag, status));
                    next_k();
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&vfull[vbuf]);
                    mbar_arrive(&empty[stage]);
                }
                stage += 2;
                if (stage > F::kStages) {
                    stage = 1;
                    phase ^= 1;
                }
                vbuf ^= 1;
                vphase ^= vbuf ^ 1;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ------------------------------------------------------------ softmax
        // A wait that gives up sets the abort flag: the loops then run without
        // waiting through every segment that was published, so that every barrier still has
        // all its warps.
        const int half = warp >> 2, ht = threadIdx.x & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_tm = tmem + lanes + F::s_col(half), o_tm = tmem + lanes + F::o_col(half);
        const int G = a.group;

        // 16 bytes number c of a 256-byte row of this warp, in the places of the row's query parts
        auto staged = [&](int row, int c) {
            return reinterpret_cast<uint4 *>(smem + (2 * half + (c >> 3)) * F::kQPart +
                                             ((warp & 3) * 32 + row) * kDim + (((c & 7) ^ (row & 7)) << 4));
        };
        uint32_t sphase = 0, ophase = 0;
        uint32_t kstage = 0, vbuf = 0;  // of the segment's first tile
        // K and V are released here, by one warp of the half that used a tile last
        // (a commit costs the issuer ~175 cycles): a half's scores are complete after
        // the product and the scores issued before them.
        const bool releases = (warp & 3) == 0 && lane == 0;
        for (;; segs.release()) {
            const Segment *sg = segs.next_published();
            if (sg == nullptr) break;
            const int n = sg->count[half];
            const bool dual = sg->dual;
            // this thread's row of the sequence and head; up to 64 doubled rows are
            // in the other warps of half B, which have another scheduler
            const int shift = dual ? (half == 1 && sg->rows_end - sg->row0 <= 64 ? 64 : 0) : half * kHalfRows;
            const int r = sg->row0 + (dual ? (ht + shift) % kHalfRows : ht + shift);
            const bool live = r < sg->rows_end;
            const bool any_live = __any_sync(0xFFFFFFFFu, live);
            const int tok = r / G, head = sg->hk * G + (r - tok * G);
            const int64_t q_row = sg->q0 + tok;
            float m_run = -INFINITY, l_run = 0.0f;
            if (n > 0) {
                // The row's query: power of two that takes its largest channel to
                // [128, 256), two E4M3 parts, K-major with the 128-byte swizzle.  The warp
                // fetches two rows at a time (a thread its own row would touch 32 lines with
                // each load) and hands them out through the rows' own places in shared memory.
                // (This runs once per segment, from instructions that are no longer in the
                // cache: short loops, since each new line of code costs more than its work.)
                const int64_t at = live ? q_row * a.q_stride + static_cast<int64_t>(head) * kDim : -1;
#pragma unroll 1
                for (int i = 0; i < 16; ++i) {
                    const int64_t from = __shfl_sync(0xFFFFFFFFu, at, 2 * i + (lane >> 4));
                    cp_async_16(staged(2 * i + (lane >> 4), lane & 15),
                                a.q + (from >= 0 ? from : 0) + (lane & 15) * 8, from >= 0 ? 16 : 0);
                }
                cp_async_wait_all();
                __syncwarp();
                uint32_t top = 0;
#pragma unroll 1
                for (int c = 0; c < 16; ++c) top = max(top, amax_bits8(*staged(lane, c)));
                const int e = max(static_cast<int>(top >> 7) - 127, -100);
                const float up = __uint_as_float(static_cast<uint32_t>(7 - e + 127) << 23);
                const float scale = fmaxf(
                    a.scale * 1.4426950408889634f * __uint_as_float(static_cast<uint32_t>(e - 7 + 127) << 23),
                    kMinScale);
                // Parts of 16 channels take the places of their row's 16-byte pieces c and
                // 8 + c, so the first 8 pieces move to registers and the last go first.
                uint4 u[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) u[c] = *staged(lane, c);
#pragma unroll 1
                for (int c = 7; c >= 0; --c) {
                    uint4 x0, x1;
                    if (c >= 4) {
                        x0 = *staged(lane, 2 * c);
                        x1 = *staged(lane, 2 * c + 1);
                    } else {
                        x0 = u[6];
                        x1 = u[7];
#pragma unroll
                        for (int k = 7; k >= 2; --k) u[k] = u[k - 2];
                    }
                    uint2 hi[2], lo[2];
                    split8(x0, up, hi[0], lo[0]);
                    split8(x1, up, hi[1], lo[1]);
                    *staged(lane, c) = make_uint4(hi[0].x, hi[0].y, hi[1].x, hi[1].y);
                    *staged(lane, 8 + c) = make_uint4(lo[0].x, lo[0].y, lo[1].x, lo[1].y);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&qfull[half]);

                // columns of tile t0 that the row sees, 128 fewer per tile
                int seen = (live ? (a.causal ? min(sg->limit0 + tok, sg->len - 1) : sg->len - 1) : -1) + 1 -
                           (sg->t0 + (dual ? half : 0)) * kTile;
                const int step = dual ? 2 * kTile : kTile;
                for (int j = 0; j < n; ++j, seen -= step) {
                    mbar_wait(&sfull[half], sphase, abort_flag, status);
                    sphase ^= 1;
                    if (releases && (dual || half == 1)) {
                        const int t = dual ? 2 * j + half : j;
                        mbar_arrive(&empty[(kstage + 2 * t) % F::kStages]);
                        if (j > 0) mbar_arrive(&vempty[(vbuf + (dual ? 0 : t - 1) + (dual ? half : 0)) & 1]);
                    }
                    if (!any_live) {  // what the tensor memory holds for these rows goes nowhere
                        if (lane < 2) mbar_arrive(&pfull[2 * half + lane]);
                        continue;
                    }
                    tc_fence_after_sync();
                    float v[128];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(s_tm + 32 * c, v + 32 * c);
                    tmem_ld_wait<128>(v);
                    if (__any_sync(0xFFFFFFFFu, seen < kTile)) {
#pragma unroll
                        for (int c = 0; c < 128; ++c) v[c] = c < seen ? v[c] : -INFINITY;
                    }
                    float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                    for (int c = 4; c < 128; c += 8)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mx[k] = fmaxf(mx[k], c + 4 + k < 128 ? fmaxf(v[c + k], v[c + 4 + k]) : v[c + k]);
                    const float z = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
                    const bool move = z > m_run + kRescaleAt;  // always from -inf, if anything is seen
                    if (__any_sync(0xFFFFFFFFu, move)) {
                        const float f = move ? ex2(m_run - z) : 1.0f;
                        if (move) m_run = z;
                        l_run *= f;
                        if (j > 0) {
                            // the product that wrote O is complete: it was issued before these scores
#pragma unroll 1
                            for (int c = 0; c < 128; c += 16) {
                                float o[16];
                                tmem_ld<16>(o_tm + c, o);
                                tmem_ld_wait<16>(o);
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] *= f;
                                tmem_st16(o_tm + c, reinterpret_cast<const uint32_t *>(o));
                            }
                        }
                    }
                    const float neg = m_run == -INFINITY ? 0.0f : kWeightLog2 - m_run;
                    const float2 s2 = make_float2(scale, scale), n2 = make_float2(neg, neg);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int c = 0; c < 128; c += 64) {
                        uint32_t p[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            float2 x = ffma2(make_float2(v[c + 2 * k], v[c + 2 * k + 1]), s2, n2);
                            x.x = ex2(x.x);
                            x.y = ex2(x.y);
                            sum[k & 1] = fadd2(sum[k & 1], x);
                            p[k] = pack_f16(x.x, x.y);
                        }
                        tmem_st32(s_tm + c / 2, p);
                        tmem_st_wait();
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&pfull[2 * half + c / 64]);
                    }
                    sum[0] = fadd2(sum[0], sum[1]);
                    l_run += sum[0].x + sum[0].y;
                }
                mbar_wait(&ofull[half], ophase, abort_flag, status);
                ophase ^= 1;
                if (releases && (dual || half == 1)) mbar_arrive(&vempty[(vbuf + (dual ? half : n - 1)) & 1]);
                tc_fence_after_sync();
            }
            const int tiles = sg->t1 - sg->t0;
            kstage = (kstage + 2 * tiles) % F::kStages;
            vbuf = (vbuf + tiles) & 1;

            float *b_max = reinterpret_cast<float *>(smem + F::kRowOff), *b_sum = b_max + kHalfRows;
            float4 *b_out = reinterpret_cast<float4 *>(smem);  // [32 groups of 4 channels][128 rows]
            float f_a = 1.0f, f_b = 0.0f;
            if (dual) {
                named_barrier(3, 256);  // both halves' MMAs are done with the queries
                if (half == 1) {
                    const int row = r - sg->row0;
                    if (n > 0 && any_live) {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            float o[32];
                            tmem_ld32(o_tm + 32 * c, o);
                            tmem_ld_wait<32>(o);
                            if (live) {
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    b_out[(8 * c + k) * kHalfRows + row] =
                                        make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                            }
                        }
                    }
                    b_max[row] = m_run;
                    b_sum[row] = l_run;
                    named_barrier(3, 256);
                    named_barrier(3, 256);  // half A has read it
                    continue;
                }
                named_barrier(3, 256);
                const float m_b = b_max[ht], m = fmaxf(m_run, m_b);
                if (m_b > -INFINITY) {
                    f_a = ex2(m_run - m);
                    f_b = ex2(m_b - m);
                    l_run = fmaf(l_run, f_a, b_sum[ht] * f_b);
                    m_run = m;
                }
            }
            // O of this thread's row, 32 channels from 32 c on, with half B's where there is one
            auto output = [&](int c, float *o) {
                tmem_ld32(o_tm + 32 * c, o);
                tmem_ld_wait<32>(o);
                if (f_b == 0.0f) return;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float4 v = b_out[(8 * c + k) * kHalfRows + ht];
                    o[4 * k] = fmaf(o[4 * k], f_a, v.x * f_b);
                    o[4 * k + 1] = fmaf(o[4 * k + 1], f_a, v.y * f_b);
                    o[4 * k + 2] = fmaf(o[4 * k + 2], f_a, v.z * f_b);
                    o[4 * k + 3] = fmaf(o[4 * k + 3], f_a, v.w * f_b);
                }
            };
            // 32 channels of the output: o times `f` (which takes the 2^8 of V back) in BF16,
            // to the row's place in shared memory; then all rows of the warp, two at a time.
            // (Of doubled halves that memory has B's output: they store directly.)
            uint16_t *out_row = a.out + q_row * a.out_stride + static_cast<int64_t>(head) * kDim;
            auto store = [&](int c, const float *o, float f) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float t[8];
#pragma unroll
                    for (int d = 0; d < 8; ++d) t[d] = f != 0.0f ? o[8 * k + d] * f : 0.0f;
                    const uint4 v = pack_bf16x8(t);
                    if (!dual)
                        *staged(lane, 4 * c + k) = v;
                    else if (live)
                        reinterpret_cast<uint4 *>(out_row)[4 * c + k] = v;
                }
            };
            auto flush = [&] {
                if (dual) return;
                __syncwarp();
                const int64_t at = live ? out_row - a.out : -1;
#pragma unroll 2
                for (int i = 0; i < 16; ++i) {
                    const int64_t to = __shfl_sync(0xFFFFFFFFu, at, 2 * i + (lane >> 4));
                    if (to >= 0)
                        *reinterpret_cast<uint4 *>(a.out + to + (lane & 15) * 8) = *staged(2 * i + (lane >> 4), lane & 15);
                }
                __syncwarp();
            };
            auto store_lse = [&](float m, float l) {
                if (live && a.lse != nullptr)
                    a.lse[q_row * a.q_heads + head] =
                        l > 0.0f ? (m - kWeightLog2 + log2f(l)) * 0.69314718055994531f : -INFINITY;
            };
            if (sg->whole) {
                const float f = l_run > 0.0f ? __fdividef(256.0f, l_run) : 0.0f;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    float o[32];
                    output(c, o);
                    store(c, o, f);
                }
                flush();
                store_lse(m_run, l_run);
                if (dual) named_barrier(3, 256);
                continue;
            }
            // partial: this CTA's slot 1 if the item begins here, else slot 0
            const int c_first = sg->c_first, c_last = sg->c_last;
            auto slot = [&](int i) {
                return partials + (static_cast<int64_t>(2 * i + (i == c_first ? 1 : 0)) * 2 + half) * F::kPartial;
            };
            float *mine = slot(blockIdx.x);
            if (n > 0 && any_live) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    float o[32];
                    output(c, o);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        __stcg(reinterpret_cast<float4 *>(mine) + (8 * c + k) * kHalfRows + ht,
                               make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]));
                }
            }
            __stcg(mine + kHalfRows * kDim + ht, m_run);
            __stcg(mine + kHalfRows * (kDim + 1) + ht, l_run);
            if (dual) named_barrier(3, 256);
            __threadfence();
            named_barrier(1 + half, 128);
            if (ht == 0) {
                int *counter = counters + 2 * c_first + half;
                const bool last = atomicAdd(counter, 1) == c_last - c_first;
                if (last) *counter = 0;
                shared_last[half] = last;
                __threadfence();
            }
            named_barrier(1 + half, 128);
            if (!shared_last[half] || !any_live) continue;
            // join in the order of the CTAs, a row per thread
            float m = -INFINITY, l = 0.0f;
#pragma unroll 4
            for (int i = c_first; i <= c_last; ++i) m = fmaxf(m, __ldcg(slot(i) + kHalfRows * kDim + ht));
#pragma unroll 4
            for (int i = c_first; i <= c_last; ++i) {
                const float *p = slot(i) + kHalfRows * kDim + ht;
                const float mi = __ldcg(p), li = __ldcg(p + kHalfRows);
                l += mi > -INFINITY ? ex2(mi - m) * li : 0.0f;
            }
            const float f = l > 0.0f ? __fdividef(256.0f, l) : 0.0f;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                float o[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = 0.0f;
#pragma unroll 2
                for (int i = c_first; i <= c_last; ++i) {
                    const float *p = slot(i);
                    const float mi = __ldcg(p + kHalfRows * kDim + ht);
                    float4 v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[k] = __ldcg(reinterpret_cast<const float4 *>(p) + (8 * c + k) * kHalfRows + ht);
                    // without a maximum, its O may never have been written
                    const bool some = mi > -INFINITY;
                    const float fi = ex2(mi - m);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        o[4 * k] = some ? fmaf(fi, v[k].x, o[4 * k]) : o[4 * k];
                        o[4 * k + 1] = some ? fmaf(fi, v[k].y, o[4 * k + 1]) : o[4 * k + 1];
                        o[4 * k + 2] = some ? fmaf(fi, v[k].z, o[4 * k + 2]) : o[4 * k + 2];
                        o[4 * k + 3] = some ? fmaf(fi, v[k].w, o[4 * k + 3]) : o[4 * k + 3];
                    }
                }
                store(c, o, f);
            }
            flush();
            store_lse(m, l);
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace attn
}  // namespace fp8bq
