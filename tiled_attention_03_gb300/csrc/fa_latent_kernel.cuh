// fa_latent_kernel.cuh -- attention of a batch's new tokens over a paged cache of one
// latent row per token (the absorbed form of latent attention), on sm_103a.
//
// A row of the cache has DL latent elements and 64 rotary ones. Every head's key is the
// whole row and its value the latent part, so with q the absorbed query of a (token, head)
// pair
//     s_j = scale q . row_j,   O = sum_j softmax(s)_j row_j[0 .. DL),   LSE = ln sum_j exp(s_j)
// and all heads of all new tokens of a sequence are rows of one problem that reads each
// cached row once.
//
// Both products are taken transposed, S^T = K Q^T (64 keys x R rows) and O^T += V^T P^T
// (DL x R in slices of 128), because O of 128 rows and 512 columns would fill tensor memory
// by itself and leave no columns for S: with R <= 64 rows as the N of both products O^T takes
// DL / 128 * R columns (twice that for R <= 32, see below). A tile of 64 keys comes into shared memory once, by TMA from the
// pages, and is the K-major A operand of the first product and, read with its latent columns as
// M, the MN-major A operand of the second. It comes and goes in parts of 128 columns (the last
// with the rotary ones), each with its own barriers: the scores start on the first part, and
// the part of a slice of O^T that is done is loaded anew while the next slice is computed.
//
// S^T arrives with keys in lanes, 16 lanes of each warp's 32 (the layout of M = 64), and is
// read as 16 x 256 bit fragments: a thread holds 2 keys of each of R / 4 rows. The weights
// p = exp2(s scale log2 e - ref) go to shared memory through transposing 8 x 8 stores, as the
// K-major B operand of the second product; blocks of up to 32 rows hand them over as two 16-bit parts
// side by side, with columns of O^T for each that are added at the end. The reference of a row is lazy: it moves only
// when a score passes it by 2^8, so a tile costs the four warps one barrier with a vote and
// no row maximum; when it does move, the row's l and its column of O^T are rescaled.
//
// The work is cut as in fa_paged_kernel.cuh: all blocks of rows with all their key tiles,
// and kTicks more for a block's start and end, form one line, of which every worker takes an
// equal share; pieces of cut blocks are joined by a second kernel. A worker is G = 1 or 2
// CTAs that take the same tiles for R rows each, side by side, so that with more rows than R the
// second reads them from L2.
//
// What bounds it: with one block per sequence the chain of a tile, scores, softmax and product, as
// two tiles of 74 KB are all that shared memory holds at DL = 512: 8 sequences of 32768 rows, 32 heads, take
// 61 us, 5.0 TB/s, of which 13.5 are the start, the last output and the merge, and take 59 to 65
// without any key loads. With more blocks the products, 36 of M = 64 and 16 of M = 128 at 33 and 49 cycles at
// least, 1,970 of a tile's 2,300 cycles (1000 tokens of 16 heads on 14000 rows: 456 us, 1,110
// TFLOP/s; 433 without any key loads).
//
// Warps (256 threads): 0-3 softmax and outputs, 4 key tiles, 5 issuer of S^T, 6 issuer of
// O^T, 7 scheduler and Q tiles. What the issuers' branches and descriptors come from is taken
// from one lane by a shuffle, so that the compiler knows it to be the warp's and the products
// are issued from uniform registers (1000 x 16 rows on 14000 keys: 480 us at that point, 583 without).
// Every wait is bounded; on expiry the CTA records the failure, drains
// its copies and products, frees its tensor memory and returns. Waits of the softmax warps
// end in a vote before the next barrier, so that all four leave together.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "fa_divisor.cuh"
#include "fa_paged_kernel.cuh"
#include "fa_pdl.cuh"
#include "ptx.cuh"

namespace fa {
namespace latent {

constexpr int kBK = 64;     // keys per tile
constexpr int kDR = 64;     // rotary elements of a row
constexpr int kThreads = 256;
constexpr int kLoadWarp = 4, kScoreWarp = 5, kOutWarp = 6, kPlanWarp = 7;
// A block's start and end, in tiles (at 3, 4 and 6: 40 sequences of 0-16000 rows with 128 heads 53.3,
// 53.7 and 55.1 us, 96 of 0-12000 with 12 heads at DL 256 24.8, 25.2 and 26.9).
constexpr int kTicks = 3;
constexpr int kUnitSlots = 4;
constexpr int kUnitConsumers = 7;  // warps that take the pieces: all but the scheduler
constexpr int kMaxStages = 4;
constexpr int kMaxParts = 8;  // stages x parts
constexpr uint32_t kTmemCols = 512;
constexpr float kMoveAt = 8.0f;  // log2 units a score may pass its row's reference by
constexpr float kUnset = 3e38f;  // minus the reference of a row that has seen no key: any score passes it
constexpr unsigned kStatusTimeout = 4;
constexpr unsigned kStatusLayout = 2;  // shared memory base not 1024-aligned
constexpr uint32_t kTmem = 0;  // all columns of tensor memory are allocated: they start at 0

enum : int { kRoleSoftmax = 1, kRoleTma = 2, kRoleMma = 3 };

struct Params {
    void *O;
    float *LSE;
    float *part_O;     // [2 * CTAs][R][DL]: O / l of the pieces of cut blocks
    float *part_LSE;   // [2 * CTAs][R]
    paged::MergeInfo *info;  // [CTAs]
    const int *cu_q, *seq_k, *table;
    int B, H, group;   // CTAs per worker
    Divisor by_H;
    int rb_log2;       // rows of a block: group * R
    int total_q, max_pages, page_log2, num_pages, max_keys;
    int chunk;         // tokens per TMA box: min(page size, kBK)
    int page_step, page_none;  // the map's last coordinate: page * page_step; past its end
    int wl, wr;        // key j visible to the query at position i iff i - wl <= j <= i + wr
    unsigned line_most;  // the longest line of work that ascending offsets can make
    float scale_log2;
    unsigned long long wait_budget_ns;
    unsigned int *status;
    int fault_skip_k;  // test hook: every CTA skips the load at this ring position (-1: none)
};

// Shared memory: Q tiles (region after region of 64 columns, R rows of 128 bytes), the
// ring of key tiles (part after part; in a part of 128 columns groups of 8 keys with their two
// regions side by side, the rotary region's groups by themselves), the weights (R rows of 64
// keys), all with the 128-byte swizzle; then what is small.
template <int DL, int R>
struct Smem {
    static constexpr int kRegions = DL / 64 + 1;
    static constexpr int kParts = DL / 128;
    static constexpr int kAtom = 1024;                     // one region of a group
    static constexpr int kGroup = 2 * kAtom;
    static constexpr int kPart = kBK / 8 * kGroup;
    static constexpr int kTile = kParts * kPart + kBK / 8 * kAtom;
    static constexpr int kQRegion = R * 128;
    static constexpr int kQBytes = kRegions * kQRegion;
    // 16-bit parts of a weight in its product with the values, and the bytes of one part and of a buffer
    // of all. One alone puts O's error at 0.0021 where its own rounding is 0.0017 (bf16, relative,
    // root mean square). With up to 32 rows a second part costs little as R further columns of the same
    // products (8 sequences of 32768 rows 60.4 -> 61.1 us, 96 ragged ones 24.1 -> 24.5; as products of
    // its own 62.9 and 24.9). With 64 the products are the bound: at DL = 256 1000 tokens of 16 heads on
    // 14000 rows 335 -> 374 us, 40 sequences with 128 heads 39.9 -> 42.6; at DL = 512, where tensor memory
    // has no columns for it, a product of its own from the place of the tile's rotary part (which the
    // scores have used by then) 456 -> 614 and 53 -> 60. There weights are rounded, as in the forward
    // passes over whole sequences.
    static constexpr int kPParts = R <= 32 ? 2 : 1;
    static constexpr int kPPart = R * 128;
    static constexpr int kPBytes = kPParts * kPPart;
    static constexpr int kSmall = 3 * 1024;
    static constexpr int kMost = 227 * 1024 - kSmall;
    // two Q tiles (the next block's scores start while this one ends) and two buffers of weights
    // where two key tiles leave room for them, else two of weights where they do (16 sequences of 0-16000
    // rows, 20 heads, DL 512: 23.7 us, with two Q tiles in their place 25.0); the rest is for key tiles
    static constexpr int kQStages = 2 * kQBytes + 2 * kTile + 2 * kPBytes <= kMost ? 2 : 1;
    static constexpr int kPBufs = kQStages * kQBytes + 2 * kTile + 2 * kPBytes <= kMost ? 2 : 1;
    static constexpr int kFit = (kMost - kQStages * kQBytes - kPBufs * kPBytes) / kTile;
    // an even number, so that a slot of the ring has one buffer of scores and of weights
    static constexpr int kStages = (kFit < kMaxStages ? kFit : kMaxStages) / 2 * 2;
    static_assert(kStages >= 2, "shared memory");
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + kQStages * kQBytes;
    static constexpr int kP = kK + kStages * kTile;
    static constexpr int kBar = kP + kPBufs * kPBytes;
    static constexpr int kMisc = kBar + 48 * 8;        // TMEM address, abort flag
    static constexpr int kScan = kMisc + 16;           // 8 warp sums, the start of the share
    static constexpr int kRing = kScan + 64;           // kUnitSlots pieces
    static constexpr int kLimits = kRing + kUnitSlots * 64;  // first and last key of each row
    static constexpr int kFactor = kLimits + R * 8;    // a number per row
    static constexpr int kRef = kFactor + R * 4;       // minus the reference of each row
    static constexpr int kRed = kRef + R * 4;          // one per softmax warp and row
    static constexpr int kBytes = kRed + 4 * R * 4;
    static_assert(kRing % 16 == 0 && kLimits % 16 == 0 && kBytes - kBar <= kSmall, "layout");
    // more than half of the SM's shared memory: one CTA (and one holder of all 512
    // TMEM columns) per SM
    static constexpr int kAlloc = kBytes > 120 * 1024 ? kBytes : 120 * 1024;
    static constexpr uint32_t kTmemO = 0;
    static constexpr int kOCols = kPParts * R;  // of a slice of O^T: for each part of the weights the rows
    static constexpr uint32_t kTmemS = DL / 128 * kOCols;
    static_assert(kTmemS + 2 * R <= kTmemCols, "TMEM columns");
};

enum : int {
    kBarQFull = 0,                         // + stage (2)
    kBarQEmpty = 2,                        // + stage (2)
    kBarKFull = 4,                         // + stage and part
    kBarKEmpty = kBarKFull + kMaxParts,    // + stage and part
    kBarSFull = kBarKEmpty + kMaxParts,    // + buffer (2)
    kBarPFull = kBarSFull + 2,             // + buffer (2): weights written, scores read
    kBarPVDone = kBarPFull + 2,            // + buffer (2)
    kBarOFree = kBarPVDone + 2,
    kBarUnitFull = kBarOFree + 1,               // + slot
    kBarUnitEmpty = kBarUnitFull + kUnitSlots,  // + slot
    kBarDrain = kBarUnitEmpty + kUnitSlots,     // + issuer (2)
    kNumBars = kBarDrain + 2,
};
static_assert(kNumBars <= 48, "barrier slots");

// One piece of a block: n key tiles from j0 on (none: no row sees a key) for this CTA's
// rows r0 .. r0 + rows - 1 of sequence b, counted over (token, head) pairs.
struct Piece {
    int b, r0, rows;
    int j0, n;
    int lo_key, hi_key;  // the first and last key that any row of the block sees
    int q_off, nk;       // token i of the sequence stands at key position i + q_off
    int row0;            // the first row of all rows (token * H + head)
    int slot;            // partial slot, or -1: the whole block, written to O and LSE
};
static_assert(sizeof(Piece) <= 64, "ring slot");

struct Seq {
    int q0, nq, nk;
};
__device__ __forceinline__ Seq load_seq(int b, const Params &p) {
    Seq s{0, 0, 0};
    if (b >= p.B) return s;
    s.q0 = min(max(p.cu_q[b], 0), p.total_q);
    s.nq = min(max(p.cu_q[b + 1], s.q0), p.total_q) - s.q0;
    s.nk = min(max(p.seq_k[b], 0), p.max_keys);
    return s;
}
// Key tiles j0 .. j1 and keys lo .. hi that rows r0 .. r1 - 1 of a sequence see.
__device__ __forceinline__ void range_of(const Seq &s, int r0, int r1, const Params &p, int &lo, int &hi,
                                         int &j0, int &j1) {
    const int t0 = p.by_H.of(r0), tl = p.by_H.of(r1 - 1), q_off = s.nk - s.nq;
    lo = max(0, t0 + q_off - p.wl);
    hi = min(s.nk - 1, tl + q_off + p.wr);
    j0 = lo / kBK;
    j1 = hi < lo ? j0 - 1 : hi / kBK;
}
__device__ __forceinline__ int blocks_of(const Seq &s, const Params &p) {
    return (s.nq * p.H + (1 << p.rb_log2) - 1) >> p.rb_log2;
}
__device__ __forceinline__ int block_tiles(const Seq &s, int blk, const Params &p) {
    int lo, hi, j0, j1;
    range_of(s, blk << p.rb_log2, min((blk + 1) << p.rb_log2, s.nq * p.H), p, lo, hi, j0, j1);
    return j1 - j0 + 1;
}

// Ticks of sequence s (every thread of the warp calls it with its own). Those of many
// blocks are summed by the whole warp one after the other.
__device__ __forceinline__ unsigned seq_work(const Seq &s, const Params &p) {
    const int nb = blocks_of(s, p);
    unsigned w = 0;
    constexpr int kOwn = 4;
    if (nb <= kOwn)
        for (int x = 0; x < nb; ++x) w += block_tiles(s, x, p) + kTicks;
    unsigned todo = __ballot_sync(0xffffffffu, nb > kOwn);
    const int lane = threadIdx.x & 31;
    while (todo != 0) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const Seq o{0, __shfl_sync(0xffffffffu, s.nq, src), __shfl_sync(0xffffffffu, s.nk, src)};
        const int n = __shfl_sync(0xffffffffu, nb, src);
        unsigned part = 0;
        for (int x = lane; x < n; x += 32) part = paged::add_work(part, block_tiles(o, x, p) + kTicks);
        part = paged::warp_sum_work(part);
        if (lane == src) w = part;
    }
    return w;
}

__device__ __forceinline__ void record_timeout(const Params &p, volatile int *abort_flag, int role, int unit) {
    *abort_flag = 1;
    if (atomicCAS(p.status, 0u, kStatusTimeout) == 0u) {
        p.status[1] = static_cast<unsigned>(role);
        p.status[2] = static_cast<unsigned>(unit);
        p.status[3] = blockIdx.x;
        __threadfence();
    }
}

// 16 lanes x N / 4 runs of 256 bits, as 8-column blocks of two registers for lanes t / 4 and two
// for lanes t / 4 + 8, columns 2 (t mod 4) and the next: thread t's part of a 16 x 2N tile.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// 32 lanes x 16 consecutive columns, and the wait for them.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
// Four 8 x 8 matrices of 16-bit elements, stored transposed: lane i gives the address of row i mod 8
// of matrix i / 8.
__device__ __forceinline__ void store_transposed(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a),
                 "r"(b), "r"(c), "r"(d)
                 : "memory");
}
// Barrier of the four softmax warps, and whether any of their threads voted yes.
__device__ __forceinline__ bool any_of(bool mine) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(mine))
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

template <int DL, int R, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    fa_latent_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmR, const __grid_constant__ Params p) {
    using L = Smem<DL, R>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *const smem = smem_raw;
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + L::kBar;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);
    constexpr int kStart = kThreads / 32;  // its sequence, ticks into it, q0, nq, nk
    volatile unsigned *scan = reinterpret_cast<volatile unsigned *>(smem + L::kScan);
    auto bar = [bar0](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    auto sQ = [sbase](int k) { return sbase + L::kQ + (k % L::kQStages) * L::kQBytes; };
    auto sK = [sbase](int t) { return sbase + L::kK + (t % L::kStages) * L::kTile; };
    auto sP = [sbase](int t) { return sbase + L::kP + (t % L::kPBufs) * L::kPBytes; };
    auto slot_of = [smem](int k) {
        return reinterpret_cast<Piece *>(smem + L::kRing + (k % kUnitSlots) * 64);
    };
    // (from one lane: the compiler then knows that the roles' branches are the warp's)
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
    const int lane = threadIdx.x & 31;
    const uint64_t budget = p.wait_budget_ns;
    // worker w's CTAs stand side by side; numbered worker by worker within each place of the
    // group, so that a cut block's pieces have consecutive numbers
    const int workers = gridDim.x / p.group, worker = blockIdx.x / p.group, sub = blockIdx.x % p.group;
    const int cta = sub * workers + worker;

    if ((sbase & 1023u) != 0) {
        after_previous();
        if (threadIdx.x == 0) {
            atomicCAS(p.status, 0u, kStatusLayout);
            p.info[cta].last_cta = -1;
        }
        return;
    }
    // what needs nothing of the kernel before
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    if (threadIdx.x == kLoadWarp * 32) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(kBarQFull + s), 1);
            mbar_init(bar(kBarQEmpty + s), 1);
            mbar_init(bar(kBarSFull + s), 1);
            mbar_init(bar(kBarPFull + s), 128);
            mbar_init(bar(kBarPVDone + s), 1);
            mbar_init(bar(kBarDrain + s), 1);
        }
        for (int s = 0; s < L::kStages * L::kParts; ++s) {
            mbar_init(bar(kBarKFull + s), 1);
            mbar_init(bar(kBarKEmpty + s), 1);
        }
        mbar_init(bar(kBarOFree), 128);
        for (int k = 0; k < kUnitSlots; ++k) {
            mbar_init(bar(kBarUnitFull + k), 1);
            mbar_init(bar(kBarUnitEmpty + k), kUnitConsumers);
        }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmR);
    }
    after_previous();
    let_next_start();

    // ---- this worker's share of the line of work: ticks w0 .. w1 - 1 of W
    auto scanned = [&](unsigned w, unsigned &all) -> unsigned {  // sum of w up to this thread, and of all
        unsigned incl = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl = paged::add_work(incl, x);
        }
        __syncthreads();
        if (lane == 31) scan[warp] = incl;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        unsigned before = 0;
        all = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) before = paged::add_work(before, scan[i]);
            all = paged::add_work(all, scan[i]);
        }
        return paged::add_work(before, incl);
    };
    const Seq seq0 = load_seq(static_cast<int>(threadIdx.x), p);
    const unsigned work0 = seq_work(seq0, p);
    unsigned W, incl0 = scanned(work0, W);
    for (int b0 = kThreads; b0 < p.B; b0 += kThreads) {
        unsigned more;
        scanned(seq_work(load_seq(b0 + static_cast<int>(threadIdx.x), p), p), more);
        W = paged::add_work(W, more);
    }
    // more than an ordered batch of these sizes can have: offsets in no order, the batch is left alone
    if (W > p.line_most) W = 0;
    const unsigned T = (W + workers - 1) / workers;
    const unsigned w0 = min(worker * T, W), w1 = min(w0 + T, W);
    auto start_at = [&](int b, const Seq &s, unsigned incl, unsigned w) {
        if (incl - w <= w0 && w0 < incl) {
            scan[kStart] = static_cast<unsigned>(b);
            scan[kStart + 1] = w0 - (incl - w);
            scan[kStart + 2] = static_cast<unsigned>(s.q0);
            scan[kStart + 3] = static_cast<unsigned>(s.nq);
            scan[kStart + 4] = static_cast<unsigned>(s.nk);
        }
    };
    if (w0 < w1) {
        start_at(static_cast<int>(threadIdx.x), seq0, incl0, work0);
        unsigned carry = 0;
        for (int b0 = kThreads; b0 < p.B; b0 += kThreads) {
            unsigned all;
            if (b0 == kThreads) scanned(work0, carry);
            const int b = b0 + static_cast<int>(threadIdx.x);
            const Seq s = load_seq(b, p);
            const unsigned w = seq_work(s, p);
            const unsigned incl = carry + scanned(w, all);
            start_at(b, s, incl, w);
            carry += all;
        }
    }
    const bool idle = w0 >= w1 || *tmem_slot != kTmem;  // nothing left for this worker
    if (idle && threadIdx.x == 0) {
        p.info[cta].last_cta = -1;
        if (*tmem_slot != kTmem) atomicCAS(p.status, 0u, kStatusLayout);
    }
    __syncthreads();
    constexpr uint32_t tmem = kTmem;

    // The k-th piece of this CTA (every role walks the same pieces). b < 0: no more.
    auto take = [&](int k, bool &ok) -> Piece {
        Piece P{};
        P.b = -1;
        const int slot = k % kUnitSlots;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarUnitFull + slot), (k / kUnitSlots) & 1,
                                                       abort_flag, budget));
        if (!ok) return P;
        P = *slot_of(k);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarUnitEmpty + slot));
        return P;
    };

    if (idle) {
        // (frees its tensor memory below)
    } else if (warp == kPlanWarp) {
        // ================================================================ scheduler and Q tiles
        // the block that holds tick w0, by the whole warp, and the ticks `rem` of it that
        // belong to the worker before
        int b = static_cast<int>(scan[kStart]), blk = 0, rem = static_cast<int>(scan[kStart + 1]);
        Seq s{static_cast<int>(scan[kStart + 2]), static_cast<int>(scan[kStart + 3]),
              static_cast<int>(scan[kStart + 4])};
        int nb = blocks_of(s, p);
        for (int x0 = 0; x0 < nb && nb > 1; x0 += 32) {
            const int n = x0 + lane < nb ? block_tiles(s, x0 + lane, p) + kTicks : 0;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, rem < incl);
            if (hit != 0) {
                const int at = __ffs(hit) - 1;
                blk = x0 + at;
                rem -= __shfl_sync(0xffffffffu, incl - n, at);
                break;
            }
            rem -= __shfl_sync(0xffffffffu, incl, 31);
        }
        unsigned w = w0;
        bool ok = true;
        paged::MergeInfo info{};
        info.last_cta = -1;
        int pieces = 0;
        // Finds the k-th piece and publishes it (by the whole warp, uniformly).
        auto publish = [&](int k) -> Piece {
            Piece P{};
            P.b = -1;
            const int slot = k % kUnitSlots;
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarUnitEmpty + slot),
                                                           ((k / kUnitSlots) & 1) ^ 1, abort_flag, budget));
            if (!ok) return P;
            while (w < w1 && P.b < 0) {
                int lo, hi, j0, j1;
                const int nrows = s.nq * p.H, first_row = blk << p.rb_log2;
                range_of(s, first_row, min(first_row + (1 << p.rb_log2), nrows), p, lo, hi, j0, j1);
                const int n = j1 - j0 + 1;
                const int len = min(n + kTicks - rem, static_cast<int>(w1 - w));
                // this share's tiles of the block: ja .. je - 1
                const int ja = max(rem - kTicks, 0), je = rem + len - kTicks;
                const int r0 = first_row + sub * R, rows = min(r0 + R, nrows) - r0;
                if (rows > 0 && (n == 0 ? rem == 0 : je > ja)) {
                    P.b = b;
                    P.r0 = r0;
                    P.rows = rows;
                    P.lo_key = lo;
                    P.hi_key = hi;
                    P.q_off = s.nk - s.nq;
                    P.nk = s.nk;
                    P.row0 = s.q0 * p.H + r0;
                    P.j0 = j0 + ja;
                    P.n = n == 0 ? 0 : je - ja;
                    const bool starts = ja == 0, ends = n == 0 || je == n;
                    P.slot = starts && ends ? -1 : 2 * cta + (pieces > 0);
                    if (n > 0) ++pieces;
                    if (starts && !ends) {
                        info.last_cta = sub * workers + static_cast<int>((w - rem + kTicks + n - 1) / T);
                        info.slot = P.slot;
                        info.slot_rows = R;
                        info.rows = rows;
                        info.tok0 = 0;
                        info.head0 = P.row0;
                    }
                }
                w += len;
                rem = 0;
                if (++blk == nb) {
                    blk = 0;
                    while (w < w1 && ++b < p.B) {
                        s = load_seq(b, p);
                        nb = blocks_of(s, p);
                        if (nb > 0) break;
                    }
                    if (b >= p.B) w = w1;
                }
            }
            if (lane == 0) {
                *slot_of(k) = P;
                mbar_arrive(bar(kBarUnitFull + slot));
            }
            __syncwarp();
            return P;
        };
        int q_loads = 0;
        for (int k = 0; ok; ++k) {
            const Piece P = publish(k);
            if (!ok || P.b < 0) break;
            if (P.n == 0) continue;
            const int qs = q_loads % L::kQStages;
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarQEmpty + qs), ((q_loads / L::kQStages) & 1) ^ 1,
                                                           abort_flag, budget));
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(bar(kBarQFull + qs), L::kQBytes);
            __syncwarp();
            if (lane < L::kRegions)
                tma_load_3d(sQ(q_loads) + lane * L::kQRegion, &tmQ, bar(kBarQFull + qs), 64 * lane, 0, P.row0);
            __syncwarp();
            ++q_loads;
        }
        if (lane == 0) {
            p.info[cta] = info;
            if (!ok) record_timeout(p, abort_flag, kRoleTma, -1);
            for (int st = 0; st < L::kQStages; ++st)
                if (q_loads > st) {
                    const int last = q_loads - 1 - ((q_loads - 1 - st) % L::kQStages);
                    mbar_wait_bounded(bar(kBarQFull + st), (last / L::kQStages) & 1, nullptr, budget);
                }
        }
    } else if (warp == kLoadWarp) {
        // ================================================================ key tiles
        // Chunks of key tile j that hold a key of the piece's block; chunk `lane`'s page and
        // first token in it. Returns the ballot of the chunks to load.
        auto chunk_of = [&](const Piece &P, int j, int &page, int &tok) -> uint32_t {
            const int k0 = j * kBK + lane * p.chunk;
            const bool need = lane * p.chunk < kBK && k0 + p.chunk > P.lo_key && k0 <= P.hi_key;
            page = 0;
            tok = k0 & ((1 << p.page_log2) - 1);
            if (need) {
                page = p.table[static_cast<size_t>(P.b) * p.max_pages + (k0 >> p.page_log2)];
                // a page number outside the cache reads as zeros
                page = page >= 0 && page < p.num_pages ? page * p.page_step : p.page_none;
            }
            return __ballot_sync(0xffffffffu, need);
        };
        int t = 0, issued = 0;  // tiles, and their parts
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const Piece P = take(k, ok);
            if (!ok || P.b < 0) break;
            if (P.n == 0) continue;
            int page, tok;
            uint32_t need = chunk_of(P, P.j0, page, tok);
            for (int x = 0; ok && x < P.n; ++x, ++t) {
                const int st = t % L::kStages * L::kParts;
                // the next tile's page numbers are on their way while this one waits
                int page_n = 0, tok_n = 0;
                uint32_t need_n = 0;
                if (x + 1 < P.n) need_n = chunk_of(P, P.j0 + x + 1, page_n, tok_n);
                const uint32_t keys = static_cast<uint32_t>(__popc(need)) * p.chunk;
#pragma unroll
                for (int part = 0; part < L::kParts; ++part) {
                    ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarKEmpty + st + part),
                                                                         ((t / L::kStages) & 1) ^ 1, abort_flag, budget));
                    if (!ok) break;
                    ++issued;
                    if (t == p.fault_skip_k) continue;
                    const bool last = part + 1 == L::kParts;
                    const uint32_t full = bar(kBarKFull + st + part);
                    if (lane == 0) mbar_arrive_expect_tx(full, keys * (last ? 384 : 256));
                    __syncwarp();
                    if ((need >> lane) & 1u) {
                        paged::tma_load_5d(sK(t) + part * L::kPart + lane * (p.chunk >> 3) * L::kGroup, &tmK, full, 0,
                                           0, 2 * part, tok >> 3, page);
                        if (last)
                            paged::tma_load_5d(sK(t) + L::kParts * L::kPart + lane * (p.chunk >> 3) * L::kAtom, &tmR,
                                               full, 0, 0, L::kRegions - 1, tok >> 3, page);
                    }
                    __syncwarp();
                }
                page = page_n;
                tok = tok_n;
                need = need_n;
            }
        }
        if (lane == 0) {
            if (!ok) record_timeout(p, abort_flag, kRoleTma, -1);
            // copies in flight: the last one of every barrier, all within one budget
            const uint64_t t0 = global_timer_ns();
            for (int st = 0; st < L::kStages; ++st)
                for (int part = 0; part < L::kParts; ++part) {
                    const int n = (issued - part + L::kParts - 1) / L::kParts;  // tiles whose part was issued
                    if (n <= st) continue;
                    const int last = n - 1 - ((n - 1 - st) % L::kStages);
                    const uint64_t spent = global_timer_ns() - t0;
                    mbar_wait_bounded(bar(kBarKFull + st * L::kParts + part), (last / L::kStages) & 1, nullptr,
                                      spent < budget ? budget - spent : 0);
                }
        }
    } else if (warp == kScoreWarp || warp == kOutWarp) {
        // ================================================================ issuers of the products
        const bool scores = warp == kScoreWarp;
        constexpr uint32_t idesc_s = idesc_f16_ab(BF16, kBK, R, false, false);
        constexpr uint32_t idesc_o = idesc_f16_ab(BF16, 128, L::kOCols, true, false);
        // a value that all lanes have, from one of them: the compiler then keeps what follows from
        // it in uniform registers, which the products take their descriptors from
        auto one = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
        auto wait = [&](int b, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait_bounded(bar(b), parity, abort_flag, budget));
        };
        // Latent columns of rows r0 .. r1 - 1 of key tile t: 0 times whatever the page holds there
        // must be 0.
        auto zero_rows = [&](int t, int r0, int r1) {
            uint8_t *base = smem + L::kK + (t % L::kStages) * L::kTile;
            constexpr int kPer = DL / 8;  // 16-byte pieces of a row
            for (int c = r0 * kPer + lane; c < r1 * kPer; c += 32) {
                const int r = c / kPer, x = c % kPer;
                *reinterpret_cast<uint4 *>(base + (x >> 4) * L::kPart + (r >> 3) * L::kGroup + ((x >> 3) & 1) * L::kAtom +
                                           (r & 7) * 128 + (x & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
        };
        int t = 0, live = 0;  // key tiles, and pieces with tiles, so far
        bool ok = true;
        int k = 0;
        for (; ok; ++k) {
            const Piece P = take(k, ok);
            const int pb = one(P.b), n = one(P.n), j0 = one(P.j0), lo = one(P.lo_key), hi = one(P.hi_key);
            if (!ok || pb < 0) break;
            if (n == 0) continue;
            if (scores) {
                ok = wait(kBarQFull + live % L::kQStages, (live / L::kQStages) & 1);
                const uint64_t db = paged::tile_desc<128>(sQ(live), 16, 1024);
                for (int x = 0; ok && x < n; ++x, ++t) {
                    const uint32_t phase = (t / L::kStages) & 1;
                    const int st = t % L::kStages * L::kParts;
                    // the scores before in this buffer have been read
                    if (t >= 2) ok = wait(kBarPFull + t % 2, (t / 2 - 1) & 1);
                    if (!ok) break;
                    const uint32_t d = kTmem + L::kTmemS + (t % 2) * R;
                    const uint64_t da = paged::tile_desc<128>(sK(t), 16, L::kGroup);
                    const uint64_t dr = paged::tile_desc<128>(sK(t) + L::kParts * L::kPart, 16, L::kAtom);
#pragma unroll
                    for (int part = 0; part < L::kParts; ++part) {
                        ok = ok && wait(kBarKFull + st + part, phase);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                umma_f16_ss(d, da + part * (L::kPart >> 4) + (c / 4) * (L::kAtom >> 4) + (c % 4) * 2,
                                            db + (2 * part + c / 4) * (L::kQRegion >> 4) + (c % 4) * 2, idesc_s,
                                            part > 0 || c > 0 ? 1u : 0u);
                            if (part + 1 == L::kParts) {
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    umma_f16_ss(d, dr + c * 2, db + 2 * L::kParts * (L::kQRegion >> 4) + c * 2, idesc_s,
                                                1u);
                                umma_commit(bar(kBarSFull + t % 2));
                            }
                        }
                        __syncwarp();
                    }
                }
                if (ok) {
                    if (elect_one()) umma_commit(bar(kBarQEmpty + live % L::kQStages));
                    __syncwarp();
                }
            } else {
                for (int x = 0; ok && x < n; ++x, ++t) {
                    // the tile's rows a .. b hold keys lo .. hi: the product takes the steps of 16 that
                    // have one of them, whose other rows become 0 (hidden keys' scores, which may be read
                    // meanwhile, are not looked at)
                    const int kv0 = (j0 + x) * kBK, a = max(lo - kv0, 0), b = min(hi - kv0, kBK - 1);
                    const int c0 = a / 16, c1 = b / 16, st = t % L::kStages * L::kParts;
                    if ((a & 15) != 0 || (b & 15) != 15) {
                        for (int part = 0; ok && part < L::kParts; ++part)
                            ok = wait(kBarKFull + st + part, (t / L::kStages) & 1);
                        if (!ok) break;
                        zero_rows(t, c0 * 16, a);
                        zero_rows(t, b + 1, c1 * 16 + 16);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    ok = wait(kBarPFull + t % 2, (t / 2) & 1);
                    if (ok && x == 0 && live > 0) ok = wait(kBarOFree, (live - 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t da = paged::tile_desc<128>(sK(t), L::kAtom, L::kGroup);
                    const uint64_t db = paged::tile_desc<128>(sP(t), 16, 1024);
                    if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < L::kParts; ++s) {
#pragma unroll
                            for (int c = 0; c < kBK / 16; ++c)
                                if (c >= c0 && c <= c1)
                                    umma_f16_ss(kTmem + L::kTmemO + s * L::kOCols,
                                                da + s * (L::kPart >> 4) + c * ((2 * L::kGroup) >> 4), db + c * 2,
                                                idesc_o, x > 0 || c > c0 ? 1u : 0u);
                            umma_commit(bar(kBarKEmpty + st + s));
                        }
                        umma_commit(bar(kBarPVDone + t % 2));
                    }
                    __syncwarp();
                }
            }
            ++live;
        }
        if (!ok && lane == 0) record_timeout(p, abort_flag, kRoleMma, k);
        const int drain = kBarDrain + (scores ? 0 : 1);
        if (elect_one()) umma_commit(bar(drain));
        __syncwarp();
        if (lane == 0) mbar_wait_bounded(bar(drain), 0, nullptr, budget);
        __syncwarp();
    } else if (warp < 4) {
        // ================================================================ softmax and outputs
        constexpr int kOwn = R / 4;  // rows of which this thread holds two keys
        const uint32_t tl = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        const float sl2 = p.scale_log2;
        const int kq = lane >> 2, cq = lane & 3;
        // its i-th row
        auto row_of = [cq](int i) { return 8 * (i >> 1) + 2 * cq + (i & 1); };
        int2 *limits = reinterpret_cast<int2 *>(smem + L::kLimits);
        float *factor = reinterpret_cast<float *>(smem + L::kFactor);
        float *ref = reinterpret_cast<float *>(smem + L::kRef);
        float *red = reinterpret_cast<float *>(smem + L::kRed);
        bool dead = false;  // a wait has run out
        auto wait = [&](int b, uint32_t parity) {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar(b), parity, abort_flag, budget))) {
                dead = true;
                *abort_flag = 1;
            }
        };
        int t = 0, live = 0, k = 0;
        while (true) {
            bool ok;
            const Piece P = take(k, ok);
            ++k;
            if (!ok) dead = true;
            if (any_of(dead || P.b < 0)) break;
            const int tid = threadIdx.x;
            if (P.n == 0) {  // no row sees a key
                for (int c = tid; c < P.rows * (DL / 8); c += 128)
                    reinterpret_cast<uint4 *>(p.O)[static_cast<size_t>(P.row0) * (DL / 8) + c] = make_uint4(0, 0, 0, 0);
                if (tid < P.rows) p.LSE[P.row0 + tid] = -INFINITY;
                continue;
            }
            if (tid < R) {
                const int i = p.by_H.of(P.r0 + min(tid, P.rows - 1)) + P.q_off;
                limits[tid] = make_int2(max(0, i - p.wl), min(P.nk - 1, i + p.wr));
            }
            softmax_sync();
            // a tile with keys in [lo_last, hi_first] only is visible to every row
            const int lo_last = limits[P.rows - 1].x, hi_first = limits[0].y;
            // minus the row's reference, also in ref[]; kUnset before there is one, -inf (weights 0)
            // for rows that are not there
            float nm[kOwn], l[kOwn];
#pragma unroll
            for (int i = 0; i < kOwn; ++i) nm[i] = l[i] = 0.f;  // (set on the first tile)
            bool broken = false;
            for (int x0 = 0; x0 < P.n; ++x0, ++t) {
                const uint32_t tS = tl + L::kTmemS + (t % 2) * R;
                const int key = (P.j0 + x0) * kBK + warp * 16 + kq;  // and key + 8
                const bool whole = (P.j0 + x0) * kBK >= lo_last && (P.j0 + x0) * kBK + kBK - 1 <= hi_first;
                wait(kBarSFull + t % 2, (t / 2) & 1);
                tc_fence_after();
                float x[R / 2];
                // s scale log2 e - reference; -inf for hidden keys
                auto load = [&]() -> float {
                    uint32_t s[R / 2];
                    tmem_ld_frag(tS, s);
                    float top = -INFINITY;
#pragma unroll
                    for (int c = 0; c < R / 2; c += 2) {
                        // registers c, c + 1: rows i, i + 1 of block c / 4; key (+ 8 for odd c / 2)
                        const int i = (c >> 2) * 2;
                        x[c] = __uint_as_float(s[c]);
                        x[c + 1] = __uint_as_float(s[c + 1]);
                        ffma2(x[c], x[c + 1], sl2, sl2, nm[i], nm[i + 1]);
                    }
                    if (!whole) {
#pragma unroll
                        for (int i = 0; i < kOwn; ++i) {
                            const int2 lim = limits[row_of(i)];
                            const int c = (i >> 1) * 4 + (i & 1);
                            if (key < lim.x || key > lim.y) x[c] = -INFINITY;
                            if (key + 8 < lim.x || key + 8 > lim.y) x[c + 2] = -INFINITY;
                        }
                    }
#pragma unroll
                    for (int c = 0; c < R / 2; c += 2) top = max3f(top, x[c], x[c + 1]);
                    return top;
                };
                // a block's first tile sets the references
                bool move = x0 == 0;
                if (!move) move = any_of(load() > kMoveAt || dead);
                if (move) {
                    if (any_of(dead)) {
                        broken = true;
                        break;
                    }
                    // ---- references move: each row's maximum of this tile, through the buffer of the
                    // weights (free once the product before has completed; O^T then holds the sum
                    // through the tile before): entry (row, 8 warp + kq), 32 to a row
                    if (t > 0) wait(kBarPVDone + (t - 1) % 2, ((t - 1) / 2) & 1);
                    float *most = reinterpret_cast<float *>(smem + L::kP + (t % L::kPBufs) * L::kPBytes);
                    {
                        uint32_t s[R / 2];
                        tmem_ld_frag(tS, s);
#pragma unroll
                        for (int i = 0; i < kOwn; ++i) {
                            const int c = (i >> 1) * 4 + (i & 1);
                            const int2 lim = limits[row_of(i)];
                            const float a = key < lim.x || key > lim.y ? -INFINITY : __uint_as_float(s[c]);
                            const float b = key + 8 < lim.x || key + 8 > lim.y ? -INFINITY : __uint_as_float(s[c + 2]);
                            // (a row's 16-byte pieces stand in an order of their own: fewer bank conflicts)
                            most[row_of(i) * 32 + ((warp * 8 + kq) ^ ((row_of(i) & 7) << 2))] = fmaxf(a, b);
                        }
                    }
                    softmax_sync();
                    constexpr int kShare = 128 / R;  // threads of a row
                    const int own_row = tid / kShare;
                    float own_max = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 8 / kShare; ++i) {
                        const float4 v = *reinterpret_cast<const float4 *>(
                            most + own_row * 32 + (((tid % kShare + i * kShare) ^ (own_row & 7)) << 2));
                        own_max = fmaxf(own_max, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
                    }
#pragma unroll
                    for (int o = 1; o < kShare; o <<= 1)
                        own_max = fmaxf(own_max, __shfl_xor_sync(0xffffffffu, own_max, o));
                    if (tid % kShare == 0) {
                        const float old = x0 == 0 ? (own_row < P.rows ? kUnset : -INFINITY) : ref[own_row];
                        const float m = own_max * sl2;
                        const bool above = m > -old;  // above the reference (or the first)
                        factor[own_row] = above ? ex2_approx(-m - old) : 1.f;
                        ref[own_row] = above ? -m : old;
                    }
                    softmax_sync();
#pragma unroll
                    for (int i = 0; i < kOwn; i += 2) {
                        const float2 f = *reinterpret_cast<const float2 *>(factor + row_of(i));
                        const float2 n = *reinterpret_cast<const float2 *>(ref + row_of(i));
                        l[i] *= f.x, l[i + 1] *= f.y;
                        nm[i] = n.x, nm[i + 1] = n.y;
                    }
                    if (x0 > 0) {
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < DL / 128 * L::kOCols; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(tl + L::kTmemO + c, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * factor[c % R + e]);
                            tmem_st16(tl + L::kTmemO + c, o);
                        }
                        tmem_st_wait();
                    }
                    load();
                }
                // ---- weights: l keeps the fp32 values, the product takes 16 bits, or the sum of two parts of
                // 16 bits (see kPParts)
#pragma unroll
                for (int c = 0; c < R / 2; ++c) x[c] = ex2_approx(x[c]);
#pragma unroll
                for (int i = 0; i < kOwn; i += 2) {
                    const int c = i * 2;
                    fadd2(l[i], l[i + 1], x[c], x[c + 1]);
                    fadd2(l[i], l[i + 1], x[c + 2], x[c + 3]);
                }
                // the product with the weights before in this buffer has completed
                if (t >= L::kPBufs) wait(kBarPVDone + (t - L::kPBufs) % 2, ((t - L::kPBufs) / 2) & 1);
                const uint32_t base = sP(t);
#pragma unroll
                for (int b = 0; b < R / 8; b += 2) {
                    const int c = 4 * b;
                    const int r = 8 * (b + (lane >> 4)) + (lane & 7), octet = 2 * warp + ((lane >> 3) & 1);
                    const uint32_t at = base + r * 128 + ((octet ^ (r & 7)) << 4);
                    if constexpr (L::kPParts == 2) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) two_parts<BF16>(x[c + 2 * e], x[c + 2 * e + 1], hi[e], lo[e]);
                        store_transposed(at, hi[0], hi[1], hi[2], hi[3]);
                        store_transposed(at + L::kPPart, lo[0], lo[1], lo[2], lo[3]);
                    } else {
                        store_transposed(at, pack2<BF16>(x[c], x[c + 1]), pack2<BF16>(x[c + 2], x[c + 3]),
                                         pack2<BF16>(x[c + 4], x[c + 5]), pack2<BF16>(x[c + 6], x[c + 7]));
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(bar(kBarPFull + t % 2));
            }
            if (broken) break;
            // ---- epilogue: O / l rounded to 16 bit, LSE = ln 2 (m + log2 l); a piece of a
            // cut block keeps both in fp32 for the merge
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
                if (kq == 0) red[warp * R + row_of(i)] = l[i];
            }
            softmax_sync();
            float sum = 0.f, m = 0.f;
            if (tid < R) {
                sum = (red[tid] + red[R + tid]) + (red[2 * R + tid] + red[3 * R + tid]);
                m = -ref[tid];
                factor[tid] = sum == 0.f ? 0.f : 1.f / sum;
            }
            wait(kBarPVDone + (t - 1) % 2, ((t - 1) / 2) & 1);
            if (any_of(dead)) break;
            if (tid < P.rows) {
                const float lse = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994530942f;
                if (P.slot < 0)
                    p.LSE[P.row0 + tid] = lse;
                else
                    p.part_LSE[static_cast<size_t>(P.slot) * R + tid] = lse;
            }
            tc_fence_after();
            // lane = a column of O, register = a row
            const size_t row0 = P.slot < 0 ? static_cast<size_t>(P.row0) : static_cast<size_t>(P.slot) * R;
            const size_t at0 = row0 * DL + warp * 32 + lane;
            constexpr int kParts = L::kParts;
            // 32 rows (or R) of a slice of O^T at a time (with the next ones asked for ahead the code is
            // twice as long, 8 % slower at 128 heads)
            constexpr int kAtOnce = R < 32 ? R : 32, kSteps = R / kAtOnce * kParts;
#pragma unroll 1
            for (int x = 0; x < kSteps; ++x) {
                const int part = x * kAtOnce / R, r0 = x * kAtOnce % R, left = P.rows - r0;
                if (left <= 0) continue;
                uint32_t o[kAtOnce];
                auto columns = [&](int at, uint32_t(&o)[kAtOnce]) {
                    if constexpr (kAtOnce == 32) {
                        tmem_ld32(tl + L::kTmemO + at, o);
                        tmem_ld_wait(o);
                    } else {
                        tmem_ld16(tl + L::kTmemO + at, o);
                    }
                };
                columns(part * L::kOCols + r0, o);
                if constexpr (L::kPParts == 2) {
                    uint32_t more[kAtOnce];
                    columns(part * L::kOCols + R + r0, more);
#pragma unroll
                    for (int e = 0; e < kAtOnce; ++e)
                        o[e] = __float_as_uint(__uint_as_float(o[e]) + __uint_as_float(more[e]));
                }
                float y[kAtOnce];
                // a row without keys: 0, whatever its column holds
#pragma unroll
                for (int e = 0; e < kAtOnce; e += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(factor + r0 + e);
                    y[e] = f.x == 0.f ? 0.f : __uint_as_float(o[e]) * f.x;
                    y[e + 1] = f.y == 0.f ? 0.f : __uint_as_float(o[e + 1]) * f.y;
                    y[e + 2] = f.z == 0.f ? 0.f : __uint_as_float(o[e + 2]) * f.z;
                    y[e + 3] = f.w == 0.f ? 0.f : __uint_as_float(o[e + 3]) * f.w;
                }
                const size_t at = at0 + static_cast<size_t>(r0) * DL + part * 128;
                if (P.slot < 0) {
                    uint16_t *to = static_cast<uint16_t *>(p.O) + at;
#pragma unroll
                    for (int e = 0; e < kAtOnce; e += 2) {
                        const uint32_t two = pack2<BF16>(y[e], y[e + 1]);
                        if (e < left) to[e * DL] = static_cast<uint16_t>(two);
                        if (e + 1 < left) to[(e + 1) * DL] = static_cast<uint16_t>(two >> 16);
                    }
                } else {
                    float *to = p.part_O + at;
#pragma unroll
                    for (int e = 0; e < kAtOnce; ++e)
                        if (e < left) to[e * DL] = y[e];
                }
            }
            tc_fence_before();
            mbar_arrive(bar(kBarOFree));
            ++live;
        }
        if (dead && lane == 0) record_timeout(p, abort_flag, kRoleSoftmax, k);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(*tmem_slot, kTmemCols);
    }
}

// Joins the pieces of the cut blocks. With O_s, LSE_s of piece s
//     LSE = ln sum_s exp(LSE_s)          O = sum_s exp(LSE_s - LSE) O_s
// around the largest LSE_s, in a fixed order. Every thread block lists the cut blocks in shared memory,
// with the rows before each, and takes every gridDim-th batch of the rows. A thread holds four
// columns of a row; with fewer rows than there are places for them, several groups of DL / 4
// threads share a row's pieces and are summed at the end. Bound by latency: statistics and the first
// pieces are asked for together. (A block per row, most of which found nothing to do, took 14 us for 32 rows
// of 8 sequences in 20 pieces.)
struct MergeParams {
    const paged::MergeInfo *info;
    const float *part_O, *part_LSE;
    void *O;
    float *LSE;
    int ctas;
};
constexpr int kMergeThreads = 512;
constexpr int kMergeMost = 512;  // CTAs at most
constexpr int kMergeBlocks = 2;  // per SM

template <int DL, bool BF16>
__global__ void __launch_bounds__(kMergeThreads, kMergeBlocks) fa_latent_merge_kernel(const MergeParams p) {
    constexpr int kAcross = DL / 4, kPlaces = kMergeThreads / kAcross;
    __shared__ float4 sums[kMergeThreads];
    __shared__ int before[kMergeMost], warp_rows[kMergeThreads / 32];
    __shared__ int4 units[kMergeMost];  // pieces, first slot, rows of a slot, first row of all
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    after_previous();
    let_next_start();
    // rows of the cut blocks up to this one's
    static_assert(kMergeMost == kMergeThreads, "a CTA per thread");
    int rows = 0;
    if (tid < p.ctas) {
        const paged::MergeInfo u = p.info[tid];
        rows = u.last_cta >= 0 ? u.rows : 0;
        units[tid] = make_int4(u.last_cta - tid + 1, u.slot, u.slot_rows, u.head0);
    }
    int incl = rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) warp_rows[warp] = incl;
    __syncthreads();
    int total_rows = 0;
#pragma unroll
    for (int i = 0; i < kMergeThreads / 32; ++i) {
        if (i < warp) incl += warp_rows[i];
        total_rows += warp_rows[i];
    }
    before[tid] = incl - rows;
    __syncthreads();
    int groups = 1;  // per row
    while (groups < kPlaces && total_rows * groups * 2 <= static_cast<int>(gridDim.x) * kPlaces) groups *= 2;
    const int per_block = kPlaces / groups;
    const int place = tid / kAcross, col = tid % kAcross, group = place % groups;
    for (int x0 = blockIdx.x * per_block; x0 < total_rows; x0 += gridDim.x * per_block) {
        const bool there = x0 + place / groups < total_rows;
        const int x = min(x0 + place / groups, total_rows - 1);
        // the last CTA with no more than x rows before it: its block
        int c = 0;
#pragma unroll
        for (int step = kMergeMost / 2; step > 0; step >>= 1)
            if (before[c + step] <= x) c += step;
        const int4 u = units[c];
        const int row = x - before[c], n = u.x;
        auto at = [&](int s) { return static_cast<size_t>(s == 0 ? u.y : 2 * (c + s)) * u.z + row; };
        constexpr int kBatch = 4;  // pieces in flight
        float4 o[kBatch];
        float w[kBatch];
        auto fetch = [&](int s0) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int s = min(s0 + i * groups, n - 1);
                o[i] = *reinterpret_cast<const float4 *>(p.part_O + at(s) * DL + 4 * col);
                w[i] = p.part_LSE[at(s)];
            }
        };
        const float first = lane < n ? p.part_LSE[at(lane)] : -INFINITY;
        fetch(group);
        float m = first, total = 0.f;
        for (int s = lane + 32; s < n; s += 32) m = fmaxf(m, p.part_LSE[at(s)]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        // the weight of a piece; one that saw nothing weighs 0, one with NaN NaN
        auto weight = [&](float x) { return x == -INFINITY ? 0.f : expf(x - m); };
        total = weight(first);
        for (int s = lane + 32; s < n; s += 32) total += weight(p.part_LSE[at(s)]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s0 = group; s0 < n; s0 += kBatch * groups) {
            if (s0 != group) fetch(s0);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const float f = s0 + i * groups < n ? weight(w[i]) : 0.f;
                if (f == 0.f) continue;  // (a piece that saw nothing, or none)
                acc.x = fmaf(f, o[i].x, acc.x);
                acc.y = fmaf(f, o[i].y, acc.y);
                acc.z = fmaf(f, o[i].z, acc.z);
                acc.w = fmaf(f, o[i].w, acc.w);
            }
        }
        if (groups > 1) {
            sums[tid] = acc;
            __syncthreads();
            if (group == 0)
                for (int g = 1; g < groups; ++g) {
                    const float4 v = sums[tid + g * kAcross];
                    acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
                }
            __syncthreads();
        }
        if (!there || group != 0) continue;
        const bool none = total == 0.f;
        const float inv = none ? 0.f : 1.f / total;
        const size_t g = static_cast<size_t>(u.w) + row;
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.O) + g * DL + 4 * col) =
            make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
        if (col == 0) p.LSE[g] = none ? -INFINITY : m + logf(total);
    }
}

}  // namespace latent
}  // namespace fa
