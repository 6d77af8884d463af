// fa_paged_kernel.cuh -- attention of a batch's new tokens over a paged K/V cache, for
// head dimensions 32, 64, 128 and 256 on sm_103a.
//
// The method is that of fa_fwd1t_kernel.cuh (128-row Q tile, K/V blocks of bn(D) keys,
// S in two or three TMEM buffers, online softmax with a lazily moved reference max, P
// in tensor memory, O divided by l once). What differs:
//   * K and V tiles are gathered from pages: the tile's keys are cut into chunks of
//     min(page size, bn) tokens, lane c of the producer warp reads chunk c's page number
//     and issues its TMA box; chunks that hold no key of the unit are not read. A box is
//     five-dimensional (64 columns, 8 tokens, column region, group of 8 tokens, page and
//     head), so that one copy brings all of a chunk's columns: with one copy per chunk and region
//     pages of 16 tokens took 886 us where pages of 128 took 823 (the chunk named below).
//   * Rows of a unit are (token, head) pairs: the pf query heads of one K/V head (or
//     a divisor of them when there are more than 128) for 128 / pf tokens, token-major
//     in the tile, so that every K/V tile is read once for all of them, at one token
//     per sequence as well as in a chunk of a prompt.
//   * The work is cut by K/V tiles, not by units: all units (sequence, head group,
//     tile of tokens) with all their visible K/V tiles, and kChunkTicks more for each unit's
//     start and end, form one line of W ticks, and CTA c takes ticks c T .. c T + T - 1 of it
//     (T = ceil(W / CTAs)). Every CTA gets the same share whatever the lengths are,
//     without counters.
//     A unit cut by a share's end leaves one partial (O / l and LSE, fp32) per piece,
//     which fa_paged_merge_kernel joins in the order of the pieces: at most two pieces
//     per CTA are partial, so the workspace depends on the SM count and D alone. The
//     lengths are read on the device, so a captured call follows them.
//   * Keys that no row of the unit sees (past the sequence's end in its last page, or
//     before a window) may hold anything, NaN included: their scores are replaced
//     before the maximum, and their V rows are zeroed in shared memory before the product.
//   * A row that sees no key (a sequence without keys, or more queries than keys under
//     a mask) gets O = 0 and LSE = -inf.
//
// Warps (256 threads; a ninth warp would cost the softmax its registers): 0-3 softmax, 4
// scheduler (walks the CTA's share and publishes its pieces, one ahead) and Q and K
// producer, 5 issuer of S = Q K^T, 6 V producer, 7 issuer of O += P V. A softmax warp
// none of whose rows exists (decode: pf rows of 128) passes its blocks on without
// touching them.
//
// Two warps issue the products because the tensor pipe holds only about one operation
// ahead: a single issuer spent 1,032 cycles of a 128-key tile at d = 128 issuing and 410 in
// its waits for P, V and K (with clock reads in the code), while the softmax waited 498 of
// 1,771 for scores. With two, the waits of one fall into the products of the
// other. What one thread's issue order used to give is then a barrier: S(t) goes into the
// TMEM buffer of P(t - 3) once the product with P(t - 3) has completed. The scores run
// ahead by the three buffers (two at d = 256), across units as well. 2048 queries on
// 32048 keys, 32 / 8 heads: 790 -> 700 us at d = 128, 768 -> 690 us at d = 256 (16 / 4
// heads), each pair on one board; from board to board the d = 128 case takes 680 to 740. At d <= 64 the softmax sets the pace and a second issuer only took its
// instruction slots (620 and 657 us): one warp issues both there.
// Every wait is bounded; on expiry the CTA records the failure, drains its copies and
// MMAs, frees its tensor memory and returns.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "fa_mask.cuh"
#include "fa_pdl.cuh"
#include "fa_tmem_max.cuh"
#include "ptx.cuh"

namespace fa {
namespace paged {

constexpr int kBM = 128;  // rows per unit (TMEM lanes)
__host__ __device__ constexpr int bn(int D) { return D == 256 ? 64 : 128; }  // keys per tile
constexpr int kThreads = 256;
// A unit's start and end (its first scores, its last product, its outputs) in tiles:
// measured 3 to 4.5 us against 0.8 us for a tile of 64 keys at d = 256 and 0.94 us for one
// of 128 at d = 128. Of 5, 3 and 8: 12 sequences of 1-700 new tokens at d = 256 154.3, 164.0 and
// 156.8 us, 2048 tokens on 8000 keys at d = 128 176.2, 168.6 and 179.6.
constexpr int kChunkTicks = 5;
constexpr int kQKWarp = 4;
constexpr int kScoreWarp = 5;
constexpr int kVWarp = 6;
constexpr int kOutWarp = 7;
// Q, K and V ring depths: what shared memory holds. Two Q tiles let the scores of the
// next unit start while this one ends; K is read by its scores alone, soon after it
// comes, V a few tiles later.
__host__ __device__ constexpr int q_stages(int D) { return D == 256 ? 1 : 2; }
__host__ __device__ constexpr int k_stages(int D) { return D <= 64 ? 5 : D == 128 ? 2 : 3; }
__host__ __device__ constexpr int v_stages(int D) { return D <= 64 ? 6 : D == 128 ? 3 : 2; }
constexpr int kMaxStages = 6;
constexpr int kSBufs = 3;
__host__ __device__ constexpr int s_bufs(int D) { return D == 256 ? 2 : 3; }
// Q read by S = Q K^T from TMEM at d = 256: with 64-key tiles the shared-memory form
// would need more than the SM's shared-memory bandwidth (see fa_fwd1t_kernel.cuh)
__host__ __device__ constexpr bool q_in_tmem(int D) { return D == 256; }
constexpr uint32_t kTmemCols = 512;
__host__ __device__ constexpr uint32_t tmem_o(int D) { return D == 256 ? 256u : 384u; }
constexpr uint32_t kTmemS = 0;
constexpr uint32_t kTmemQ = 128;  // d = 256 only
constexpr float kRescaleThreshold = 8.0f;  // log2 units, as in fa_fwd_kernel.cuh
constexpr unsigned kStatusTimeout = 4;
constexpr int kUnitSlots = 8;
// Whether S and O += P V are issued by a warp each.
__host__ __device__ constexpr bool two_issuers(int D) { return D >= 128; }
// Warps that take the pieces: all but the scheduler (and an idle issuer); each arrives
// once per piece.
__host__ __device__ constexpr int unit_consumers(int D) { return two_issuers(D) ? 7 : 6; }
enum : int { kRoleSoftmax = 1, kRoleTma = 2, kRoleMma = 3 };

// Written by every CTA for the merge: the unit whose first piece is this CTA's last
// one and which later CTAs continue (last_cta < 0: none).
struct MergeInfo {
    int last_cta;   // the CTA of the unit's last piece
    int slot;       // partial slot of the first piece (the others: 2 * cta)
    int rows;       // rows of the unit
    int tok0, head0;  // its first token (of all tokens) and head
    int slot_rows;  // rows of a partial slot
    int pad[2];
};

struct Params {
    void *O;
    float *LSE;
    float *part_O;     // [2 * CTAs][128][D]: O / l of the pieces of cut units
    float *part_LSE;   // [2 * CTAs][128]
    MergeInfo *info;   // [CTAs]
    const int *cu_q;   // B + 1: sequence b owns tokens cu_q[b] .. cu_q[b+1] - 1
    const int *seq_k;  // B: keys of each sequence, its new tokens included
    const int *table;  // B x max_pages page numbers
    int B, H, kv_group, pf, spaces, tpt;  // heads per unit; H / pf; tokens per unit
    int total_q, max_pages, page_log2, num_pages;
    int max_keys;      // max_pages pages of keys (a length above it counts as this)
    int chunk;         // tokens per TMA box: min(page size, bn(D))
    int page_step, head_step;  // the maps' last coordinate: page * page_step + head * head_step
    int page_none;     // one past its last value: reads as zeros
    int wl, wr;        // key j visible to the query at position i iff i - wl <= j <= i + wr
    float scale_log2;
    unsigned long long wait_budget_ns;
    unsigned int *status;
    int fault_skip_k;  // test hook: every CTA skips the K load at this ring position (-1: none)
    int infos;  // entries of info per CTA, all to be written (more than one: what the decode body has)
};

// Tiles are stored as regions of min(D, 64) columns with the swizzle of that row width. Q: region
// after region of 128 rows; K and V: groups of 8 rows, the regions of a group side by side.
template <int D>
struct Smem {
    static constexpr int kCols = D < 64 ? D : 64;
    static constexpr int kRowBytes = kCols * 2;
    static constexpr int kRegions = D / kCols;
    static constexpr int kQRegion = kBM * kRowBytes;
    static constexpr int kQBytes = kRegions * kQRegion;
    static constexpr int kAtom = 8 * kRowBytes;        // one region of a group
    static constexpr int kGroup = kRegions * kAtom;
    static constexpr int kKVBytes = bn(D) / 8 * kGroup;
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + q_stages(D) * kQBytes;
    static constexpr int kV = kK + k_stages(D) * kKVBytes;
    static constexpr int kBar = kV + v_stages(D) * kKVBytes;
    static constexpr int kNumBars = 64;
    static constexpr int kMisc = kBar + kNumBars * 8;  // TMEM address, abort flag
    static constexpr int kScan = kMisc + 16;           // 8 warp sums, start sequence and offset
    static constexpr int kUnitRing = kScan + 48;       // kUnitSlots pieces
    static_assert(kUnitRing % 16 == 0, "ring alignment");
    static constexpr int kBytes = kUnitRing + kUnitSlots * 64;
    // more than half of the SM's shared memory: one CTA (and one holder of all 512
    // TMEM columns) per SM
    static constexpr int kAlloc = kBytes + 1024 > 120 * 1024 ? kBytes + 1024 : 120 * 1024;
    static_assert(kAlloc <= 227 * 1024, "shared memory");
};

enum : int {
    kBarQFull = 0,                         // + stage (2)
    kBarQEmpty = 2,                        // + stage (2)
    kBarKFull = 4,                         // + stage
    kBarKEmpty = kBarKFull + kMaxStages,   // + stage
    kBarVFull = kBarKEmpty + kMaxStages,   // + stage
    kBarVEmpty = kBarVFull + kMaxStages,   // + stage
    kBarSFull = kBarVEmpty + kMaxStages,   // + buffer (3)
    kBarPFull = kBarSFull + kSBufs,        // + buffer (3)
    kBarPVDone = kBarPFull + kSBufs,       // + buffer (3)
    kBarODone = kBarPVDone + kSBufs,
    kBarOFree = kBarODone + 1,
    kBarUnitFull = kBarOFree + 1,               // + slot (8)
    kBarUnitEmpty = kBarUnitFull + kUnitSlots,  // + slot (8)
    kBarDrain = kBarUnitEmpty + kUnitSlots,  // + issuer (2)
    kBarQReady = kBarDrain + 2,            // Q copied into TMEM (d = 256)
    kNumBarsUsed = kBarQReady + 1,
};
static_assert(kNumBarsUsed <= Smem<256>::kNumBars, "barrier slots");

// One piece of a unit: n K/V tiles from j0 on (none: no row sees a key) of the unit with
// tokens t0 .. t0 + ceil(rows / pf) - 1 of sequence b. They are taken from tile `first` on,
// around the end to j0 again: CTAs that have come equally far then read the same tiles of
// a sequence at the same time, instead of each starting its units at key 0 at a time of
// its own (2048 queries on 32048 keys, 8 K/V heads: L2 missed 2.3 GB of the 134 MB cache).
struct Piece {
    int b, sp, t0, rows;
    int j0, n, first;
    __device__ __forceinline__ int tile(int x) const {
        const int j = first + x;
        return j < j0 + n ? j : j - n;
    }
    int lo_key, hi_key;  // the first and last key that any row of the unit sees
    int q_off, nk;       // token i of the sequence stands at key position i + q_off
    int tok0;            // the unit's first token of all tokens
    int slot;            // partial slot, or -1: the whole unit, written to O and LSE
};
static_assert(sizeof(Piece) <= 64, "ring slot");

struct Seq {
    int q0, nq, nk;
};
__device__ __forceinline__ Seq load_seq(int b, const Params &p) {
    Seq s;
    s.q0 = min(max(p.cu_q[b], 0), p.total_q);
    s.nq = min(max(p.cu_q[b + 1], s.q0), p.total_q) - s.q0;
    s.nk = min(max(p.seq_k[b], 0), p.max_keys);
    return s;
}

// K/V tiles j0 .. j1 that the rows of token tile qb see, and the keys lo .. hi.
template <int kBN>
__device__ __forceinline__ void unit_range(const Seq &s, int qb, const Params &p, int &lo, int &hi,
                                           int &j0, int &j1) {
    const int t0 = qb * p.tpt, tl = min(t0 + p.tpt, s.nq) - 1;
    const int q_off = s.nk - s.nq;
    lo = max(0, t0 + q_off - p.wl);
    hi = min(s.nk - 1, tl + q_off + p.wr);
    j0 = lo / kBN;
    j1 = hi < lo ? j0 - 1 : hi / kBN;
}
// A unit's K/V tiles (none when no row sees a key: its rows are written all the same).
template <int kBN>
__device__ __forceinline__ int unit_tiles(const Seq &s, int qb, const Params &p) {
    int lo, hi, j0, j1;
    unit_range<kBN>(s, qb, p, lo, hi, j0, j1);
    return j1 - j0 + 1;
}

__device__ __forceinline__ void record_timeout(const Params &p, volatile int *abort_flag, int role,
                                               int unit) {
    *abort_flag = 1;
    if (atomicCAS(p.status, 0u, kStatusTimeout) == 0u) {
        p.status[1] = static_cast<unsigned>(role);
        p.status[2] = static_cast<unsigned>(unit);
        p.status[3] = blockIdx.x;
        __threadfence();
    }
}

// 5-D tiled copy global -> shared, completion counted on mbarrier `bar`.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3, int32_t c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
        : "memory");
}

// Shared-memory matrix descriptor as in ptx.cuh, with the byte distances of 64-column blocks
// (MN-major operands) and of groups of 8 rows given.
template <int kRowBytes>
__device__ __forceinline__ uint64_t tile_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(kRowBytes == 128 ? 2 : 4) << 61;
    return d;
}

__device__ __forceinline__ unsigned warp_sum(unsigned v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums of ticks stay at kNoLine once they reach it. The host admits calls whose line is
// shorter, so only offsets that are not in ascending order, whose sequences overlap, get
// there: such a batch is left alone, as its sums past 32 bits would give shares nowhere.
constexpr unsigned kNoLine = 0x7fffffffu;
__device__ __forceinline__ unsigned add_work(unsigned a, unsigned b) { return min(a + b, kNoLine); }
__device__ __forceinline__ unsigned warp_sum_work(unsigned v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = add_work(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Ticks of one head group of sequence b (every thread of the warp calls it with its own
// b; b >= B gives 0). Long sequences, with many token tiles, are summed by the whole
// warp one after the other.
template <int kBN>
__device__ __forceinline__ unsigned seq_work(int b, const Params &p) {
    Seq s{0, 0, 0};
    if (b < p.B) s = load_seq(b, p);
    const int nqb = (s.nq + p.tpt - 1) / p.tpt;
    unsigned w = 0;
    constexpr int kOwn = 4;
    if (nqb <= kOwn)
        for (int qb = 0; qb < nqb; ++qb) w += unit_tiles<kBN>(s, qb, p) + kChunkTicks;
    unsigned todo = __ballot_sync(0xffffffffu, nqb > kOwn);
    const int lane = threadIdx.x & 31;
    while (todo != 0) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const Seq o{0, __shfl_sync(0xffffffffu, s.nq, src), __shfl_sync(0xffffffffu, s.nk, src)};
        const int n = __shfl_sync(0xffffffffu, nqb, src);
        unsigned part = 0;
        for (int qb = lane; qb < n; qb += 32) part += unit_tiles<kBN>(o, qb, p) + kChunkTicks;
        part = warp_sum(part);
        if (lane == src) w = part;
    }
    return w;
}

// A CTA of the kernel.
template <int D, bool BF16>
__device__ __forceinline__ void chunk_cta(const CUtensorMap &tmQ, const CUtensorMap &tmK, const CUtensorMap &tmV,
                                          const Params &p, uint8_t *smem_raw) {
    using L = Smem<D>;
    constexpr int kBN = bn(D);
    constexpr uint32_t kTmemO = tmem_o(D);
    constexpr int kSB = s_bufs(D);
    constexpr bool kQT = q_in_tmem(D);
    constexpr int kKStages = k_stages(D);
    constexpr int kVStages = v_stages(D);
    constexpr int kQStages = q_stages(D);
    static_assert(kQT ? (kSB * kBN <= static_cast<int>(kTmemQ) && kTmemQ + D / 2 <= kTmemO)
                      : kSB * kBN <= static_cast<int>(kTmemO),
                  "TMEM columns");
    static_assert(kTmemO + D <= kTmemCols, "TMEM columns");
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + L::kBar;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);
    constexpr int kStartSeq = kThreads / 32, kStartOff = kStartSeq + 1;
    volatile unsigned *scan = reinterpret_cast<volatile unsigned *>(smem + L::kScan);
    auto bar = [bar0](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    auto sQ = [sbase](int k) { return sbase + L::kQ + (k % kQStages) * L::kQBytes; };
    auto sK = [sbase](int t) { return sbase + L::kK + (t % kKStages) * L::kKVBytes; };
    auto sV = [sbase](int t) { return sbase + L::kV + (t % kVStages) * L::kKVBytes; };
    auto slot_of = [smem](int k) {
        return reinterpret_cast<Piece *>(smem + L::kUnitRing + (k % kUnitSlots) * 64);
    };

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint64_t budget = p.wait_budget_ns;

    // ---- this CTA's share of the line of work: ticks w0 .. w1 - 1 of W. B sequences are
    // summed, and then searched for w0, one to a thread at a time.
    auto block_sum = [&](unsigned v) -> unsigned {
        v = warp_sum_work(v);
        __syncthreads();
        if (lane == 0) scan[warp] = v;
        __syncthreads();
        unsigned s = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) s = add_work(s, scan[i]);
        return s == kNoLine ? 0 : s;
    };
    for (int i = 1 + threadIdx.x; i < p.infos; i += kThreads)
        p.info[i * gridDim.x + blockIdx.x].last_cta = -1;
    unsigned mine = 0, first = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const unsigned w = seq_work<kBN>(b0 + static_cast<int>(threadIdx.x), p) * p.spaces;
        if (b0 == 0) first = w;
        mine = add_work(mine, w);
    }
    const unsigned W = block_sum(mine);
    const unsigned T = (W + gridDim.x - 1) / gridDim.x;
    const unsigned w0 = min(blockIdx.x * T, W), w1 = min(w0 + T, W);
    if (w0 >= w1) {  // nothing left for this CTA
        if (threadIdx.x == 0) p.info[blockIdx.x].last_cta = -1;
        return;
    }
    unsigned carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        const unsigned w = b0 == 0 ? first : seq_work<kBN>(b, p) * p.spaces;
        unsigned incl = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        unsigned before = carry, all = carry;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) before += scan[i];
            all += scan[i];
        }
        const unsigned lo = before + incl - w;
        if (lo <= w0 && w0 < lo + w) {
            scan[kStartSeq] = static_cast<unsigned>(b);
            scan[kStartOff] = w0 - lo;
        }
        carry = all;
        if (w0 < carry) break;
    }

    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    if (threadIdx.x == kQKWarp * 32) {
        for (int s = 0; s < kQStages; ++s) {
            mbar_init(bar(kBarQFull + s), 1);
            // Q's shared-memory copy is released by the score issuer's commit, or at d = 256
            // by the softmax threads once they have copied it into TMEM
            mbar_init(bar(kBarQEmpty + s), kQT ? 128 : 1);
        }
        mbar_init(bar(kBarQReady), 128);
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(bar(kBarKFull + s), 1);
            mbar_init(bar(kBarKEmpty + s), 1);
        }
        for (int s = 0; s < kVStages; ++s) {
            mbar_init(bar(kBarVFull + s), 1);
            mbar_init(bar(kBarVEmpty + s), 1);
        }
        for (int b = 0; b < kSB; ++b) {
            mbar_init(bar(kBarSFull + b), 1);
            mbar_init(bar(kBarPFull + b), 128);
            mbar_init(bar(kBarPVDone + b), 1);
        }
        mbar_init(bar(kBarODone), 1);
        mbar_init(bar(kBarOFree), 128);
        for (int k = 0; k < kUnitSlots; ++k) {
            mbar_init(bar(kBarUnitFull + k), 1);
            mbar_init(bar(kBarUnitEmpty + k), unit_consumers(D));
        }
        mbar_init(bar(kBarDrain + 0), 1);
        mbar_init(bar(kBarDrain + 1), 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

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

    // Chunks of K/V tile j that hold a key of the piece's unit; chunk `lane`'s page and
    // first token in it. Returns the ballot of the chunks to load.
    auto chunk_of = [&](const Piece &P, int j, int &page, int &tok) -> uint32_t {
        const int k0 = j * kBN + lane * p.chunk;
        const bool need = lane * p.chunk < kBN && k0 + p.chunk > P.lo_key && k0 <= P.hi_key;
        page = 0;
        tok = k0 & ((1 << p.page_log2) - 1);
        if (need) {
            page = p.table[static_cast<size_t>(P.b) * p.max_pages + (k0 >> p.page_log2)];
            // a page number outside the cache reads as zeros
            const int hkv = P.sp * p.pf / p.kv_group;
            page = page >= 0 && page < p.num_pages ? page * p.page_step + hkv * p.head_step : p.page_none;
        }
        return __ballot_sync(0xffffffffu, need);
    };
    auto load_chunks = [&](const CUtensorMap *map, uint32_t dst, uint32_t full, uint32_t need, int page,
                           int tok) {
        if (lane == 0)
            mbar_arrive_expect_tx(full, static_cast<uint32_t>(__popc(need)) * p.chunk * (L::kGroup / 8));
        __syncwarp();
        if ((need >> lane) & 1u)
            tma_load_5d(dst + lane * p.chunk * (L::kGroup / 8), map, full, 0, 0, 0, tok >> 3, page);
        __syncwarp();
    };

    if (warp == kQKWarp) {
        // ================================================================ scheduler, Q and K
        // the unit that holds tick w0, by the whole warp: head group sp, token tile qb, and
        // the ticks `rem` of it that belong to the CTA before
        int b = static_cast<int>(scan[kStartSeq]), sp, qb = 0, rem;
        Seq s = load_seq(b, p);
        int nqb = (s.nq + p.tpt - 1) / p.tpt;
        {
            unsigned per = 0;
            for (int x = lane; x < nqb; x += 32) per += unit_tiles<kBN>(s, x, p) + kChunkTicks;
            per = warp_sum(per);
            sp = static_cast<int>(scan[kStartOff] / per);
            rem = static_cast<int>(scan[kStartOff] - sp * per);
            for (int x0 = 0; x0 < nqb; x0 += 32) {
                const int n = x0 + lane < nqb ? unit_tiles<kBN>(s, x0 + lane, p) + kChunkTicks : 0;
                int incl = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                const unsigned hit = __ballot_sync(0xffffffffu, rem < incl);
                if (hit != 0) {
                    const int at = __ffs(hit) - 1;
                    qb = x0 + at;
                    rem -= __shfl_sync(0xffffffffu, incl - n, at);
                    break;
                }
                rem -= __shfl_sync(0xffffffffu, incl, 31);
            }
        }
        unsigned w = w0;
        bool ok = true;
        MergeInfo info{};
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
                unit_range<kBN>(s, qb, p, lo, hi, j0, j1);
                const int n = j1 - j0 + 1;
                const int len = min(n + kChunkTicks - rem, static_cast<int>(w1 - w));
                // this share's tiles of the unit: ja .. je - 1
                const int ja = max(rem - kChunkTicks, 0), je = rem + len - kChunkTicks;
                if (n == 0 ? rem == 0 : je > ja) {
                    P.b = b;
                    P.sp = sp;
                    P.t0 = qb * p.tpt;
                    P.rows = (min(P.t0 + p.tpt, s.nq) - P.t0) * p.pf;
                    P.lo_key = lo;
                    P.hi_key = hi;
                    P.q_off = s.nk - s.nq;
                    P.nk = s.nk;
                    P.tok0 = s.q0 + P.t0;
                    P.j0 = j0 + ja;
                    P.n = n == 0 ? 0 : je - ja;
                    P.first = n == 0 ? 0 : P.j0 + static_cast<int>((w - w0) % P.n);
                    const bool starts = ja == 0, ends = n == 0 || je == n;
                    P.slot = starts && ends ? -1 : 2 * static_cast<int>(blockIdx.x) + (pieces > 0);
                    if (n > 0) ++pieces;
                    if (starts && !ends) {
                        info.last_cta = static_cast<int>((w - rem + kChunkTicks + n - 1) / T);
                        info.slot = P.slot;
                        info.slot_rows = kBM;
                        info.rows = P.rows;
                        info.tok0 = P.tok0;
                        info.head0 = sp * p.pf;
                    }
                }
                w += len;
                rem = 0;
                if (++qb == nqb) {
                    qb = 0;
                    if (++sp == p.spaces) {
                        sp = 0;
                        while (w < w1 && ++b < p.B) {
                            s = load_seq(b, p);
                            nqb = (s.nq + p.tpt - 1) / p.tpt;
                            if (nqb > 0) break;
                        }
                        if (b >= p.B) w = w1;
                    }
                }
            }
            if (lane == 0) {
                *slot_of(k) = P;
                mbar_arrive(bar(kBarUnitFull + slot));
            }
            __syncwarp();
            return P;
        };
        int t = 0, q_loads = 0;
        Piece N = publish(0);
        for (int k = 0; ok && N.b >= 0; ++k) {
            const Piece P = N;
            N = publish(k + 1);
            if (!ok) break;
            if (P.n == 0) continue;
            const int qs = q_loads % kQStages;
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarQEmpty + qs), ((q_loads / kQStages) & 1) ^ 1,
                                                           abort_flag, budget));
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(kBarQFull + qs), static_cast<uint32_t>(p.pf * p.tpt) *
                                                               L::kRowBytes * L::kRegions);
                for (int g = 0; g < L::kRegions; ++g)
                    tma_load_3d(sQ(q_loads) + g * L::kQRegion, &tmQ, bar(kBarQFull + qs), L::kCols * g,
                                P.sp * p.pf, P.tok0);
            }
            ++q_loads;
            int page, tok;
            uint32_t need = chunk_of(P, P.tile(0), page, tok);
            for (int x = 0; x < P.n; ++x, ++t) {
                const int st = t % kKStages;
                // the next tile's page numbers are on their way while this one waits
                int page_n = 0, tok_n = 0;
                uint32_t need_n = 0;
                if (x + 1 < P.n) need_n = chunk_of(P, P.tile(x + 1), page_n, tok_n);
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarKEmpty + st), ((t / kKStages) & 1) ^ 1,
                                                               abort_flag, budget));
                if (!ok) break;
                if (t != p.fault_skip_k) load_chunks(&tmK, sK(t), bar(kBarKFull + st), need, page, tok);
                page = page_n;
                tok = tok_n;
                need = need_n;
            }
        }
        if (lane == 0) {
            p.info[blockIdx.x] = info;
            if (!ok) record_timeout(p, abort_flag, kRoleTma, -1);
            for (int st = 0; st < kQStages; ++st)
                if (q_loads > st) {
                    const int last = q_loads - 1 - ((q_loads - 1 - st) % kQStages);
                    mbar_wait_bounded(bar(kBarQFull + st), (last / kQStages) & 1, nullptr, budget);
                }
            for (int st = 0; st < kKStages; ++st)
                if (t > st) {
                    const int last = t - 1 - ((t - 1 - st) % kKStages);
                    mbar_wait_bounded(bar(kBarKFull + st), (last / kKStages) & 1, nullptr, budget);
                }
        }
    } else if (warp == kVWarp) {
        // ================================================================ V
        int t = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const Piece P = take(k, ok);
            if (!ok || P.b < 0) break;
            int page, tok;
            uint32_t need = chunk_of(P, P.tile(0), page, tok);
            for (int x = 0; x < P.n; ++x, ++t) {
                const int st = t % kVStages;
                int page_n = 0, tok_n = 0;
                uint32_t need_n = 0;
                if (x + 1 < P.n) need_n = chunk_of(P, P.tile(x + 1), page_n, tok_n);
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarVEmpty + st), ((t / kVStages) & 1) ^ 1,
                                                               abort_flag, budget));
                if (!ok) break;
                load_chunks(&tmV, sV(t), bar(kBarVFull + st), need, page, tok);
                page = page_n;
                tok = tok_n;
                need = need_n;
            }
        }
        if (lane == 0) {
            if (!ok) record_timeout(p, abort_flag, kRoleTma, -1);
            for (int s = 0; s < kVStages; ++s)
                if (t > s) {
                    const int last = t - 1 - ((t - 1 - s) % kVStages);
                    mbar_wait_bounded(bar(kBarVFull + s), (last / kVStages) & 1, nullptr, budget);
                }
        }
    } else if (warp == kScoreWarp || (warp == kOutWarp && two_issuers(D))) {
        // ================================================================ issuers of the products
        const bool scores = warp == kScoreWarp;
        constexpr uint32_t idesc_s = idesc_f16_ab(BF16, kBM, kBN, false, false);
        constexpr uint32_t idesc_o = idesc_f16_ab(BF16, kBM, D, false, true);
        constexpr int kSteps = L::kCols / 16;  // K-steps of 16 columns per region
        auto wait = [&](int b, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait_bounded(bar(b), parity, abort_flag, budget));
        };
        auto commit = [&](int b) {
            if (elect_one()) umma_commit(bar(b));
            __syncwarp();
        };
        // S(t) = Q K_t^T into S buffer t mod kSB; Q from shared memory, or from TMEM.
        auto issue_s = [&](int t, int q) {
            tc_fence_after();
            const uint64_t dq = tile_desc<L::kRowBytes>(sQ(q), 16, L::kAtom);
            const uint64_t dk = tile_desc<L::kRowBytes>(sK(t), 16, L::kGroup);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t offq = (k / kSteps) * (L::kQRegion >> 4) + (k % kSteps) * 2;
                    const uint32_t offk = (k / kSteps) * (L::kAtom >> 4) + (k % kSteps) * 2;
                    if constexpr (kQT)
                        umma_f16_ts(tmem + kTmemS + (t % kSB) * kBN, tmem + kTmemQ + k * 8, dk + offk,
                                    idesc_s, k > 0 ? 1u : 0u);
                    else
                        umma_f16_ss(tmem + kTmemS + (t % kSB) * kBN, dq + offq, dk + offk, idesc_s,
                                    k > 0 ? 1u : 0u);
                }
                umma_commit(bar(kBarSFull + t % kSB));
                umma_commit(bar(kBarKEmpty + t % kKStages));  // K is read by S only
            }
            __syncwarp();
        };
        // O (+)= P(t) V_t, P read from the first kBN / 2 columns of S buffer t mod kSB.
        auto issue_pv = [&](int t, bool first_tile) {
            tc_fence_after();
            const uint64_t dv = tile_desc<L::kRowBytes>(sV(t), L::kAtom, L::kGroup);
            const uint32_t acc0 = first_tile ? 0u : 1u;
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kBN / 16; ++k)
                    umma_f16_ts(tmem + kTmemO, tmem + kTmemS + (t % kSB) * kBN + k * 8,
                                dv + k * ((2 * L::kGroup) >> 4), idesc_o, k > 0 ? 1u : acc0);
                umma_commit(bar(kBarPVDone + t % kSB));
                umma_commit(bar(kBarVEmpty + t % kVStages));
            }
            __syncwarp();
        };
        // Rows of V tile t (keys kv0 ..) outside keys lo .. hi: 0 times whatever the page
        // holds there must be 0.
        auto zero_rows = [&](int t, int kv0, int lo, int hi) {
            const uint4 z = make_uint4(0, 0, 0, 0);
            uint8_t *base = smem + L::kV + (t % kVStages) * L::kKVBytes;
            constexpr int kPer = D / 8;  // 16-byte pieces of a row
            auto zero = [&](int r0, int r1) {
                for (int c = r0 * kPer + lane; c < r1 * kPer; c += 32) {
                    const int r = c / kPer, x = c % kPer;  // a row's regions are kAtom apart
                    *reinterpret_cast<uint4 *>(base + (r >> 3) * L::kGroup + (r & 7) * L::kRowBytes +
                                               (x / (L::kRowBytes / 16)) * L::kAtom +
                                               (x % (L::kRowBytes / 16)) * 16) = z;
                }
            };
            zero(0, min(max(lo - kv0, 0), kBN));
            zero(min(max(hi + 1 - kv0, 0), kBN), kBN);
            fence_proxy_async_smem();
            __syncwarp();
        };
        int t = 0, live = 0;  // K/V tiles, and pieces with tiles, so far
        bool ok = true;
        int k = 0;
        for (; ok; ++k) {
            const Piece P = take(k, ok);
            if (!ok || P.b < 0) break;
            if (P.n == 0) continue;
            auto q_ready = [&] {
                return wait(kQT ? kBarQReady : kBarQFull + live % kQStages, (live / kQStages) & 1);
            };
            auto k_ready = [&](int tk) { return wait(kBarKFull + tk % kKStages, (tk / kKStages) & 1); };
            auto output = [&](int x) {
                ok = wait(kBarVFull + t % kVStages, (t / kVStages) & 1);
                if (!ok) return;
                const int kv0 = P.tile(x) * kBN;
                if (kv0 < P.lo_key || kv0 + kBN - 1 > P.hi_key)
                    zero_rows(t, kv0, P.lo_key, P.hi_key);  // while the softmax is still at this tile
                ok = wait(kBarPFull + t % kSB, (t / kSB) & 1);
                if (ok && x == 0 && live > 0) ok = wait(kBarOFree, (live - 1) & 1);
                if (ok) issue_pv(t, x == 0);
            };
            if constexpr (!two_issuers(D)) {
                ok = q_ready();
                for (int x = 0; ok && x < P.n && x < kSB; ++x) {
                    ok = k_ready(t + x);
                    if (ok) issue_s(t + x, live);
                }
                for (int x = 0; ok && x < P.n; ++x, ++t) {
                    output(x);
                    if (ok && x + kSB < P.n) {
                        ok = k_ready(t + kSB);
                        if (ok) issue_s(t + kSB, live);  // after the product with P(t), in issue order
                    }
                }
                if (ok) {
                    commit(kBarQEmpty + live % kQStages);
                    commit(kBarODone);
                }
            } else if (scores) {
                ok = q_ready();
                for (int x = 0; ok && x < P.n; ++x, ++t) {
                    ok = k_ready(t);
                    // the buffer's last P has been multiplied (one wait per use, and the
                    // next use's product needs this S: the phases cannot run ahead)
                    if (ok && t >= kSB) ok = wait(kBarPVDone + t % kSB, (t / kSB - 1) & 1);
                    if (ok) issue_s(t, live);
                }
                if (ok && !kQT) commit(kBarQEmpty + live % kQStages);
            } else {
                for (int x = 0; ok && x < P.n; ++x, ++t) output(x);
                if (ok) commit(kBarODone);
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
        // ================================================================ softmax warpgroup
        const int row = threadIdx.x & 127;
        const uint32_t tl = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        const float sl2 = p.scale_log2;
        const int row_tok = row / p.pf, row_head = row - row_tok * p.pf;
        // d = 256: copy the k-th live piece's Q tile from shared memory into TMEM, this
        // thread's row into its lane (128-byte swizzle: 16-byte chunk c of row r sits
        // at chunk c ^ (r mod 8) of the row), then release both copies' barriers.
        auto copy_q = [&](int k) -> bool {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarQFull), k & 1, abort_flag, budget)))
                return false;
#pragma unroll
            for (int g = 0; g < L::kRegions; ++g) {
                uint32_t w[32];
                const uint8_t *src = smem + L::kQ + g * L::kQRegion + row * 128;
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(src + ((c ^ (row & 7)) << 4));
                    w[4 * c] = v.x;
                    w[4 * c + 1] = v.y;
                    w[4 * c + 2] = v.z;
                    w[4 * c + 3] = v.w;
                }
                tmem_st32(tl + kTmemQ + g * 32, w);
            }
            tmem_st_wait();
            mbar_arrive(bar(kBarQEmpty));
            tc_fence_before();
            mbar_arrive(bar(kBarQReady));
            return true;
        };
        int k = 0;  // pieces taken
        bool ok = true;
        auto out_row = [&](const Piece &P) {
            return (static_cast<size_t>(P.tok0) + row_tok) * p.H + P.sp * p.pf + row_head;
        };
        // The next piece with tiles (b < 0: none); pieces without get O = 0, LSE = -inf.
        auto next_live = [&]() -> Piece {
            while (true) {
                const Piece P = take(k, ok);
                ++k;
                if (!ok || P.b < 0 || P.n > 0) return P;
                if (row < P.rows) {
                    const size_t g = out_row(P);
                    const uint32_t z[8] = {};
                    uint8_t *orow = reinterpret_cast<uint8_t *>(p.O) + g * (D * 2);
                    for (int c = 0; c < D / 16; ++c) st_global_v8(orow + c * 32, z);
                    p.LSE[g] = -INFINITY;
                }
            }
        };
        int t = 0, live = 0;
        Piece P = next_live();
        if (ok && kQT && P.b >= 0) ok = copy_q(0);
        while (ok && P.b >= 0) {
            const int i = P.t0 + row_tok;
            const bool active = row < P.rows;
            const bool warp_active = warp * 32 < P.rows;
            const int lo_i = max(0, i + P.q_off - p.wl);
            const int hi_i = min(P.nk - 1, i + P.q_off + p.wr);
            // a tile with keys in [lo_last, hi_first] only is visible to every row
            const int tl_i = P.t0 + (P.rows - 1) / p.pf;
            const int lo_last = max(0, tl_i + P.q_off - p.wl);
            const int hi_first = min(P.nk - 1, P.t0 + P.q_off + p.wr);
            float m = -INFINITY, l = 0.f;
            for (int x0 = 0; x0 < P.n; ++x0, ++t) {
                const uint32_t tS = tl + kTmemS + (t % kSB) * kBN;
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarSFull + t % kSB), (t / kSB) & 1,
                                                               abort_flag, budget));
                if (!ok) break;
                if (!warp_active) {
                    // no row here: S is passed on as it is (an MMA row depends on its own
                    // A row alone, and these rows are not stored)
                    mbar_arrive(bar(kBarPFull + t % kSB));
                    continue;
                }
                tc_fence_after();
                float x[kBN];
                const int kv0 = P.tile(x0) * kBN;
                float m_tile;
                if (kv0 >= lo_last && kv0 + kBN - 1 <= hi_first) {
                    // every key visible: the TMEM loads reduce each 32-column run to
                    // its maximum
                    float mr[kBN / 32];
#pragma unroll
                    for (int h = 0; h < kBN; h += 64) {
                        uint32_t a[32], b[32];
                        tmem_ld32_max(tS + h, a, mr[h / 32]);
                        tmem_ld32_max(tS + h + 32, b, mr[h / 32 + 1]);
                        tmem_ld_max_wait(a, mr[h / 32]);
                        tmem_ld_max_wait(b, mr[h / 32 + 1]);
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            x[h + c] = __uint_as_float(a[c]);
                            x[h + c + 32] = __uint_as_float(b[c]);
                        }
                    }
                    float mm = mr[0];
#pragma unroll
                    for (int c = 1; c < kBN / 32; ++c) mm = fmaxf(mm, mr[c]);
                    m_tile = mm * sl2;
                } else {
#pragma unroll
                    for (int h = 0; h < kBN; h += 64) {
                        uint32_t a[32], b[32];
                        tmem_ld32(tS + h, a);
                        tmem_ld32(tS + h + 32, b);
                        tmem_ld_wait(a);
                        tmem_ld_wait(b);
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            x[h + c] = __uint_as_float(a[c]);
                            x[h + c + 32] = __uint_as_float(b[c]);
                        }
                    }
                    mask_outside_run(x, lo_i - kv0, hi_i - kv0, -INFINITY);
                    float ma = fmaxf(x[0], x[1]), mb = fmaxf(x[2], x[3]);
#pragma unroll
                    for (int c = 4; c < kBN; c += 4) {
                        ma = max3f(ma, x[c], x[c + 1]);
                        mb = max3f(mb, x[c + 2], x[c + 3]);
                    }
                    m_tile = fmaxf(ma, mb) * sl2;
                }
                if (!active) m_tile = -INFINITY;  // a row that is not there moves no reference
                const float m_old = m;
                if (m_tile > m + kRescaleThreshold) m = m_tile;
                const float corr = m != m_old ? ex2_approx(m_old - m) : 1.f;
                const float nm = m == -INFINITY ? 0.f : -m;
                float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
                for (int c = 0; c < kBN; c += 2) {
                    ffma2(x[c], x[c + 1], sl2, sl2, nm, nm);
                    x[c] = ex2_approx(x[c]);
                    x[c + 1] = ex2_approx(x[c + 1]);
                }
#pragma unroll
                for (int c = 0; c < kBN; c += 4) {
                    fadd2(s0, s1, x[c], x[c + 1]);
                    fadd2(s2, s3, x[c + 2], x[c + 3]);
                }
                // P(j) as 16-bit pairs over the first kBN / 2 columns of the buffer: the operand
                // type of the product, as in the library's other forwards; l keeps the fp32
                // values. The rounding puts O's error at 0.0024 where its own is 0.0017 (bf16,
                // relative, root mean square). A second part beside it, what the rounding left,
                // gave 0.0017 and took 988 us for 727 (2048 tokens on 32048 keys, d = 128).
#pragma unroll
                for (int h = 0; h < kBN; h += 64) {
                    uint32_t pk[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) pk[e] = pack2<BF16>(x[h + 2 * e], x[h + 2 * e + 1]);
                    tmem_st16(tS + h / 2, pk);
                    tmem_st16(tS + h / 2 + 16, pk + 16);
                }
                l = l * corr + ((s0 + s1) + (s2 + s3));
                // The reference max moved: O holds the sum through block j-1 once that
                // product completes; rescale this row's O before P(j) is released.
                if (x0 > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
                    const int tp = t - 1;
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarPVDone + tp % kSB), (tp / kSB) & 1,
                                                                   abort_flag, budget));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tl + kTmemO + c * 32, o);
                        tmem_ld_wait(o);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float a0 = __uint_as_float(o[e]), a1 = __uint_as_float(o[e + 1]);
                            fmul2(a0, a1, corr, corr);
                            o[e] = __float_as_uint(a0);
                            o[e + 1] = __float_as_uint(a1);
                        }
                        tmem_st32(tl + kTmemO + c * 32, o);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(bar(kBarPFull + t % kSB));
            }
            if (!ok) break;
            Piece N{};
            if constexpr (kQT) {
                // every S of this piece has completed (its last S buffer was read), so
                // the next piece's Q can replace this one's in TMEM during the epilogue
                N = next_live();
                if (ok && N.b >= 0) ok = copy_q(live + 1);
                if (!ok) break;
            }
            // ---- epilogue: O / l rounded to 16 bit, LSE = ln 2 (m + log2 l); a piece of
            // a cut unit keeps both in fp32 for the merge
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kBarODone), live & 1, abort_flag, budget));
            if (!ok) break;
            if (warp_active) {
                tc_fence_after();
                const float inv_l = l == 0.f ? 0.f : 1.f / l;
                const float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
                if (P.slot < 0) {
                    const size_t grow = out_row(P);
                    uint8_t *orow = reinterpret_cast<uint8_t *>(p.O) + grow * (D * 2);
#pragma unroll 2
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tl + kTmemO + c * 32, o);
                        tmem_ld_wait(o);
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            pk[e] = pack2<BF16>(__uint_as_float(o[2 * e]) * inv_l,
                                                __uint_as_float(o[2 * e + 1]) * inv_l);
                        if (l == 0.f) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) pk[e] = 0;
                        }
                        if (active) {
                            st_global_v8(orow + c * 64, pk);
                            st_global_v8(orow + c * 64 + 32, pk + 8);
                        }
                    }
                    if (active) p.LSE[grow] = lse;
                } else {
                    const size_t prow = static_cast<size_t>(P.slot) * kBM + row;
                    float *orow = p.part_O + prow * D;
#pragma unroll 2
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tl + kTmemO + c * 32, o);
                        tmem_ld_wait(o);
                        if (active) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(o[e]) * inv_l);
#pragma unroll
                            for (int q = 0; q < 4; ++q) st_global_v8(orow + c * 32 + q * 8, o + q * 8);
                        }
                    }
                    if (active) p.part_LSE[prow] = lse;
                }
            }
            tc_fence_before();
            mbar_arrive(bar(kBarOFree));
            ++live;
            if constexpr (!kQT) N = next_live();
            P = N;
        }
        if (!ok && lane == 0) record_timeout(p, abort_flag, kRoleSoftmax, k);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    fa_paged_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    after_previous();
    let_next_start();
    chunk_cta<D, BF16>(tmQ, tmK, tmV, p, smem_raw);
}

// Joins the pieces of the cut units, block c the unit that starts in worker c's share: with O_s, LSE_s of piece s
//     LSE = ln sum_s exp(LSE_s)          O = sum_s exp(LSE_s - LSE) O_s
// around the largest LSE_s (blockIdx.y shares a unit's rows). A row is summed by one warp, or
// by 2 .. 8 over as many runs of its pieces when there are fewer rows than warps, always in
// the same order. Bound by latency: every worker has a block of its own, all of them resident
// at once, and a unit's statistics and outputs are requested together, kMergeBatch pieces
// of a warp at a time (304 blocks that took several workers each in turn: 13 us after a
// decode kernel of 157 us, against about 3).
struct MergeParams {
    const MergeInfo *info;
    const float *part_O, *part_LSE;
    void *O;
    float *LSE;
    int H, pf;
    int ctas;  // > 0: either body's pieces, a block per decode worker; the chunk body had this many CTAs
};

constexpr int kMergeWarps = 8;

template <int D, bool BF16>
__global__ void __launch_bounds__(kMergeWarps * 32) fa_paged_merge_kernel(const MergeParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kV = D / 32;  // consecutive columns per lane
    constexpr int kMergeBatch = D <= 128 ? 4 : 2;
    __shared__ float red_o[kMergeWarps][D];
    __shared__ float red_m[kMergeWarps], red_w[kMergeWarps];
    after_previous();
    let_next_start();
    int c = blockIdx.x, part = blockIdx.y, parts = gridDim.y;
    MergeInfo u = p.info[c];
    if (p.ctas > 0) {
        // a unit of the chunk body is shared by every p.ctas-th block
        const MergeInfo chunk = p.info[c % p.ctas];
        if (chunk.last_cta >= 0 && chunk.slot_rows == kBM) {
            u = chunk;
            part += c / p.ctas * parts;
            parts *= gridDim.x / p.ctas;
            c %= p.ctas;
        }
    }
    if (u.last_cta < 0) return;
    const int n = u.last_cta - c + 1;
    int ways = 1;  // warps per row
    while (ways < kMergeWarps && u.rows * ways * 2 <= kMergeWarps) ways *= 2;
    const int per = (n + ways - 1) / ways, run = warp % ways;
    const int s_lo = min(run * per, n), s_hi = min(s_lo + per, n);
    for (int row0 = part * (kMergeWarps / ways); row0 < u.rows; row0 += parts * (kMergeWarps / ways)) {
        const int row = row0 + warp / ways;
        const bool there = row < u.rows;
        auto prow = [&](int s) {
            return static_cast<size_t>(s == 0 ? u.slot : 2 * (c + s)) * u.slot_rows + row;
        };
        float m = -INFINITY, wsum = 0.f, acc[kV];
#pragma unroll
        for (int e = 0; e < kV; ++e) acc[e] = 0.f;
        for (int s0 = s_lo; there && s0 < s_hi; s0 += kMergeBatch) {
            const int ns = min(kMergeBatch, s_hi - s0);
            float o[kMergeBatch][kV];
#pragma unroll
            for (int s = 0; s < kMergeBatch; ++s) {
                const float *src = p.part_O + prow(s0 + min(s, ns - 1)) * D + lane * kV;
#pragma unroll
                for (int e = 0; e < kV; ++e) o[s][e] = src[e];
            }
            // lane s the statistic of piece s0 + s; an empty piece (-inf) weighs 0
            const float x = lane < ns ? p.part_LSE[prow(s0 + lane)] : -INFINITY;
            float top = x;
#pragma unroll
            for (int d = kMergeBatch / 2; d > 0; d >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float m_new = fmaxf(m, __shfl_sync(0xffffffffu, top, 0));
            const float f = m == -INFINITY ? 0.f : expf(m - m_new);
            m = m_new;
            wsum *= f;
#pragma unroll
            for (int e = 0; e < kV; ++e) acc[e] *= f;
            const float w = x == -INFINITY ? 0.f : expf(x - m);
#pragma unroll
            for (int s = 0; s < kMergeBatch; ++s) {
                const float ws = __shfl_sync(0xffffffffu, w, s);
                if (s >= ns) break;
                wsum += ws;
#pragma unroll
                for (int e = 0; e < kV; ++e) acc[e] = fmaf(ws, o[s][e], acc[e]);
            }
        }
        if (ways > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kV; ++e) red_o[warp][lane * kV + e] = acc[e];
            if (lane == 0) red_m[warp] = m, red_w[warp] = wsum;
            __syncthreads();
            if (run == 0) {
                float top = m;
                for (int i = 1; i < ways; ++i) top = fmaxf(top, red_m[warp + i]);
                float total = 0.f;
#pragma unroll
                for (int e = 0; e < kV; ++e) acc[e] = 0.f;
                for (int i = 0; i < ways; ++i) {
                    // a run that saw nothing adds nothing; one with NaN adds it
                    if (red_m[warp + i] == -INFINITY && red_w[warp + i] == 0.f) continue;
                    const float f = red_m[warp + i] == top ? 1.f : expf(red_m[warp + i] - top);
                    total = fmaf(f, red_w[warp + i], total);
#pragma unroll
                    for (int e = 0; e < kV; ++e) acc[e] = fmaf(f, red_o[warp + i][lane * kV + e], acc[e]);
                }
                m = top;
                wsum = total;
            }
        }
        if (!there || run != 0) continue;
        const bool none = wsum == 0.f;
        const float inv = none ? 0.f : 1.f / wsum;
#pragma unroll
        for (int e = 0; e < kV; ++e) acc[e] *= inv;
        const int i = row / p.pf;
        const size_t g = (static_cast<size_t>(u.tok0) + i) * p.H + u.head0 + (row - i * p.pf);
        uint16_t *orow = reinterpret_cast<uint16_t *>(p.O) + g * D + lane * kV;
        if constexpr (kV == 1) {
            orow[0] = static_cast<uint16_t>(pack2<BF16>(acc[0], 0.f) & 0xffffu);
        } else {
#pragma unroll
            for (int e = 0; e < kV; e += 2)
                *reinterpret_cast<uint32_t *>(orow + e) = pack2<BF16>(acc[e], acc[e + 1]);
        }
        if (lane == 0) p.LSE[g] = none ? -INFINITY : m + logf(wsum);
    }
}

}  // namespace paged
}  // namespace fa
