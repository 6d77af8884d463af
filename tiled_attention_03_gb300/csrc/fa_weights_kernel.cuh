// fa_weights_kernel.cuh -- the attention weight that the new tokens of a batch give to each key of
// a paged cache, for head dimensions 32, 64, 128 and 256 on sm_103a.
//
// For key j of a K/V head, over the new tokens i of its sequence that see it and the query
// heads h of the group,
//     a_j = sum_{i, h} exp(scale q_{i,h} . k_j - LSE_{i,h}),
// with the LSE that the attention of the same tokens left. No row maximum and no normalisation
// are needed: LSE is both. A key that was there before gets a_j added, one of the call's
// own tokens is set to it, so a slot's former content does not matter.
//
// The scores are taken transposed, S^T = K Q^T (128 keys x R rows): keys stand in the lanes of
// tensor memory, so that the sum over rows is a sum over one thread's registers, and a tile of
// keys, the M operand, is read once for all rows of its sequence and K/V head. A unit is one tile
// of 128 or 256 keys of one K/V head with all tiles of R rows that see it; CTA c takes every gridDim-th
// unit from c on (every other time from the end of the run: units of one sequence grow lighter along
// the keys under a causal mask). That shares them evenly, needs no counters, and gives every
// key to one thread: one addition per key and call, so the result is the same every time (keys
// of pages that several sequences share get one addition each, in any order).
//
// What bounds it: single steps read K once, by HBM (8 sequences of 32768 keys of 8 heads of 128: 88
// us, 6.1 TB/s); short or narrow ones by the 1,400 cycles that a unit costs its issuer, in waits and in
// instructions that are fetched anew (lanes that wait for a barrier each, and units handed out 32 at a
// time, made both slower, by 2 and 8 %). Chunks: a tile of 128 x 128 scores takes about 1,150 cycles, of which
// the products take 528 and the exponentials as long; computing some of those by multiply-adds made it
// slower (10 of 32: by 13 %), as the sums wait for tensor memory and for each other more than for a pipe.
//
// Warps (640 threads): 0-15 are four teams of four that sum every fourth tile of rows (of units with
// one: every fourth unit), as one team's loads from tensor memory and exponentials wait for each
// other; 16 finds units, 32 at a time, 17 issues the products, 18 loads queries and their LSE, 19 loads
// keys; the loaders ask for page numbers one tile ahead, and for LSEs one or, where units have many tiles,
// three (2048 tokens on 6000 keys: 126 us with one, 118 with three).
// Every wait is bounded; on expiry the CTA records the failure, drains its copies and
// products, frees its tensor memory and returns.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "fa_divisor.cuh"
#include "fa_paged_kernel.cuh"
#include "fa_pdl.cuh"
#include "ptx.cuh"

namespace fa {
namespace weights {

// Keys of a tile: 128, or 256 (two products, one behind the other) for narrow tiles of rows, where what
// a unit costs besides its products is most of it (8 sequences of 32768 keys 88.4 us, with 128 88.7;
// 100 of 0-12000 at d = 64 20.4 and 25.0; with tiles of 64 rows 128 are better, 16 sequences of
// 6000-9000 keys and 40 rows 27.1 and 29.6).
constexpr int tile_keys(int d, int rows) { return rows == 16 && d <= 128 ? 256 : 128; }
constexpr int kTeams = 4;
constexpr int kThreads = (4 * kTeams + 4) * 32;
constexpr int kPlanWarp = 4 * kTeams, kIssueWarp = kPlanWarp + 1, kQWarp = kPlanWarp + 2, kKWarp = kPlanWarp + 3;
constexpr int kUnitSlots = 16;  // more than a loader's look-ups and tiles together
constexpr int kUnitConsumers = 4 * kTeams + 3;  // warps that take the units: all but the one that finds them
constexpr int kMaxStages = 8;
constexpr int kBufs = 4;  // of scores
constexpr int kLses = 8;  // of their rows' LSE: more, as queries are loaded after the LSE before them
// A team's tiles follow each other by kTeams, so it meets every use of its buffer and slots: a wait
// tells two uses of a barrier apart only when they follow each other.
static_assert(kBufs == kTeams && (kTeams & (kTeams - 1)) == 0 && kLses % kTeams == 0, "buffers of a team");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmem = 0;  // all columns are allocated: they start at 0
constexpr unsigned kStatusTimeout = 4;
constexpr unsigned kStatusLayout = 2;  // shared memory base not 1024-aligned
enum : int { kRoleSum = 1, kRoleTma = 2, kRoleMma = 3 };

struct Params {
    float *weights;    // page x H_kv x page_size
    const float *LSE;
    const int *cu_q, *seq_k, *table;
    int B, H, H_kv, pf, subs, tpt;  // heads and tokens of a tile of rows; tiles of heads per group
    int total_q, max_pages, page_log2, num_pages, max_keys;
    int chunk;         // tokens per TMA box: min(page size, keys of a tile)
    int page_step, head_step, page_none;  // the map's last coordinate; past its end
    Divisor by_heads, by_tpt, by_subs;  // by H_kv, tpt and subs
    int wl, wr;        // key j visible to the query at position i iff i - wl <= j <= i + wr
    float scale_log2;
    unsigned long long wait_budget_ns;
    unsigned int *status;
    int fault_skip_k;  // test hook: every CTA skips the load at this ring position (-1: none)
};

template <int D, int R>
struct Smem {
    using P = paged::Smem<D>;  // the layout of key tiles: groups of 8 rows, their regions side by side
    static constexpr int kBK = tile_keys(D, R);
    static constexpr int kHalves = kBK / 128;
    static constexpr int kTile = kBK / 8 * P::kGroup;
    static constexpr int kQRegion = R * P::kRowBytes;
    static constexpr int kQBytes = P::kRegions * kQRegion;
    static constexpr int kSmall = 9728;
    static constexpr int kMost = 227 * 1024 - kSmall;
    // up to four tiles of queries that leave four of keys; two of keys where one is 64 KB, or where
    // units have many tiles of rows, which then come faster than keys
    static constexpr int kQFit = (kMost - (D == 256 || R == 128 ? 2 : 4) * kTile / kHalves) / kQBytes;
    static constexpr int kQStages = kQFit < 4 ? kQFit : 4;
    static constexpr int kKFit = (kMost - kQStages * kQBytes) / kTile;
    static constexpr int kKStages = kKFit < kMaxStages ? kKFit : kMaxStages;
    static_assert(kQStages >= 2 && kKStages >= 2, "shared memory");
    static constexpr int kK = 0;
    static constexpr int kQ = kK + kKStages * kTile;
    static constexpr int kBar = kQ + kQStages * kQBytes;
    static constexpr int kMisc = kBar + 96 * 8;              // TMEM address, abort flag
    static constexpr int kRing = kMisc + 16;                 // kUnitSlots units
    static constexpr int kLse = kRing + kUnitSlots * 64;     // kLses x R, times -log2 e
    static constexpr int kSums = kLse + kLses * R * 4;       // two units' sums of three teams
    static constexpr int kBlind = kSums + 2 * (kTeams - 1) * kBK * 4;  // a bit per row of an LSE slot
    static constexpr int kBlindWords = (R + 31) / 32;
    static constexpr int kBytes = kBlind + kLses * kBlindWords * 4;
    static_assert(kBufs * kHalves * R <= kTmemCols, "TMEM columns");
    static_assert(kLse % 16 == 0 && kBytes - kBar <= kSmall, "layout");
    static constexpr int kAlloc = kBytes > 120 * 1024 ? kBytes : 120 * 1024;  // one CTA per SM
};

enum : int {
    kBarKFull = 0,                         // + stage
    kBarKEmpty = kBarKFull + kMaxStages,   // + stage
    kBarQFull = kBarKEmpty + kMaxStages,   // + stage (4)
    kBarQEmpty = kBarQFull + 4,            // + stage (4)
    kBarSFull = kBarQEmpty + 4,            // + buffer
    kBarSEmpty = kBarSFull + kBufs,        // + buffer
    kBarLFull = kBarSEmpty + kBufs,        // + LSE slot
    kBarLEmpty = kBarLFull + kLses,        // + LSE slot
    kBarSumFull = kBarLEmpty + kLses,      // + slot (2)
    kBarSumEmpty = kBarSumFull + 2,        // + slot (2)
    kBarUnitFull = kBarSumEmpty + 2,            // + slot
    kBarUnitEmpty = kBarUnitFull + kUnitSlots,  // + slot
    kBarDrain = kBarUnitEmpty + kUnitSlots,
    kNumBars = kBarDrain + 1,
};
static_assert(kNumBars <= 96, "barrier slots");

// A tile of keys of K/V head h of sequence b, and its n tiles of rows from the first-th on
// (tile r: tokens from r / subs * tpt on, heads from r mod subs * pf on).
struct Unit {
    int b, h, j;
    int first, n;
    int q0, nq, nk, q_off;  // token i of the sequence stands at key position i + q_off
    int fresh;              // keys from here on are the call's own
};
static_assert(sizeof(Unit) <= 64, "ring slot");

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
// The first tile of keys that a token of the sequence sees, and how many follow.
template <int kBK>
__device__ __forceinline__ int first_tile(const Seq &s, const Params &p) {
    return max(0, s.nk - s.nq - p.wl) / kBK;
}
template <int kBK>
__device__ __forceinline__ int key_tiles(const Seq &s, const Params &p) {
    return s.nq == 0 || s.nk == 0 ? 0 : max(0, (s.nk - 1) / kBK - first_tile<kBK>(s, p) + 1);
}
// Tokens lo .. hi (hi < lo: none) see a key of keys k0 .. k1.
__device__ __forceinline__ void tokens_of(const Unit &u, int k0, int k1, const Params &p, int &lo, int &hi) {
    lo = max(0, k0 - u.q_off - p.wr);
    hi = min(u.nq - 1, k1 - u.q_off + p.wl);
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

// 16 or 32 columns of this warp's lanes; and the wait for them.
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }
__device__ __forceinline__ void ld_cols_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void ld_cols_wait(uint32_t (&r)[32]) { tmem_ld_wait(r); }

template <int D, int R, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    fa_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ Params p) {
    using L = Smem<D, R>;
    using P = typename L::P;
    constexpr int kBK = L::kBK, kHalves = L::kHalves;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *const smem = smem_raw;
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + L::kBar;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kMisc + 4);
    auto bar = [bar0](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    auto sK = [sbase](int t) { return sbase + L::kK + (t % L::kKStages) * L::kTile; };
    auto sQ = [sbase](int t) { return sbase + L::kQ + (t % L::kQStages) * L::kQBytes; };
    float *const lse_ring = reinterpret_cast<float *>(smem + L::kLse);
    uint32_t *const blind_ring = reinterpret_cast<uint32_t *>(smem + L::kBlind);  // 1: the row's LSE is -infinity
    // (from one lane: the compiler then knows that the roles' branches are the warp's)
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
    const int lane = threadIdx.x & 31;
    const uint64_t budget = p.wait_budget_ns;

    if ((sbase & 1023u) != 0) {
        after_previous();
        if (threadIdx.x == 0) atomicCAS(p.status, 0u, kStatusLayout);
        return;
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    if (threadIdx.x == kPlanWarp * 32) {
        for (int s = 0; s < L::kKStages; ++s) {
            mbar_init(bar(kBarKFull + s), 1);
            mbar_init(bar(kBarKEmpty + s), 1);
        }
        for (int s = 0; s < L::kQStages; ++s) {
            mbar_init(bar(kBarQFull + s), 1);
            mbar_init(bar(kBarQEmpty + s), 1);
        }
        for (int s = 0; s < kBufs; ++s) {
            mbar_init(bar(kBarSFull + s), 1);
            mbar_init(bar(kBarSEmpty + s), 128);
        }
        for (int s = 0; s < kLses; ++s) {
            mbar_init(bar(kBarLFull + s), 32);
            mbar_init(bar(kBarLEmpty + s), 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(kBarSumFull + s), 128 * (kTeams - 1));
            mbar_init(bar(kBarSumEmpty + s), 128);
        }
        for (int k = 0; k < kUnitSlots; ++k) {
            mbar_init(bar(kBarUnitFull + k), 1);
            mbar_init(bar(kBarUnitEmpty + k), kUnitConsumers);
        }
        mbar_init(bar(kBarDrain), 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    after_previous();
    let_next_start();
    const bool idle = *tmem_slot != kTmem;
    if (idle && threadIdx.x == 0) atomicCAS(p.status, 0u, kStatusLayout);

    auto slot_of = [smem](int k) { return reinterpret_cast<Unit *>(smem + L::kRing + (k % kUnitSlots) * 64); };
    auto wait = [&](int b, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait_bounded(bar(b), parity, abort_flag, budget)) != 0;
    };
    auto one = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    // The k-th unit of this CTA (every role walks the same ones). b < 0: no more.
    auto take = [&](int k, bool &ok) -> Unit {
        Unit u{};
        u.b = -1;
        const int slot = k % kUnitSlots;
        ok = wait(kBarUnitFull + slot, (k / kUnitSlots) & 1);
        if (!ok) return u;
        u = *slot_of(k);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarUnitEmpty + slot));
        u.b = one(u.b);
        u.n = one(u.n);
        return u;
    };

    if (idle) {
        // (frees its tensor memory below)
    } else if (warp == kPlanWarp) {
        // ================================================================ units
        // Units are numbered sequence by sequence, tile by tile, head by head (the heads of a tile lie
        // beside each other, and CTAs side by side read them at the same time). Each lane holds one
        // sequence of the 32 from b0 on, with its units and those before it from `base` on, and
        // looks up one of this CTA's next 32 units among them.
        // The i-th is in the i-th run of gridDim units, from its front or, for odd i, from its end: where
        // units grow lighter, who has a heavy one has a light one next.
        auto unit_of = [&](long long i) {
            return i * gridDim.x + (i & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        };
        // A sequence's tokens begin where those of the sequences before it end, at the earliest, so that
        // offsets in no order make no more work than ordered ones. What is left of them are its
        // last ones: they keep their positions.
        long long base = 0, next = lane;
        bool ok = true;
        int k = 0, claimed = 0;
        for (int b0 = 0; ok && b0 < p.B; b0 += 32) {
            Seq s = load_seq(b0 + lane, p);
            int ends = s.nq > 0 ? s.q0 + s.nq : 0;  // the most of the sequences' ends up to this one
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, ends, o);
                if (lane >= o) ends = max(ends, x);
            }
            int before_me = __shfl_up_sync(0xffffffffu, ends, 1);
            before_me = max(lane > 0 ? before_me : 0, claimed);
            const int fresh = s.nk - s.nq, lost = min(max(before_me - s.q0, 0), s.nq);
            s.q0 += lost;
            s.nq -= lost;
            claimed = max(claimed, __shfl_sync(0xffffffffu, ends, 31));
            const int tiles = key_tiles<kBK>(s, p);
            long long incl = static_cast<long long>(tiles) * p.H_kv;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            const long long before = incl - static_cast<long long>(tiles) * p.H_kv;
            const long long all = __shfl_sync(0xffffffffu, incl, 31);
            while (ok) {
                const long long rel = unit_of(next) - base;
                // the last sequence with no more than rel units before it
                int at = 0;
#pragma unroll
                for (int step = 16; step > 0; step >>= 1)
                    if (__shfl_sync(0xffffffffu, before, at + step) <= rel) at += step;
                Unit u{};
                u.b = b0 + at;
                u.q0 = __shfl_sync(0xffffffffu, s.q0, at);
                u.nq = __shfl_sync(0xffffffffu, s.nq, at);
                u.nk = __shfl_sync(0xffffffffu, s.nk, at);
                const int x = static_cast<int>(rel - __shfl_sync(0xffffffffu, before, at));
                const int found = __popc(__ballot_sync(0xffffffffu, rel < all));  // of the 32 units
                const int y = p.by_heads.of(max(x, 0));
                u.h = x - y * p.H_kv;
                u.q_off = u.nk - u.nq;
                u.fresh = __shfl_sync(0xffffffffu, fresh, at);
                u.j = y + first_tile<kBK>(Seq{0, u.nq, u.nk}, p);
                int lo, hi;
                tokens_of(u, u.j * kBK, min(u.j * kBK + kBK, u.nk) - 1, p, lo, hi);
                u.first = p.by_tpt.of(lo) * p.subs;
                u.n = hi < lo ? 0 : (p.by_tpt.of(hi) + 1) * p.subs - u.first;
                for (int i = 0; ok && i < found; ++i, ++k) {
                    const int slot = k % kUnitSlots;
                    ok = wait(kBarUnitEmpty + slot, ((k / kUnitSlots) & 1) ^ 1);
                    if (ok && lane == i) {
                        *slot_of(k) = u;
                        mbar_arrive(bar(kBarUnitFull + slot));
                    }
                    __syncwarp();
                }
                next += found;
                if (found < 32) break;
            }
            base += all;
        }
        if (ok) {
            const int slot = k % kUnitSlots;
            ok = wait(kBarUnitEmpty + slot, ((k / kUnitSlots) & 1) ^ 1);
            if (ok && lane == 0) {
                Unit u{};
                u.b = -1;
                *slot_of(k) = u;
                mbar_arrive(bar(kBarUnitFull + slot));
            }
            __syncwarp();
        }
        if (!ok && lane == 0) record_timeout(p, abort_flag, kRoleTma, -3);
    } else if (warp == kKWarp) {
        // ================================================================ key tiles
        bool ok = true;
        int k = 0, t = 0;
        // The next unit with rows: its chunk `lane` of the tile, and that chunk's page.
        struct Tile {
            int b, h, k0, page;
            bool need;
        };
        auto next = [&]() -> Tile {
            Tile n{-1, 0, 0, 0, false};
            while (true) {
                const Unit u = take(k, ok);
                ++k;
                if (!ok || u.b < 0) return n;
                if (u.n == 0) continue;
                n.b = u.b;
                n.h = u.h;
                n.k0 = u.j * kBK + lane * p.chunk;
                n.need = lane * p.chunk < kBK && n.k0 < u.nk;
                if (n.need) n.page = p.table[static_cast<size_t>(u.b) * p.max_pages + (n.k0 >> p.page_log2)];
                return n;
            }
        };
        Tile now = next();
        while (ok && now.b >= 0) {
            const Tile after = next();
            if (!ok) break;
            // a page number outside the cache reads as zeros
            const int page = now.page >= 0 && now.page < p.num_pages ? now.page * p.page_step + now.h * p.head_step
                                                                     : p.page_none;
            const unsigned all = __ballot_sync(0xffffffffu, now.need);
            const int st = t % L::kKStages;
            ok = wait(kBarKEmpty + st, ((t / L::kKStages) & 1) ^ 1);
            if (!ok) break;
            if (t != p.fault_skip_k) {
                if (lane == 0)
                    mbar_arrive_expect_tx(bar(kBarKFull + st),
                                          static_cast<uint32_t>(__popc(all)) * p.chunk * (P::kGroup / 8));
                __syncwarp();
                if (now.need)
                    paged::tma_load_5d(sK(t) + lane * p.chunk * (P::kGroup / 8), &tmK, bar(kBarKFull + st), 0, 0, 0,
                                       (now.k0 & ((1 << p.page_log2) - 1)) >> 3, page);
                __syncwarp();
            }
            ++t;
            now = after;
        }
        if (lane == 0) {
            if (!ok) record_timeout(p, abort_flag, kRoleTma, -1);
            for (int s2 = 0; s2 < L::kKStages; ++s2)
                if (t > s2) {
                    const int last = t - 1 - ((t - 1 - s2) % L::kKStages);
                    mbar_wait_bounded(bar(kBarKFull + s2), (last / L::kKStages) & 1, nullptr, budget);
                }
        }
    } else if (warp == kQWarp) {
        // ================================================================ queries and their LSE
        bool ok = true;
        int k = 0, i = 0;
        constexpr int kOwn = (R + 31) / 32;
        // this lane's rows of a tile: token and head
        int tok[kOwn], head[kOwn];
#pragma unroll
        for (int y = 0; y < kOwn; ++y) {
            tok[y] = (lane + 32 * y) / p.pf;
            head[y] = lane + 32 * y - tok[y] * p.pf;
        }
        Unit u{};
        int x = 0;
        bool end = false;
        // A tile of rows: its first token of all (< 0: no more) and head, and its LSEs.
        struct Tile {
            int row0, h0;
            float v[kOwn];
        };
        auto next = [&](Tile &n) {
            n.row0 = -1;
            if (end) return;
            while (x >= u.n) {
                u = take(k, ok);
                ++k;
                x = 0;
                if (!ok || u.b < 0) {
                    end = true;
                    return;
                }
            }
            const int r = u.first + x++;
            const int ts = p.by_subs.of(r), t0 = ts * p.tpt;
            n.h0 = (u.h * p.subs + r - ts * p.subs) * p.pf;
            n.row0 = u.q0 + t0;
#pragma unroll
            for (int y = 0; y < kOwn; ++y) {
                n.v[y] = -INFINITY;
                if (tok[y] < p.tpt && t0 + tok[y] < u.nq)
                    n.v[y] = p.LSE[(static_cast<size_t>(n.row0) + tok[y]) * p.H + n.h0 + head[y]];
            }
        };
        auto load = [&](const Tile &n) {
            const int st = i % L::kQStages;
            ok = ok && wait(kBarQEmpty + st, ((i / L::kQStages) & 1) ^ 1);
            if (!ok) return;
            if (lane == 0)
                mbar_arrive_expect_tx(bar(kBarQFull + st),
                                      static_cast<uint32_t>(p.pf * p.tpt) * P::kRowBytes * P::kRegions);
            __syncwarp();
            if (lane < P::kRegions)
                tma_load_3d(sQ(i) + lane * L::kQRegion, &tmQ, bar(kBarQFull + st), P::kCols * lane, n.h0, n.row0);
            __syncwarp();
            ++i;
        };
        // row c: token c / pf, head c mod pf. Minus the LSE; rows that saw nothing are marked, as no
        // number added to any score, NaN and infinity among them, would make their weights 0
        auto store = [&](const Tile &n) {
            const int slot = (i - 1) % kLses;
            ok = ok && wait(kBarLEmpty + slot, (((i - 1) / kLses) & 1) ^ 1);
            if (!ok) return;
#pragma unroll
            for (int y = 0; y < kOwn; ++y) {
                const uint32_t none = __ballot_sync(0xffffffffu, n.v[y] == -INFINITY);
                if (lane == 0) blind_ring[slot * L::kBlindWords + y] = none;
                if (lane + 32 * y < R) lse_ring[slot * R + lane + 32 * y] = n.v[y] * -1.4426950408889634f;
            }
            mbar_arrive(bar(kBarLFull + slot));
        };
        if constexpr (R >= 64) {
            // LSEs three tiles ahead, in variables of their own, as a copy would wait for them
            Tile n0, n1, n2;
            next(n0);
            next(n1);
            next(n2);
            bool more = true;
            auto step = [&](Tile &n) {
                more = more && ok && n.row0 >= 0;
                if (!more) return;
                load(n);
                store(n);
                if (ok) next(n);
            };
            while (more) {
                step(n0);
                step(n1);
                step(n2);
            }
        } else {
            Tile n;
            next(n);
            while (ok && n.row0 >= 0) {
                load(n);
                const Tile now = n;
                next(n);
                store(now);
            }
        }
        if (lane == 0) {
            if (!ok) record_timeout(p, abort_flag, kRoleTma, -2);
            for (int s = 0; s < L::kQStages; ++s)
                if (i > s) {
                    const int last = i - 1 - ((i - 1 - s) % L::kQStages);
                    mbar_wait_bounded(bar(kBarQFull + s), (last / L::kQStages) & 1, nullptr, budget);
                }
        }
    } else if (warp == kIssueWarp) {
        // ================================================================ S^T = K Q^T
        constexpr uint32_t idesc = idesc_f16_ab(BF16, 128, R, false, false);
        constexpr int kSteps = P::kCols / 16;  // K-steps of 16 columns per region
        int t = 0, i = 0, k = 0;
        bool ok = true;
        for (; ok; ++k) {
            const Unit u = take(k, ok);
            if (!ok || u.b < 0) break;
            if (u.n == 0) continue;
            ok = wait(kBarKFull + t % L::kKStages, (t / L::kKStages) & 1);
            const uint64_t dk = paged::tile_desc<P::kRowBytes>(sK(t), 16, P::kGroup);
            for (int x = 0; ok && x < u.n; ++x, ++i) {
                ok = wait(kBarQFull + i % L::kQStages, (i / L::kQStages) & 1);
                if (ok) ok = wait(kBarSEmpty + i % kBufs, ((i / kBufs) & 1) ^ 1);
                if (!ok) break;
                tc_fence_after();
                const uint64_t dq = paged::tile_desc<P::kRowBytes>(sQ(i), 16, P::kAtom);
                const uint32_t d = kTmem + (i % kBufs) * kHalves * R;
                if (elect_one()) {
#pragma unroll
                    for (int c = 0; c < kHalves * D / 16; ++c) {
                        constexpr int kOf = D / 16;
                        umma_f16_ss(d + c / kOf * R,
                                    dk + c / kOf * (16 * P::kGroup >> 4) + (c % kOf / kSteps) * (P::kAtom >> 4) +
                                        (c % kSteps) * 2,
                                    dq + (c % kOf / kSteps) * (L::kQRegion >> 4) + (c % kSteps) * 2, idesc,
                                    c % kOf > 0 ? 1u : 0u);
                    }
                    umma_commit(bar(kBarSFull + i % kBufs));
                    umma_commit(bar(kBarQEmpty + i % L::kQStages));
                }
                __syncwarp();
            }
            if (ok) {
                if (elect_one()) umma_commit(bar(kBarKEmpty + t % L::kKStages));
                __syncwarp();
                ++t;
            }
        }
        if (!ok && lane == 0) record_timeout(p, abort_flag, kRoleMma, k);
        if (elect_one()) umma_commit(bar(kBarDrain));
        __syncwarp();
        if (lane == 0) mbar_wait_bounded(bar(kBarDrain), 0, nullptr, budget);
        __syncwarp();
    } else {
        // ================================================================ sums over rows
        const int team = warp >> 2;
        const int own = threadIdx.x & 127;
        const uint32_t tl = kTmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const float sl2 = p.scale_log2;
        float *const sums = reinterpret_cast<float *>(smem + L::kSums);
        int i = 0, k = 0, joined = 0;  // tiles of rows; units; those that the teams share
        bool ok = true;
        for (; ok; ++k) {
            const Unit u = take(k, ok);
            if (!ok || u.b < 0) break;
            if (u.n == 0) continue;
            const int me = (team - i) & (kTeams - 1);  // tiles me, me + kTeams, ... of the unit are this team's
            if (u.n == 1 && me != 0) {
                ++i;
                continue;
            }
            // this thread's keys; their pages; the tokens that see them, and those that see every key of the tile
            int key[kHalves], page[kHalves], lo[kHalves], hi[kHalves], all_lo, all_hi, x1, x2;
#pragma unroll
            for (int y = 0; y < kHalves; ++y) {
                key[y] = u.j * kBK + 128 * y + own;
                page[y] = -1;
                if (key[y] < u.nk && me == 0)
                    page[y] = p.table[static_cast<size_t>(u.b) * p.max_pages + (key[y] >> p.page_log2)];
                tokens_of(u, key[y], key[y], p, lo[y], hi[y]);
            }
            tokens_of(u, u.j * kBK + kBK - 1, u.j * kBK + kBK - 1, p, all_lo, x1);
            tokens_of(u, u.j * kBK, u.j * kBK, p, x2, all_hi);
            float a[kHalves][4];
#pragma unroll
            for (int y = 0; y < kHalves; ++y) a[y][0] = a[y][1] = a[y][2] = a[y][3] = 0.f;
            for (int x = me; ok && x < u.n; x += kTeams) {
                const int at = i + x, buf = at % kBufs, t0 = p.by_subs.of(u.first + x) * p.tpt;
                ok = wait(kBarLFull + at % kLses, (at / kLses) & 1);
                if (ok) ok = wait(kBarSFull + buf, (at / kBufs) & 1);
                if (!ok) break;
                tc_fence_after();
                // rows that see this key, and whether that is every row of the tile for all keys (rows
                // behind the sequence's last token may hold anything: they are not looked at)
                const bool whole = t0 >= all_lo && t0 + p.tpt - 1 <= all_hi && p.tpt * p.pf == R;
                const float *lse = lse_ring + at % kLses * R;
                // (a bit per row: comparing the LSEs themselves cost registers, 116 -> 139 us for 2048 tokens on
                // 6000 keys, the bits 118)
                uint32_t blinds[L::kBlindWords], any_blind = 0;
#pragma unroll
                for (int w = 0; w < L::kBlindWords; ++w) any_blind |= blinds[w] = blind_ring[at % kLses * L::kBlindWords + w];
                constexpr int kCols = R < 32 ? R : 32, kLoads = kHalves * R / kCols;
                uint32_t r[2][kCols];  // the next columns come while these are summed
                ld_cols(tl + buf * kHalves * R, r[0]);
#pragma unroll
                for (int z = 0; z < kLoads; ++z) {
                    const int h = z * kCols % R, half = z * kCols / R;
                    uint32_t(&now)[kCols] = r[z & 1];
                    ld_cols_wait(now);
                    if (z + 1 < kLoads) ld_cols(tl + buf * kHalves * R + (z + 1) * kCols, r[(z + 1) & 1]);
                    float y[kCols];
#pragma unroll
                    for (int c = 0; c < kCols; c += 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(lse + h + c);
                        y[c] = __uint_as_float(now[c]), y[c + 1] = __uint_as_float(now[c + 1]);
                        y[c + 2] = __uint_as_float(now[c + 2]), y[c + 3] = __uint_as_float(now[c + 3]);
                        ffma2(y[c], y[c + 1], sl2, sl2, v.x, v.y);
                        ffma2(y[c + 2], y[c + 3], sl2, sl2, v.z, v.w);
                    }
                    if (z + 1 == kLoads) {  // scores and LSE are read: the next ones may come
                        tc_fence_before();
                        mbar_arrive(bar(kBarSEmpty + buf));
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(kBarLEmpty + at % kLses));
                    }
                    if (!whole || any_blind != 0) {
                        const int c_lo = (lo[half] - t0) * p.pf, c_hi = min(hi[half] - t0 + 1, p.tpt) * p.pf;
                        // ones from bit n on, for n of 0 to 32
                        auto from = [](int n) { return __funnelshift_lc(0u, ~0u, min(max(n, 0), 32)); };
                        const uint32_t sees = from(c_lo - h) & ~from(c_hi - h) & ~blinds[h / 32];
#pragma unroll
                        for (int c = 0; c < kCols; ++c)
                            if ((sees >> c & 1) == 0) y[c] = -INFINITY;
                    }
#pragma unroll
                    for (int c = 0; c < kCols; ++c) y[c] = ex2_approx(y[c]);
#pragma unroll
                    for (int c = 0; c < kCols; c += 4) {
                        fadd2(a[half][0], a[half][1], y[c], y[c + 1]);
                        fadd2(a[half][2], a[half][3], y[c + 2], y[c + 3]);
                    }
                }
            }
            i += u.n;
            if (!ok) break;
            float sum[kHalves];
#pragma unroll
            for (int y = 0; y < kHalves; ++y) sum[y] = (a[y][0] + a[y][1]) + (a[y][2] + a[y][3]);
            if (u.n > 1) {
                // the other teams hand their sums to the first
                const int slot = joined % 2;
                float *const sum_of = sums + slot * (kTeams - 1) * kBK + own;
                // (the first as well, as the others may not have handed it those of two units ago)
                ok = wait(kBarSumEmpty + slot, ((joined / 2) & 1) ^ 1);
                if (!ok) break;
                if (me != 0) {
#pragma unroll
                    for (int y = 0; y < kHalves; ++y) sum_of[(me - 1) * kBK + 128 * y] = sum[y];
                    mbar_arrive(bar(kBarSumFull + slot));
                } else {
                    ok = wait(kBarSumFull + slot, (joined / 2) & 1);
                    if (!ok) break;
#pragma unroll
                    for (int o = 0; o < kTeams - 1; ++o)
#pragma unroll
                        for (int y = 0; y < kHalves; ++y) sum[y] += sum_of[o * kBK + 128 * y];
                    mbar_arrive(bar(kBarSumEmpty + slot));
                }
                ++joined;
                if (me != 0) continue;
            }
#pragma unroll
            for (int y = 0; y < kHalves; ++y)
                if (key[y] < u.nk && page[y] >= 0 && page[y] < p.num_pages) {
                    float *w = p.weights + ((static_cast<size_t>(page[y]) * p.H_kv + u.h) << p.page_log2) +
                               (key[y] & ((1 << p.page_log2) - 1));
                    if (key[y] >= u.fresh)
                        *w = sum[y];
                    else
                        atomicAdd(w, sum[y]);
                }
        }
        if (!ok && lane == 0) record_timeout(p, abort_flag, kRoleSum, k);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(*tmem_slot, kTmemCols);
    }
}

}  // namespace weights
}  // namespace fa
