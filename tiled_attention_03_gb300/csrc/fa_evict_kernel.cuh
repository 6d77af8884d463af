// fa_evict_kernel.cuh -- eviction from a paged K/V cache: for each sequence that is longer than
// the budget and each K/V head, the keys to keep (the first ones, the recent ones, and of
// those between the ones of the largest weight) move together, in their order, to the front of the
// sequence's pages, with their values and weights.
//
// A cluster of 1 .. 8 CTAs takes a sequence and head. It first selects, each CTA on its part of the
// slots: weights as ordered 32-bit numbers, histograms of 8 bits at a time summed over the
// cluster through distributed shared memory, from the top digit down until the kept ones are
// exactly told apart; where equal weights remain, 8 bits of the index at a time, lowest first. What
// is kept is then a comparison with two numbers; one bit per slot of it goes to every CTA.
//
// Then it moves, in place, each CTA its own columns of all rows (of 64 or 128 bytes where rows are
// that wide), so that none waits for another. Row r of what is kept comes from a slot >= r: rounds of
// consecutive rows are taken in order, and a round is written once it, and so all before, has
// been read. The next rounds' rows are on their way meanwhile (asynchronous copies to shared memory):
// they lie behind everything that this round writes. One block barrier a round orders all of that. (With
// whole rows per CTA and slots shared among the cluster a round was small and took a cluster barrier
// and 1.5 to 2 us: 16 sequences of 5000 to 20000 keys cut to 8192 took 295 us; rounds of
// consecutive slots instead of rows, fewer bytes in flight where few are kept, 174; this 127, 4.8 TB/s.)
//
// Bound by memory: rows and weights are read and written once.
#pragma once

#include <cstdint>

#include "fa_copy.cuh"
#include "fa_pdl.cuh"
#include "ptx.cuh"

namespace fa {
namespace evict {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kDepth = 3;             // rounds of rows in shared memory
constexpr int kPages = 2048;          // page numbers that stay there
constexpr int kWords = 2048;          // 32 slots each: a window of slots whose bits are known
constexpr int kWindow = kWords * 32;

struct Params {
    uint16_t *k, *v;
    float *weights;  // page x H_kv x page_size
    long long page_stride, token_stride, head_stride;
    const int *seq_k, *table;
    int *seq_out;
    int H_kv, d;
    int rows;        // of a round (at most kThreads)
    int piece_log2;  // 16-byte pieces of a CTA's columns: 2^piece_log2
    int keys;        // weights of a CTA that stay in shared memory (a multiple of 4)
    int max_pages, page_log2, num_pages, max_keys;
    int budget, first, recent;
};

struct Shared {
    unsigned hist[2][256];          // of this CTA, read by the cluster
    unsigned part[kWarps / 4][256];
    int pages[kPages];
    unsigned bits[kWords];          // of the window: 1 = kept (written by the cluster)
    int before[kWords + 1];         // kept slots of the window before each word
    int warp_sum[kWarps];
    int found[3];                   // digit, still to take, its count
};
constexpr int kSharedBytes = (static_cast<int>(sizeof(Shared)) + 127) / 128 * 128;
// behind it: the weights' ordered forms, and later, in their place, the rows of kDepth rounds and
// their lists (one more: it is made while the round before is still read): a kept row's first elements
// before and after, -1 where its page is not in the cache, and its weight
constexpr int kLists = kDepth + 1;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// An address of this CTA's shared memory as CTA `rank` of the cluster has it.
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ unsigned ld_cluster(uint32_t addr) {
    unsigned v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, int v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Larger for a larger weight; equal for -0 and 0; NaN counts as -infinity.
__device__ __forceinline__ uint32_t ordered(float w) {
    const uint32_t u = __float_as_uint(w != w ? -INFINITY : w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kThreads, 2) fa_evict_kernel(const Params p) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Shared &sh = *reinterpret_cast<Shared *>(smem_raw);
    uint32_t *const keys = reinterpret_cast<uint32_t *>(smem_raw + kSharedBytes);
    const uint32_t bufs = smem_u32(smem_raw) + kSharedBytes;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = static_cast<int>(cluster_rank()), ctas = static_cast<int>(cluster_size());
    const int unit = blockIdx.x / ctas, b = unit / p.H_kv, h = unit - b * p.H_kv;
    after_previous();
    let_next_start();
    const int n = min(max(p.seq_k[b], 0), p.max_keys);
    if (h == 0 && rank == 0 && tid == 0) p.seq_out[b] = min(n, p.budget);
    if (n <= p.budget) return;

    const int *table = p.table + static_cast<size_t>(b) * p.max_pages;
    const int page_mask = (1 << p.page_log2) - 1;
    // page of slot j, or -1 when its number lies outside the cache
    for (int i = tid; i < kPages && i <= (n - 1) >> p.page_log2; i += kThreads) sh.pages[i] = table[i];
    __syncthreads();
    auto page_of = [&](int j) {
        const int i = j >> p.page_log2, x = i < kPages ? sh.pages[i] : table[i];
        return x >= 0 && x < p.num_pages ? x : -1;
    };
    auto weight_at = [&](int page, int j) {
        return ((static_cast<long long>(page) * p.H_kv + h) << p.page_log2) + (j & page_mask);
    };
    auto weight_of = [&](int j) {
        const int page = page_of(j);
        return page < 0 ? 0.f : p.weights[weight_at(page, j)];
    };
    // this CTA's part of the slots, from `begin` on: whole words of bits
    const int part_slots = ((n + ctas - 1) / ctas + 31) & ~31, begin = rank * part_slots;
    const int own = max(0, min(part_slots, n - begin));

    // ---- select `want` of the slots between the first and the recent ones
    const int mid0 = p.first, mid1 = n - p.recent;
    int want = p.budget - p.first - p.recent;
    uint32_t T = 0xffffffffu;  // kept: above T, or equal and at J or before
    int J = -1;
    // ordered weights of this CTA's slots between (0, which no weight gives: not between), several
    // loads of a thread at a time
    constexpr int kBatch = 8;
    const int cached = min((own + 3) & ~3, p.keys);
    auto key_of = [&](int j) { return j >= mid0 && j < mid1 ? ordered(weight_of(j)) : 0u; };
    for (int x0 = 0; x0 < cached; x0 += kBatch * kThreads) {
        uint32_t m[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int x = x0 + i * kThreads + tid;
            m[i] = x < min(own, cached) ? key_of(begin + x) : 0u;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (x0 + i * kThreads + tid < cached) keys[x0 + i * kThreads + tid] = m[i];
    }
    if (want > 0) {
        T = 0;
        J = 0x7fffffff;
        int top = 24;  // of the index
        while (top > 0 && (n - 1) >> top == 0) top -= 8;
        // passes 0 .. 3: digits of the weight; from 4 on: of the index, among the weights equal to T
        int J0 = 0;
        for (int pass = 0, shift = 24; want > 0; ++pass) {
            const bool by_index = pass >= 4;
            if (pass == 4) shift = top;
            for (int i = tid; i < kWarps / 4 * 256; i += kThreads) (&sh.part[0][0])[i] = 0;
            __syncthreads();
            unsigned *const part = sh.part[warp / 4];
            if (by_index) {
                auto count = [&](uint32_t m, int j) {
                    if (m == T && (shift == 24 || j >> (shift + 8) == J0 >> (shift + 8))) atomicAdd(&part[(j >> shift) & 255], 1u);
                };
                for (int x = tid; x < cached; x += kThreads)
                    if (keys[x] == T) count(T, begin + x);
                for (int x = cached + tid; x < own; x += kThreads) count(key_of(begin + x), begin + x);
            } else {
                const int known = shift < 24 ? shift + 8 : 31;  // (nothing is known before the first digit)
                const uint32_t prefix = shift < 24 ? T >> known : 0u;
                auto count = [&](uint32_t m) {
                    if (m != 0 && (shift == 24 || m >> known == prefix)) atomicAdd(&part[(m >> shift) & 255u], 1u);
                };
#pragma unroll 2
                for (int x = tid * 4; x < cached; x += 4 * kThreads) {
                    const uint4 m = *reinterpret_cast<const uint4 *>(keys + x);
                    count(m.x), count(m.y), count(m.z), count(m.w);
                }
                for (int x = cached + tid; x < own; x += kThreads) count(key_of(begin + x));
            }
            __syncthreads();
            if (tid < 256) {
                unsigned c = 0;
                for (int i = 0; i < kWarps / 4; ++i) c += sh.part[i][tid];
                sh.hist[pass & 1][tid] = c;
            }
            if (ctas > 1)
                cluster_sync();
            else
                __syncthreads();
            // digit 255 - tid of a weight (the largest first), tid of an index
            const int digit = by_index ? tid : 255 - tid;
            unsigned c = 0;
            if (tid < 256)
                for (int r = 0; r < ctas; ++r) c += ld_cluster(at_rank(smem_u32(&sh.hist[pass & 1][digit]), r));
            unsigned incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            if (lane == 31) sh.warp_sum[warp] = static_cast<int>(incl);
            __syncthreads();
            for (int i = 0; i < warp && i < 8; ++i) incl += sh.warp_sum[i];
            if (tid < 256 && incl - c < static_cast<unsigned>(want) && static_cast<unsigned>(want) <= incl) {
                sh.found[0] = digit;
                sh.found[1] = want - static_cast<int>(incl - c);
                sh.found[2] = static_cast<int>(c);
            }
            __syncthreads();
            want = sh.found[1];
            const bool exact = sh.found[2] == want;  // everything with these digits is kept
            if (by_index) {
                J0 |= sh.found[0] << shift;
                if (exact || shift == 0) {
                    J = J0 | ((1 << shift) - 1);
                    break;
                }
            } else {
                T |= static_cast<uint32_t>(sh.found[0]) << shift;
                if (exact) break;  // all of them, at any index
            }
            shift -= 8;
        }
    } else if (ctas > 1) {
        cluster_sync();  // all have started: their shared memory is written below
    }

    // ---- move. A thread copies the same 16-byte piece of every kThreads / 2^piece_log2-th row.
    const int log2 = p.piece_log2, S = p.rows;
    const int piece = (rank << log2) + (tid & ((1 << log2) - 1)), per_row = p.d / 8;  // of a key
    uint16_t *const mine = (piece < per_row ? p.k + piece * 8 : p.v + (piece - per_row) * 8) + h * p.head_stride;
    const int row0 = tid >> log2, row_step = kThreads >> log2;
    const uint32_t buf_bytes = static_cast<uint32_t>(S) << (log2 + 4);
    longlong2 *const list_at = reinterpret_cast<longlong2 *>(smem_raw + kSharedBytes + kDepth * buf_bytes);
    float *const list_w = reinterpret_cast<float *>(list_at + kLists * S);
    auto element = [&](int page, int j) { return page * p.page_stride + (j & page_mask) * p.token_stride; };
    int done = 0;  // kept rows of earlier windows
    for (int window = 0; window < n; window += kWindow) {
        const int end = min(n, window + kWindow), words = (end - window + 31) / 32;
        // ---- its bits: of the first window each CTA's part, whose weights may be in shared memory;
        // of others (whose weights nothing has been written over) a warp's words in turn
        const int w_first = window == 0 ? begin / 32 + warp : rank * kWarps + warp;
        const int w_end = window == 0 ? min((begin + own + 31) / 32, words) : words;
        const int w_step = window == 0 ? kWarps : kWarps * ctas;
        for (int i = w_first; i < w_end; i += w_step) {
            const int j = window + i * 32 + lane;
            bool kept = false;
            if (j < end) {
                kept = j < mid0 || j >= mid1;
                if (!kept) {
                    const uint32_t m = window == 0 && j - begin < cached ? keys[j - begin] : ordered(weight_of(j));
                    kept = m > T || (m == T && j <= J);
                }
            }
            const unsigned word = __ballot_sync(0xffffffffu, kept);
            if (lane < ctas) st_cluster(at_rank(smem_u32(&sh.bits[i]), lane), static_cast<int>(word));
        }
        if (ctas > 1)
            cluster_sync();
        else
            __syncthreads();
        // ---- kept slots before each word
        constexpr int kOwn = kWords / kThreads;
        int c[kOwn], sum = 0;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            c[i] = sum;
            sum += tid * kOwn + i < words ? __popc(sh.bits[tid * kOwn + i]) : 0;
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) sh.warp_sum[warp] = incl;
        __syncthreads();
        for (int i = 0; i < warp; ++i) incl += sh.warp_sum[i];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) sh.before[tid * kOwn + i] = incl - sum + c[i];
        if (tid == kThreads - 1) sh.before[kWords] = incl;
        __syncthreads();

        const int rows = sh.before[kWords], rounds = (rows + S - 1) / S;
        float w_next = 0.f;  // the weight of this thread's row of the round listed last
        int w_at = -1;
        // the places of round t's rows before and after
        auto list = [&](int t) {
            if (w_at >= 0) list_w[w_at] = w_next;
            w_at = -1;
            const int row = t * S + tid;
            if (tid >= S || row >= rows) return;
            // the last word with no more than `row` kept slots before it, and its bit of that rank
            int word = 0;
#pragma unroll
            for (int step = kWords / 2; step > 0; step >>= 1)
                if (sh.before[word + step] <= row) word += step;
            int rank_in = row - sh.before[word], bit = 0;
            const unsigned bits = sh.bits[word];
#pragma unroll
            for (int step = 16; step > 0; step >>= 1) {
                const int below = __popc((bits >> bit) & ((1u << step) - 1));
                if (rank_in >= below) bit += step, rank_in -= below;
            }
            const int at = t % kLists * S + tid, from = window + word * 32 + bit, to = done + row;
            const int page = page_of(from), page_to = page_of(to);
            list_at[at] = make_longlong2(page < 0 ? -1 : element(page, from), page_to < 0 ? -1 : element(page_to, to));
            if (rank == 0) {
                w_at = at;
                w_next = page < 0 ? 0.f : p.weights[weight_at(page, from)];
            }
        };
        auto load = [&](int t) {
            const int count = min(S, rows - t * S);
            const longlong2 *list = list_at + t % kLists * S;
            uint32_t to = bufs + t % kDepth * buf_bytes + tid * 16;
#pragma unroll 4
            for (int row = row0; row < count; row += row_step, to += kThreads * 16) {
                const long long from = list[row].x;
                copy16_or_zero(to, mine + max(from, 0ll), from >= 0);
            }
            copies_commit();
        };
#pragma unroll
        for (int t = 0; t + 1 < kDepth; ++t) {
            list(t);
            __syncthreads();
            if (t < rounds)
                load(t);
            else
                copies_commit();
        }
        for (int t = 0; t < rounds; ++t) {
            const int ahead = t + kDepth - 1;
            copies_wait<kDepth - 2>();  // round t is there
            list(ahead);
            __syncthreads();  // for all threads; and the round before has left its buffer
            if (ahead < rounds)
                load(ahead);
            else
                copies_commit();
            const int dest = t * S, count = min(S, rows - dest);
            const longlong2 *at = list_at + t % kLists * S;
            const uint8_t *staged = smem_raw + kSharedBytes + t % kDepth * buf_bytes + tid * 16;
#pragma unroll 4
            for (int row = row0; row < count; row += row_step, staged += kThreads * 16) {
                const long long to = at[row].y;
                if (to >= 0) *reinterpret_cast<uint4 *>(mine + to) = *reinterpret_cast<const uint4 *>(staged);
            }
            if (rank == 0 && tid < count) {
                const int j = done + dest + tid, page = page_of(j);
                if (page >= 0) p.weights[weight_at(page, j)] = list_w[t % kLists * S + tid];
            }
        }
        done += rows;
        // the bits are read no more (nor does anybody leave while they may be written)
        if (ctas > 1 && end < n)
            cluster_sync();
        else
            __syncthreads();
    }
}

}  // namespace evict
}  // namespace fa
