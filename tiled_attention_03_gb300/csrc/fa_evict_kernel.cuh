// fa_evict_kernel.cuh -- eviction from a paged K/V cache: for each sequence that is longer than
// the budget and each K/V head, the keys to keep (the first ones, the recent ones, and of
// those between the ones of the largest weight) move together, in their order, to the front of the
// sequence's pages, with their values and weights.
//
// A cluster of 1 .. 8 CTAs takes a sequence and head. It first selects: weights as ordered 32-bit
// numbers, histograms of 8 bits at a time summed over the cluster through distributed
// shared memory, from the top digit down until the kept ones are exactly told apart; where equal
// weights remain, 8 bits of the index at a time, lowest first. What is kept is then a
// comparison with two numbers, which every thread can make for its own slot.
//
// Then it moves, in place. Slot j's row goes to a slot <= j, so rounds of consecutive slots are
// taken in order, and a row may be written once the round it was read in, and so all before, has
// been read by the whole cluster: one cluster barrier per round, which also carries the CTAs' counts.
// The next round's rows are loaded (asynchronous copies to shared memory) before the
// barrier: they lie behind everything that this round writes.
//
// Bound by memory: rows are read and written once, weights read once. Weights and page numbers
// stay in shared memory as far as they fit, so that nothing but the rows is waited for between
// rounds, and rounds are as large as what is left allows.
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
constexpr int kBufBytes = 64 * 1024;  // rows of a round (two rounds are in flight)
constexpr int kKept = 16384;          // weights of this CTA that stay in shared memory
constexpr int kPages = 2048;          // page numbers that do

struct Params {
    uint16_t *k, *v;
    float *weights;  // page x H_kv x page_size
    long long page_stride, token_stride, head_stride;
    const int *seq_k, *table;
    int *seq_out;
    int H_kv, d, slots;  // slots: of a CTA in a round
    int max_pages, page_log2, num_pages, max_keys;
    int budget, first, recent;
};

struct Shared {
    float w_all[kKept];
    int pages[kPages];
    unsigned hist[2][256];          // of this CTA, read by the cluster
    unsigned part[kWarps / 4][256];
    int counts[2][kMaxCluster];     // kept rows of each CTA in a round, written by each
    int warp_sum[kWarps];
    int found[3];                   // digit, still to take, its count
    long long src[2][kThreads];     // kept rows of a round: first element, -1: not in the cache
    long long dst[kThreads];
    float w[2][kThreads];
};
constexpr int kSharedBytes = (static_cast<int>(sizeof(Shared)) + 127) / 128 * 128 + 2 * kBufBytes;

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

__global__ void __launch_bounds__(kThreads, 1) fa_evict_kernel(const Params p) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Shared &sh = *reinterpret_cast<Shared *>(smem_raw);
    uint8_t *const bufs = smem_raw + kSharedBytes - 2 * kBufBytes;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = static_cast<int>(cluster_rank()), ctas = static_cast<int>(cluster_size());
    const int unit = blockIdx.x / ctas, b = unit / p.H_kv, h = unit - b * p.H_kv;
    after_previous();
    let_next_start();
    const int n = min(max(p.seq_k[b], 0), p.max_keys);
    if (h == 0 && rank == 0 && tid == 0) p.seq_out[b] = min(n, p.budget);
    if (n <= p.budget) return;

    const int S = p.slots, round = S * ctas, rounds = (n + round - 1) / round;
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
    // this CTA's x-th slot
    auto slot = [&](int x) { return x / S * round + rank * S + x % S; };
    const int own = rounds * S;

    // ---- select `want` of the slots between the first and the recent ones
    const int mid0 = p.first, mid1 = n - p.recent;
    int want = p.budget - p.first - p.recent;
    uint32_t T = 0xffffffffu;  // kept: above T, or equal and at J or before
    int J = -1;
    // weights of this CTA's slots, several loads of a thread at a time
    constexpr int kBatch = 8;
    for (int x0 = 0; x0 < own && x0 < kKept; x0 += kBatch * kThreads) {
        float w[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int x = x0 + i * kThreads + tid, j = slot(x);
            w[i] = x < own && x < kKept && j < n ? weight_of(j) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (x0 + i * kThreads + tid < kKept) sh.w_all[x0 + i * kThreads + tid] = w[i];
    }
    __syncthreads();
    auto own_weight = [&](int x, int j) { return x < kKept ? sh.w_all[x] : weight_of(j); };
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
            for (int x = tid; x < own; x += kThreads) {
                const int j = slot(x);
                if (j < mid0 || j >= mid1) continue;
                const uint32_t m = ordered(own_weight(x, j));
                const uint32_t v = by_index ? static_cast<uint32_t>(j) : m;
                const uint32_t known = by_index ? static_cast<uint32_t>(J0) : T;
                if ((by_index && m != T) || (shift < 24 && v >> (shift + 8) != known >> (shift + 8))) continue;
                atomicAdd(&sh.part[warp / 4][(v >> shift) & 255u], 1u);
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
    }

    // ---- move
    const int row_bytes = p.d * 2, pieces = row_bytes / 16;  // of a key, and of a value
    // Finds the kept ones of round t's slots and starts their copies. Returns their number.
    auto load = [&](int t) -> int {
        const int x = t * S + tid, j = t * round + rank * S + tid, buf = t & 1;
        bool kept = false;
        float w = 0.f;
        int page = -1;
        if (tid < S && j < n) {
            page = page_of(j);
            w = own_weight(x, j);
            kept = j < mid0 || j >= mid1;
            if (!kept) {
                const uint32_t m = ordered(w);
                kept = m > T || (m == T && j <= J);
            }
        }
        const unsigned mask = __ballot_sync(0xffffffffu, kept);
        if (lane == 0) sh.warp_sum[warp] = __popc(mask);
        __syncthreads();
        int at = __popc(mask & ((1u << lane) - 1)), count = 0;
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) at += sh.warp_sum[i];
            count += sh.warp_sum[i];
        }
        if (kept) {
            sh.src[buf][at] = page < 0 ? -1 : page * p.page_stride + (j & page_mask) * p.token_stride + h * p.head_stride;
            sh.w[buf][at] = w;
        }
        if (tid < ctas) st_cluster(at_rank(smem_u32(&sh.counts[buf][rank]), tid), count);
        __syncthreads();
        const uint32_t base = smem_u32(bufs) + buf * kBufBytes;
        for (int c = tid; c < count * pieces * 2; c += kThreads) {
            const int row = c / (2 * pieces), y = c - row * 2 * pieces;
            const long long src = sh.src[buf][row];
            const uint16_t *from = (y < pieces ? p.k : p.v) + (src < 0 ? 0 : src) + (y < pieces ? y : y - pieces) * 8;
            copy16_or_zero(base + c * 16, from, src >= 0);
        }
        copies_commit();
        return count;
    };
    int before = 0;  // kept rows of earlier rounds
    int count = load(0);
    for (int t = 0; t < rounds; ++t) {
        int next = 0;
        if (t + 1 < rounds) {
            next = load(t + 1);
            copies_wait<1>();
        } else {
            copies_wait<0>();
        }
        // this round has been read by all
        if (ctas > 1)
            cluster_sync();
        else
            __syncthreads();
        int dest = before;
        for (int r = 0; r < ctas; ++r) {
            const int c = sh.counts[t & 1][r];
            if (r < rank) dest += c;
            before += c;
        }
        if (tid < count) {
            const int j = dest + tid, page = page_of(j);
            sh.dst[tid] = page < 0 ? -1 : page * p.page_stride + (j & page_mask) * p.token_stride + h * p.head_stride;
            if (page >= 0) p.weights[weight_at(page, j)] = sh.w[t & 1][tid];
        }
        __syncthreads();
        const uint4 *rows = reinterpret_cast<const uint4 *>(bufs + (t & 1) * kBufBytes);
        for (int c = tid; c < count * pieces * 2; c += kThreads) {
            const int row = c / (2 * pieces), y = c - row * 2 * pieces;
            const long long dst = sh.dst[row];
            if (dst >= 0)
                *reinterpret_cast<uint4 *>((y < pieces ? p.k : p.v) + dst + (y < pieces ? y : y - pieces) * 8) = rows[c];
        }
        __syncthreads();
        count = next;
    }
    if (ctas > 1) cluster_sync();  // nobody leaves while its shared memory may be read or written
}

}  // namespace evict
}  // namespace fa
