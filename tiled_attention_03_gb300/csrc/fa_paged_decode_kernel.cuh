// fa_paged_decode_kernel.cuh -- attention of few new tokens per sequence over a paged
// K/V cache (decode steps): at most 16 rows (query heads of one K/V head x tokens) a unit.
//
// Such a unit reads every key once for a handful of products, so memory bounds it, and
// at short or ragged lengths latency does. The 128-row tile of fa_paged_kernel.cuh fills
// 1 / 8 of its rows at best and runs its units one after the other per SM; here a warp is
// the worker: it streams its own keys through a ring of asynchronous 16-byte copies in
// shared memory, multiplies with mma.sync (m16n8k16, fp32 accumulators in registers, the
// rows' 16 x d outputs among them) and keeps its own online softmax. No barrier is shared,
// and the latencies of one warp's unit hide behind the other warps' streams.
//
// The work is cut as in fa_paged_kernel.cuh, with warps in place of CTAs: all units with all
// their K/V tiles of kKeys keys form one line, a unit taking kUnitTicks more than its
// tiles (its start and end cost that much), and worker w takes ticks w T .. w T + T - 1. A unit
// that several workers share is joined by fa_paged_merge_kernel.
//
// Which of the two a batch is for depends on its longest sequence, which only the device
// knows: many rows of one sequence in units of 16 read its keys again and again. A batch of
// no more than max_new tokens goes to the decode kernel. With a few per sequence on average (or
// one, or less: most sequences of a batch of fixed size may have none) one kernel holds both
// bodies and takes the chunks' if a sequence has more than max_new new tokens. 256 tokens of one of
// 256 sequences, on 30000 keys, take 120 us so, and 718 in units of 16 rows; 64 sequences of 100
// keys with a token each 13.6 us, 13.2 with the decode kernel alone, and 15.1 with two
// launches, one of which returns at once.
//
// Measured with the merge, in a graph: 8 x 32768 keys, 32 / 8 heads, d 128: 162 us (6.6 TB/s);
// 128 ragged sequences, window 4096, 16 / 4 heads, d 64: 34 us (4.6 TB/s; the tcgen05 tile
// took 84 us); 4 sequences of 60-1000 keys, d 128: 12.2 us.
//
// Keys that no row of the unit sees are not read: their rows are filled with zeros in
// shared memory, whatever the pages hold.
#pragma once

#include "fa_copy.cuh"
#include "fa_paged_kernel.cuh"

namespace fa {
namespace paged {

constexpr int kSmallRows = 16;  // rows of a unit at most

template <int D>
struct Small {
    static constexpr int kKeys = D <= 64 ? 32 : 16;  // keys per tile
    static constexpr int kWarps = D == 256 ? 4 : 8;
    static constexpr int kStages = 3;
    static constexpr int kRowBytes = D * 2;
    static constexpr int kTileBytes = kKeys * kRowBytes;
    static constexpr int kChunks = D / 8;            // 16-byte chunks per row
    static constexpr int kCopyRows = 32 / kChunks;   // rows per copy instruction of a warp
    static constexpr int kRing = kWarps * kStages * 2 * kTileBytes;
    // Q as A operands stays in registers, except at d = 256, where it would take 64 next
    // to the outputs' 128: there each warp keeps its rows in shared memory
    static constexpr bool kQShared = D == 256;
    static constexpr int kQBytes = kQShared ? kSmallRows * kRowBytes : 0;
    static constexpr int kScan = kRing + kWarps * kQBytes;  // 256 prefixes, 256 works, warp sums
    static constexpr int kBytes = kScan + 2 * 256 * 4 + 64;
    static_assert(kBytes <= 227 * 1024, "shared memory");
};
// A unit's start and end (its rows in, its outputs out, the drained ring between) in tiles. 128 ragged
// sequences at d 64: 34.2 us, 35.6 with 2 and 34.4 with 8; 8 x 32768 keys 161.0, 162.0 and 164.5.
constexpr int kUnitTicks = 4;

// 16-byte chunk c of row r of a tile sits at chunk c ^ swizzle(r): the 8 rows that one
// ldmatrix reads fall into different banks.
template <int D>
__device__ __forceinline__ uint32_t tile_at(int row, int chunk) {
    const int x = D == 32 ? (row >> 1) & 3 : row & 7;
    return static_cast<uint32_t>(row * Small<D>::kRowBytes + ((chunk ^ x) << 4));
}

__device__ __forceinline__ void ldmatrix4(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t at, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

struct SmallParams {
    const uint16_t *Q;
    void *O;
    float *LSE;
    float *part_O;    // [2 * workers][16][D]
    float *part_LSE;  // [2 * workers][16]
    MergeInfo *info;  // [workers]
    const uint16_t *k, *v;
    long long page_stride, token_stride, head_stride;
    const int *cu_q, *seq_k, *table;
    int B, H, kv_group, pf, spaces, tpt;
    int total_q, max_pages, page_log2, num_pages, max_keys;
    int wl, wr;
    float scale_log2;
    int min_ticks;
};

// K/V tiles of a unit (token tile qb of a sequence), from tile j0 on, and its keys lo .. hi.
template <int kKeys>
__device__ __forceinline__ int small_unit(const Seq &s, int qb, const SmallParams &p, int &lo, int &hi,
                                          int &j0) {
    const int t0 = qb * p.tpt, tl = min(t0 + p.tpt, s.nq) - 1;
    const int q_off = s.nk - s.nq;
    lo = max(0, t0 + q_off - p.wl);
    hi = min(s.nk - 1, tl + q_off + p.wr);
    j0 = lo / kKeys;
    return hi < lo ? 0 : hi / kKeys - j0 + 1;  // tiles
}
__device__ __forceinline__ Seq small_seq(int b, const SmallParams &p) {
    Seq s;
    s.q0 = min(max(p.cu_q[b], 0), p.total_q);
    s.nq = min(max(p.cu_q[b + 1], s.q0), p.total_q) - s.q0;
    s.nk = min(max(p.seq_k[b], 0), p.max_keys);
    return s;
}
// Units of a sequence per head group (mostly one: the division is worth avoiding).
__device__ __forceinline__ int small_units(const Seq &s, const SmallParams &p) {
    return s.nq <= p.tpt ? min(s.nq, 1) : (s.nq + p.tpt - 1) / p.tpt;
}
// Ticks of one head group of a sequence: its units' tiles and kUnitTicks each.
template <int kKeys>
__device__ __forceinline__ unsigned small_work(const Seq &s, const SmallParams &p) {
    const int nqb = small_units(s, p);
    unsigned w = 0;
    for (int qb = 0; qb < nqb; ++qb) {
        int lo, hi, j0;
        w += small_unit<kKeys>(s, qb, p, lo, hi, j0) + kUnitTicks;
    }
    return w;
}

// A CTA of the decode kernel: the shares of its first kWarps warps. EITHER: false, with nothing
// done, if a sequence has more than max_new new tokens (for every warp of the block alike).
template <int D, bool BF16, bool EITHER>
__device__ __forceinline__ bool decode_cta(const SmallParams &p, uint8_t *small_smem, int max_new) {
    using L = Small<D>;
    constexpr int kKeys = L::kKeys, kWarps = L::kWarps, kThr = kWarps * 32;
    unsigned *pre = reinterpret_cast<unsigned *>(small_smem + L::kScan);
    unsigned *wrk = pre + 256;
    unsigned *sums = wrk + 256;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = smem_u32(small_smem) + warp * L::kStages * 2 * L::kTileBytes;
    // neighbouring shares on different SMs: few shares still use all of them
    const unsigned worker = warp * gridDim.x + blockIdx.x;
    const unsigned workers = kWarps * gridDim.x;

    // ---- this warp's share: ticks w0 .. w1 - 1 of W, and the sequence b that holds w0, `off`
    // ticks into it. Up to 128 sequences every warp finds its own, one to four to a lane,
    // without a barrier; more are summed and searched by the block.
    unsigned W, T, w0, w1, off = 0, per = 0;  // per: ticks of one head group of sequence b
    int b = -1;
    Seq s{0, 0, 0};
    constexpr int kOwn = 4;
    if (p.B <= 32 * kOwn) {
        const int own = (p.B + 31) >> 5;
        Seq q[kOwn];
        unsigned w[kOwn], sum = 0;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            q[i] = Seq{0, 0, 0};
            if (i < own && own * lane + i < p.B) q[i] = small_seq(own * lane + i, p);
        }
        if constexpr (EITHER) {
            int longest = q[0].nq;
#pragma unroll
            for (int i = 1; i < kOwn; ++i) longest = max(longest, q[i].nq);
            if (__any_sync(0xffffffffu, longest > max_new)) return false;
            if (warp >= kWarps) return true;
        }
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            w[i] = 0;
            if (i < own) w[i] = small_work<kKeys>(q[i], p);
            sum = add_work(sum, w[i] * p.spaces);
        }
        unsigned incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl = add_work(incl, y);
        }
        W = __shfl_sync(0xffffffffu, incl, 31);
        if (W == kNoLine) W = 0;
        T = max((W + workers - 1) / workers, static_cast<unsigned>(p.min_ticks));
        w0 = min(worker * T, W);
        w1 = min(w0 + T, W);
        unsigned lo = incl - sum;
        const unsigned hit = __ballot_sync(0xffffffffu, lo <= w0 && w0 < incl);
        if (w0 < w1) {
            // in the lane that holds w0: which of its sequences
            int at = 0;
            Seq mine = q[0];
            per = w[0];
#pragma unroll
            for (int i = 0; i < kOwn - 1; ++i)
                if (at == i && i + 1 < own && w0 >= lo + w[i] * p.spaces) {
                    lo += w[i] * p.spaces;
                    at = i + 1;
                    mine = q[i + 1];
                    per = w[i + 1];
                }
            const int src = __ffs(hit) - 1;
            b = own * src + __shfl_sync(0xffffffffu, at, src);
            off = w0 - __shfl_sync(0xffffffffu, lo, src);
            per = __shfl_sync(0xffffffffu, per, src);
            s.q0 = __shfl_sync(0xffffffffu, mine.q0, src);
            s.nq = __shfl_sync(0xffffffffu, mine.nq, src);
            s.nk = __shfl_sync(0xffffffffu, mine.nk, src);
        }
    } else {
        unsigned mine = 0, first = 0, carry = 0;
        bool longer = false;
        for (int x = threadIdx.x; x < p.B && (!EITHER || warp < kWarps); x += kThr) {
            const Seq q = small_seq(x, p);
            if (EITHER && q.nq > max_new) {
                longer = true;
                break;
            }
            const unsigned w = small_work<kKeys>(q, p) * p.spaces;
            if (x < kThr) first = w;
            mine = add_work(mine, w);
        }
        __syncwarp();
        mine = warp_sum_work(mine);
        if (lane == 0 && warp < kWarps) sums[warp] = mine;
        if constexpr (EITHER) {
            if (__syncthreads_or(longer)) return false;
            if (warp >= kWarps) return true;
        } else {
            __syncthreads();
        }
        W = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) W = add_work(W, sums[i]);
        if (W == kNoLine) W = 0;
        T = max((W + workers - 1) / workers, static_cast<unsigned>(p.min_ticks));
        w0 = min(worker * T, W);
        w1 = min(w0 + T, W);
        for (int b0 = 0; b0 < p.B; b0 += kThr) {
            const int x = b0 + static_cast<int>(threadIdx.x);
            const unsigned w = b0 == 0 ? first : x < p.B ? small_work<kKeys>(small_seq(x, p), p) * p.spaces : 0;
            unsigned incl = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            __syncthreads();
            if (lane == 31) sums[warp] = incl;
            __syncthreads();
            unsigned before = carry;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                if (i < warp) before += sums[i];
                carry += sums[i];
            }
            pre[threadIdx.x] = before + incl - w;
            wrk[threadIdx.x] = w;
            __syncthreads();
            if (b < 0 && w0 < w1) {
#pragma unroll
                for (int i = 0; i < kWarps; ++i) {
                    const unsigned lo = pre[32 * i + lane];
                    const unsigned hit = __ballot_sync(0xffffffffu, lo <= w0 && w0 < lo + wrk[32 * i + lane]);
                    if (hit != 0) {
                        const int at = 32 * i + __ffs(hit) - 1;
                        b = b0 + at;
                        off = w0 - pre[at];
                    }
                }
            }
            // the block's largest share start is its last warp's
            if (((kWarps - 1) * gridDim.x + blockIdx.x) * static_cast<unsigned long long>(T) < carry) break;
        }
        if (b >= 0) {
            s = small_seq(b, p);
            per = small_work<kKeys>(s, p);
        }
    }
    MergeInfo info{};
    info.last_cta = -1;
    if (b < 0) {
        if (lane == 0) p.info[worker] = info;
        return true;
    }

    int nqb = small_units(s, p), qb = 0, sp;
    int skip;  // ticks of the current unit before this share
    {
        sp = static_cast<int>(off / per);
        skip = static_cast<int>(off - sp * per);
        for (; qb < nqb - 1; ++qb) {
            int lo, hi, j0;
            const int n = small_unit<kKeys>(s, qb, p, lo, hi, j0) + kUnitTicks;
            if (skip < n) break;
            skip -= n;
        }
    }
    const float sl2 = p.scale_log2;
    const int r0 = lane >> 2, c0 = (lane & 3) * 2;  // this lane's rows r0, r0 + 8; first column
    const long long copy_off =
        static_cast<long long>(lane / L::kChunks) * p.token_stride + (lane % L::kChunks) * 8;
    const long long copy_step = L::kCopyRows * p.token_stride;
    int pieces = 0;
    for (unsigned w = w0; w < w1;) {
        int lo, hi, j0;
        const int n = small_unit<kKeys>(s, qb, p, lo, hi, j0);
        const int len = min(n + kUnitTicks - skip, static_cast<int>(w1 - w));
        const int ja = max(skip - kUnitTicks, 0), je = skip + len - kUnitTicks;  // tiles ja .. je - 1
        const int t0 = qb * p.tpt;
        const int rows = (min(t0 + p.tpt, s.nq) - t0) * p.pf;
        const int tok0 = s.q0 + t0, head0 = sp * p.pf;
        auto out_row = [&](int r) {
            const int i = r / p.pf;
            return (static_cast<size_t>(tok0) + i) * p.H + head0 + (r - i * p.pf);
        };
        if (n == 0) {
            if (skip == 0) {  // no row sees a key
                for (int r = 0; r < rows; ++r) {
                    uint32_t *o = reinterpret_cast<uint32_t *>(p.O) + out_row(r) * (D / 2);
                    for (int c = lane; c < D / 2; c += 32) o[c] = 0;
                    if (lane == 0) p.LSE[out_row(r)] = -INFINITY;
                }
            }
        } else if (je > ja) {
            const int q_off = s.nk - s.nq;
            const bool both = rows > 8;
            const long long head_off = static_cast<long long>(head0 / p.kv_group) * p.head_stride + copy_off;
            const int *table = p.table + static_cast<size_t>(b) * p.max_pages;
            int page_base = -64, pages = 0;  // this lane's page number: of page page_base + lane
            auto issue = [&](int j, int slot) {
                if (j < je) {
                    const int kv0 = (j0 + j) * kKeys;
                    const uint32_t dk = ring + slot * 2 * L::kTileBytes, dv = dk + L::kTileBytes;
#pragma unroll
                    for (int g = 0; g < kKeys / 8; ++g) {
                        const int key0 = kv0 + 8 * g;
                        const int pi = key0 >> p.page_log2;
                        if (pi < page_base || pi >= page_base + 32) {
                            page_base = pi;
                            pages = pi + lane <= (hi >> p.page_log2) ? table[pi + lane] : -1;
                        }
                        const int page = __shfl_sync(0xffffffffu, pages, pi - page_base);
                        const bool known = page >= 0 && page < p.num_pages;
                        const long long at = (known ? page : 0) * p.page_stride +
                                             (key0 & ((1 << p.page_log2) - 1)) * p.token_stride + head_off;
                        const uint16_t *pk = p.k + at, *pv = p.v + at;
                        const bool all = known && key0 >= lo && key0 + 7 <= hi;
#pragma unroll
                        for (int i = 0; i < 8 / L::kCopyRows; ++i) {
                            const int row = i * L::kCopyRows + lane / L::kChunks;
                            const uint32_t d = tile_at<D>(8 * g + row, lane % L::kChunks);
                            if (all) {
                                copy16(dk + d, pk);
                                copy16(dv + d, pv);
                            } else {
                                const int key = key0 + row;
                                const bool there = known && key >= lo && key <= hi;
                                copy16_or_zero(dk + d, there ? pk : p.k, there);
                                copy16_or_zero(dv + d, there ? pv : p.v, there);
                            }
                            pk += copy_step;
                            pv += copy_step;
                        }
                    }
                }
                copies_commit();
            };
            __syncwarp();  // every lane is done with the ring of the piece before
            const uint32_t q_tile = smem_u32(small_smem) + L::kRing + warp * L::kQBytes;
            if constexpr (L::kQShared) {
#pragma unroll
                for (int i = 0; i < kSmallRows / L::kCopyRows; ++i) {
                    const int r = i * L::kCopyRows + lane / L::kChunks;
                    copy16_or_zero(q_tile + tile_at<D>(r, lane % L::kChunks),
                                   p.Q + out_row(r < rows ? r : 0) * D + (lane % L::kChunks) * 8, r < rows);
                }
            }
            // Q as the A operand of every k-step: rows r0 and r0 + 8, columns c0 and c0 + 8 (on
            // its way while the first copies look up their pages)
            uint32_t qa[L::kQShared ? 1 : D / 16][4];
            if constexpr (!L::kQShared) {
                const uint32_t *q0 =
                    reinterpret_cast<const uint32_t *>(p.Q + out_row(r0 < rows ? r0 : 0) * D + c0);
                const uint32_t *q1 =
                    reinterpret_cast<const uint32_t *>(p.Q + out_row(r0 + 8 < rows ? r0 + 8 : 0) * D + c0);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    qa[k][0] = r0 < rows ? q0[8 * k] : 0;
                    qa[k][1] = r0 + 8 < rows ? q1[8 * k] : 0;
                    qa[k][2] = r0 < rows ? q0[8 * k + 4] : 0;
                    qa[k][3] = r0 + 8 < rows ? q1[8 * k + 4] : 0;
                }
            }
#pragma unroll
            for (int i = 0; i < L::kStages - 1; ++i) issue(ja + i, i);
            float o[D / 8][4];
#pragma unroll
            for (int c = 0; c < D / 8; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
            float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
            const int i0 = t0 + r0 / p.pf + q_off, i1 = t0 + (r0 + 8) / p.pf + q_off;
            const int lo0 = i0 - p.wl, hi0 = min(s.nk - 1, i0 + p.wr);
            const int lo1 = i1 - p.wl, hi1 = min(s.nk - 1, i1 + p.wr);
            // a tile with keys in [lo_last, hi_first] only is visible to every row
            const int lo_last = t0 + (rows - 1) / p.pf + q_off - p.wl;
            const int hi_first = min(s.nk - 1, t0 + q_off + p.wr);
            for (int j = ja, slot = 0; j < je; ++j) {
                copies_wait<L::kStages - 2>();
                __syncwarp();
                issue(j + L::kStages - 1, slot == 0 ? L::kStages - 1 : slot - 1);
                const uint32_t sk = ring + slot * 2 * L::kTileBytes, sv = sk + L::kTileBytes;
                slot = slot + 1 == L::kStages ? 0 : slot + 1;
                const int kv0 = (j0 + j) * kKeys;
                // scores in two chains of products, of the even and of the odd steps: one chain
                // of d / 16 dependent products is most of a lone warp's time
                float x[kKeys / 8][4], y[kKeys / 8][4];
#pragma unroll
                for (int c = 0; c < kKeys / 8; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[c][e] = y[c][e] = 0.f;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t(&a)[4] = qa[L::kQShared ? 0 : k];
                    if constexpr (L::kQShared) ldmatrix4(q_tile + tile_at<D>(lane & 15, 2 * k + (lane >> 4)), a);
#pragma unroll
                    for (int c = 0; c < kKeys / 16; ++c) {
                        uint32_t kb[4];
                        ldmatrix4(sk + tile_at<D>(16 * c + (lane & 7) + ((lane >> 4) << 3),
                                                  2 * k + ((lane >> 3) & 1)),
                                  kb);
                        mma16816<BF16>(k & 1 ? y[2 * c] : x[2 * c], a, kb[0], kb[1]);
                        mma16816<BF16>(k & 1 ? y[2 * c + 1] : x[2 * c + 1], a, kb[2], kb[3]);
                    }
                }
#pragma unroll
                for (int c = 0; c < kKeys / 8; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[c][e] += y[c][e];
                if (kv0 < lo_last || kv0 + kKeys - 1 > hi_first) {
#pragma unroll
                    for (int c = 0; c < kKeys / 8; ++c)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int key = kv0 + 8 * c + c0 + e;
                            if (key < lo0 || key > hi0) x[c][e] = -INFINITY;
                            if (key < lo1 || key > hi1) x[c][2 + e] = -INFINITY;
                        }
                }
                // rows that are not there have scores of 0 and see what they may: harmless
                float t0m = -INFINITY, t1m = -INFINITY;
#pragma unroll
                for (int c = 0; c < kKeys / 8; ++c) {
                    t0m = max3f(t0m, x[c][0], x[c][1]);
                    if (both) t1m = max3f(t1m, x[c][2], x[c][3]);
                }
                t0m = fmaxf(t0m, __shfl_xor_sync(0xffffffffu, t0m, 1));
                t0m = fmaxf(t0m, __shfl_xor_sync(0xffffffffu, t0m, 2)) * sl2;
                const float m0_old = m0, m1_old = m1;
                if (t0m > m0 + kRescaleThreshold) m0 = t0m;
                if (both) {
                    t1m = fmaxf(t1m, __shfl_xor_sync(0xffffffffu, t1m, 1));
                    t1m = fmaxf(t1m, __shfl_xor_sync(0xffffffffu, t1m, 2)) * sl2;
                    if (t1m > m1 + kRescaleThreshold) m1 = t1m;
                }
                if (__any_sync(0xffffffffu, m0 != m0_old || m1 != m1_old)) {
                    const float f0 = m0 != m0_old ? ex2_approx(m0_old - m0) : 1.f;
                    const float f1 = !both ? f0 : m1 != m1_old ? ex2_approx(m1_old - m1) : 1.f;
                    l0 *= f0;
                    l1 *= f1;
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) {
                        fmul2(o[c][0], o[c][1], f0, f0);
                        fmul2(o[c][2], o[c][3], f1, f1);
                    }
                }
                const float n0 = m0 == -INFINITY ? 0.f : -m0, n1 = m1 == -INFINITY ? 0.f : -m1;
                // P as the sum of two parts of 16 bits, the operand type of the product. With 8 rows or
                // fewer the second part takes the place of rows 8 to 15, whose outputs are added at the
                // end; with more it is multiplied by itself.
                // P goes into its product with V as hi + lo, two parts of 16 bits (the operand type):
                // hi alone put O's error at 0.0023 where its own rounding is 0.0017 (bf16, relative,
                // root mean square). Up to 8 rows, lo is rows 8 to 15 of the operand, whose outputs are
                // added at the end: the same products; with more rows lo is multiplied by itself (16
                // sequences of 3 tokens, 12 rows a unit: 17.9 -> 18.8 us). l keeps the fp32 values.
                uint32_t pa[kKeys / 16][4];
#pragma unroll
                for (int c = 0; c < kKeys / 8; ++c) {
                    ffma2(x[c][0], x[c][1], sl2, sl2, n0, n0);
                    x[c][0] = ex2_approx(x[c][0]);
                    x[c][1] = ex2_approx(x[c][1]);
                    l0 += x[c][0] + x[c][1];
                    two_parts<BF16>(x[c][0], x[c][1], pa[c / 2][(c & 1) * 2], pa[c / 2][(c & 1) * 2 + 1]);
                }
                auto product = [&](const uint32_t (&a)[kKeys / 16][4]) {
#pragma unroll
                    for (int c = 0; c < D / 16; ++c)
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k) {
                            uint32_t vb[4];
                            ldmatrix4_trans(sv + tile_at<D>(16 * k + (lane & 15), 2 * c + (lane >> 4)), vb);
                            mma16816<BF16>(o[2 * c], a[k], vb[0], vb[1]);
                            mma16816<BF16>(o[2 * c + 1], a[k], vb[2], vb[3]);
                        }
                };
                if (both) {
                    uint32_t pb[kKeys / 16][4];
#pragma unroll
                    for (int c = 0; c < kKeys / 8; ++c) {
                        ffma2(x[c][2], x[c][3], sl2, sl2, n1, n1);
                        x[c][2] = ex2_approx(x[c][2]);
                        x[c][3] = ex2_approx(x[c][3]);
                        l1 += x[c][2] + x[c][3];
                        uint32_t *hi = pa[c / 2] + (c & 1) * 2, *lo = pb[c / 2] + (c & 1) * 2;
                        lo[0] = hi[1];
                        two_parts<BF16>(x[c][2], x[c][3], hi[1], lo[1]);
                    }
                    product(pb);
                }
                product(pa);
            }
            copies_wait<0>();
            if (!both) {
#pragma unroll
                for (int c = 0; c < D / 8; ++c) fadd2(o[c][0], o[c][1], o[c][2], o[c][3]);
            }
            // ---- O / l and LSE = ln 2 (m + log2 l) of the piece
            const bool starts = ja == 0, ends = je == n;
            const int slot = starts && ends ? -1 : 2 * static_cast<int>(worker) + (pieces > 0);
            ++pieces;
            if (starts && !ends) {
                info.last_cta = static_cast<int>((w - skip + kUnitTicks + n - 1) / T);
                info.slot = slot;
                info.slot_rows = kSmallRows;
                info.rows = rows;
                info.tok0 = tok0;
                info.head0 = head0;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = r0 + 8 * h;
                float l = h ? l1 : l0;
                const float m = h ? m1 : m0;
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const float lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
                if (r >= rows) continue;
                if (slot < 0) {
                    const size_t row = out_row(r);
                    uint32_t *dst = reinterpret_cast<uint32_t *>(p.O) + (row * D + c0) / 2;
#pragma unroll
                    for (int c = 0; c < D / 8; ++c)
                        dst[4 * c] = l == 0.f ? 0u : pack2<BF16>(o[c][2 * h] * inv, o[c][2 * h + 1] * inv);
                    if (c0 == 0) p.LSE[row] = lse;
                } else {
                    const size_t row = static_cast<size_t>(slot) * kSmallRows + r;
                    float *dst = p.part_O + row * D + c0;
#pragma unroll
                    for (int c = 0; c < D / 8; ++c)
                        *reinterpret_cast<float2 *>(dst + 8 * c) =
                            l == 0.f ? make_float2(0.f, 0.f)
                                     : make_float2(o[c][2 * h] * inv, o[c][2 * h + 1] * inv);
                    if (c0 == 0) p.part_LSE[row] = lse;
                }
            }
        }
        w += len;
        skip = 0;
        if (++qb == nqb) {
            qb = 0;
            if (++sp == p.spaces) {
                sp = 0;
                while (w < w1 && ++b < p.B) {
                    s = small_seq(b, p);
                    nqb = small_units(s, p);
                    if (nqb > 0) break;
                }
                if (b >= p.B) break;
            }
        }
    }
    if (lane == 0) p.info[worker] = info;
    return true;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(Small<D>::kWarps * 32, 1)
    fa_paged_decode_kernel(const __grid_constant__ SmallParams p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    after_previous();
    let_next_start();
    decode_cta<D, BF16, false>(p, smem_raw, 0);
}

// Decode or chunks (see above), by the longest sequence.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    fa_paged_either_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ SmallParams s,
                           const __grid_constant__ Params p, int max_new) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    after_previous();
    let_next_start();
    if (!decode_cta<D, BF16, true>(s, smem_raw, max_new)) chunk_cta<D, BF16>(tmQ, tmK, tmV, p, smem_raw);
}

}  // namespace paged
}  // namespace fa
