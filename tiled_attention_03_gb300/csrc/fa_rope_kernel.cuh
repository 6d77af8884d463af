// fa_rope_kernel.cuh -- norms of queries and keys per head with their rotary positions
// (forward and backward), and the append of keys and values to a paged cache.
//
// A row is one head of one token: d 16-bit elements, held by d / 8 lanes of 16 bytes
// each (a "group"; d <= 256, so a warp holds 256 / d rows). With A_i, B_i the products of
// weight and cosine or sine of element i, and x_p its partner in the rotated pair,
//     y_i = r (x_i A_i + x_p B_i),   r = 1 / sqrt(mean(x^2) + eps),
// so that a row costs one sum of squares over the group and two multiply-adds per
// element; A and B serve every head of a token.
//
// The phase of a pair is position * step in 64-bit fixed point turns: the product's wrap
// around 2^64 is the exact reduction by whole turns, and the upper bits, as a signed
// number of half turns in [-1, 1), go through sincospif.
//
// A warp works alone on an equal share of the line of all tokens' stages (a stage is a few
// heads of one tensor of one token). Its lanes compute a token's cosines and sines once;
// the rows stream through a ring of asynchronous 16-byte copies into shared memory, kDepth -
// 1 stages ahead and across tokens, so that the bytes in flight do not cost registers
// and no block barrier stops them. Partners in another lane (half layout) are read from
// the ring as well.
//
// Bound by memory, 4 bytes per element forward and 6 backward, and beside it by its own
// instructions (61 and 67 % of issue slots). B4 N4096 d128 bf16, replayed in a graph:
// forward of 32+32 heads 87 us (6.2 TB/s), backward of 32+8 heads 92 us (5.5 TB/s). Without
// norm and rotation the forward took as long, without its stores or its loads 69 us. A
// block per few tokens with an angle barrier took 161 and 152 us, a warp per whole token 99
// and 133 us.
#pragma once

#include <cstdint>

#include "fa.h"
#include "fa_copy.cuh"
#include "fa_pdl.cuh"
#include "ptx.cuh"

namespace fa {
namespace rope {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 128;  // d / 2
constexpr int kDepth = 4;       // stages of the ring (kDepth - 1 in flight)
constexpr int kRows = 2;        // rows per group and stage, forward

// A (batch, head, token, d) tensor of 16-bit elements, strides >= 0; null: not there.
struct Rows {
    uint16_t *p;
    long long batch, head, token;
};

struct Params {
    Rows q, k, q_out, k_out;       // backward: inputs, and the gradients of the outputs in
    Rows dq, dk;                   // backward: gradients of the inputs
    Rows v;                        // append
    int H, H_kv, H_v;              // heads of q, k, v (0: not there)
    int N;                         // tokens per batch entry
    int tokens;                    // B * N
    const int *positions;          // null: token index in its batch entry
    const unsigned long long *steps;
    int half_r;                    // rotated pairs
    float magnitude, eps;
    const uint16_t *wq, *wk;       // null: not normalised
    // a token's stages: s_q of queries, then s_k of keys, then s_v of values; all tokens'
    int s_q, s_k, s_v;
    long long stages;
    // paged
    uint16_t *kc, *vc;
    long long page_stride, token_stride, head_stride;
    const int *cu_q, *seq_k, *table;
    int B, max_pages, page_log2, num_pages;
    float *part;                   // backward: [blocks][2][D] partial weight gradients
};

template <bool BF16>
__device__ __forceinline__ void unpack2(uint32_t w, float &lo, float &hi) {
    if constexpr (BF16) {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xffff0000u);
    } else {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(lo), "=f"(hi)
            : "r"(w));
    }
}

// Two floats in one 64-bit register pair. The rows stay packed from their 16-bit words to
// the result's: every multiply and add below is one instruction for two elements.
using f2 = uint64_t;
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 both(float x) { return f2_pack(x, x); }

template <bool BF16>
__device__ __forceinline__ f2 unpack_pair(uint32_t w) {
    float lo, hi;
    unpack2<BF16>(w, lo, hi);
    return f2_pack(lo, hi);
}
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &v, f2 (&x)[4]) {
    x[0] = unpack_pair<BF16>(v.x);
    x[1] = unpack_pair<BF16>(v.y);
    x[2] = unpack_pair<BF16>(v.z);
    x[3] = unpack_pair<BF16>(v.w);
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack_pair(f2 x) {
    float lo, hi;
    f2_unpack(x, lo, hi);
    return pack2<BF16>(lo, hi);
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const f2 (&y)[4]) {
    return make_uint4(pack_pair<BF16>(y[0]), pack_pair<BF16>(y[1]), pack_pair<BF16>(y[2]),
                      pack_pair<BF16>(y[3]));
}
__device__ __forceinline__ f2 swapped(f2 x) {
    float lo, hi;
    f2_unpack(x, lo, hi);
    return f2_pack(hi, lo);
}
template <bool BF16>
__device__ __forceinline__ float load1(const uint16_t *p) {
    float lo, hi;
    unpack2<BF16>(*p, lo, hi);
    return lo;
}

// How the partner of a rotated element is found: beside it (interleaved), in another
// lane at the same place (half layout, pair distance a multiple of 8 elements), or
// anywhere in the row (half layout, other distances).
enum : int { kBeside = 0, kLane = 1, kAnywhere = 2 };

template <int D>
struct Geometry {
    static constexpr int kLanes = D / 8;          // lanes per row
    static constexpr int kGroups = 32 / kLanes;   // rows of a warp at a time
};

// The partner of element i among 2 half_r rotated ones (i itself past them).
template <int MODE>
__device__ __forceinline__ int partner(int i, int half_r) {
    if (i >= 2 * half_r) return i;
    if (MODE == kBeside) return i ^ 1;
    return i < half_r ? i + half_r : i - half_r;
}

// Cosines and sines (times the magnitude) of one token's pairs, by the whole warp.
__device__ __forceinline__ void angles(float (&cs)[2][kMaxPairs], const Params &p, int pos) {
    __syncwarp();
    for (int j = threadIdx.x & 31; j < p.half_r; j += 32) {
        const long long phase = static_cast<long long>(
            static_cast<unsigned long long>(static_cast<long long>(pos)) * p.steps[j]);
        float s, c;
        sincospif(static_cast<float>(phase) * 0x1p-63f, &s, &c);
        cs[0][j] = c * p.magnitude;
        cs[1][j] = s * p.magnitude;
    }
    __syncwarp();
}

// Coefficients of elements 8 l + e: C the cosine, S the sine of the partner (negative in
// the first element of a pair; TRANSPOSED: in the second); C = 1, S = -0 past the rotated ones
// (0 x -0 added leaves the sign of a zero as it is).
template <int MODE, bool TRANSPOSED>
__device__ __forceinline__ void coefficients(const float (&cs)[2][kMaxPairs], int half_r, int l,
                                             f2 (&C)[4], f2 (&S)[4]) {
    if constexpr (MODE == kLane) {
        const bool first = 8 * l < half_r, rotated = 8 * l < 2 * half_r;
        const int j = first ? 8 * l : 8 * l - half_r;
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const float4 one = make_float4(1.f, 1.f, 1.f, 1.f), zero = make_float4(-0.f, -0.f, -0.f, -0.f);
            const float4 c = rotated ? *reinterpret_cast<const float4 *>(&cs[0][j + 2 * e]) : one;
            const float4 s = rotated ? *reinterpret_cast<const float4 *>(&cs[1][j + 2 * e]) : zero;
            const f2 sign = both(rotated && first != TRANSPOSED ? -1.f : 1.f);
            C[e] = f2_pack(c.x, c.y), C[e + 1] = f2_pack(c.z, c.w);
            S[e] = mul2(f2_pack(s.x, s.y), sign), S[e + 1] = mul2(f2_pack(s.z, s.w), sign);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float c[2], t[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int i = 8 * l + 2 * e + x;
                c[x] = 1.f;
                t[x] = -0.f;
                if (i < 2 * half_r) {
                    const bool first = MODE == kBeside ? x == 0 : i < half_r;
                    const int j = MODE == kBeside ? i >> 1 : (first ? i : i - half_r);
                    c[x] = cs[0][j];
                    t[x] = first != TRANSPOSED ? -cs[1][j] : cs[1][j];
                }
            }
            C[e] = f2_pack(c[0], c[1]);
            S[e] = f2_pack(t[0], t[1]);
        }
    }
}

// The weight at elements 8 l + e (1 without one), and at their partners.
template <bool BF16>
__device__ __forceinline__ void weights(const uint16_t *w, int l, f2 (&x)[4]) {
    if (w == nullptr) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = both(1.f);
    } else {
        unpack8<BF16>(__ldg(reinterpret_cast<const uint4 *>(w + 8 * l)), x);
    }
}
template <bool BF16, int MODE>
__device__ __forceinline__ void partner_weights(const uint16_t *w, int half_r, int l, f2 (&x)[4]) {
    if (w == nullptr) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = both(1.f);
    } else if (MODE == kLane) {
        weights<BF16>(w, partner<MODE>(8 * l, half_r) / 8, x);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[e] = f2_pack(load1<BF16>(w + partner<MODE>(8 * l + 2 * e, half_r)),
                           load1<BF16>(w + partner<MODE>(8 * l + 2 * e + 1, half_r)));
    }
}

// A row in the ring: this lane's 16 bytes and its elements' partners. `at`: the lane's
// own place; the row's first lane is at - l.
template <int D, bool BF16, int MODE>
__device__ __forceinline__ void read_row(const uint4 *at, int half_r, int l, int partner_l, f2 (&x)[4],
                                         f2 (&xp)[4]) {
    unpack8<BF16>(*at, x);
    if constexpr (MODE == kBeside) {
#pragma unroll
        for (int e = 0; e < 4; ++e) xp[e] = swapped(x[e]);
    } else if constexpr (MODE == kLane) {
        unpack8<BF16>(at[partner_l - l], xp);
    } else {
        const uint16_t *row = reinterpret_cast<const uint16_t *>(at - l);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            xp[e] = f2_pack(load1<BF16>(row + partner<MODE>(8 * l + 2 * e, half_r)),
                            load1<BF16>(row + partner<MODE>(8 * l + 2 * e + 1, half_r)));
    }
    if (2 * half_r < D) {  // no partner: not even an infinity times 0 (pairs are whole: 2 half_r is even)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (8 * l + 2 * e >= 2 * half_r) xp[e] = 0;
    }
}

// Sum over the lanes of a group, of two values at once.
template <int D>
__device__ __forceinline__ f2 group_sum(f2 v) {
#pragma unroll
    for (int o = Geometry<D>::kLanes / 2; o > 0; o >>= 1) {
        float a, b;
        f2_unpack(v, a, b);
        v = add2(v, f2_pack(__shfl_xor_sync(0xffffffffu, a, o), __shfl_xor_sync(0xffffffffu, b, o)));
    }
    return v;
}

// sum_e a_e b_e over this lane's 8 elements.
__device__ __forceinline__ float dot8(const f2 (&a)[4], const f2 (&b)[4]) {
    const f2 s = add2(fma2(a[2], b[2], mul2(a[0], b[0])), fma2(a[3], b[3], mul2(a[1], b[1])));
    float x, y;
    f2_unpack(s, x, y);
    return x + y;
}

// Where token m stands: its position, and in an append whether it belongs to a sequence
// and the first element of its slot in the cache (-1: none). By the whole warp; the
// sequence of token m is the number of sequences that end at or before m.
struct Place {
    int pos;
    bool live;
    long long slot;
};
template <bool PAGED>
__device__ __forceinline__ Place place(const Params &p, int m, int n) {
    Place r{0, true, -1};
    if constexpr (!PAGED) {
        r.pos = p.positions ? __ldg(p.positions + m) : n;
    } else {
        // every lane probes the end of one of 32 parts of what is left to search
        int before = 0;
        for (int left = p.B; left > 0;) {
            const int step = (left + 31) >> 5;
            const int last = (static_cast<int>(threadIdx.x & 31) + 1) * step;
            const bool past = last <= left && p.cu_q[before + last] <= m;
            const int parts = __popc(__ballot_sync(0xffffffffu, past));
            before += parts * step;
            left = min(step - 1, left - parts * step);
        }
        r.live = false;
        if (before < p.B) {
            const int first = p.cu_q[before], end = p.cu_q[before + 1];
            const long long at = static_cast<long long>(p.seq_k[before]) - (end - m);
            if (m >= first && m < end) {
                r.live = true;
                r.pos = static_cast<int>(at);
                const long long page = at >> p.page_log2;
                if (at >= 0 && page < p.max_pages) {
                    const int x = p.table[static_cast<long long>(before) * p.max_pages + page];
                    if (x >= 0 && x < p.num_pages)
                        r.slot = x * p.page_stride + (at & ((1ll << p.page_log2) - 1)) * p.token_stride;
                }
            }
        }
    }
    return r;
}

// A warp's part of a token: token m = (b, n), its stages s .. end - 1, with `left` stages
// of the warp's share from s on. m >= 0 while there is one.
struct Item {
    int m, b, n, s, end;
    long long left;
    __device__ __forceinline__ void place_token(const Params &p) {
        end = static_cast<int>(min(static_cast<long long>(p.s_q + p.s_k + p.s_v), s + left));
        b = p.N == p.tokens ? 0 : m / p.N;
        n = m - b * p.N;
    }
    // this warp's share: the w-th of `warps` equal ones
    __device__ __forceinline__ void first(const Params &p, long long w, long long warps) {
        const long long x = p.stages * w / warps;
        left = p.stages * (w + 1) / warps - x;
        const int per = p.s_q + p.s_k + p.s_v;
        m = static_cast<int>(x / per);
        s = static_cast<int>(x - static_cast<long long>(m) * per);
        if (left > 0) place_token(p);
    }
    // the next token (its stages from 0 on)
    __device__ __forceinline__ void next(const Params &p, int done) {
        left -= done;
        ++m;
        s = 0;
        if (left > 0) place_token(p);
    }
};

// The run of an item's stages from stage s on that belong to one tensor (0 queries, 1
// keys, 2 values): its stages, and the head of its first row (this lane's group adds g).
struct Run {
    int kind, stages, head, heads;
};
template <int kStageHeads>
__device__ __forceinline__ Run run_of(const Params &p, int s, int end) {
    Run r;
    r.kind = s < p.s_q ? 0 : s < p.s_q + p.s_k ? 1 : 2;
    const int first = r.kind == 0 ? 0 : r.kind == 1 ? p.s_q : p.s_q + p.s_k;
    const int count = r.kind == 0 ? p.s_q : r.kind == 1 ? p.s_k : p.s_v;
    r.stages = min(end, first + count) - s;
    r.head = (s - first) * kStageHeads;
    r.heads = r.kind == 0 ? p.H : r.kind == 1 ? p.H_kv : p.H_v;
    return r;
}

__device__ __forceinline__ uint16_t *row_at(const Rows &t, const Item &i, int h) {
    return t.p + i.b * t.batch + i.n * t.token + h * t.head;
}

// The walk of a warp's copies, ahead of its products: row pointers of up to two tensors
// that step from stage to stage, set anew only where a run ends.
template <int kTensors, int kStageHeads>
struct Ahead {
    Item at;
    int done;                       // stages of this token taken into runs
    int stages;                     // left in this run (0: nothing more to copy)
    int h, heads;                   // this lane's first head of the stage, and their number
    const uint16_t *src[kTensors];  // its row
    long long head[kTensors];       // elements between heads (-1: a tensor that is not there)

    // which(kind, i): the i-th tensor of a run of that kind
    template <typename Which>
    __device__ __forceinline__ void run(const Params &p, int g, int l, const Which &which) {
        const Run r = run_of<kStageHeads>(p, at.s, at.end);
        stages = r.stages;
        done += r.stages;
        at.s += r.stages;
        h = r.head + g;
        heads = r.heads;
#pragma unroll
        for (int i = 0; i < kTensors; ++i) {
            const Rows &t = which(r.kind, i);
            src[i] = row_at(t, at, h) + 8 * l;
            head[i] = t.p ? t.head : -1;
        }
    }
    template <typename Which>
    __device__ __forceinline__ void start(const Params &p, int g, int l, const Which &which) {
        stages = done = 0;
        if (at.left > 0) run(p, g, l, which);
    }
    template <typename Which>
    __device__ __forceinline__ void next(const Params &p, int g, int l, const Which &which) {
        h += kStageHeads;
#pragma unroll
        for (int i = 0; i < kTensors; ++i) src[i] += kStageHeads * head[i];
        if (--stages == 0) {
            if (at.s < at.end) {
                run(p, g, l, which);
            } else {
                at.next(p, done);
                start(p, g, l, which);
            }
        }
    }
};

// Forward (PAGED = false) and append (PAGED = true).
template <int D, bool BF16, int MODE, bool PAGED>
__global__ void __launch_bounds__(kThreads, 2) fa_norm_rope_kernel(const Params p) {
    using G = Geometry<D>;
    constexpr int U = kRows;
    constexpr int kStageHeads = G::kGroups * U;
    __shared__ uint4 ring[kWarps][kDepth][U][32];
    __shared__ __align__(16) float cs_all[kWarps][2][kMaxPairs];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane % G::kLanes, g = lane / G::kLanes;
    const long long warps = static_cast<long long>(gridDim.x) * kWarps;
    const long long share = static_cast<long long>(blockIdx.x) * kWarps + warp;
    float(&cs)[2][kMaxPairs] = cs_all[warp];
    const int partner_l = MODE == kLane ? partner<MODE>(8 * l, p.half_r) / 8 : l;
    auto which = [&](int kind, int) -> const Rows & { return kind == 0 ? p.q : kind == 1 ? p.k : p.v; };

    after_previous();
    let_next_start();
    Item at;
    at.first(p, share, warps);
    Ahead<1, kStageHeads> in;
    in.at = at;
    in.start(p, g, l, which);
    auto issue = [&](int slot) {
        if (in.stages > 0) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (in.h + u * G::kGroups < in.heads)
                    copy16(smem_u32(&ring[warp][slot][u][lane]), in.src[0] + u * G::kGroups * in.head[0]);
            in.next(p, g, l, which);
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) issue(i);

    int slot = 0;
    for (; at.left > 0; at.next(p, at.end - at.s)) {
        const Place where = place<PAGED>(p, at.m, at.n);
        angles(cs, p, where.pos);
        for (int s = at.s; s < at.end;) {
            const Run run = run_of<kStageHeads>(p, s, at.end);
            s += run.stages;
            const uint16_t *w = run.kind == 0 ? p.wq : p.wk;
            // values, and rows neither normalised nor rotated, go through bit by bit (in the
            // append alone: the dense forward of 16,384 x 64 rows took 88.5 us with it, 87.7 without)
            const bool as_is = PAGED && (run.kind == 2 || (w == nullptr && p.half_r == 0));
            f2 A[4], Bc[4];
            if (!as_is) {
                f2 wt[4];
                coefficients<MODE, false>(cs, p.half_r, l, A, Bc);
                weights<BF16>(w, l, wt);
#pragma unroll
                for (int e = 0; e < 4; ++e) A[e] = mul2(A[e], wt[e]);
                partner_weights<BF16, MODE>(w, p.half_r, l, wt);
#pragma unroll
                for (int e = 0; e < 4; ++e) Bc[e] = mul2(Bc[e], wt[e]);
            }
            int h = run.head + g;
            // heads of this run that are stored: none where the token has no place
            int heads = run.heads;
            long long dst_head;
            uint16_t *dst;
            if (PAGED && run.kind > 0) {
                if (where.slot < 0) heads = 0;
                dst_head = p.head_stride;
                dst = (run.kind == 1 ? p.kc : p.vc) + where.slot + h * dst_head + 8 * l;
            } else {
                if (PAGED && !where.live) heads = 0;
                const Rows &t = run.kind == 0 ? p.q_out : p.k_out;
                dst_head = t.head;
                dst = row_at(t, at, h) + 8 * l;
            }
            for (int j = 0; j < run.stages; ++j) {
                copies_wait<kDepth - 2>();
                __syncwarp();  // the stage is there, and the one before has been read
                issue((slot + kDepth - 1) % kDepth);
                const uint4(&stage)[U][32] = ring[warp][slot];
                slot = (slot + 1) % kDepth;
                uint4 out[U];
                if (as_is) {
#pragma unroll
                    for (int u = 0; u < U; ++u) out[u] = stage[u][lane];
                } else {
                    f2 y[U][4], yp[U][4], r = both(1.f);
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        read_row<D, BF16, MODE>(&stage[u][lane], p.half_r, l, partner_l, y[u], yp[u]);
                    if (w) {
                        static_assert(U == 2, "the rows' sums go through the lanes as one pair");
                        float s0, s1;
                        f2_unpack(group_sum<D>(f2_pack(dot8(y[0], y[0]), dot8(y[1], y[1]))), s0, s1);
                        r = f2_pack(rsqrtf(s0 * (1.f / D) + p.eps), rsqrtf(s1 * (1.f / D) + p.eps));
                    }
                    float r0, r1;
                    f2_unpack(r, r0, r1);
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const f2 ru = both(u == 0 ? r0 : r1);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            y[u][e] = mul2(fma2(y[u][e], A[e], mul2(yp[u][e], Bc[e])), ru);
                        out[u] = pack8<BF16>(y[u]);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (h + u * G::kGroups < heads)
                        *reinterpret_cast<uint4 *>(dst + u * G::kGroups * dst_head) = out[u];
                h += kStageHeads;
                dst += kStageHeads * dst_head;
            }
        }
    }
    copies_wait<0>();
}

// Backward: dx of every row, and per block the sums of u z over its rows. The split of
// the rows over blocks depends on the sizes alone, so the sums are the same every time.
template <int D, bool BF16, int MODE>
__global__ void __launch_bounds__(kThreads, 2) fa_norm_rope_bwd_kernel(const Params p) {
    using G = Geometry<D>;
    constexpr int kStageHeads = G::kGroups;
    __shared__ uint4 ring[kWarps][kDepth][2][32];  // gradient and input rows
    __shared__ __align__(16) float cs_all[kWarps][2][kMaxPairs];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane % G::kLanes, g = lane / G::kLanes;
    const long long warps = static_cast<long long>(gridDim.x) * kWarps;
    const long long share = static_cast<long long>(blockIdx.x) * kWarps + warp;
    float(&cs)[2][kMaxPairs] = cs_all[warp];
    const int partner_l = MODE == kLane ? partner<MODE>(8 * l, p.half_r) / 8 : l;
    f2 dwq[4], dwk[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) dwq[e] = dwk[e] = 0;
    auto which = [&](int kind, int i) -> const Rows & {
        return i == 0 ? (kind == 0 ? p.q_out : p.k_out) : kind == 0 ? p.q : p.k;
    };

    after_previous();
    let_next_start();
    Item at;
    at.first(p, share, warps);
    Ahead<2, kStageHeads> in;
    in.at = at;
    in.start(p, g, l, which);
    auto issue = [&](int slot) {
        if (in.stages > 0) {
            if (in.h < in.heads) {
                copy16(smem_u32(&ring[warp][slot][0][lane]), in.src[0]);
                if (in.head[1] >= 0) copy16(smem_u32(&ring[warp][slot][1][lane]), in.src[1]);
            }
            in.next(p, g, l, which);
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) issue(i);

    int slot = 0;
    for (; at.left > 0; at.next(p, at.end - at.s)) {
        angles(cs, p, place<false>(p, at.m, at.n).pos);
        f2 C[4], S[4];
        coefficients<MODE, true>(cs, p.half_r, l, C, S);
        for (int s = at.s; s < at.end;) {
            const Run run = run_of<kStageHeads>(p, s, at.end);
            s += run.stages;
            const uint16_t *w = run.kind == 0 ? p.wq : p.wk;
            const Rows &t = run.kind == 0 ? p.dq : p.dk;
            int h = run.head + g;
            uint16_t *dst = row_at(t, at, h) + 8 * l;
            f2 wt[4], dw[4];
            weights<BF16>(w, l, wt);
#pragma unroll
            for (int e = 0; e < 4; ++e) dw[e] = 0;
            for (int j = 0; j < run.stages; ++j) {
                copies_wait<kDepth - 2>();
                __syncwarp();
                issue((slot + kDepth - 1) % kDepth);
                const uint4(&stage)[2][32] = ring[warp][slot];
                slot = (slot + 1) % kDepth;
                const bool there = h < run.heads;
                f2 o[4], yp[4];
                read_row<D, BF16, MODE>(&stage[0][lane], p.half_r, l, partner_l, o, yp);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = fma2(o[e], C[e], mul2(yp[e], S[e]));
                if (w) {
                    f2 x8[4], uw[4];
                    unpack8<BF16>(stage[1][lane], x8);
#pragma unroll
                    for (int e = 0; e < 4; ++e) uw[e] = mul2(o[e], wt[e]);
                    float xx, ux;
                    f2_unpack(group_sum<D>(f2_pack(dot8(x8, x8), dot8(uw, x8))), xx, ux);
                    const float r = rsqrtf(xx * (1.f / D) + p.eps);
                    const f2 rr = both(r), k = both(-ux * (1.f / D) * r * r);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f2 z = mul2(x8[e], rr);
                        if (there) dw[e] = fma2(o[e], z, dw[e]);  // a row that is not there adds nothing
                        o[e] = fma2(z, k, mul2(uw[e], rr));
                    }
                }
                if (there) *reinterpret_cast<uint4 *>(dst) = pack8<BF16>(o);
                h += kStageHeads;
                dst += kStageHeads * t.head;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (run.kind == 0) dwq[e] = add2(dwq[e], dw[e]);
                else dwk[e] = add2(dwk[e], dw[e]);
            }
        }
    }
    copies_wait<0>();
    if (p.part == nullptr) return;
    // the groups' sums, column by column, in one order
    float *red = reinterpret_cast<float *>(&ring[0][0][0][0]);
    constexpr int kAll = kWarps * G::kGroups;
    auto reduce = [&](const f2 (&dw)[4], int which_w) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float a, b;
            f2_unpack(dw[e], a, b);
            *reinterpret_cast<float2 *>(&red[threadIdx.x * 8 + 2 * e]) = make_float2(a, b);
        }
        __syncthreads();
        if (threadIdx.x < D) {
            float s = 0.f;
            for (int r = 0; r < kAll; ++r) s += red[r * D + threadIdx.x];
            p.part[(static_cast<size_t>(blockIdx.x) * 2 + which_w) * D + threadIdx.x] = s;
        }
    };
    reduce(dwq, 0);
    reduce(dwk, 1);
}

// Weight gradients: column c of the blocks' sums, added in one order; 32 columns a block.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads)
    fa_norm_rope_sum_kernel(const float *part, int blocks, int D, float *dwq, float *dwk) {
    __shared__ float red[32][33];
    after_previous();
    let_next_start();
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
    float s = 0.f;
    for (int b = r; b < blocks; b += 32) s += part[static_cast<size_t>(b) * 2 * D + c];
    red[r][threadIdx.x & 31] = s;
    __syncthreads();
    // warp r: column r of the tile
    float v = red[threadIdx.x & 31][r];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) {
        const int col = blockIdx.x * 32 + r;
        float *dw = col < D ? dwq : dwk;
        if (dw) dw[col < D ? col : col - D] = v;
    }
}

}  // namespace rope
}  // namespace fa
