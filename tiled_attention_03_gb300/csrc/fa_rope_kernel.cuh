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
// A warp works alone: an item is one token (or a part of its heads, when there are few
// tokens), whose cosines and sines its lanes compute once; the rows stream through a ring
// of asynchronous 16-byte copies into shared memory, kDepth - 1 stages ahead and across
// items, so that the bytes in flight do not cost registers and no block barrier stops
// them. Partners in another lane (half layout) are read from the ring as well.
//
// Bound by memory: 4 bytes per element forward, 6 backward.
#pragma once

#include <cstdint>

#include "fa.h"
#include "fa_pdl.cuh"
#include "ptx.cuh"

namespace fa {
namespace rope {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 128;  // d / 2
constexpr int kDepth = 4;       // stages of the ring (kDepth - 1 in flight)
constexpr int kRows = 2;        // rows per group and stage, forward

// A (batch, head, token, d) tensor of 16-bit elements; null: not there.
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
    // a token's stages: s_q of queries, then s_k of keys, then s_v of values; an item is
    // `per_item` of them, `chunks` items a token
    int s_q, s_k, s_v, per_item, chunks;
    long long items;
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
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
    unpack2<BF16>(v.x, x[0], x[1]);
    unpack2<BF16>(v.y, x[2], x[3]);
    unpack2<BF16>(v.z, x[4], x[5]);
    unpack2<BF16>(v.w, x[6], x[7]);
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
    return make_uint4(pack2<BF16>(y[0], y[1]), pack2<BF16>(y[2], y[3]), pack2<BF16>(y[4], y[5]),
                      pack2<BF16>(y[6], y[7]));
}
template <bool BF16>
__device__ __forceinline__ float load1(const uint16_t *p) {
    float lo, hi;
    unpack2<BF16>(*p, lo, hi);
    return lo;
}

// 16-byte asynchronous copy global -> shared (past L1), and its groups.
__device__ __forceinline__ void copy16(uint4 *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
// the first element of a pair); C = 1, S = 0 past the rotated ones.
template <int MODE>
__device__ __forceinline__ void coefficients(const float (&cs)[2][kMaxPairs], int half_r, int l,
                                             float (&C)[8], float (&S)[8]) {
    if constexpr (MODE == kLane) {
        const bool first = 8 * l < half_r, rotated = 8 * l < 2 * half_r;
        const int j = first ? 8 * l : 8 * l - half_r;
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            const float4 one = make_float4(1.f, 1.f, 1.f, 1.f), zero = make_float4(0.f, 0.f, 0.f, 0.f);
            const float4 c = rotated ? *reinterpret_cast<const float4 *>(&cs[0][j + e]) : one;
            const float4 s = rotated ? *reinterpret_cast<const float4 *>(&cs[1][j + e]) : zero;
            C[e] = c.x, C[e + 1] = c.y, C[e + 2] = c.z, C[e + 3] = c.w;
            S[e] = first ? -s.x : s.x, S[e + 1] = first ? -s.y : s.y;
            S[e + 2] = first ? -s.z : s.z, S[e + 3] = first ? -s.w : s.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = 8 * l + e;
            C[e] = 1.f;
            S[e] = 0.f;
            if (i < 2 * half_r) {
                const bool first = MODE == kBeside ? (e & 1) == 0 : i < half_r;
                const int j = MODE == kBeside ? i >> 1 : (first ? i : i - half_r);
                C[e] = cs[0][j];
                const float s = cs[1][j];
                S[e] = first ? -s : s;
            }
        }
    }
}

// The weight at elements 8 l + e (1 without one), and at their partners.
template <bool BF16>
__device__ __forceinline__ void weights(const uint16_t *w, int l, float (&x)[8]) {
    if (w == nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 1.f;
    } else {
        unpack8<BF16>(__ldg(reinterpret_cast<const uint4 *>(w + 8 * l)), x);
    }
}
template <bool BF16, int MODE>
__device__ __forceinline__ void partner_weights(const uint16_t *w, int half_r, int l, float (&x)[8]) {
    if (w == nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 1.f;
    } else if (MODE == kLane) {
        weights<BF16>(w, partner<MODE>(8 * l, half_r) / 8, x);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = load1<BF16>(w + partner<MODE>(8 * l + e, half_r));
    }
}

// A row in the ring: this lane's 16 bytes and its elements' partners. `at`: the lane's
// own place; the row's first lane is at - l.
template <int D, bool BF16, int MODE>
__device__ __forceinline__ void read_row(const uint4 *at, int half_r, int l, int partner_l,
                                         float (&x)[8], float (&xp)[8]) {
    unpack8<BF16>(*at, x);
    if constexpr (MODE == kBeside) {
#pragma unroll
        for (int e = 0; e < 8; ++e) xp[e] = x[e ^ 1];
    } else if constexpr (MODE == kLane) {
        unpack8<BF16>(at[partner_l - l], xp);
    } else {
        const uint16_t *row = reinterpret_cast<const uint16_t *>(at - l);
#pragma unroll
        for (int e = 0; e < 8; ++e) xp[e] = load1<BF16>(row + partner<MODE>(8 * l + e, half_r));
    }
    if (2 * half_r < D) {  // no partner: not even an infinity times 0
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (8 * l + e >= 2 * half_r) xp[e] = 0.f;
    }
}

// Sum over the lanes of a group.
template <int D>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = Geometry<D>::kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// sum_e a_e b_e in four chains of two.
__device__ __forceinline__ float dot8(const float (&a)[8], const float (&b)[8]) {
    float s0 = a[0], s1 = a[1], t0 = a[4], t1 = a[5];
    fmul2(s0, s1, b[0], b[1]);
    fmul2(t0, t1, b[4], b[5]);
    float u0 = a[2], u1 = a[3], v0 = a[6], v1 = a[7];
    ffma2(u0, u1, b[2], b[3], s0, s1);
    ffma2(v0, v1, b[6], b[7], t0, t1);
    fadd2(u0, u1, v0, v1);
    return u0 + u1;
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
        int before = 0;
        for (int b = threadIdx.x & 31; b < p.B; b += 32) before += p.cu_q[b + 1] <= m;
        before = __reduce_add_sync(0xffffffffu, before);
        r.live = false;
        if (before < p.B) {
            const int first = p.cu_q[before];
            const long long at = static_cast<long long>(p.seq_k[before]) - (p.cu_q[before + 1] - m);
            if (m >= first) {
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

// A walk over stages: stage s of item `item`, whose token is m = (b, n).
struct Cursor {
    long long item;
    int m, b, n, s, end;
    __device__ __forceinline__ void start(const Params &p, long long x) {
        item = x;
        m = b = n = s = end = 0;
        if (x >= p.items) return;
        m = p.chunks == 1 ? static_cast<int>(x) : static_cast<int>(x / p.chunks);
        s = static_cast<int>(x - static_cast<long long>(m) * p.chunks) * p.per_item;
        end = min(s + p.per_item, p.s_q + p.s_k + p.s_v);
        b = p.N == p.tokens ? 0 : m / p.N;
        n = m - b * p.N;
    }
    __device__ __forceinline__ bool more(const Params &p) const { return item < p.items; }
    __device__ __forceinline__ void next(const Params &p, long long warps) {
        if (++s == end) start(p, item + warps);
    }
};

__device__ __forceinline__ const uint16_t *row_at(const Rows &t, const Cursor &c) {
    return t.p + c.b * t.batch + c.n * t.token;
}

// Forward (PAGED = false) and append (PAGED = true).
template <int D, bool BF16, int MODE, bool PAGED>
__global__ void __launch_bounds__(kThreads, 3) fa_norm_rope_kernel(const Params p) {
    using G = Geometry<D>;
    constexpr int U = kRows;
    constexpr int kStageHeads = G::kGroups * U;
    __shared__ uint4 ring[kWarps][kDepth][U][32];
    __shared__ __align__(16) float cs_all[kWarps][2][kMaxPairs];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane % G::kLanes, g = lane / G::kLanes;
    const long long warps = static_cast<long long>(gridDim.x) * kWarps;
    float(&cs)[2][kMaxPairs] = cs_all[warp];
    const int partner_l = MODE == kLane ? partner<MODE>(8 * l, p.half_r) / 8 : l;

    // rows of a stage: head first + u * groups + g of the stage's tensor
    auto issue = [&](const Cursor &c, int slot) {
        if (c.more(p)) {
            const bool is_q = c.s < p.s_q, is_k = !is_q && (!PAGED || c.s < p.s_q + p.s_k);
            const Rows &t = is_q ? p.q : is_k ? p.k : p.v;
            const int heads = is_q ? p.H : is_k ? p.H_kv : p.H_v;
            const int first = (c.s - (is_q ? 0 : is_k ? p.s_q : p.s_q + p.s_k)) * kStageHeads + g;
            const uint16_t *src = row_at(t, c) + 8 * l;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = first + u * G::kGroups;
                if (h < heads) copy16(&ring[warp][slot][u][lane], src + h * t.head);
            }
        }
        copy_commit();
    };

    Cursor in, at;
    in.start(p, static_cast<long long>(blockIdx.x) * kWarps + warp);
    at = in;
    after_previous();
    let_next_start();
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) {
        issue(in, i);
        if (in.more(p)) in.next(p, warps);
    }
    float A[8], Bc[8];
    Place where{0, false, -1};
    long long known = -1;  // the item whose angles are in cs
    int kind = -1;         // the tensor whose coefficients are in A and Bc
    int i = 0;
    for (; at.more(p); at.next(p, warps), ++i) {
        const bool is_q = at.s < p.s_q, is_k = !is_q && (!PAGED || at.s < p.s_q + p.s_k);
        if (known != at.item) {
            known = at.item;
            kind = -1;
            where = place<PAGED>(p, at.m, at.n);
            angles(cs, p, where.pos);
        }
        const uint16_t *w = is_q ? p.wq : p.wk;
        if (kind != (is_q ? 0 : 1) && (is_q || is_k)) {
            kind = is_q ? 0 : 1;
            float wt[8];
            coefficients<MODE>(cs, p.half_r, l, A, Bc);
            weights<BF16>(w, l, wt);
#pragma unroll
            for (int e = 0; e < 8; ++e) A[e] *= wt[e];
            partner_weights<BF16, MODE>(w, p.half_r, l, wt);
#pragma unroll
            for (int e = 0; e < 8; ++e) Bc[e] *= wt[e];
        }
        const int heads = is_q ? p.H : is_k ? p.H_kv : p.H_v;
        const int first = (at.s - (is_q ? 0 : is_k ? p.s_q : p.s_q + p.s_k)) * kStageHeads + g;
        uint16_t *dst;
        long long head_stride;
        bool store = true;
        if (PAGED && !is_q) {
            store = where.slot >= 0;
            dst = (is_k ? p.kc : p.vc) + (store ? where.slot : 0);
            head_stride = p.head_stride;
        } else {
            if (PAGED) store = where.live;
            const Rows &t = is_q ? p.q_out : p.k_out;
            dst = const_cast<uint16_t *>(row_at(t, at));
            head_stride = t.head;
        }
        dst += 8 * l;
        copy_wait<kDepth - 2>();
        __syncwarp();  // the stage is there, and the one of the previous round has been read
        issue(in, (i + kDepth - 1) % kDepth);
        if (in.more(p)) in.next(p, warps);
        const uint4(&stage)[U][32] = ring[warp][i % kDepth];
        uint4 out[U];
        if (PAGED && !is_q && !is_k) {
#pragma unroll
            for (int u = 0; u < U; ++u) out[u] = stage[u][lane];
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[8], xp[8], r = 1.f;
                read_row<D, BF16, MODE>(&stage[u][lane], p.half_r, l, partner_l, x, xp);
                if (w) r = rsqrtf(group_sum<D>(dot8(x, x)) * (1.f / D) + p.eps);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    fmul2(xp[e], xp[e + 1], Bc[e], Bc[e + 1]);
                    ffma2(x[e], x[e + 1], A[e], A[e + 1], xp[e], xp[e + 1]);
                    fmul2(x[e], x[e + 1], r, r);
                }
                out[u] = pack8<BF16>(x);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = first + u * G::kGroups;
            if (store && h < heads) *reinterpret_cast<uint4 *>(dst + h * head_stride) = out[u];
        }
    }
    copy_wait<0>();
}

// Backward: dx of every row, and per block the sums of u z over its rows. The split of
// the rows over blocks depends on the sizes alone, so the sums are the same every time.
template <int D, bool BF16, int MODE>
__global__ void __launch_bounds__(kThreads, 2) fa_norm_rope_bwd_kernel(const Params p) {
    using G = Geometry<D>;
    __shared__ uint4 ring[kWarps][kDepth][2][32];  // gradient and input rows
    __shared__ __align__(16) float cs_all[kWarps][2][kMaxPairs];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane % G::kLanes, g = lane / G::kLanes;
    const long long warps = static_cast<long long>(gridDim.x) * kWarps;
    float(&cs)[2][kMaxPairs] = cs_all[warp];
    const int partner_l = MODE == kLane ? partner<MODE>(8 * l, p.half_r) / 8 : l;
    float dwq[8], dwk[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.f;

    auto issue = [&](const Cursor &c, int slot) {
        if (c.more(p)) {
            const bool is_q = c.s < p.s_q;
            const int h = (c.s - (is_q ? 0 : p.s_q)) * G::kGroups + g;
            if (h < (is_q ? p.H : p.H_kv)) {
                const Rows &dy = is_q ? p.q_out : p.k_out, &x = is_q ? p.q : p.k;
                copy16(&ring[warp][slot][0][lane], row_at(dy, c) + h * dy.head + 8 * l);
                if (is_q ? p.wq != nullptr : p.wk != nullptr)
                    copy16(&ring[warp][slot][1][lane], row_at(x, c) + h * x.head + 8 * l);
            }
        }
        copy_commit();
    };

    Cursor in, at;
    in.start(p, static_cast<long long>(blockIdx.x) * kWarps + warp);
    at = in;
    after_previous();
    let_next_start();
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) {
        issue(in, i);
        if (in.more(p)) in.next(p, warps);
    }
    float C[8], S[8], wt[8];
    long long known = -1;
    int kind = -1, i = 0;
    for (; at.more(p); at.next(p, warps), ++i) {
        const bool is_q = at.s < p.s_q;
        const uint16_t *w = is_q ? p.wq : p.wk;
        if (known != at.item) {
            known = at.item;
            angles(cs, p, place<false>(p, at.m, at.n).pos);
            coefficients<MODE>(cs, p.half_r, l, C, S);
        }
        if (kind != (is_q ? 0 : 1)) {
            kind = is_q ? 0 : 1;
            weights<BF16>(w, l, wt);
        }
        const int h = (at.s - (is_q ? 0 : p.s_q)) * G::kGroups + g;
        const bool there = h < (is_q ? p.H : p.H_kv);
        const Rows &dx = is_q ? p.dq : p.dk;
        copy_wait<kDepth - 2>();
        __syncwarp();  // the stage is there, and the one of the previous round has been read
        issue(in, (i + kDepth - 1) % kDepth);
        if (in.more(p)) in.next(p, warps);
        const uint4(&stage)[2][32] = ring[warp][i % kDepth];
        float o[8], yp[8];
        read_row<D, BF16, MODE>(&stage[0][lane], p.half_r, l, partner_l, o, yp);
        // the transposed rotation: the sine's sign is the other one
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            fmul2(yp[e], yp[e + 1], -S[e], -S[e + 1]);
            ffma2(o[e], o[e + 1], C[e], C[e + 1], yp[e], yp[e + 1]);
        }
        if (w) {
            float x[8], uw[8];
            unpack8<BF16>(stage[1][lane], x);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                uw[e] = o[e], uw[e + 1] = o[e + 1];
                fmul2(uw[e], uw[e + 1], wt[e], wt[e + 1]);
            }
            const float r = rsqrtf(group_sum<D>(dot8(x, x)) * (1.f / D) + p.eps);
            const float k = -group_sum<D>(dot8(uw, x)) * (1.f / D) * r * r * r;
            auto add = [&](float(&dw)[8]) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    float z0 = x[e], z1 = x[e + 1];
                    fmul2(z0, z1, r, r);
                    ffma2(z0, z1, o[e], o[e + 1], dw[e], dw[e + 1]);
                    dw[e] = z0, dw[e + 1] = z1;
                }
            };
            if (there) {  // a row that is not there adds nothing
                if (is_q) add(dwq);
                else add(dwk);
            }
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                fmul2(uw[e], uw[e + 1], r, r);
                ffma2(x[e], x[e + 1], k, k, uw[e], uw[e + 1]);
                o[e] = x[e], o[e + 1] = x[e + 1];
            }
        }
        if (there)
            *reinterpret_cast<uint4 *>(const_cast<uint16_t *>(row_at(dx, at)) + h * dx.head + 8 * l) =
                pack8<BF16>(o);
    }
    copy_wait<0>();
    if (p.part == nullptr) return;
    // the groups' sums, column by column, in one order
    float *red = reinterpret_cast<float *>(&ring[0][0][0][0]);
    constexpr int kAll = kWarps * G::kGroups;
    auto reduce = [&](const float (&dw)[8], int which) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) red[threadIdx.x * 8 + e] = dw[e];
        __syncthreads();
        if (threadIdx.x < D) {
            float s = 0.f;
            for (int r = 0; r < kAll; ++r) s += red[r * D + threadIdx.x];
            p.part[(static_cast<size_t>(blockIdx.x) * 2 + which) * D + threadIdx.x] = s;
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
