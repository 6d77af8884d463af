// fa_rope_kernel.cuh -- norms of queries and keys per head with their rotary positions
// (forward and backward), and the append of keys and values to a paged cache.
//
// A row is one head of one token: d 16-bit elements, held by d / 8 lanes of 16 bytes
// each (a "group"; d <= 256, so a group lies in one warp). With A_i, B_i the products of
// weight and cosine or sine of element i, and x_p its partner in the rotated pair,
//     y_i = r (x_i A_i + x_p B_i),   r = 1 / sqrt(mean(x^2) + eps),
// so that a row costs one sum of squares over the group and two multiply-adds per
// element; A and B serve every head of a token. The partner's elements come from another
// lane as packed words (half layout) or sit beside their own (interleaved).
//
// The phase of a pair is position * step in 64-bit fixed point turns: the product's wrap
// around 2^64 is the exact reduction by whole turns, and the upper bits, as a signed
// number of half turns in [-1, 1), go through sincospif. A block computes the cosines and
// sines of its T tokens once, into shared memory.
//
// Bound by memory: 4 bytes per element forward, 6 backward, against about 10 operations.
#pragma once

#include <cstdint>

#include "fa.h"
#include "ptx.cuh"

namespace fa {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;     // tokens per block
constexpr int kMaxPairs = 128;    // d / 2

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
    long long tokens;              // B * N
    const int *positions;          // null: token index in its batch entry
    const unsigned long long *steps;
    int half_r;                    // rotated pairs
    float magnitude, eps;
    const uint16_t *wq, *wk;       // null: not normalised
    int T, chunk, chunks;          // tokens per block; heads per block; blocks per token tile
    // paged
    uint16_t *kc, *vc;
    long long page_stride, token_stride, head_stride;
    const int *cu_q, *seq_k, *table;
    int B, max_pages, page_log2, num_pages;
    // backward
    float *part;                   // [blocks][2][D] partial weight gradients
    long long tiles;               // token tiles x chunks
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

// How the partner of a rotated element is found: beside it (interleaved), in another
// lane at the same place (half layout, pair distance a multiple of 8 elements), or
// anywhere (half layout, other distances: through shared memory).
enum : int { kBeside = 0, kLane = 1, kAnywhere = 2 };

template <int D>
struct Geometry {
    static constexpr int kLanes = D / 8;               // lanes per row
    static constexpr int kGroups = kThreads / kLanes;  // rows in flight per block
};

// The partner of element i among r = 2 half_r rotated ones (i itself past them).
template <int MODE>
__device__ __forceinline__ int partner(int i, int half_r) {
    if (i >= 2 * half_r) return i;
    if (MODE == kBeside) return i ^ 1;
    return i < half_r ? i + half_r : i - half_r;
}

template <int D>
struct Shared {
    float cs[2][kMaxTokens][kMaxPairs];        // magnitude times cosine, sine
    uint4 stage[kThreads];                     // kAnywhere: raw rows
    float red[kThreads * 8];                   // backward: weight gradients of the groups
    int pos[kMaxTokens];
    long long cache_off[kMaxTokens];           // append: first element of the token's slot, or -1
    int live[kMaxTokens];                      // append: the token belongs to a sequence
};

// cos and sin of the block's tokens. `pos` is set and synchronised.
template <int D>
__device__ __forceinline__ void angles(Shared<D> &sh, const Params &p, int T) {
    for (int x = threadIdx.x; x < T * p.half_r; x += kThreads) {
        const int t = x / p.half_r, j = x - t * p.half_r;
        const long long phase = static_cast<long long>(
            static_cast<unsigned long long>(static_cast<long long>(sh.pos[t])) * p.steps[j]);
        float s, c;
        sincospif(static_cast<float>(phase) * 0x1p-63f, &s, &c);
        sh.cs[0][t][j] = c * p.magnitude;
        sh.cs[1][t][j] = s * p.magnitude;
    }
}

// Signed coefficients of element i = 8 l + e: cosine C and sine S of the partner (S is
// negative in the first element of a pair), C = 1 and S = 0 past the rotated ones.
template <int D, int MODE>
__device__ __forceinline__ void coefficients(const Shared<D> &sh, const Params &p, int t, int l,
                                             float (&C)[8], float (&S)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int i = 8 * l + e;
        C[e] = 1.f;
        S[e] = 0.f;
        if (i < 2 * p.half_r) {
            const bool first = MODE == kBeside ? (e & 1) == 0 : i < p.half_r;
            const int j = MODE == kBeside ? i >> 1 : (first ? i : i - p.half_r);
            C[e] = sh.cs[0][t][j];
            const float s = sh.cs[1][t][j];
            S[e] = first ? -s : s;
        }
    }
}

// The partners' values of this lane's 8 elements (raw row words v of the group).
template <int D, bool BF16, int MODE>
__device__ __forceinline__ void partners(Shared<D> &sh, const Params &p, const uint4 &v, int l,
                                         int src_lane, const float (&x)[8], float (&xp)[8]) {
    if constexpr (MODE == kBeside) {
#pragma unroll
        for (int e = 0; e < 8; ++e) xp[e] = x[e ^ 1];
    } else if constexpr (MODE == kLane) {
        uint4 w;
        w.x = __shfl_sync(0xffffffffu, v.x, src_lane);
        w.y = __shfl_sync(0xffffffffu, v.y, src_lane);
        w.z = __shfl_sync(0xffffffffu, v.z, src_lane);
        w.w = __shfl_sync(0xffffffffu, v.w, src_lane);
        unpack8<BF16>(w, xp);
    } else {
        __syncwarp();
        sh.stage[threadIdx.x] = v;
        __syncwarp();
        const uint16_t *row = reinterpret_cast<const uint16_t *>(&sh.stage[threadIdx.x - l]);
#pragma unroll
        for (int e = 0; e < 8; ++e) xp[e] = load1<BF16>(row + partner<MODE>(8 * l + e, p.half_r));
    }
    if (2 * p.half_r < D) {  // no partner: not even an infinity times 0
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (8 * l + e >= 2 * p.half_r) xp[e] = 0.f;
    }
}

// Sum over the lanes of a group.
template <int D>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = Geometry<D>::kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ uint4 load_row(const uint16_t *p, bool there) {
    return there ? __ldcs(reinterpret_cast<const uint4 *>(p)) : make_uint4(0, 0, 0, 0);
}

// Where the tokens t0 .. t0 + T - 1 stand; warp t sets token t. Append: also their slots
// in the cache. The sequence of token m is the number of sequences that end at or before m.
template <int D, bool PAGED>
__device__ __forceinline__ void places(Shared<D> &sh, const Params &p, long long t0, int T) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp >= T) return;
    const long long m = t0 + warp;
    if constexpr (!PAGED) {
        if (lane == 0 && m < p.tokens)
            sh.pos[warp] = p.positions ? p.positions[m] : static_cast<int>(m % p.N);
    } else {
        int before = 0;
        for (int b = lane; b < p.B; b += 32) before += p.cu_q[b + 1] <= m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
        if (lane == 0) {
            int pos = 0, live = 0;
            long long off = -1;
            if (m < p.tokens && before < p.B) {
                const long long first = p.cu_q[before], end = p.cu_q[before + 1];
                const long long at = static_cast<long long>(p.seq_k[before]) - (end - m);
                if (m >= first) {
                    live = 1;
                    pos = static_cast<int>(at);
                    const long long page = at >> p.page_log2;
                    if (at >= 0 && page < p.max_pages) {
                        const int n = p.table[static_cast<long long>(before) * p.max_pages + page];
                        if (n >= 0 && n < p.num_pages)
                            off = n * p.page_stride + (at & ((1ll << p.page_log2) - 1)) * p.token_stride;
                    }
                }
            }
            sh.pos[warp] = pos;
            sh.live[warp] = live;
            sh.cache_off[warp] = off;
        }
    }
}

// Forward (PAGED = false) and append (PAGED = true).
template <int D, bool BF16, int MODE, bool PAGED>
__global__ void __launch_bounds__(kThreads) fa_norm_rope_kernel(const Params p) {
    using G = Geometry<D>;
    __shared__ Shared<D> sh;
    const int T = p.T, per = G::kGroups / T;  // groups per token
    const long long tile = blockIdx.x / p.chunks;
    const int h0 = static_cast<int>(blockIdx.x % p.chunks) * p.chunk, h1 = h0 + p.chunk;
    places<D, PAGED>(sh, p, tile * T, T);
    __syncthreads();
    angles<D>(sh, p, T);
    __syncthreads();
    const int group = threadIdx.x / G::kLanes, l = threadIdx.x % G::kLanes;
    const int t = group / per, g = group % per;
    const long long m = tile * T + t;
    const bool there = m < p.tokens && (!PAGED || sh.live[t] != 0);
    const long long b = m / p.N, n = m - b * p.N;
    const int src_lane = (threadIdx.x & 31) - l + partner<MODE>(8 * l, p.half_r) / 8;
    constexpr int U = 4;  // rows in flight per group

    float C[8], S[8];
    coefficients<D, MODE>(sh, p, t, l, C, S);
    // heads a .. z of one tensor: first = its first head among all
    auto rows = [&](const Rows &in, const Rows &out, const uint16_t *w, int first, int heads,
                    bool to_cache) {
        const int a = max(h0 - first, 0), z = min(h1 - first, heads);
        if (a >= z) return;
        float A[8], Bc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = 8 * l + e;
            A[e] = C[e] * (w ? load1<BF16>(w + i) : 1.f);
            Bc[e] = S[e] * (w ? load1<BF16>(w + partner<MODE>(i, p.half_r)) : 1.f);
        }
        const uint16_t *src = in.p + b * in.batch + n * in.token + 8 * l;
        const bool store = there && (!to_cache || sh.cache_off[t] >= 0);
        uint16_t *dst = (to_cache ? p.kc + sh.cache_off[t] : out.p + b * out.batch + n * out.token) + 8 * l;
        const long long dst_head = to_cache ? p.head_stride : out.head;
        for (int h = a; h < z; h += per * U) {  // uniform over the block
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int hh = h + g + u * per;
                v[u] = load_row(src + hh * in.head, there && hh < z);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (h + u * per >= z) break;
                const int hh = h + g + u * per;
                float x[8], xp[8], r = 1.f;
                unpack8<BF16>(v[u], x);
                partners<D, BF16, MODE>(sh, p, v[u], l, src_lane, x, xp);
                if (w) {
                    float s = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) s = fmaf(x[e], x[e], s);
                    r = rsqrtf(group_sum<D>(s) * (1.f / D) + p.eps);
                }
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = r * fmaf(x[e], A[e], xp[e] * Bc[e]);
                if (store && hh < z) *reinterpret_cast<uint4 *>(dst + hh * dst_head) = pack8<BF16>(y);
            }
        }
    };
    rows(p.q, p.q_out, p.wq, 0, p.H, false);
    rows(p.k, p.k_out, p.wk, p.H, p.H_kv, PAGED);
    if constexpr (PAGED) {
        const int first = p.H + p.H_kv;
        const int a = max(h0 - first, 0), z = min(h1 - first, p.H_v);
        if (there && sh.cache_off[t] >= 0)
            for (int h = a + g; h < z; h += per)
                *reinterpret_cast<uint4 *>(p.vc + sh.cache_off[t] + h * p.head_stride + 8 * l) =
                    load_row(p.v.p + n * p.v.token + h * p.v.head + 8 * l, true);
    }
}

// Backward: dx of every row, and per block the sums of u z over its rows. A block walks
// tiles blockIdx.x, + gridDim.x, ...: the split depends on the sizes alone.
template <int D, bool BF16, int MODE>
__global__ void __launch_bounds__(kThreads) fa_norm_rope_bwd_kernel(const Params p) {
    using G = Geometry<D>;
    __shared__ Shared<D> sh;
    const int T = p.T, per = G::kGroups / T;
    const int group = threadIdx.x / G::kLanes, l = threadIdx.x % G::kLanes;
    const int t = group / per, g = group % per;
    const int src_lane = (threadIdx.x & 31) - l + partner<MODE>(8 * l, p.half_r) / 8;
    constexpr int U = 2;
    float dwq[8], dwk[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.f;

    for (long long x = blockIdx.x; x < p.tiles; x += gridDim.x) {
        const long long tile = x / p.chunks;
        const int h0 = static_cast<int>(x % p.chunks) * p.chunk, h1 = h0 + p.chunk;
        __syncthreads();
        places<D, false>(sh, p, tile * T, T);
        __syncthreads();
        angles<D>(sh, p, T);
        __syncthreads();
        const long long m = tile * T + t;
        const bool there = m < p.tokens;
        const long long b = m / p.N, n = m - b * p.N;
        float C[8], S[8];
        coefficients<D, MODE>(sh, p, t, l, C, S);
        auto rows = [&](const Rows &in, const Rows &dy, const Rows &dx, const uint16_t *w, int first,
                        int heads, float (&dw)[8]) {
            const int a = max(h0 - first, 0), z = min(h1 - first, heads);
            if (a >= z) return;
            float wt[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) wt[e] = w ? load1<BF16>(w + 8 * l + e) : 1.f;
            const uint16_t *xs = w ? in.p + b * in.batch + n * in.token + 8 * l : nullptr;
            const uint16_t *ys = dy.p + b * dy.batch + n * dy.token + 8 * l;
            uint16_t *ds = dx.p + b * dx.batch + n * dx.token + 8 * l;
            for (int h = a; h < z; h += per * U) {
                uint4 vy[U], vx[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int hh = h + g + u * per;
                    vy[u] = load_row(ys + hh * dy.head, there && hh < z);
                    vx[u] = w ? load_row(xs + hh * in.head, there && hh < z) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (h + u * per >= z) break;
                    const int hh = h + g + u * per;
                    float y[8], yp[8], o[8];
                    unpack8<BF16>(vy[u], y);
                    partners<D, BF16, MODE>(sh, p, vy[u], l, src_lane, y, yp);
                    // the transposed rotation: the sine's sign is the other one
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] = fmaf(y[e], C[e], -(yp[e] * S[e]));
                    if (w) {
                        float xx[8], s = 0.f, c = 0.f;
                        unpack8<BF16>(vx[u], xx);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            s = fmaf(xx[e], xx[e], s);
                            c = fmaf(o[e] * wt[e], xx[e], c);
                        }
                        const float r = rsqrtf(group_sum<D>(s) * (1.f / D) + p.eps);
                        const float k = group_sum<D>(c) * (1.f / D) * r * r;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            dw[e] = fmaf(o[e], xx[e] * r, dw[e]);
                            o[e] = r * fmaf(-k, xx[e], o[e] * wt[e]);
                        }
                    }
                    if (there && hh < z) *reinterpret_cast<uint4 *>(ds + hh * dx.head) = pack8<BF16>(o);
                }
            }
        };
        rows(p.q, p.q_out, p.dq, p.wq, 0, p.H, dwq);
        rows(p.k, p.k_out, p.dk, p.wk, p.H, p.H_kv, dwk);
    }
    if (p.part == nullptr) return;
    auto reduce = [&](const float (&dw)[8], int which) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) sh.red[threadIdx.x * 8 + e] = dw[e];
        __syncthreads();
        if (threadIdx.x < D) {
            float s = 0.f;
            for (int r = 0; r < G::kGroups; ++r) s += sh.red[r * D + threadIdx.x];
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
