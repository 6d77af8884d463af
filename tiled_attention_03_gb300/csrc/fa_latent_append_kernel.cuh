// fa_latent_append_kernel.cuh -- the append of new tokens to a paged cache of latent rows: the
// latent normalised, the rotary part of the key and those of the queries rotated.
//
// An item is one token's row of the cache, or up to kHeads of its queries' rotary parts; a warp
// takes an equal share of the line of items, so that a token's place in the cache and its angles
// are found once for its items of the warp. With r = 1 / sqrt(mean(c^2) + eps) over the DL
// latent elements the row is (c r w, rotated k_rope); rotations are those of fa_rope_kernel.cuh
// (exact phases, a row of 64 elements to 8 lanes, partners read from a copy in shared memory).
// The loads of an item start before its place is searched for and its angles are computed.
//
// What bounds it: instructions for prompts (24 prompts of 1-2000 tokens, 12 heads, DL = 256, in
// 15.5 us, 3.5 TB/s; 20.4 with items dealt in turn, each finding its own place and angles; 15.9
// with the next item's loads ahead, which cost registers and with them warps), and for single
// tokens the latency of place, page and angles (3.3 us).
#pragma once

#include <cstdint>

#include "fa_pdl.cuh"
#include "fa_rope_kernel.cuh"

namespace fa {
namespace latent {

constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kSteps = 4;           // rows of queries per lane and item
constexpr int kHeads = 4 * kSteps;  // heads per item
// blocks an SM holds at once, by their registers (80 and 110): 24 prompts of 1-2000 tokens 15.4 us at
// DL = 256, with four 20.4; 22.0 at DL = 512, with three 26.4
constexpr int blocks_per_sm(int64_t dl) { return dl == 512 ? 2 : 3; }

struct AppendParams {
    rope::Params r;  // rotation, batch and pages; q and q_out
    const uint16_t *c, *k;
    long long c_token, k_token;
    uint16_t *data;
    int parts;        // items per token: its row, and its queries kHeads at a time
    long long items;
};

template <int DL, bool BF16, int MODE>
__global__ void __launch_bounds__(kAppendThreads) fa_latent_append_kernel(const AppendParams p) {
    using namespace rope;
    constexpr int kPer = DL / 8;                      // 16-byte pieces of a latent row
    constexpr int kOwn = kPer > 32 ? kPer / 32 : 1;   // of a lane
    static_assert(kOwn <= kSteps, "loads of an item");
    __shared__ uint4 stage_all[kAppendWarps][kSteps][32];
    __shared__ __align__(16) float cs_all[kAppendWarps][2][kMaxPairs];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane & 7, g = lane >> 3;
    uint4(&stage)[kSteps][32] = stage_all[warp];
    float(&cs)[2][kMaxPairs] = cs_all[warp];
    const int half_r = p.r.half_r;
    const int partner_l = MODE == kLane ? partner<MODE>(8 * l, half_r) / 8 : l;
    after_previous();
    let_next_start();
    // this warp's items: the w-th of equal shares of their line
    const long long w = static_cast<long long>(blockIdx.x) * kAppendWarps + warp;
    const long long warps = static_cast<long long>(gridDim.x) * kAppendWarps;
    const long long begin = p.items * w / warps, end = p.items * (w + 1) / warps;
    if (begin >= end) return;
    int m = static_cast<int>(begin / p.parts), part = static_cast<int>(begin - static_cast<long long>(m) * p.parts);
    uint4 in[kSteps], k_in = make_uint4(0, 0, 0, 0);
    auto load = [&](int m, int part, uint4(&in)[kSteps], uint4 &k_in) {
        if (part == 0) {
            const uint4 *src = reinterpret_cast<const uint4 *>(p.c + m * p.c_token);
#pragma unroll
            for (int x = 0; x < kOwn; ++x)
                in[x] = lane + 32 * x < kPer ? src[lane + 32 * x] : make_uint4(0, 0, 0, 0);
            if (g == 0) k_in = reinterpret_cast<const uint4 *>(p.k + m * p.k_token)[l];
        } else {
            const int h0 = (part - 1) * kHeads + g;
            const uint16_t *src = p.r.q.p + m * p.r.q.token + h0 * p.r.q.head + 8 * l;
#pragma unroll
            for (int x = 0; x < kSteps; ++x)
                if (h0 + 4 * x < p.r.H) in[x] = *reinterpret_cast<const uint4 *>(src + 4 * x * p.r.q.head);
        }
    };
    int placed = -1;
    Place where{0, false, -1};
    f2 C[4], S[4];
    for (long long i = begin; i < end; ++i, part = part + 1 < p.parts ? part + 1 : 0, m += part == 0) {
        load(m, part, in, k_in);
        const int h0 = (part - 1) * kHeads + g;
        if (m != placed) {
            placed = m;
            where = place<true>(p.r, m, 0);
            if (half_r > 0) {
                angles(cs, p.r, where.pos);
                coefficients<MODE, false>(cs, half_r, l, C, S);
            }
        }
        // a row's 8 elements of this lane from its staged copy, rotated
        auto rotated = [&](const uint4 *at) -> uint4 {
            f2 x[4], xp[4];
            read_row<64, BF16, MODE>(at, half_r, l, partner_l, x, xp);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = fma2(xp[e], S[e], mul2(x[e], C[e]));
            return pack8<BF16>(x);
        };
        if (part == 0) {
            if (half_r > 0) {
                stage[0][lane] = k_in;
                __syncwarp();
                k_in = rotated(&stage[0][lane]);
                __syncwarp();
            }
            if (p.r.wk != nullptr) {
                float sum = 0.f;
                f2 x[kOwn][4];
#pragma unroll
                for (int y = 0; y < kOwn; ++y) {
                    unpack8<BF16>(in[y], x[y]);
                    sum += dot8(x[y], x[y]);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const f2 inv = both(rsqrtf(sum * (1.f / DL) + p.r.eps));
#pragma unroll
                for (int y = 0; y < kOwn; ++y) {
                    f2 w[4];
                    if (lane + 32 * y < kPer) {
                        weights<BF16>(p.r.wk, lane + 32 * y, w);
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[y][e] = mul2(mul2(x[y][e], inv), w[e]);
                        in[y] = pack8<BF16>(x[y]);
                    }
                }
            }
            if (where.slot >= 0) {
                uint4 *dst = reinterpret_cast<uint4 *>(p.data + where.slot);
#pragma unroll
                for (int x = 0; x < kOwn; ++x)
                    if (lane + 32 * x < kPer) dst[lane + 32 * x] = in[x];
                if (g == 0) dst[kPer + l] = k_in;
            }
        } else if (where.live) {
            if (half_r > 0) {
#pragma unroll
                for (int x = 0; x < kSteps; ++x) stage[x][lane] = in[x];
                __syncwarp();
            }
            uint16_t *dst = p.r.q_out.p + m * p.r.q_out.token + h0 * p.r.q_out.head + 8 * l;
#pragma unroll
            for (int x = 0; x < kSteps; ++x)
                if (h0 + 4 * x < p.r.H)
                    *reinterpret_cast<uint4 *>(dst + 4 * x * p.r.q_out.head) =
                        half_r > 0 ? rotated(&stage[x][lane]) : in[x];
            __syncwarp();
        }
    }
}

}  // namespace latent
}  // namespace fa
