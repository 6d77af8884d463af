// fa_rope_api.cu -- fa_rope_steps, fa_qk_norm_rope, fa_qk_norm_rope_backward and
// fa_paged_append: argument checks and launches of the kernels of fa_rope_kernel.cuh.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_host.h"
#include "fa_paged_host.h"
#include "fa_pdl.cuh"
#include "fa_rope_kernel.cuh"

namespace {

using fa::rope::Params;
using fa::rope::Rows;

constexpr int64_t kLimit = int64_t{1} << 29;  // tokens, and heads of a call

// One tensor of a call: its sizes, whether it is written, and the tensor it may be in
// place of (an index into the list; -1: none).
struct Tensor {
    const fa_rows *r;
    int64_t B, heads, N;
    bool written;
    int twin;
};

bool there(const fa_rows *r) { return r != nullptr && r->data != nullptr; }

// Elements from the first to the last of a tensor, or 0 when that does not fit 2^60.
int64_t extent(const Tensor &t, int64_t d) {
    const int64_t st[3] = {t.r->batch, t.r->head, t.r->token}, n[3] = {t.B, t.heads, t.N};
    double e = 0;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1) e += static_cast<double>(n[i] - 1) * static_cast<double>(st[i]);
    if (e > 1e18) return 0;
    int64_t sum = d;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1) sum += (n[i] - 1) * st[i];
    return sum;
}

// Whether no two elements of a written tensor share a place.
bool injective(const Tensor &t, int64_t d) {
    const int64_t n[3] = {t.B, t.heads, t.N}, st[3] = {t.r->batch, t.r->head, t.r->token};
    return fa_host::span_apart(n, st, d) > 0;
}

// Slices of one fused buffer: equal strides of tokens and batch entries (those there are
// more than one of), the larger a multiple of the smaller, s; each tensor's part of a
// token is shorter than s, and the two parts lie at different places modulo s.
bool interleaved(const Tensor &a, const Tensor &b, int64_t d) {
    if ((a.N > 1 && a.r->token != b.r->token) || (a.B > 1 && a.r->batch != b.r->batch)) return false;
    const int64_t token = a.N > 1 ? a.r->token : 0, batch = a.B > 1 ? a.r->batch : 0;
    const int64_t s = token > 0 && (batch == 0 || token < batch) ? token : batch;
    if (s < 1 || token % s != 0 || batch % s != 0) return false;
    const int64_t span_a = a.heads > 1 ? (a.heads - 1) * a.r->head + d : d;
    const int64_t span_b = b.heads > 1 ? (b.heads - 1) * b.r->head + d : d;
    const intptr_t bytes = reinterpret_cast<intptr_t>(b.r->data) - reinterpret_cast<intptr_t>(a.r->data);
    int64_t off = (bytes / 2) % s;
    if (off < 0) off += s;
    return off >= span_a && off + span_b <= s;
}

// The descriptors of a call: alignment, strides, and what is written overlaps nothing
// else (but the tensor it replaces, or its neighbours in a fused buffer).
fa_status check_tensors(const Tensor *t, int count, int64_t d) {
    for (int i = 0; i < count; ++i) {
        if (!there(t[i].r)) continue;
        const fa_rows &r = *t[i].r;
        if (!fa_host::aligned16(r.data)) return FA_ERR_INVALID_ARG;
        const int64_t st[3] = {r.batch, r.head, r.token}, n[3] = {t[i].B, t[i].heads, t[i].N};
        for (int x = 0; x < 3; ++x)  // the stride of a single entry does not matter
            if (n[x] > 1 && (st[x] < 0 || st[x] % 8 != 0 || st[x] >= (int64_t{1} << 40)))
                return FA_ERR_INVALID_ARG;
        if (extent(t[i], d) == 0) return FA_ERR_UNSUPPORTED;
        if (t[i].written && !injective(t[i], d)) return FA_ERR_INVALID_ARG;
    }
    for (int i = 0; i < count; ++i) {
        if (!there(t[i].r) || !t[i].written) continue;
        for (int j = 0; j < count; ++j) {
            if (j == i || !there(t[j].r) || (t[j].written && j < i)) continue;
            const fa_rows &a = *t[i].r, &b = *t[j].r;
            if (!fa_host::overlaps(a.data, static_cast<size_t>(extent(t[i], d)) * 2, b.data,
                                   static_cast<size_t>(extent(t[j], d)) * 2))
                continue;
            if (j == t[i].twin && a.data == b.data && (t[i].B == 1 || a.batch == b.batch) &&
                (t[i].heads == 1 || a.head == b.head) && (t[i].N == 1 || a.token == b.token))
                continue;
            if (!interleaved(t[i], t[j], d)) return FA_ERR_INVALID_ARG;
        }
    }
    return FA_OK;
}

// Buffers that are only read (small arrays) against every written tensor.
bool hits_written(const void *p, size_t n, const Tensor *t, int count, int64_t d) {
    if (p == nullptr || n == 0) return false;
    for (int i = 0; i < count; ++i)
        if (there(t[i].r) && t[i].written &&
            fa_host::overlaps(p, n, t[i].r->data, static_cast<size_t>(extent(t[i], d)) * 2))
            return true;
    return false;
}

fa_status check_rope(const fa_norm_rope &r, int64_t d) {
    if (r.rotary_dim < 0 || r.rotary_dim > d || r.rotary_dim % 2 != 0) return FA_ERR_INVALID_ARG;
    if (r.layout != FA_ROPE_HALF && r.layout != FA_ROPE_INTERLEAVED) return FA_ERR_INVALID_ARG;
    if (r.rotary_dim > 0 && (r.steps == nullptr || !fa_host::aligned16(r.steps))) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(r.magnitude) || !std::isfinite(r.eps) || r.eps < 0.f) return FA_ERR_INVALID_ARG;
    if (!fa_host::aligned16(r.q_weight) || !fa_host::aligned16(r.k_weight)) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

bool known(int64_t d) { return d == 32 || d == 64 || d == 128 || d == 256; }

fa_status device_of(int *dev, fa_host::DeviceInfo *di) {
    if (cudaGetDevice(dev) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    *di = fa_host::device_info(*dev);
    if (di->err == cudaErrorInvalidDevice) return FA_ERR_UNSUPPORTED;
    if (di->err != cudaSuccess) return FA_ERR_CUDA;
    return di->cc_major == 10 && di->cc_minor == 3 ? FA_OK : FA_ERR_UNSUPPORTED;
}

bool absent_or_on(const void *p, int dev) { return p == nullptr || fa_host::on_device(p, dev); }

// The stride of a dimension of one entry may be anything: 0 here, so that the kernels see
// none below 0.
Rows rows_of(const fa_rows *r, int64_t B, int64_t heads, int64_t N) {
    if (!there(r)) return Rows{nullptr, 0, 0, 0};
    return Rows{static_cast<uint16_t *>(r->data), B > 1 ? r->batch : 0, heads > 1 ? r->head : 0,
                N > 1 ? r->token : 0};
}

void set_rope(Params &p, const fa_norm_rope &r) {
    p.steps = reinterpret_cast<const unsigned long long *>(r.steps);
    p.half_r = static_cast<int>(r.rotary_dim / 2);
    p.magnitude = r.magnitude;
    p.eps = r.eps;
    p.wq = static_cast<const uint16_t *>(r.q_weight);
    p.wk = static_cast<const uint16_t *>(r.k_weight);
}

int mode_of(const fa_norm_rope &r) {
    if (r.layout == FA_ROPE_INTERLEAVED) return fa::rope::kBeside;
    return r.rotary_dim % 16 == 0 ? fa::rope::kLane : fa::rope::kAnywhere;
}

// The stages of a token, `rows` rows per group each, and the blocks of a launch. Up to
// `resident` blocks (what the SMs hold at once) every warp takes a stage at least; more,
// up to `most`, in whole waves of them, only where their warps still have kLongShare stages each:
// blocks that start as others end even out what the SMs get, but a share that is shorter is
// mostly its start (24 prompts appended at d 64: 25.6 us with shares of 28, 29.5 us with 14),
// and blocks of equal length past the last whole wave run by themselves (forward, 32 + 8 heads,
// d 128: 69,000 stages in a little over a wave took 36.8 us, in one 24.7). Against resident blocks
// alone, forward at d 128: 32 + 32 heads 260,000 stages 85.6 and 96.2 us, 137,000 47.3 and 48.1;
// 32 + 8 heads 300,000 stages 97.0 and 105.2; tokens of few stages pay for the more starts (16 +
// 2 heads, 5 stages a token, 300,000 in all: 112.3 and 109.2).
// The backward keeps to resident blocks: its longer start and end and the sums of more
// blocks cost more than they even out (92 us, 97 to 104 us with more).
constexpr int kLongShare = 28;
unsigned set_stages(Params &p, int64_t d, int rows, long long resident, long long most) {
    const int heads = static_cast<int>(256 / d) * rows;
    auto stages = [heads](int h) { return (h + heads - 1) / heads; };
    p.s_q = stages(p.H);
    p.s_k = stages(p.H_kv);
    p.s_v = stages(p.H_v);
    p.stages = static_cast<long long>(p.tokens) * (p.s_q + p.s_k + p.s_v);
    const long long each = (p.stages + fa::rope::kWarps - 1) / fa::rope::kWarps;
    const long long waves = p.stages / (fa::rope::kWarps * kLongShare * resident);
    const long long blocks = waves > 1 ? waves * resident : each < resident ? each : resident;
    return static_cast<unsigned>(blocks < most ? blocks : most);
}

template <int D, bool BF16, bool PAGED>
cudaError_t forward_mode(const Params &p, int mode, unsigned g, cudaStream_t st) {
    using namespace fa::rope;
    auto *k = mode == kBeside ? fa_norm_rope_kernel<D, BF16, kBeside, PAGED>
              : mode == kLane ? fa_norm_rope_kernel<D, BF16, kLane, PAGED>
                              : fa_norm_rope_kernel<D, BF16, kAnywhere, PAGED>;
    return fa::launch_after(k, g, kThreads, 0, st, p);
}
template <int D, bool BF16>
cudaError_t backward_mode(const Params &p, int mode, unsigned g, cudaStream_t st) {
    using namespace fa::rope;
    auto *k = mode == kBeside ? fa_norm_rope_bwd_kernel<D, BF16, kBeside>
              : mode == kLane ? fa_norm_rope_bwd_kernel<D, BF16, kLane>
                              : fa_norm_rope_bwd_kernel<D, BF16, kAnywhere>;
    return fa::launch_after(k, g, kThreads, 0, st, p);
}
template <bool PAGED>
cudaError_t forward(const Params &p, int64_t d, bool bf16, int mode, unsigned g, cudaStream_t st) {
    switch (d) {
        case 32: return bf16 ? forward_mode<32, true, PAGED>(p, mode, g, st) : forward_mode<32, false, PAGED>(p, mode, g, st);
        case 64: return bf16 ? forward_mode<64, true, PAGED>(p, mode, g, st) : forward_mode<64, false, PAGED>(p, mode, g, st);
        case 128: return bf16 ? forward_mode<128, true, PAGED>(p, mode, g, st) : forward_mode<128, false, PAGED>(p, mode, g, st);
        default: return bf16 ? forward_mode<256, true, PAGED>(p, mode, g, st) : forward_mode<256, false, PAGED>(p, mode, g, st);
    }
}
cudaError_t backward(const Params &p, int64_t d, bool bf16, int mode, unsigned g, cudaStream_t st) {
    switch (d) {
        case 32: return bf16 ? backward_mode<32, true>(p, mode, g, st) : backward_mode<32, false>(p, mode, g, st);
        case 64: return bf16 ? backward_mode<64, true>(p, mode, g, st) : backward_mode<64, false>(p, mode, g, st);
        case 128: return bf16 ? backward_mode<128, true>(p, mode, g, st) : backward_mode<128, false>(p, mode, g, st);
        default: return bf16 ? backward_mode<256, true>(p, mode, g, st) : backward_mode<256, false>(p, mode, g, st);
    }
}

// Resident blocks per SM (the kernels' launch bounds).
constexpr int kBlocksPerSm = 2;
// Blocks of a backward launch at most: each leaves 2 d partial sums.
constexpr int kBackwardBlocksPerSm = 2;

// What the two dense calls check alike: sizes, and which of q and k are there.
fa_status check_sizes(int64_t B, int64_t *H, int64_t *H_kv, int64_t N, int64_t d, fa_dtype dtype,
                      const fa_rows *q, const fa_rows *k) {
    if (B < 1 || N < 1 || d < 1) return FA_ERR_INVALID_ARG;
    if (!there(q)) *H = 0;
    if (!there(k)) *H_kv = 0;
    if (*H == 0 && *H_kv == 0) return FA_ERR_INVALID_ARG;
    if ((there(q) && *H < 1) || (there(k) && *H_kv < 1)) return FA_ERR_INVALID_ARG;
    if (dtype != FA_DTYPE_FP16 && dtype != FA_DTYPE_BF16) return FA_ERR_INVALID_ARG;
    if (!known(d)) return FA_ERR_UNSUPPORTED;
    if (B > kLimit || N > kLimit || B * N > kLimit || *H > (1 << 20) || *H_kv > (1 << 20))
        return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

}  // namespace

extern "C" {

fa_status fa_rope_steps(const double *frequencies, int64_t n, uint64_t *steps) {
    if (frequencies == nullptr || steps == nullptr || n < 1) return FA_ERR_INVALID_ARG;
    for (int64_t j = 0; j < n; ++j)
        if (!std::isfinite(frequencies[j]) || !(std::fabs(frequencies[j]) < 1048576.0))
            return FA_ERR_INVALID_ARG;
    for (int64_t j = 0; j < n; ++j) {
        const double turns = std::fabs(frequencies[j]) * 0.15915494309189533577;  // 1 / (2 pi)
        const double part = turns - std::floor(turns);  // exact (turns >= 0): [0, 1)
        const double fixed = std::nearbyint(part * 18446744073709551616.0);
        const uint64_t step = fixed >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(fixed);
        steps[j] = frequencies[j] < 0 ? 0 - step : step;
    }
    return FA_OK;
}

fa_status fa_qk_norm_rope(const fa_rows *q, const fa_rows *k, const fa_rows *q_out,
                          const fa_rows *k_out, const fa_norm_rope *rope, const int32_t *positions,
                          int64_t B, int64_t H, int64_t H_kv, int64_t N, int64_t d, fa_dtype dtype,
                          void *stream) {
    if (rope == nullptr || there(q) != there(q_out) || there(k) != there(k_out)) return FA_ERR_INVALID_ARG;
    fa_status s = check_sizes(B, &H, &H_kv, N, d, dtype, q, k);
    if (s == FA_OK) s = check_rope(*rope, d);
    if (s != FA_OK) return s;
    const Tensor t[] = {{q, B, H, N, false, -1}, {k, B, H_kv, N, false, -1},
                        {q_out, B, H, N, true, 0}, {k_out, B, H_kv, N, true, 1}};
    s = check_tensors(t, 4, d);
    if (s != FA_OK) return s;
    if (!fa_host::aligned4(positions)) return FA_ERR_INVALID_ARG;
    const size_t wbytes = static_cast<size_t>(d) * 2;
    if (hits_written(positions, static_cast<size_t>(B * N) * 4, t, 4, d) ||
        hits_written(rope->rotary_dim > 0 ? rope->steps : nullptr,
                     static_cast<size_t>(rope->rotary_dim) * 4, t, 4, d) ||
        hits_written(rope->q_weight, wbytes, t, 4, d) || hits_written(rope->k_weight, wbytes, t, 4, d))
        return FA_ERR_INVALID_ARG;
    int dev = 0;
    fa_host::DeviceInfo di;
    s = device_of(&dev, &di);
    if (s != FA_OK) return s;
    for (const Tensor &x : t)
        if (there(x.r) && !fa_host::on_device(x.r->data, dev)) return FA_ERR_INVALID_ARG;
    if (!absent_or_on(positions, dev) || !absent_or_on(rope->rotary_dim > 0 ? rope->steps : nullptr, dev) ||
        !absent_or_on(rope->q_weight, dev) || !absent_or_on(rope->k_weight, dev))
        return FA_ERR_INVALID_ARG;
    fa_host::take_fault_position();  // nothing here waits: an armed test hook is spent
    Params p{};
    p.q = rows_of(q, B, H, N);
    p.k = rows_of(k, B, H_kv, N);
    p.q_out = rows_of(q_out, B, H, N);
    p.k_out = rows_of(k_out, B, H_kv, N);
    p.H = static_cast<int>(H);
    p.H_kv = static_cast<int>(H_kv);
    p.N = static_cast<int>(N);
    p.tokens = static_cast<int>(B * N);
    p.positions = positions;
    set_rope(p, *rope);
    const unsigned blocks = set_stages(p, d, fa::rope::kRows, di.sm_count * kBlocksPerSm,
                                       int64_t{1} << 30);
    if (forward<false>(p, d, dtype == FA_DTYPE_BF16, mode_of(*rope), blocks,
                       static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return FA_ERR_CUDA;
    fa_host::count_launches(1);
    return FA_OK;
}

size_t fa_qk_norm_rope_backward_workspace_bytes(int64_t d) {
    if (!known(d)) return 0;
    return static_cast<size_t>(fa_host::sm_count_or_default()) * kBackwardBlocksPerSm * 2 * static_cast<size_t>(d) * sizeof(float);
}

fa_status fa_qk_norm_rope_backward(const fa_rows *q, const fa_rows *k, const fa_rows *dq_out,
                                   const fa_rows *dk_out, const fa_rows *dq, const fa_rows *dk,
                                   float *dq_weight, float *dk_weight, const fa_norm_rope *rope,
                                   const int32_t *positions, int64_t B, int64_t H, int64_t H_kv,
                                   int64_t N, int64_t d, fa_dtype dtype, void *workspace,
                                   size_t workspace_bytes, void *stream) {
    if (rope == nullptr || there(dq_out) != there(dq) || there(dk_out) != there(dk)) return FA_ERR_INVALID_ARG;
    fa_status s = check_sizes(B, &H, &H_kv, N, d, dtype, dq, dk);
    if (s == FA_OK) s = check_rope(*rope, d);
    if (s != FA_OK) return s;
    // a weight needs its input and its gradient; without one neither is used
    const bool wq = H > 0 && rope->q_weight != nullptr, wk = H_kv > 0 && rope->k_weight != nullptr;
    if (wq != (dq_weight != nullptr) || wk != (dk_weight != nullptr)) return FA_ERR_INVALID_ARG;
    if ((wq && !there(q)) || (wk && !there(k))) return FA_ERR_INVALID_ARG;
    const fa_rows *xq = wq ? q : nullptr, *xk = wk ? k : nullptr;
    const Tensor t[] = {{xq, B, H, N, false, -1}, {xk, B, H_kv, N, false, -1},
                        {dq_out, B, H, N, false, -1}, {dk_out, B, H_kv, N, false, -1},
                        {dq, B, H, N, true, 2}, {dk, B, H_kv, N, true, 3}};
    s = check_tensors(t, 6, d);
    if (s != FA_OK) return s;
    if (!fa_host::aligned4(positions) || !fa_host::aligned4(dq_weight) || !fa_host::aligned4(dk_weight))
        return FA_ERR_INVALID_ARG;
    const size_t need = fa_qk_norm_rope_backward_workspace_bytes(d);
    if ((wq || wk) && (workspace == nullptr || !fa_host::aligned16(workspace) || workspace_bytes < need))
        return FA_ERR_INVALID_ARG;
    const size_t wbytes = static_cast<size_t>(d) * 2, gbytes = static_cast<size_t>(d) * 4;
    const struct {
        const void *p;
        size_t n;
        bool written;
    } small[] = {{positions, static_cast<size_t>(B * N) * 4, false},
                 {rope->rotary_dim > 0 ? rope->steps : nullptr, static_cast<size_t>(rope->rotary_dim) * 4, false},
                 {rope->q_weight, wbytes, false},
                 {rope->k_weight, wbytes, false},
                 {dq_weight, gbytes, true},
                 {dk_weight, gbytes, true},
                 {wq || wk ? workspace : nullptr, need, true}};
    for (int i = 0; i < 7; ++i) {
        if (hits_written(small[i].p, small[i].n, t, 6, d)) return FA_ERR_INVALID_ARG;
        if (!small[i].written || small[i].p == nullptr) continue;
        for (int j = 0; j < 7; ++j)
            if (j != i && small[j].p != nullptr &&
                fa_host::overlaps(small[i].p, small[i].n, small[j].p, small[j].n))
                return FA_ERR_INVALID_ARG;
        for (const Tensor &x : t)
            if (there(x.r) && fa_host::overlaps(small[i].p, small[i].n, x.r->data,
                                                static_cast<size_t>(extent(x, d)) * 2))
                return FA_ERR_INVALID_ARG;
    }
    int dev = 0;
    fa_host::DeviceInfo di;
    s = device_of(&dev, &di);
    if (s != FA_OK) return s;
    for (const Tensor &x : t)
        if (there(x.r) && !fa_host::on_device(x.r->data, dev)) return FA_ERR_INVALID_ARG;
    for (const auto &x : small)
        if (!absent_or_on(x.p, dev)) return FA_ERR_INVALID_ARG;
    fa_host::take_fault_position();  // nothing here waits: an armed test hook is spent
    Params p{};
    p.q = rows_of(xq, B, H, N);
    p.k = rows_of(xk, B, H_kv, N);
    p.q_out = rows_of(dq_out, B, H, N);
    p.k_out = rows_of(dk_out, B, H_kv, N);
    p.dq = rows_of(dq, B, H, N);
    p.dk = rows_of(dk, B, H_kv, N);
    p.H = static_cast<int>(H);
    p.H_kv = static_cast<int>(H_kv);
    p.N = static_cast<int>(N);
    p.tokens = static_cast<int>(B * N);
    p.positions = positions;
    set_rope(p, *rope);
    if (!wq) p.wq = nullptr;
    if (!wk) p.wk = nullptr;
    p.part = wq || wk ? static_cast<float *>(workspace) : nullptr;
    const unsigned blocks = set_stages(p, d, 1, di.sm_count * kBlocksPerSm, di.sm_count * kBackwardBlocksPerSm);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (backward(p, d, dtype == FA_DTYPE_BF16, mode_of(*rope), blocks, st) != cudaSuccess) return FA_ERR_CUDA;
    fa_host::count_launches(1);
    if (p.part != nullptr) {
        if (fa::launch_after(fa::rope::fa_norm_rope_sum_kernel, static_cast<unsigned>(2 * d / 32),
                             fa::rope::kSumThreads, 0, st, static_cast<const float *>(p.part),
                             static_cast<int>(blocks), static_cast<int>(d), dq_weight, dk_weight) != cudaSuccess)
            return FA_ERR_CUDA;
        fa_host::count_launches(1);
    }
    return FA_OK;
}

fa_status fa_paged_append(const fa_rows *q, const fa_rows *k, const fa_rows *v, const fa_rows *q_out,
                          const fa_paged_cache *cache, const int32_t *block_table, int64_t max_pages,
                          const int32_t *cu_seqlens_q, const int32_t *seqlens_k, int64_t B, int64_t H,
                          int64_t total_q, const fa_norm_rope *rope, void *stream) {
    if (cache == nullptr || B < 1 || total_q < 0 || max_pages < 0 || there(q) != there(q_out))
        return FA_ERR_INVALID_ARG;
    size_t cache_bytes = 0;
    fa_status s = fa_host::check_cache(*cache, &cache_bytes);
    if (s != FA_OK) return s;
    if (cache->k == cache->v) return FA_ERR_INVALID_ARG;  // a key and a value for each place
    const int64_t d = cache->d, H_kv = cache->H_kv;
    const fa_norm_rope plain{nullptr, 0, FA_ROPE_INTERLEAVED, 1.f, nullptr, nullptr, 0.f};
    const fa_norm_rope &r = rope ? *rope : plain;
    s = check_rope(r, d);
    if (s != FA_OK) return s;
    if (!there(q)) H = 0;
    if (there(q) && H < 1) return FA_ERR_INVALID_ARG;
    if (total_q == 0) return FA_OK;  // no new tokens: nothing to do
    if (!there(k) || !there(v) || !cu_seqlens_q || !seqlens_k || (!block_table && max_pages > 0))
        return FA_ERR_INVALID_ARG;
    if (!fa_host::aligned4(block_table) || !fa_host::aligned4(cu_seqlens_q) || !fa_host::aligned4(seqlens_k))
        return FA_ERR_INVALID_ARG;
    if (total_q > kLimit || B > kLimit || H > (1 << 20) || max_pages > kLimit ||
        max_pages * cache->page_size > (int64_t{1} << 31))
        return FA_ERR_UNSUPPORTED;
    const Tensor t[] = {{q, 1, H, total_q, false, -1}, {k, 1, H_kv, total_q, false, -1},
                        {v, 1, H_kv, total_q, false, -1}, {q_out, 1, H, total_q, true, 0}};
    s = check_tensors(t, 4, d);
    if (s != FA_OK) return s;
    // k and v of the cache may be interleaved with each other (as the caller lays them
    // out), but neither touches anything else
    const size_t wbytes = static_cast<size_t>(d) * 2;
    const struct {
        const void *p;
        size_t n;
    } small[] = {{r.rotary_dim > 0 ? r.steps : nullptr, static_cast<size_t>(r.rotary_dim) * 4},
                 {r.q_weight, wbytes},
                 {r.k_weight, wbytes},
                 {max_pages > 0 ? block_table : nullptr, static_cast<size_t>(B * max_pages) * 4},
                 {cu_seqlens_q, static_cast<size_t>(B + 1) * 4},
                 {seqlens_k, static_cast<size_t>(B) * 4}};
    for (const auto &x : small)
        if (hits_written(x.p, x.n, t, 4, d)) return FA_ERR_INVALID_ARG;
    for (const void *c : {cache->k, cache->v}) {
        for (const auto &x : small)
            if (x.p != nullptr && fa_host::overlaps(c, cache_bytes, x.p, x.n)) return FA_ERR_INVALID_ARG;
        for (const Tensor &x : t)
            if (there(x.r) && fa_host::overlaps(c, cache_bytes, x.r->data,
                                                static_cast<size_t>(extent(x, d)) * 2))
                return FA_ERR_INVALID_ARG;
    }
    int dev = 0;
    fa_host::DeviceInfo di;
    s = device_of(&dev, &di);
    if (s != FA_OK) return s;
    for (const Tensor &x : t)
        if (there(x.r) && !fa_host::on_device(x.r->data, dev)) return FA_ERR_INVALID_ARG;
    for (const auto &x : small)
        if (!absent_or_on(x.p, dev)) return FA_ERR_INVALID_ARG;
    if (!fa_host::on_device(cache->k, dev) || !fa_host::on_device(cache->v, dev)) return FA_ERR_INVALID_ARG;
    fa_host::take_fault_position();  // nothing here waits: an armed test hook is spent
    Params p{};
    p.q = rows_of(q, 1, H, total_q);
    p.k = rows_of(k, 1, H_kv, total_q);
    p.v = rows_of(v, 1, H_kv, total_q);
    p.q_out = rows_of(q_out, 1, H, total_q);
    p.H = static_cast<int>(H);
    p.H_kv = p.H_v = static_cast<int>(H_kv);
    p.N = static_cast<int>(total_q);
    p.tokens = static_cast<int>(total_q);
    set_rope(p, r);
    p.kc = static_cast<uint16_t *>(cache->k);
    p.vc = static_cast<uint16_t *>(cache->v);
    p.page_stride = cache->page_stride;
    p.token_stride = cache->token_stride;
    p.head_stride = cache->head_stride;
    p.cu_q = cu_seqlens_q;
    p.seq_k = seqlens_k;
    p.table = block_table;
    p.B = static_cast<int>(B);
    p.max_pages = static_cast<int>(max_pages);
    while ((int64_t{1} << p.page_log2) < cache->page_size) ++p.page_log2;
    p.num_pages = static_cast<int>(cache->num_pages);
    const unsigned blocks = set_stages(p, d, fa::rope::kRows, di.sm_count * kBlocksPerSm,
                                       int64_t{1} << 30);
    if (forward<true>(p, d, cache->dtype == FA_DTYPE_BF16, mode_of(r), blocks,
                      static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return FA_ERR_CUDA;
    fa_host::count_launches(1);
    return FA_OK;
}

}  // extern "C"
