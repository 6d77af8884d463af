// fa_paged_api.cu -- fa_forward_paged: argument checks, tensor maps and launches of the
// paged attention kernel and its merge (fa_paged_kernel.cuh).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "fa.h"
#include "fa_host.h"
#include "fa_paged_decode_kernel.cuh"
#include "fa_paged_host.h"
#include "fa_paged_kernel.cuh"

namespace {

using fa_host::align256;

constexpr int kMaxDevices = 64;

// Ticks of a decode worker's share at least: shorter ones cut a unit into more pieces to merge. Of 8,
// 4 and 16: 4 sequences of 60-1000 keys 12.4, 10.7 and 16.5 us, one of 10000 keys 18.9, 21.5 and
// 19.1, 32 of 4000 keys with one K/V head 18.8, 19.7 and 19.9.
constexpr int kMinTicks = 8;

struct Configured {
    std::once_flag once;
    cudaError_t err = cudaSuccess;
};
Configured g_configured[kMaxDevices];

// Shared memory of the kernel that holds both bodies.
template <int D>
constexpr int kEitherSmem = fa::paged::Smem<D>::kAlloc > fa::paged::Small<D>::kBytes ? fa::paged::Smem<D>::kAlloc
                                                                                     : fa::paged::Small<D>::kBytes;

template <int D, bool BF16>
cudaError_t opt_in() {
    cudaError_t e = cudaFuncSetAttribute(fa::paged::fa_paged_kernel<D, BF16>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, fa::paged::Smem<D>::kAlloc);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fa::paged::fa_paged_decode_kernel<D, BF16>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, fa::paged::Small<D>::kBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fa::paged::fa_paged_either_kernel<D, BF16>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kEitherSmem<D>);
    return e;
}

bool configured(int dev) {
    Configured &c = g_configured[dev];
    std::call_once(c.once, [&c] {
        cudaError_t e = opt_in<32, false>();
        if (e == cudaSuccess) e = opt_in<32, true>();
        if (e == cudaSuccess) e = opt_in<64, false>();
        if (e == cudaSuccess) e = opt_in<64, true>();
        if (e == cudaSuccess) e = opt_in<128, false>();
        if (e == cudaSuccess) e = opt_in<128, true>();
        if (e == cudaSuccess) e = opt_in<256, false>();
        if (e == cudaSuccess) e = opt_in<256, true>();
        c.err = e;
    });
    return c.err == cudaSuccess;
}

// Two partial results per worker, and what the merge needs to know of each. The chunk
// kernel has a worker of 128 rows per SM, the decode kernel eight (four at d = 256) of 16.
constexpr int kMaxWorkersPerSm = 8;
static_assert(fa::paged::kBM == kMaxWorkersPerSm * fa::paged::kSmallRows, "one layout for both kernels");
struct Layout {
    size_t lse, o, bytes;  // info at 0
};
Layout layout_of(int64_t d, int64_t sms) {
    const size_t rows = static_cast<size_t>(2 * sms) * fa::paged::kBM;
    Layout l;
    l.lse = align256(static_cast<size_t>(sms) * kMaxWorkersPerSm * sizeof(fa::paged::MergeInfo));
    l.o = l.lse + align256(rows * sizeof(float));
    l.bytes = l.o + rows * static_cast<size_t>(d) * sizeof(float);
    return l;
}

// What a call runs: decode, chunks, or whichever the device finds (see
// fa_paged_decode_kernel.cuh); and the merge.
struct Plan {
    bool decode, chunk;
    int max_new;
    unsigned merge_rows;  // blocks of the merge per decode unit
    fa::paged::SmallParams small;
    fa::paged::Params p;
    fa::paged::MergeParams merge;
    CUtensorMap q, k, v;
    unsigned sms;
};

template <int D, bool BF16>
cudaError_t launch(const Plan &x, cudaStream_t st) {
    using namespace fa::paged;
    using S = Small<D>;
    fa::paged::Params p = x.p;
    p.infos = x.decode ? S::kWarps : 1;
    const cudaError_t e =
        !x.chunk ? fa::launch_after(fa_paged_decode_kernel<D, BF16>, dim3(x.sms), S::kWarps * 32, S::kBytes, st, x.small)
        : !x.decode
            ? fa::launch_after(fa_paged_kernel<D, BF16>, dim3(x.sms), kThreads, Smem<D>::kAlloc, st, x.q, x.k, x.v, p)
            : fa::launch_after(fa_paged_either_kernel<D, BF16>, dim3(x.sms), kThreads, kEitherSmem<D>, st, x.q, x.k, x.v,
                               x.small, p, x.max_new);
    if (e != cudaSuccess) return e;
    // a block per worker; a unit of the chunk kernel has 128 rows to share among several
    const dim3 grid(x.decode ? x.sms * S::kWarps : x.sms, !x.chunk ? 1 : x.decode ? x.merge_rows : 16);
    return fa::launch_after(fa_paged_merge_kernel<D, BF16>, grid, kMergeWarps * 32, 0, st, x.merge);
}

fa_status run(const void *Q, void *O, float *LSE, const fa_paged_cache *cache, const int32_t *table,
              int64_t max_pages, const int32_t *cu_q, const int32_t *seq_k, int64_t B, int64_t H,
              int64_t total_q, float scale, fa_mask_mode mask_mode, int64_t window_left,
              int64_t window_right, void *workspace, size_t workspace_bytes, void *stream) {
    // ---- host-side checks: nothing is enqueued on failure
    if (cache == nullptr || B < 1 || H < 1 || total_q < 0 || max_pages < 0) return FA_ERR_INVALID_ARG;
    size_t cache_bytes = 0;
    const fa_status cs = fa_host::check_cache(*cache, &cache_bytes);
    if (cs != FA_OK) return cs;
    const int64_t d = cache->d, H_kv = cache->H_kv;
    if (H % H_kv != 0) return FA_ERR_INVALID_ARG;
    if (mask_mode != FA_MASK_NONE && mask_mode != FA_MASK_CAUSAL && mask_mode != FA_MASK_WINDOW)
        return FA_ERR_INVALID_ARG;
    if (mask_mode == FA_MASK_WINDOW && (window_left < 0 || window_right < 0)) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
    if (total_q == 0) return FA_OK;  // no query rows: nothing to do
    if (!Q || !O || !LSE || !cu_q || !seq_k || (!table && max_pages > 0)) return FA_ERR_INVALID_ARG;
    if (!fa_host::aligned16(Q) || !fa_host::aligned32(O) || !fa_host::aligned4(LSE) ||
        !fa_host::aligned4(cu_q) || !fa_host::aligned4(seq_k) || !fa_host::aligned4(table))
        return FA_ERR_INVALID_ARG;
    // Heads of a unit: all query heads of one K/V head, or a divisor of them.
    const int64_t group = H / H_kv;
    int64_t pf = group;
    if (pf > fa::paged::kBM)
        for (pf = fa::paged::kBM; group % pf != 0;) --pf;
    // Few tokens: the decode kernel, whose units re-read a sequence's keys kMaxReads times at
    // most. A few tokens per sequence on average: whichever kernel suits the longest, as it
    // turns out on the device (with no more tokens than sequences, too: most may have none).
    constexpr int64_t kMaxReads = 2;
    const bool small = pf <= fa::paged::kSmallRows;
    const int64_t tpt_small = small ? fa::paged::kSmallRows / pf : 0, tpt = fa::paged::kBM / pf;
    const int64_t max_new = kMaxReads * tpt_small;
    const bool steps_only = small && total_q <= max_new;
    const bool either = small && !steps_only && total_q <= B * tpt_small;
    const bool decode = steps_only || either, chunked = !steps_only;
    const int64_t spaces = H / pf;
    const int64_t max_keys = max_pages * cache->page_size;
    // Size limits of this implementation: 32-bit token and key indices, and a line of
    // work below 2^31 tiles.
    const int64_t kLimit = int64_t{1} << 29;
    if (total_q > kLimit || max_pages > kLimit || max_keys > kLimit || B > kLimit || H > kLimit ||
        total_q * H > 0x7fffffffLL)
        return FA_ERR_UNSUPPORTED;
    auto line = [&](int64_t tokens, int64_t keys) {  // ticks of a line of work at most
        return static_cast<double>(spaces) * static_cast<double>(total_q / tokens + B) *
               static_cast<double>(max_keys / keys + 8);
    };
    if ((decode && line(tpt_small, d <= 64 ? 32 : 16) > 2147483647.0) ||
        (chunked && line(tpt, fa::paged::bn(static_cast<int>(d))) > 2147483647.0))
        return FA_ERR_UNSUPPORTED;
    const Layout lay = layout_of(d, fa_host::sm_count_or_default());
    if (workspace == nullptr || !fa_host::aligned32(workspace) || workspace_bytes < lay.bytes)
        return FA_ERR_INVALID_ARG;
    const size_t tbytes = static_cast<size_t>(total_q) * H * d * 2;
    const size_t lbytes = static_cast<size_t>(total_q) * H * sizeof(float);
    const size_t cubytes = static_cast<size_t>(B + 1) * 4, skbytes = static_cast<size_t>(B) * 4;
    const size_t tabytes = static_cast<size_t>(B) * max_pages * 4;
    struct Buf {
        const void *p;
        size_t n;
    };
    const Buf in[] = {{Q, tbytes}, {cache->k, cache_bytes}, {cache->v, cache_bytes},
                      {cu_q, cubytes}, {seq_k, skbytes}, {table, tabytes}};
    const Buf out[] = {{O, tbytes}, {LSE, lbytes}, {workspace, lay.bytes}};
    for (int i = 0; i < 3; ++i) {
        for (const Buf &b : in)
            if (b.n > 0 && fa_host::overlaps(out[i].p, out[i].n, b.p, b.n)) return FA_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (fa_host::overlaps(out[i].p, out[i].n, out[j].p, out[j].n)) return FA_ERR_INVALID_ARG;
    }

    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    const fa_host::DeviceInfo di = fa_host::device_info(dev);
    if (di.err == cudaErrorInvalidDevice || dev >= kMaxDevices) return FA_ERR_UNSUPPORTED;
    if (di.err != cudaSuccess) return FA_ERR_CUDA;
    if (!(di.cc_major == 10 && di.cc_minor == 3)) return FA_ERR_UNSUPPORTED;
    const void *all[] = {Q, O, LSE, cu_q, seq_k, cache->k, cache->v, workspace};
    for (const void *x : all)
        if (!fa_host::on_device(x, dev)) return FA_ERR_INVALID_ARG;
    if (max_pages > 0 && !fa_host::on_device(table, dev)) return FA_ERR_INVALID_ARG;
    if (!configured(dev)) return FA_ERR_CUDA;

    const bool bf16 = cache->dtype == FA_DTYPE_BF16;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    int page_log2 = 0;
    while ((int64_t{1} << page_log2) < cache->page_size) ++page_log2;
    // "all keys" is a window wider than any offset
    const int64_t every = total_q + max_keys;
    int64_t wl = every, wr = every;
    if (mask_mode == FA_MASK_CAUSAL) wr = 0;
    if (mask_mode == FA_MASK_WINDOW) {
        wl = window_left < every ? window_left : every;
        wr = window_right < every ? window_right : every;
    }
    const float scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    Plan x{};
    x.decode = decode;
    x.chunk = chunked;
    x.max_new = static_cast<int>(max_new);
    x.merge_rows = total_q <= B ? 1 : 4;
    x.sms = static_cast<unsigned>(di.sm_count);
    fa::paged::MergeInfo *info = reinterpret_cast<fa::paged::MergeInfo *>(ws);
    float *part_LSE = reinterpret_cast<float *>(ws + lay.lse), *part_O = reinterpret_cast<float *>(ws + lay.o);
    x.merge.info = info;
    x.merge.part_LSE = part_LSE;
    x.merge.part_O = part_O;
    x.merge.O = O;
    x.merge.LSE = LSE;
    x.merge.H = static_cast<int>(H);
    x.merge.pf = static_cast<int>(pf);
    x.merge.ctas = either ? di.sm_count : 0;
    const int fault = fa_host::take_fault_position();  // the decode kernel has no wait to run out
    // what both kernels' parameters have alike
    auto common = [&](auto &p) {
        p.O = O;
        p.LSE = LSE;
        p.part_O = part_O;
        p.part_LSE = part_LSE;
        p.info = info;
        p.cu_q = cu_q;
        p.seq_k = seq_k;
        p.table = table;
        p.B = static_cast<int>(B);
        p.H = static_cast<int>(H);
        p.kv_group = static_cast<int>(group);
        p.pf = static_cast<int>(pf);
        p.spaces = static_cast<int>(spaces);
        p.total_q = static_cast<int>(total_q);
        p.max_pages = static_cast<int>(max_pages);
        p.page_log2 = page_log2;
        p.num_pages = static_cast<int>(cache->num_pages);
        p.max_keys = static_cast<int>(max_keys);
        p.wl = static_cast<int>(wl);
        p.wr = static_cast<int>(wr);
        p.scale_log2 = scale_log2;
    };
    if (decode) {
        fa::paged::SmallParams &p = x.small;
        common(p);
        p.Q = static_cast<const uint16_t *>(Q);
        p.k = static_cast<const uint16_t *>(cache->k);
        p.v = static_cast<const uint16_t *>(cache->v);
        p.page_stride = cache->page_stride;
        p.token_stride = cache->token_stride;
        p.head_stride = cache->head_stride;
        p.tpt = static_cast<int>(tpt_small);
        p.min_ticks = kMinTicks;
    }
    if (chunked) {
        fa::paged::Params &p = x.p;
        common(p);
        const int kbn = fa::paged::bn(static_cast<int>(d));
        const int64_t box = cache->page_size < kbn ? cache->page_size : kbn;
        fa_host::PageSteps steps;
        if (!fa_host::page_steps(*cache, &steps) ||
            !fa_host::make_map_rows(&x.q, Q, bf16, total_q, H, d, static_cast<uint32_t>(pf),
                                    static_cast<uint32_t>(tpt)) ||
            !fa_host::make_map_pages(&x.k, cache->k, *cache, steps, static_cast<uint32_t>(box)) ||
            !fa_host::make_map_pages(&x.v, cache->v, *cache, steps, static_cast<uint32_t>(box)))
            return FA_ERR_CUDA;
        p.tpt = static_cast<int>(tpt);
        p.chunk = static_cast<int>(box);
        p.page_step = static_cast<int>(steps.page);
        p.head_step = static_cast<int>(steps.head);
        p.page_none = static_cast<int>(steps.count);
        p.wait_budget_ns = fa_host::wait_budget();
        p.status = di.status;
        p.fault_skip_k = fault;
    }
    cudaError_t e;
    switch (d) {
        case 32: e = bf16 ? launch<32, true>(x, st) : launch<32, false>(x, st); break;
        case 64: e = bf16 ? launch<64, true>(x, st) : launch<64, false>(x, st); break;
        case 128: e = bf16 ? launch<128, true>(x, st) : launch<128, false>(x, st); break;
        default: e = bf16 ? launch<256, true>(x, st) : launch<256, false>(x, st); break;
    }
    if (e != cudaSuccess) return FA_ERR_CUDA;
    fa_host::count_launches(2);
    return FA_OK;
}

}  // namespace

extern "C" {

size_t fa_forward_paged_workspace_bytes(int64_t d) {
    if (d != 32 && d != 64 && d != 128 && d != 256) return 0;
    return layout_of(d, fa_host::sm_count_or_default()).bytes;
}

fa_status fa_forward_paged(const void *Q, void *O, float *LSE, const fa_paged_cache *cache,
                           const int32_t *block_table, int64_t max_pages,
                           const int32_t *cu_seqlens_q, const int32_t *seqlens_k, int64_t B,
                           int64_t H, int64_t total_q, float scale, fa_mask_mode mask_mode,
                           int64_t window_left, int64_t window_right, void *workspace,
                           size_t workspace_bytes, void *stream) {
    return run(Q, O, LSE, cache, block_table, max_pages, cu_seqlens_q, seqlens_k, B, H, total_q, scale,
               mask_mode, window_left, window_right, workspace, workspace_bytes, stream);
}

}  // extern "C"
