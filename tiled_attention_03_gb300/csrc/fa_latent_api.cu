// fa_latent_api.cu -- fa_forward_latent: argument checks, tensor maps and launches of the
// latent attention kernel and its merge (fa_latent_kernel.cuh).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "fa.h"
#include "fa_host.h"
#include "fa_latent_kernel.cuh"
#include "fa_paged_host.h"
#include "fa_pdl.cuh"

namespace {

using fa_host::align256;

constexpr int kMaxDevices = 64;
constexpr int kMaxRows = 64;  // rows of a CTA's block at most

// Two partial results per CTA, and what the merge needs to know of each.
struct Layout {
    size_t lse, o, bytes;  // info at 0
};
Layout layout_of(int64_t dl, int64_t sms) {
    const size_t rows = static_cast<size_t>(2 * sms) * kMaxRows;
    Layout l;
    l.lse = align256(static_cast<size_t>(sms) * sizeof(fa::paged::MergeInfo));
    l.o = l.lse + align256(rows * sizeof(float));
    l.bytes = l.o + rows * static_cast<size_t>(dl) * sizeof(float);
    return l;
}

struct Plan {
    int rows;  // of a CTA's block: 16, 32 or 64
    unsigned ctas;
    fa::latent::Params p;
    fa::latent::MergeParams merge;
    CUtensorMap q, k, r;  // k: two regions of 64 columns at a time; r: one
    unsigned sms;
};

template <int DL, int R, bool BF16>
cudaError_t launch_rows(const Plan &x, int dev, cudaStream_t st) {
    using namespace fa::latent;
    constexpr int kAlloc = Smem<DL, R>::kAlloc;
    static std::once_flag once[kMaxDevices];
    static cudaError_t opted[kMaxDevices];
    std::call_once(once[dev], [dev] {
        opted[dev] = cudaFuncSetAttribute(fa_latent_kernel<DL, R, BF16>,
                                          cudaFuncAttributeMaxDynamicSharedMemorySize, kAlloc);
    });
    if (opted[dev] != cudaSuccess) return opted[dev];
    return fa::launch_after(fa_latent_kernel<DL, R, BF16>, dim3(x.ctas), kThreads, kAlloc, st, x.q, x.k, x.r, x.p);
}

template <int DL, bool BF16>
cudaError_t launch(const Plan &x, int dev, cudaStream_t st) {
    const cudaError_t e = x.rows == 16   ? launch_rows<DL, 16, BF16>(x, dev, st)
                          : x.rows == 32 ? launch_rows<DL, 32, BF16>(x, dev, st)
                                         : launch_rows<DL, 64, BF16>(x, dev, st);
    if (e != cudaSuccess) return e;
    return fa::launch_after(fa::latent::fa_latent_merge_kernel<DL, BF16>, dim3(fa::latent::kMergeBlocks * x.sms), fa::latent::kMergeThreads,
                            0, st, x.merge);
}

fa_status run(const void *Q, void *O, float *LSE, const fa_latent_cache *cache, const int32_t *table,
              int64_t max_pages, const int32_t *cu_q, const int32_t *seq_k, int64_t B, int64_t H,
              int64_t total_q, float scale, fa_mask_mode mask_mode, int64_t window_left,
              int64_t window_right, void *workspace, size_t workspace_bytes, void *stream) {
    // ---- host-side checks: nothing is enqueued on failure
    if (cache == nullptr || B < 1 || H < 1 || total_q < 0 || max_pages < 0) return FA_ERR_INVALID_ARG;
    size_t cache_bytes = 0;
    fa_paged_cache rows{};
    const fa_status cs = fa_host::check_latent(*cache, &rows, &cache_bytes);
    if (cs != FA_OK) return cs;
    const int64_t dl = cache->d_latent, d = rows.d;
    if (mask_mode != FA_MASK_NONE && mask_mode != FA_MASK_CAUSAL && mask_mode != FA_MASK_WINDOW)
        return FA_ERR_INVALID_ARG;
    if (mask_mode == FA_MASK_WINDOW && (window_left < 0 || window_right < 0)) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
    if (total_q == 0) return FA_OK;  // no query rows: nothing to do
    if (!Q || !O || !LSE || !cu_q || !seq_k || (!table && max_pages > 0)) return FA_ERR_INVALID_ARG;
    if (!fa_host::aligned16(Q) || !fa_host::aligned32(O) || !fa_host::aligned4(LSE) ||
        !fa_host::aligned4(cu_q) || !fa_host::aligned4(seq_k) || !fa_host::aligned4(table))
        return FA_ERR_INVALID_ARG;
    const int64_t max_keys = max_pages * cache->page_size;
    // Size limits of this implementation: 32-bit row and key indices, and a line of work
    // below 2^31 tiles.
    const int64_t kLimit = int64_t{1} << 29;
    if (total_q > kLimit || max_pages > kLimit || max_keys > kLimit || B > kLimit || H > kLimit ||
        total_q * H > (int64_t{1} << 30))
        return FA_ERR_UNSUPPORTED;
    // Rows of a CTA's block: as many as a sequence has on average, 16, 32 or 64 (at each: 4 short
    // sequences of 16 rows 10.8, 10.8 and 12.2 us; 8 of 32768 keys and 32 rows 98, 61 and 63; 40 with
    // 128 rows 116, 74 and 53); with more than one and a half blocks of 64, two CTAs side by side (40
    // sequences with 128 rows 53.3 us, with single CTAs 55.3; one of 16000 rows 456 either way; 8 of
    // 32768 keys and 32 rows, where the second CTA has none, 61 alone and 92 in pairs).
    const int64_t all_rows = total_q * H;
    const int r = all_rows <= 16 * B ? 16 : all_rows <= 32 * B ? 32 : 64;
    const int group = all_rows > 96 * B ? 2 : 1;
    const double line = (static_cast<double>(all_rows) / (r * group) + static_cast<double>(B)) *
                        (static_cast<double>(max_keys) / fa::latent::kBK + 1 + fa::latent::kTicks);
    if (line > 2147483640.0) return FA_ERR_UNSUPPORTED;
    const int sms = fa_host::sm_count_or_default();
    const Layout lay = layout_of(dl, sms);
    if (workspace == nullptr || !fa_host::aligned32(workspace) || workspace_bytes < lay.bytes)
        return FA_ERR_INVALID_ARG;
    const struct {
        const void *p;
        size_t n;
    } in[] = {{Q, static_cast<size_t>(all_rows * d) * 2},
              {cache->data, cache_bytes},
              {cu_q, static_cast<size_t>(B + 1) * 4},
              {seq_k, static_cast<size_t>(B) * 4},
              {table, static_cast<size_t>(B * max_pages) * 4}},
      out[] = {{O, static_cast<size_t>(all_rows * dl) * 2},
               {LSE, static_cast<size_t>(all_rows) * sizeof(float)},
               {workspace, lay.bytes}};
    for (int i = 0; i < 3; ++i) {
        for (const auto &b : in)
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
    if (!(di.cc_major == 10 && di.cc_minor == 3) || di.sm_count > fa::latent::kMergeMost) return FA_ERR_UNSUPPORTED;
    const void *all[] = {Q, O, LSE, cu_q, seq_k, cache->data, workspace};
    for (const void *x : all)
        if (!fa_host::on_device(x, dev)) return FA_ERR_INVALID_ARG;
    if (max_pages > 0 && !fa_host::on_device(table, dev)) return FA_ERR_INVALID_ARG;

    const bool bf16 = cache->dtype == FA_DTYPE_BF16;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    // "all keys" is a window wider than any offset
    const int64_t every = total_q + max_keys;
    int64_t wl = every, wr = every;
    if (mask_mode == FA_MASK_CAUSAL) wr = 0;
    if (mask_mode == FA_MASK_WINDOW) {
        wl = window_left < every ? window_left : every;
        wr = window_right < every ? window_right : every;
    }
    Plan x{};
    x.rows = r;
    x.sms = static_cast<unsigned>(di.sm_count);
    x.ctas = x.sms / group * group;
    fa::latent::Params &p = x.p;
    fa_host::PageSteps steps;
    const int64_t box = cache->page_size < fa::latent::kBK ? cache->page_size : fa::latent::kBK;
    if (!fa_host::page_steps(rows, &steps) ||
        !fa_host::make_map_rows(&x.q, Q, bf16, all_rows, 1, d, 1, static_cast<uint32_t>(r)) ||
        !fa_host::make_map_pages(&x.k, cache->data, rows, steps, static_cast<uint32_t>(box), 2) ||
        !fa_host::make_map_pages(&x.r, cache->data, rows, steps, static_cast<uint32_t>(box), 1))
        return FA_ERR_CUDA;
    p.O = O;
    p.LSE = LSE;
    p.part_O = reinterpret_cast<float *>(ws + lay.o);
    p.part_LSE = reinterpret_cast<float *>(ws + lay.lse);
    p.info = reinterpret_cast<fa::paged::MergeInfo *>(ws);
    p.cu_q = cu_q;
    p.seq_k = seq_k;
    p.table = table;
    p.B = static_cast<int>(B);
    p.H = static_cast<int>(H);
    p.group = group;
    p.by_H = fa::divisor(H);
    while ((1 << p.rb_log2) < r * group) ++p.rb_log2;
    p.total_q = static_cast<int>(total_q);
    p.max_pages = static_cast<int>(max_pages);
    while ((int64_t{1} << p.page_log2) < cache->page_size) ++p.page_log2;
    p.num_pages = static_cast<int>(cache->num_pages);
    p.max_keys = static_cast<int>(max_keys);
    p.chunk = static_cast<int>(box);
    p.page_step = static_cast<int>(steps.page);
    p.page_none = static_cast<int>(steps.count);
    p.wl = static_cast<int>(wl);
    p.wr = static_cast<int>(wr);
    p.line_most = static_cast<unsigned>(line) + 1;
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    p.wait_budget_ns = fa_host::wait_budget();
    p.status = di.status;
    p.fault_skip_k = fa_host::take_fault_position();
    x.merge.info = p.info;
    x.merge.part_O = p.part_O;
    x.merge.part_LSE = p.part_LSE;
    x.merge.O = O;
    x.merge.LSE = LSE;
    x.merge.ctas = static_cast<int>(x.ctas);
    cudaError_t e;
    switch (dl) {
        case 128: e = bf16 ? launch<128, true>(x, dev, st) : launch<128, false>(x, dev, st); break;
        case 256: e = bf16 ? launch<256, true>(x, dev, st) : launch<256, false>(x, dev, st); break;
        default: e = bf16 ? launch<512, true>(x, dev, st) : launch<512, false>(x, dev, st); break;
    }
    if (e != cudaSuccess) return FA_ERR_CUDA;
    fa_host::count_launches(2);
    return FA_OK;
}

}  // namespace

extern "C" {

size_t fa_forward_latent_workspace_bytes(int64_t d_latent) {
    if (d_latent != 128 && d_latent != 256 && d_latent != 512) return 0;
    return layout_of(d_latent, fa_host::sm_count_or_default()).bytes;
}

fa_status fa_forward_latent(const void *Q, void *O, float *LSE, const fa_latent_cache *cache,
                            const int32_t *block_table, int64_t max_pages,
                            const int32_t *cu_seqlens_q, const int32_t *seqlens_k, int64_t B,
                            int64_t H, int64_t total_q, float scale, fa_mask_mode mask_mode,
                            int64_t window_left, int64_t window_right, void *workspace,
                            size_t workspace_bytes, void *stream) {
    return run(Q, O, LSE, cache, block_table, max_pages, cu_seqlens_q, seqlens_k, B, H, total_q, scale,
               mask_mode, window_left, window_right, workspace, workspace_bytes, stream);
}

}  // extern "C"
