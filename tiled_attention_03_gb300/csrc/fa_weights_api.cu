// fa_weights_api.cu -- fa_paged_weights: argument checks, tensor maps and launch of the kernel
// that sums attention weights per key (fa_weights_kernel.cuh).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "fa.h"
#include "fa_host.h"
#include "fa_paged_host.h"
#include "fa_pdl.cuh"
#include "fa_weights_kernel.cuh"

namespace {

constexpr int kMaxDevices = 64;

struct Plan {
    int rows;
    unsigned sms;
    fa::weights::Params p;
    CUtensorMap q, k;
};

template <int D, int R, bool BF16>
cudaError_t launch_rows(const Plan &x, int dev, cudaStream_t st) {
    using namespace fa::weights;
    constexpr int kAlloc = Smem<D, R>::kAlloc;
    static std::once_flag once[kMaxDevices];
    static cudaError_t opted[kMaxDevices];
    std::call_once(once[dev], [dev] {
        opted[dev] = cudaFuncSetAttribute(fa_weights_kernel<D, R, BF16>,
                                          cudaFuncAttributeMaxDynamicSharedMemorySize, kAlloc);
    });
    if (opted[dev] != cudaSuccess) return opted[dev];
    return fa::launch_after(fa_weights_kernel<D, R, BF16>, dim3(x.sms), kThreads, kAlloc, st, x.q, x.k, x.p);
}

// Rows of a tile at most: what leaves shared memory for two tiles of queries and of keys.
constexpr int most_rows(int64_t d) { return d == 256 ? 64 : 128; }

template <int D, bool BF16>
cudaError_t launch(const Plan &x, int dev, cudaStream_t st) {
    if (x.rows == 16) return launch_rows<D, 16, BF16>(x, dev, st);
    if constexpr (most_rows(D) > 64)
        if (x.rows == 128) return launch_rows<D, 128, BF16>(x, dev, st);
    return launch_rows<D, 64, BF16>(x, dev, st);
}

}  // namespace

extern "C" fa_status fa_paged_weights(const void *Q, const float *LSE, float *weights,
                                      const fa_paged_cache *cache, const int32_t *block_table,
                                      int64_t max_pages, const int32_t *cu_seqlens_q,
                                      const int32_t *seqlens_k, int64_t B, int64_t H, int64_t total_q,
                                      float scale, fa_mask_mode mask_mode, int64_t window_left,
                                      int64_t window_right, void *stream) {
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
    if (!Q || !LSE || !weights || !cu_seqlens_q || !seqlens_k || (!block_table && max_pages > 0))
        return FA_ERR_INVALID_ARG;
    if (!fa_host::aligned16(Q) || !fa_host::aligned4(LSE) || !fa_host::aligned4(weights) ||
        !fa_host::aligned4(cu_seqlens_q) || !fa_host::aligned4(seqlens_k) || !fa_host::aligned4(block_table))
        return FA_ERR_INVALID_ARG;
    const int64_t max_keys = max_pages * cache->page_size;
    const int64_t kLimit = int64_t{1} << 29;
    if (total_q > kLimit || max_pages > kLimit || max_keys > kLimit || B > kLimit || H > kLimit ||
        total_q * H > (int64_t{1} << 30) || (max_keys / 128 + 1) * H_kv > (int64_t{1} << 30))
        return FA_ERR_UNSUPPORTED;
    // Rows of a tile: a sequence's on average (new tokens x query heads of a K/V head), 16, 64 or
    // 128; of them the heads of a group, or a divisor of them, for as many tokens as fit. (With 16,
    // 64 and 128: 8 sequences of 32768 keys and 4 rows 88, 96 and 158 us; 16 of 6000 to 9000 keys
    // and 40 rows 35, 27 and 33; 8192 rows of one sequence 187 with 64, 118 with 128.)
    const int64_t group = H / H_kv, all_rows = total_q * group;
    int rows = all_rows <= 16 * B ? 16 : all_rows <= 64 * B ? 64 : most_rows(d);
    int64_t pf = group < rows ? group : rows;
    while (group % pf != 0) --pf;
    const int64_t tpt = rows / pf;
    const size_t wbytes = static_cast<size_t>(cache->num_pages) * static_cast<size_t>(H_kv) *
                          static_cast<size_t>(cache->page_size) * sizeof(float);
    const struct {
        const void *p;
        size_t n;
    } in[] = {{Q, static_cast<size_t>(total_q * H * d) * 2},
              {LSE, static_cast<size_t>(total_q * H) * sizeof(float)},
              {cache->k, cache_bytes},
              {cache->v, cache_bytes},
              {cu_seqlens_q, static_cast<size_t>(B + 1) * 4},
              {seqlens_k, static_cast<size_t>(B) * 4},
              {block_table, static_cast<size_t>(B * max_pages) * 4}};
    for (const auto &b : in)
        if (b.n > 0 && fa_host::overlaps(weights, wbytes, b.p, b.n)) return FA_ERR_INVALID_ARG;

    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    const fa_host::DeviceInfo di = fa_host::device_info(dev);
    if (di.err == cudaErrorInvalidDevice || dev >= kMaxDevices) return FA_ERR_UNSUPPORTED;
    if (di.err != cudaSuccess) return FA_ERR_CUDA;
    if (!(di.cc_major == 10 && di.cc_minor == 3)) return FA_ERR_UNSUPPORTED;
    const void *all[] = {Q, LSE, weights, cu_seqlens_q, seqlens_k, cache->k};
    for (const void *x : all)
        if (!fa_host::on_device(x, dev)) return FA_ERR_INVALID_ARG;
    if (max_pages > 0 && !fa_host::on_device(block_table, dev)) return FA_ERR_INVALID_ARG;

    const bool bf16 = cache->dtype == FA_DTYPE_BF16;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // "all keys" is a window wider than any offset
    const int64_t every = total_q + max_keys;
    int64_t wl = every, wr = every;
    if (mask_mode == FA_MASK_CAUSAL) wr = 0;
    if (mask_mode == FA_MASK_WINDOW) {
        wl = window_left < every ? window_left : every;
        wr = window_right < every ? window_right : every;
    }
    Plan x{};
    x.rows = rows;
    x.sms = static_cast<unsigned>(di.sm_count);
    fa_host::PageSteps steps;
    const int64_t keys = fa::weights::tile_keys(static_cast<int>(d), rows);
    const int64_t box = cache->page_size < keys ? cache->page_size : keys;
    if (!fa_host::page_steps(*cache, &steps) ||
        !fa_host::make_map_rows(&x.q, Q, bf16, total_q, H, d, static_cast<uint32_t>(pf), static_cast<uint32_t>(tpt)) ||
        !fa_host::make_map_pages(&x.k, cache->k, *cache, steps, static_cast<uint32_t>(box)))
        return FA_ERR_CUDA;
    fa::weights::Params &p = x.p;
    p.weights = weights;
    p.LSE = LSE;
    p.cu_q = cu_seqlens_q;
    p.seq_k = seqlens_k;
    p.table = block_table;
    p.B = static_cast<int>(B);
    p.H = static_cast<int>(H);
    p.H_kv = static_cast<int>(H_kv);
    p.pf = static_cast<int>(pf);
    p.subs = static_cast<int>(group / pf);
    p.tpt = static_cast<int>(tpt);
    p.by_heads = fa::divisor(H_kv);
    p.by_tpt = fa::divisor(tpt);
    p.by_subs = fa::divisor(group / pf);
    p.total_q = static_cast<int>(total_q);
    p.max_pages = static_cast<int>(max_pages);
    while ((int64_t{1} << p.page_log2) < cache->page_size) ++p.page_log2;
    p.num_pages = static_cast<int>(cache->num_pages);
    p.max_keys = static_cast<int>(max_keys);
    p.chunk = static_cast<int>(box);
    p.page_step = static_cast<int>(steps.page);
    p.head_step = static_cast<int>(steps.head);
    p.page_none = static_cast<int>(steps.count);
    p.wl = static_cast<int>(wl);
    p.wr = static_cast<int>(wr);
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    p.wait_budget_ns = fa_host::wait_budget();
    p.status = di.status;
    p.fault_skip_k = fa_host::take_fault_position();
    cudaError_t e;
    switch (d) {
        case 32: e = bf16 ? launch<32, true>(x, dev, st) : launch<32, false>(x, dev, st); break;
        case 64: e = bf16 ? launch<64, true>(x, dev, st) : launch<64, false>(x, dev, st); break;
        case 128: e = bf16 ? launch<128, true>(x, dev, st) : launch<128, false>(x, dev, st); break;
        default: e = bf16 ? launch<256, true>(x, dev, st) : launch<256, false>(x, dev, st); break;
    }
    if (e != cudaSuccess) return FA_ERR_CUDA;
    fa_host::count_launches(1);
    return FA_OK;
}
