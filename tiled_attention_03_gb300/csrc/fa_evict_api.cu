// fa_evict_api.cu -- fa_paged_evict: argument checks and launch of the eviction kernel
// (fa_evict_kernel.cuh).
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "fa.h"
#include "fa_evict_kernel.cuh"
#include "fa_host.h"
#include "fa_paged_host.h"

namespace {
constexpr int kMaxDevices = 64;
constexpr int kMostShared = 227 * 1024;
std::once_flag g_once[kMaxDevices];
cudaError_t g_opted[kMaxDevices];
}  // namespace

extern "C" fa_status fa_paged_evict(const fa_paged_cache *cache, float *weights, const int32_t *block_table,
                                    int64_t max_pages, const int32_t *seqlens_k, int32_t *seqlens_out,
                                    int64_t B, int64_t budget, int64_t first, int64_t recent, void *stream) {
    if (cache == nullptr || B < 1 || max_pages < 0 || first < 0 || recent < 0 || budget < 0 || first > budget ||
        recent > budget - first)
        return FA_ERR_INVALID_ARG;
    size_t cache_bytes = 0;
    const fa_status cs = fa_host::check_cache(*cache, &cache_bytes);
    if (cs != FA_OK) return cs;
    if (cache->k == cache->v) return FA_ERR_INVALID_ARG;  // a key and a value for each place
    if (!weights || !seqlens_k || !seqlens_out || (!block_table && max_pages > 0)) return FA_ERR_INVALID_ARG;
    if (!fa_host::aligned4(weights) || !fa_host::aligned4(seqlens_k) || !fa_host::aligned4(seqlens_out) ||
        !fa_host::aligned4(block_table))
        return FA_ERR_INVALID_ARG;
    const int64_t kLimit = int64_t{1} << 29, max_keys = max_pages * cache->page_size;
    if (max_pages > kLimit || max_keys > kLimit || B > kLimit || cache->H_kv > kLimit ||
        B * cache->H_kv > (int64_t{1} << 27))
        return FA_ERR_UNSUPPORTED;
    const size_t wbytes = static_cast<size_t>(cache->num_pages) * static_cast<size_t>(cache->H_kv) *
                          static_cast<size_t>(cache->page_size) * sizeof(float);
    // what is written overlaps nothing else (K and V may be interleaved with each other)
    const struct {
        const void *p;
        size_t n;
        bool written;
    } bufs[] = {{cache->k, cache_bytes, true},
                {cache->v, cache_bytes, true},
                {weights, wbytes, true},
                {seqlens_out, static_cast<size_t>(B) * 4, true},
                {seqlens_k, static_cast<size_t>(B) * 4, false},
                {block_table, static_cast<size_t>(B * max_pages) * 4, false}};
    for (int i = 0; i < 6; ++i)
        for (int j = i + 1; j < 6; ++j)
            if (bufs[i].written && !(i == 0 && j == 1) && bufs[j].n > 0 &&
                fa_host::overlaps(bufs[i].p, bufs[i].n, bufs[j].p, bufs[j].n))
                return FA_ERR_INVALID_ARG;

    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    const fa_host::DeviceInfo di = fa_host::device_info(dev);
    if (di.err == cudaErrorInvalidDevice || dev >= kMaxDevices) return FA_ERR_UNSUPPORTED;
    if (di.err != cudaSuccess) return FA_ERR_CUDA;
    if (!(di.cc_major == 10 && di.cc_minor == 3)) return FA_ERR_UNSUPPORTED;
    for (const auto &x : bufs)
        if (x.n > 0 && !fa_host::on_device(x.p, dev)) return FA_ERR_INVALID_ARG;
    using namespace fa::evict;
    std::call_once(g_once[dev], [dev] {
        g_opted[dev] = cudaFuncSetAttribute(fa_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
    });
    if (g_opted[dev] != cudaSuccess) return FA_ERR_CUDA;
    fa_host::take_fault_position();  // nothing here waits: an armed test hook is spent

    Params p{};
    p.k = static_cast<uint16_t *>(cache->k);
    p.v = static_cast<uint16_t *>(cache->v);
    p.weights = weights;
    // the stride of a dimension of one entry may be anything
    p.page_stride = cache->num_pages > 1 ? cache->page_stride : 0;
    p.token_stride = cache->token_stride;
    p.head_stride = cache->H_kv > 1 ? cache->head_stride : 0;
    p.seq_k = seqlens_k;
    p.table = block_table;
    p.seq_out = seqlens_out;
    p.H_kv = static_cast<int>(cache->H_kv);
    p.d = static_cast<int>(cache->d);
    p.max_pages = static_cast<int>(max_pages);
    while ((int64_t{1} << p.page_log2) < cache->page_size) ++p.page_log2;
    p.num_pages = static_cast<int>(cache->num_pages);
    p.max_keys = static_cast<int>(max_keys);
    const int64_t most = max_keys > 0 ? max_keys : 1;
    p.budget = static_cast<int>(budget < most ? budget : most);
    p.first = static_cast<int>(first < most ? first : most);
    p.recent = static_cast<int>(recent < most ? recent : most);
    // CTAs per sequence and head: one for every 128 bytes of a row (a key and its value), twice as many
    // where that leaves SMs without one (24 units of 500 rows of 256 bytes: 12.7 us, 14.5 with no
    // more); but at least 16 KB to move for each (small budgets 9.1 us, 12.8 with at least 4 KB; those
    // 24 units 14.7 with at least 64).
    const int row_bytes = p.d * 4;
    const int64_t units = B * cache->H_kv;
    int ctas = row_bytes / 128 < kMaxCluster ? row_bytes / 128 : kMaxCluster;
    if (units * ctas < di.sm_count && ctas * 2 <= kMaxCluster) ctas *= 2;
    while (ctas > 1 && static_cast<int64_t>(p.budget) * row_bytes < ctas * 16384) ctas /= 2;
    const int columns = row_bytes / ctas;
    while ((16 << p.piece_log2) < columns) ++p.piece_log2;
    // shared memory: two CTAs to an SM; all of it where there are no two (always all: 58 -> 79 us
    // for many sequences)
    const int shared = units * ctas <= di.sm_count ? kMostShared : kMostShared / 2 / 1024 * 1024;
    const int room = (shared - kSharedBytes) / 128 * 128;
    const int rows = room / (kDepth * columns + kLists * 20);
    p.rows = rows < kThreads ? rows : kThreads;
    p.keys = room / 4;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(units * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(shared);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, fa_evict_kernel, p) != cudaSuccess) return FA_ERR_CUDA;
    fa_host::count_launches(1);
    return FA_OK;
}
