// fa_paged_host.cu -- checks and tensor maps shared by the paged-cache calls.
#include "fa_paged_host.h"

#include <cuda_runtime.h>

#include <mutex>
#include <utility>

#include "fa_host.h"

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// Swizzle and promotion as in the library's other maps: rows of 128 bytes (64 at d = 32).
bool encode(CUtensorMap *map, const void *base, bool bf16, int rank, const cuuint64_t *dims,
            const cuuint64_t *strides, const cuuint32_t *box, int64_t d) {
    EncodeTiledFn enc = encode_fn();
    if (enc == nullptr) return false;
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
               static_cast<cuuint32_t>(rank), const_cast<void *>(base), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE,
               d < 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

namespace fa_host {

int sm_count_or_default() {
    int dev = 0, sms = 152;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    else
        cudaGetLastError();
    return sms;
}

int64_t span_apart(const int64_t (&count)[3], const int64_t (&stride)[3], int64_t d) {
    int64_t n[3] = {count[0], count[1], count[2]}, s[3] = {stride[0], stride[1], stride[2]};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (s[j] > s[j + 1]) {
                std::swap(s[j], s[j + 1]);
                std::swap(n[j], n[j + 1]);
            }
    int64_t span = d;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1) {
            if (s[i] < span) return 0;
            span += (n[i] - 1) * s[i];
        }
    return span;
}

fa_status check_cache(const fa_paged_cache &c, size_t *bytes) {
    if (!c.k || !c.v || !aligned16(c.k) || !aligned16(c.v)) return FA_ERR_INVALID_ARG;
    if (c.dtype != FA_DTYPE_FP16 && c.dtype != FA_DTYPE_BF16) return FA_ERR_INVALID_ARG;
    if (c.num_pages < 1 || c.H_kv < 1 || c.page_size < 1 || c.d < 1) return FA_ERR_INVALID_ARG;
    const int64_t st[3] = {c.page_stride, c.token_stride, c.head_stride};
    const int64_t count[3] = {c.num_pages, c.page_size, c.H_kv};
    for (int i = 0; i < 3; ++i)  // the stride of a single entry does not matter
        if (count[i] > 1 && (st[i] < 1 || st[i] % 8 != 0)) return FA_ERR_INVALID_ARG;
    if (c.d != 32 && c.d != 64 && c.d != 128 && c.d != 256) return FA_ERR_UNSUPPORTED;
    if (c.page_size < kMinPage || c.page_size > (int64_t{1} << 20) || (c.page_size & (c.page_size - 1)) != 0)
        return FA_ERR_UNSUPPORTED;
    // what a tensor map and 64-bit extents hold
    if (c.num_pages >= (int64_t{1} << 31) || c.H_kv > (int64_t{1} << 20)) return FA_ERR_UNSUPPORTED;
    for (int i = 0; i < 3; ++i)
        if (count[i] > 1 && st[i] >= (int64_t{1} << 35)) return FA_ERR_UNSUPPORTED;
    double extent = 0;
    for (int i = 0; i < 3; ++i)
        if (count[i] > 1) extent += static_cast<double>(count[i] - 1) * static_cast<double>(st[i]);
    if (extent > 1e18) return FA_ERR_UNSUPPORTED;
    const int64_t span = span_apart(count, st, c.d);
    if (span == 0) return FA_ERR_INVALID_ARG;
    *bytes = static_cast<size_t>(span) * 2;
    PageSteps steps;  // the same caches for every call, whichever kernel it runs
    if (!page_steps(c, &steps)) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

bool make_map_rows(CUtensorMap *map, const void *base, bool bf16, int64_t tokens, int64_t heads,
                   int64_t d, uint32_t box_heads, uint32_t box_tokens) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d * 2),
                                   static_cast<cuuint64_t>(heads * d * 2)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(d < 64 ? d : 64), box_heads, box_tokens};
    return encode(map, base, bf16, 3, dims, strides, box, d);
}

bool page_steps(const fa_paged_cache &c, PageSteps *s) {
    const int64_t ps = c.num_pages > 1 ? c.page_stride : 0, hs = c.H_kv > 1 ? c.head_stride : 0;
    int64_t a = ps, b = hs;
    while (b != 0) {
        const int64_t r = a % b;
        a = b;
        b = r;
    }
    s->stride = a > 0 ? a : c.d;
    s->page = ps / s->stride;
    s->head = hs / s->stride;
    const double most = static_cast<double>(c.num_pages) * static_cast<double>(s->page) +
                        static_cast<double>(c.H_kv) * static_cast<double>(s->head);
    if (most >= 2147483647.0) return false;
    s->count = (c.num_pages - 1) * s->page + (c.H_kv - 1) * s->head + 1;
    return true;
}

bool make_map_pages(CUtensorMap *map, const void *base, const fa_paged_cache &c, const PageSteps &s,
                    uint32_t box_tokens) {
    const int64_t cols = c.d < 64 ? c.d : 64;
    const cuuint64_t dims[5] = {
        static_cast<cuuint64_t>(cols), 8, static_cast<cuuint64_t>(c.d / cols),
        static_cast<cuuint64_t>(c.page_size / 8), static_cast<cuuint64_t>(s.count)};
    const cuuint64_t strides[4] = {
        static_cast<cuuint64_t>(c.token_stride * 2), static_cast<cuuint64_t>(cols * 2),
        static_cast<cuuint64_t>(c.token_stride * 16), static_cast<cuuint64_t>(s.stride * 2)};
    const cuuint32_t box[5] = {static_cast<cuuint32_t>(cols), 8, static_cast<cuuint32_t>(c.d / cols),
                               box_tokens / 8, 1};
    return encode(map, base, c.dtype == FA_DTYPE_BF16, 5, dims, strides, box, c.d);
}

}  // namespace fa_host
