// fa_paged_host.h -- host-side helpers of the paged-cache calls (internal).
#pragma once

#include <cuda.h>

#include <cstddef>
#include <cstdint>

#include "fa.h"

namespace fa_host {

// SMs of the current device (152 without one).
int sm_count_or_default();
// Elements from the first to the last of a tensor of three dimensions over rows of d, if no two of
// its elements share a place, else 0: with the dimensions of more than one entry sorted by
// stride, each has to step over what the smaller ones span.
int64_t span_apart(const int64_t (&count)[3], const int64_t (&stride)[3], int64_t d);
constexpr int64_t kMinPage = 8;  // tokens per page at least: a swizzle atom of a K/V tile
// Checks a cache descriptor (not its device); bytes: the extent of k (and of v) from
// its first to its last element.
fa_status check_cache(const fa_paged_cache &c, size_t *bytes);
// 3-D TMA map over a contiguous tokens x heads x d 16-bit tensor, ordered (d, heads,
// tokens): box of min(d, 64) columns x box_heads x box_tokens.
bool make_map_rows(CUtensorMap *map, const void *base, bool bf16, int64_t tokens, int64_t heads,
                   int64_t d, uint32_t box_heads, uint32_t box_tokens);
// Page and head of a cache as one coordinate, page * page + head * head, in steps of the
// strides' greatest common divisor; count: one past its last value. False when that does
// not fit 31 bits.
struct PageSteps {
    int64_t page, head, count, stride;
};
bool page_steps(const fa_paged_cache &c, PageSteps *s);
// 5-D TMA map over one tensor of a paged cache, ordered (column in a region of min(d, 64),
// token in a group of 8, region, group of 8 tokens of a page, page and head as above): box
// of all columns of box_tokens tokens of one head of one page.
bool make_map_pages(CUtensorMap *map, const void *base, const fa_paged_cache &c, const PageSteps &s,
                    uint32_t box_tokens);

}  // namespace fa_host
