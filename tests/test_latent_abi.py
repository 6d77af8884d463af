"""Refusals of the latent-cache calls and of the two eviction calls, through the C ABI with
addresses that are never dereferenced: no GPU needed."""

import math

import pytest
import torch

import tiled_attention_03_gb300 as fa
from tiled_attention_03_gb300.binding import FaLatentCache
from test_paged_abi import (AT, FAR, INVALID, UNSUPPORTED, FaRows, cache, lib, past_checks, ref,  # noqa: F401
                            rope)

DATA = 0x200000000


def latent(**kw):
    a = dict(data=DATA, page_stride=16 * 576, token_stride=576, num_pages=100, page_size=16, d_latent=512, d_rope=64,
             dtype=1)
    a.update(kw)
    return FaLatentCache(*(a[n] for n, _ in FaLatentCache._fields_))


def attend(lib, q=AT, o=AT + FAR, lse=AT + 2 * FAR, c=None, table=AT + 3 * FAR, pages=8, cu=AT + 4 * FAR,  # noqa: F811
           lens=AT + 5 * FAR, B=3, H=4, total=20, scale=0.125, mask=1, wl=0, wr=0, ws=AT + 6 * FAR, ws_bytes=1 << 27):
    return lib.fa_forward_latent(q, o, lse, ref(latent() if c is None else c), table, pages, cu, lens, B, H, total, scale,
                                 mask, wl, wr, ws, ws_bytes, None)


def append(lib, H=4, B=3, total=20, table=AT + 5 * FAR, pages=8, cu=AT + 6 * FAR, lens=AT + 7 * FAR, c=None, r=None,  # noqa: F811
           **t):
    q = t.get("q", FaRows(AT, 0, 192, H * 192))
    x = t.get("x", FaRows(AT + FAR, 0, 0, 576))
    k = t.get("k", FaRows(AT + FAR + 512 * 2, 0, 0, 576))
    y = t.get("y", FaRows(AT + 3 * FAR + 512 * 2, 0, 576, H * 576))
    return lib.fa_latent_append(ref(q), ref(x), ref(k), ref(y), ref(latent() if c is None else c), table, pages, cu, lens,
                                B, H, total, ref(r), None)


def gather(lib, q=AT, lse=AT + FAR, w=AT + 2 * FAR, c=None, table=AT + 3 * FAR, pages=8, cu=AT + 4 * FAR,  # noqa: F811
           lens=AT + 5 * FAR, B=3, H=4, total=20, scale=0.125, mask=1, wl=0, wr=0):
    return lib.fa_paged_weights(q, lse, w, ref(cache() if c is None else c), table, pages, cu, lens, B, H, total, scale,
                                mask, wl, wr, None)


def evict(lib, c=None, w=AT, table=AT + FAR, pages=8, lens=AT + 2 * FAR, out=AT + 3 * FAR, B=3, budget=40,  # noqa: F811
          first=4, recent=16):
    return lib.fa_paged_evict(ref(cache() if c is None else c), w, table, pages, lens, out, B, budget, first, recent, None)


def no_q(**kw):
    return dict(q=FaRows(None, 0, 0, 0), y=FaRows(None, 0, 0, 0), **kw)


def turn(**kw):
    return rope(q_weight=None, **kw)


def test_good_calls_pass_the_checks(lib):  # noqa: F811
    assert past_checks(attend(lib))
    assert past_checks(append(lib)) and past_checks(append(lib, r=turn())) and past_checks(append(lib, **no_q()))
    q = FaRows(AT, 0, 192, 4 * 192)
    assert past_checks(append(lib, q=q, y=q, r=turn(k_weight=None)))  # in place
    for c in (latent(d_latent=128, token_stride=192), latent(d_latent=256), latent(num_pages=1, page_stride=-3),
              latent(token_stride=640, page_stride=16 * 640)):
        assert past_checks(attend(lib, c=c))
    assert past_checks(gather(lib)) and past_checks(gather(lib, H=64))
    one = cache(v=DATA)
    assert past_checks(gather(lib, c=one))  # values are not read
    assert past_checks(evict(lib)) and past_checks(evict(lib, budget=0, first=0, recent=0))
    assert past_checks(evict(lib, budget=20, first=4, recent=16)) and past_checks(evict(lib, budget=1 << 40))


@pytest.mark.parametrize("kw", [
    dict(data=None), dict(data=DATA + 8), dict(dtype=2), dict(num_pages=0), dict(page_size=0), dict(token_stride=0),
    dict(token_stride=572), dict(token_stride=512), dict(page_stride=4096), dict(d_latent=0), dict(d_rope=0),
    dict(d_rope=-64),
])
def test_cache_refusals(lib, kw):  # noqa: F811
    assert attend(lib, c=latent(**kw)) == INVALID
    assert append(lib, c=latent(**kw)) == INVALID


@pytest.mark.parametrize("kw", [dict(d_latent=64), dict(d_latent=384), dict(d_latent=1024, token_stride=2048, page_stride=1 << 15),
                                dict(d_rope=32), dict(d_rope=128, token_stride=640, page_stride=16 * 640),
                                dict(page_size=4), dict(page_size=24, page_stride=24 * 576)])
def test_unsupported_caches(lib, kw):  # noqa: F811
    assert attend(lib, c=latent(**kw)) == UNSUPPORTED
    assert append(lib, c=latent(**kw)) == UNSUPPORTED


@pytest.mark.parametrize("d", [0, 64, 384, 576, 1024])
def test_workspace_of_unknown_widths(lib, d):  # noqa: F811
    assert lib.fa_forward_latent_workspace_bytes(d) == 0


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(o=None), dict(lse=None), dict(table=None), dict(cu=None), dict(lens=None), dict(ws=None),
    dict(B=0), dict(H=0), dict(total=-1), dict(pages=-1), dict(scale=0.0), dict(scale=math.inf),
    dict(mask=3), dict(mask=2, wl=-1), dict(mask=2, wr=-1),
    dict(q=AT + 8), dict(o=AT + FAR + 16), dict(lse=AT + 2 * FAR + 2), dict(cu=AT + 2), dict(table=AT + 1),
    dict(ws=AT + 6 * FAR + 16), dict(ws_bytes=1000),
    dict(o=AT), dict(lse=AT + FAR + 64), dict(o=DATA), dict(ws=DATA + 32), dict(ws=AT + FAR), dict(lse=AT + 4 * FAR),
])
def test_attention_refusals(lib, kw):  # noqa: F811
    assert attend(lib, **kw) == INVALID


def test_attention_size_limits(lib):  # noqa: F811
    assert attend(lib, pages=1 << 28) == UNSUPPORTED
    assert attend(lib, total=1 << 24, H=128) == UNSUPPORTED  # 2^31 rows


@pytest.mark.parametrize("kw", [
    dict(x=FaRows(None, 0, 0, 0)), dict(k=FaRows(None, 0, 0, 0)), dict(q=FaRows(None, 0, 0, 0)),
    dict(y=FaRows(None, 0, 0, 0)), dict(H=0), dict(B=0), dict(total=-1), dict(pages=-1),
    dict(table=None), dict(cu=None), dict(lens=None), dict(lens=AT + 7 * FAR + 2),
    dict(x=FaRows(AT + FAR + 4, 0, 0, 576)), dict(k=FaRows(AT + FAR + 1024, 0, 0, 570)),
    dict(y=FaRows(AT + 3 * FAR, 0, 0, 576)),                  # heads written over each other
    dict(y=FaRows(AT + 64, 0, 192, 4 * 192)),                 # beside q, not in its place
    dict(y=FaRows(AT + FAR, 0, 64, 256)),                     # over the latents
    dict(y=FaRows(DATA, 0, 64, 256)), dict(x=FaRows(DATA, 0, 0, 576)), dict(k=FaRows(DATA + 1024, 0, 0, 576)),
    dict(lens=DATA), dict(cu=AT + 3 * FAR + 1024),
    dict(r=rope()),                                           # a weight for the queries
    dict(r=turn(rotary_dim=66)), dict(r=turn(rotary_dim=-2)), dict(r=turn(steps=None)),
    dict(r=turn(k_weight=DATA)), dict(r=turn(k_weight=0x92000004)), dict(r=turn(eps=-1.0)),
])
def test_append_refusals(lib, kw):  # noqa: F811
    assert append(lib, **kw) == INVALID


@pytest.mark.parametrize("first", ["queries", "latent"])
@pytest.mark.parametrize("d_latent,H", [(512, 4), (128, 1), (256, 16)])
def test_one_projection_of_queries_latent_and_rotary_part(lib, d_latent, H, first):  # noqa: F811
    """A token's query heads (192 wide, their rotary parts last), c and k_rope beside each other, the
    queries rotated in place: no element of one is another's, whichever comes first."""
    heads, both = 192 * H, d_latent + 64
    width, at_q, at_c = heads + both, (both if first == "latent" else 0), (heads if first == "queries" else 0)
    where = lambda i: AT + 2 * i  # noqa: E731
    q = FaRows(where(at_q + 128), 0, 192, width)
    x, k = FaRows(where(at_c), 0, 0, width), FaRows(where(at_c + d_latent), 0, 0, width)
    c = latent(d_latent=d_latent, token_stride=both, page_stride=16 * both)
    assert past_checks(append(lib, H=H, q=q, y=q, x=x, k=k, c=c))
    assert past_checks(append(lib, H=H, q=q, y=q, x=x, k=k, c=c, total=1))
    # into the queries' place from another buffer
    assert past_checks(append(lib, H=H, q=FaRows(AT + 8 * FAR, 0, 64, 64 * H), y=q, x=x, k=k, c=c))
    # but not over the latent's first or last elements, nor where the strides differ
    for off in (8 - d_latent, 56):
        over = FaRows(where(at_q + 128 + 192 * (H - 1) + off), 0, 0, width)
        assert append(lib, H=H, q=q, y=q, x=over, k=FaRows(AT + 4 * FAR, 0, 0, width), c=c) == INVALID
    assert append(lib, H=H, q=q, y=q, x=FaRows(where(at_c), 0, 0, width + 8), k=k, c=c) == INVALID


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(lse=None), dict(w=None), dict(table=None), dict(cu=None), dict(lens=None),
    dict(B=0), dict(H=0), dict(H=5), dict(total=-1), dict(pages=-1), dict(scale=-1.0), dict(scale=math.nan),
    dict(mask=3), dict(mask=2, wl=-1), dict(mask=2, wr=-1), dict(q=AT + 8), dict(lse=AT + FAR + 2), dict(w=AT + 2 * FAR + 1),
    dict(w=AT), dict(w=AT + FAR + 64), dict(w=DATA), dict(w=0x300000000), dict(w=AT + 3 * FAR), dict(w=AT + 4 * FAR),
    dict(c=cache(k=None)), dict(c=cache(head_stride=32)),
])
def test_weights_refusals(lib, kw):  # noqa: F811
    assert gather(lib, **kw) == INVALID


def test_weights_size_limits(lib):  # noqa: F811
    assert gather(lib, pages=1 << 28) == UNSUPPORTED
    assert gather(lib, c=cache(d=96, head_stride=96, token_stride=192, page_stride=4096)) == UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(w=None), dict(table=None), dict(lens=None), dict(out=None), dict(B=0), dict(pages=-1), dict(budget=-1),
    dict(first=-1), dict(recent=-1), dict(first=41, recent=0), dict(recent=41, first=0), dict(first=30, recent=11),
    dict(first=1 << 62, recent=1 << 62, budget=1 << 62),
    dict(w=AT + 2), dict(lens=AT + 2 * FAR + 1), dict(out=AT + 3 * FAR + 3),
    dict(out=AT + 2 * FAR), dict(out=AT + 2 * FAR + 8), dict(out=AT + FAR), dict(w=AT + FAR), dict(w=DATA),
    dict(w=0x300000000), dict(lens=DATA), dict(table=0x300000000), dict(out=AT),
    dict(c=cache(v=DATA)),                                    # keys and values in one place
    dict(c=cache(k=None)), dict(c=cache(token_stride=64)),
])
def test_evict_refusals(lib, kw):  # noqa: F811
    assert evict(lib, **kw) == INVALID


def test_evict_size_limits(lib):  # noqa: F811
    assert evict(lib, pages=1 << 28) == UNSUPPORTED
    assert evict(lib, B=1 << 27) == UNSUPPORTED
    assert evict(lib, c=cache(page_size=4, page_stride=4096)) == UNSUPPORTED


def test_no_tokens_need_no_pointers(lib):  # noqa: F811
    none = FaRows(None, 0, 0, 0)
    assert attend(lib, total=0, q=None, o=None, lse=None, ws=None) == fa.FA_OK
    assert append(lib, total=0, q=none, x=none, k=none, y=none, cu=None, lens=None) == fa.FA_OK
    assert gather(lib, total=0, q=None, lse=None, w=None) == fa.FA_OK


def test_null_descriptors(lib):  # noqa: F811
    assert lib.fa_forward_latent(AT, AT, AT, None, None, 0, None, None, 1, 1, 1, 1.0, 0, 0, 0, None, 0, None) == INVALID
    assert lib.fa_latent_append(None, None, None, None, None, None, 0, None, None, 1, 1, 1, None, None) == INVALID
    assert lib.fa_paged_weights(AT, AT, AT, None, None, 0, None, None, 1, 1, 1, 1.0, 0, 0, 0, None) == INVALID
    assert lib.fa_paged_evict(None, AT, None, 0, AT, AT, 1, 1, 0, 0, None) == INVALID


def test_binding_refuses_cpu_tensors():
    with pytest.raises(fa.FaError):
        fa.LatentCache(torch.zeros(2, 16, 576, dtype=torch.bfloat16), 512)
