"""Refusals of the norm-and-rotation and paged-cache calls, through the C ABI with
addresses that are never dereferenced: no GPU needed. And the rotary steps, which are
host arithmetic."""

import ctypes
import math
from fractions import Fraction

import pytest
import torch

import tiled_attention_03_gb300 as fa
from tiled_attention_03_gb300 import binding
from tiled_attention_03_gb300.binding import FaNormRope, FaPagedCache, load_library
from tiled_attention_03_gb300.build import build_library


class FaRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("head", ctypes.c_int64),
                ("token", ctypes.c_int64)]


def ref(x):
    return None if x is None else ctypes.byref(x)


INVALID, UNSUPPORTED = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
AT = 0x10000000
FAR = 0x10000000  # distance between the fake buffers


@pytest.fixture(scope="module")
def lib():
    build_library()
    return load_library()


def past_checks(rc):
    """A call whose arguments pass gets as far as the device (there is none here, or the
    addresses are not its memory)."""
    return rc in (fa.FA_ERR_CUDA, fa.FA_ERR_UNSUPPORTED) or (torch.cuda.is_available() and rc == INVALID)


def rope(**kw):
    a = dict(steps=0x90000000, rotary_dim=64, layout=0, magnitude=1.0, q_weight=0x91000000,
             k_weight=0x92000000, eps=1e-6)
    a.update(kw)
    return FaNormRope(*(a[n] for n, _ in FaNormRope._fields_))


def rows(i, H, N, d, data=None, batch=None, head=None, token=None):
    return FaRows(AT + i * FAR if data is None else data, H * N * d if batch is None else batch,
                  N * d if head is None else head, d if token is None else token)


def forward(lib, B=2, H=4, Hk=2, N=16, d=64, dtype=1, positions=0x93000000, r=None, **t):
    q = t.get("q", rows(0, H, N, d))
    k = t.get("k", rows(1, Hk, N, d))
    y = t.get("y", rows(2, H, N, d))
    z = t.get("z", rows(3, Hk, N, d))
    return lib.fa_qk_norm_rope(ref(q), ref(k), ref(y), ref(z), ref(rope() if r is None else r), positions, B, H, Hk, N, d, dtype, None)


def test_a_good_forward_passes_the_checks(lib):
    assert past_checks(forward(lib))
    none = FaRows(None, 0, 0, 0)
    assert past_checks(forward(lib, k=none, z=none, Hk=0))
    # one fused buffer: queries and keys beside each other, in place and into another one
    fused = dict(batch=16 * 8 * 64, head=64, token=8 * 64)
    q, k = rows(0, 4, 16, 64, **fused), rows(0, 2, 16, 64, data=AT + 4 * 64 * 2, **fused)
    assert past_checks(forward(lib, q=q, k=k, y=q, z=k))
    # the same with one token per batch entry, and with the batch inside the tokens
    for B, N, batch, token in ((3, 1, 8 * 64, 8), (3, 1, 8 * 64, 0), (2, 5, 8 * 64, 2 * 8 * 64)):
        q = rows(0, 4, N, 64, batch=batch, head=64, token=token)
        k = rows(0, 2, N, 64, data=AT + 4 * 64 * 2, batch=batch, head=64, token=token)
        assert past_checks(forward(lib, B=B, N=N, q=q, k=k, y=q, z=k)), (B, N)
        near = rows(0, 2, N, 64, data=AT + 3 * 64 * 2, batch=batch, head=64, token=token)
        assert forward(lib, B=B, N=N, y=q, z=near) == INVALID  # k_out over q_out's last head
        wide = rows(0, 2, N, 64, data=AT + 7 * 64 * 2, batch=batch, head=64, token=token)
        assert forward(lib, B=B, N=N, y=q, z=wide) == INVALID  # into the next token's q_out
    # a broadcast input: stride 0
    assert past_checks(forward(lib, q=rows(0, 4, 16, 64, head=0)))


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(N=0), dict(H=0), dict(Hk=-1), dict(dtype=2), dict(dtype=-1), dict(positions=0x93000002),
    dict(q=FaRows(None, 0, 0, 0)),                     # q_out without q
    dict(z=FaRows(None, 0, 0, 0)),                     # k without k_out
    dict(q=FaRows(AT + 8, 4096, 1024, 64)),            # 8-byte aligned
    dict(q=FaRows(AT, 4096, 1024, 60)),                # stride not a multiple of 8
    dict(q=FaRows(AT, 4096, -1024, 64)),
    dict(y=FaRows(AT + 2 * FAR, 4096, 0, 64)),         # heads written over each other
    dict(y=FaRows(AT + 2 * FAR, 4096, 1024, 32)),      # tokens written over each other
    dict(y=FaRows(AT + 64 * 2, 4096, 1024, 64)),       # one token behind q
    dict(y=FaRows(AT + FAR, 4096, 1024, 64)),          # q_out over k
    dict(z=FaRows(AT + 2 * FAR, 2048, 1024, 64)),      # k_out over q_out
    dict(positions=AT + 2 * FAR + 64),                 # positions inside q_out
    dict(r=rope(rotary_dim=-2)), dict(r=rope(rotary_dim=66)), dict(r=rope(rotary_dim=7)),
    dict(r=rope(steps=None)), dict(r=rope(steps=0x90000008)), dict(r=rope(layout=2)),
    dict(r=rope(magnitude=math.nan)), dict(r=rope(eps=-1.0)), dict(r=rope(eps=math.inf)),
    dict(r=rope(q_weight=0x91000002)), dict(r=rope(k_weight=AT + 2 * FAR)),
])
def test_forward_refusals(lib, kw):
    assert forward(lib, **kw) == INVALID


@pytest.mark.parametrize("d", [16, 48, 96, 512])
def test_head_dims(lib, d):
    assert forward(lib, d=d, r=rope(rotary_dim=16)) == UNSUPPORTED
    assert lib.fa_qk_norm_rope_backward_workspace_bytes(d) == 0
    assert lib.fa_forward_paged_workspace_bytes(d) == 0


def backward(lib, B=2, H=4, Hk=2, N=16, d=64, dwq=0x94000000, dwk=0x95000000, r=None, ws=0x96000000, ws_bytes=None,
             **t):
    names = ("q", "k", "dy", "dz", "dq", "dk")
    x = [t.get(n, rows(i, Hk if n in ("k", "dz", "dk") else H, N, d)) for i, n in enumerate(names)]
    if ws_bytes is None:
        ws_bytes = lib.fa_qk_norm_rope_backward_workspace_bytes(d)
    return lib.fa_qk_norm_rope_backward(*map(ref, x), dwq, dwk, ref(rope() if r is None else r), None, B, H, Hk, N, d, 1,
                                        ws, ws_bytes, None)


def test_a_good_backward_passes_the_checks(lib):
    assert past_checks(backward(lib))
    assert past_checks(backward(lib, dq=rows(2, 4, 16, 64), dk=rows(3, 2, 16, 64)))  # in place
    none = FaRows(None, 0, 0, 0)
    assert past_checks(backward(lib, q=none, k=none, dwq=None, dwk=None, r=rope(q_weight=None, k_weight=None), ws=None,
                                ws_bytes=0))


@pytest.mark.parametrize("kw", [
    dict(dwq=None), dict(dwk=None),                            # a weight without its gradient
    dict(r=rope(q_weight=None)),                               # a gradient without its weight
    dict(q=FaRows(None, 0, 0, 0)),                             # a weight without its input
    dict(dy=FaRows(None, 0, 0, 0)), dict(dk=FaRows(None, 0, 0, 0)),
    dict(ws=None), dict(ws_bytes=64), dict(ws=0x96000008), dict(ws=AT), dict(ws=AT + 4 * FAR),
    dict(dwq=0x94000002), dict(dwk=0x94000000), dict(dwq=AT + 5 * FAR),
    dict(dq=rows(0, 4, 16, 64)),                               # dq over q
    dict(dq=rows(5, 4, 16, 64)),                               # dq over dk
])
def test_backward_refusals(lib, kw):
    assert backward(lib, **kw) == INVALID


def cache(**kw):
    a = dict(k=0x200000000, v=0x300000000, page_stride=16 * 2 * 64, token_stride=2 * 64, head_stride=64,
             num_pages=100, page_size=16, H_kv=2, d=64, dtype=1)
    a.update(kw)
    return FaPagedCache(*(a[n] for n, _ in FaPagedCache._fields_))


def attend(lib, q=AT, o=AT + FAR, lse=AT + 2 * FAR, c=None, table=AT + 3 * FAR, pages=8, cu=AT + 4 * FAR,
           lens=AT + 5 * FAR, B=3, H=4, total=20, scale=0.125, mask=1, wl=0, wr=0, ws=AT + 6 * FAR, ws_bytes=1 << 26):
    return lib.fa_forward_paged(q, o, lse, ref(cache() if c is None else c), table, pages, cu, lens, B, H, total, scale, mask,
                                wl, wr, ws, ws_bytes, None)


def append(lib, H=4, B=3, total=20, table=AT + 5 * FAR, pages=8, cu=AT + 6 * FAR, lens=AT + 7 * FAR, c=None, r=None,
           **t):
    d = 64
    token = lambda i, h: FaRows(AT + i * FAR, 0, d, h * d)  # noqa: E731
    q, k, v, y = (t.get(n, token(i, h)) for i, (n, h) in enumerate((("q", H), ("k", 2), ("v", 2), ("y", H))))
    return lib.fa_paged_append(ref(q), ref(k), ref(v), ref(y), ref(cache() if c is None else c), table, pages, cu, lens, B,
                               H, total, ref(r), None)


def test_good_paged_calls_pass_the_checks(lib):
    assert past_checks(attend(lib))
    assert past_checks(append(lib))
    assert past_checks(append(lib, r=rope()))
    none = FaRows(None, 0, 0, 0)
    assert past_checks(append(lib, q=none, y=none))
    # head-major pages, and K and V of a page beside each other
    for c in (cache(token_stride=64, head_stride=16 * 64),
              cache(v=0x200000000 + 16 * 2 * 64 * 2, page_stride=2 * 16 * 2 * 64)):
        assert past_checks(attend(lib, c=c)) and past_checks(append(lib, c=c))


BAD_CACHES = [
    dict(k=None), dict(v=0x300000008), dict(dtype=3), dict(num_pages=0), dict(H_kv=0), dict(token_stride=0),
    dict(page_stride=2044), dict(head_stride=-64), dict(head_stride=32),       # heads over each other
    dict(token_stride=64),                                                     # tokens over heads
    dict(page_stride=1024),                                                    # pages over each other
]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_cache_refusals(lib, kw):
    assert attend(lib, c=cache(**kw)) == INVALID
    assert append(lib, c=cache(**kw)) == INVALID


@pytest.mark.parametrize("kw", [dict(page_size=4, page_stride=4096), dict(page_size=24, page_stride=4096),
                                dict(d=96, head_stride=96, token_stride=192, page_stride=4096)])
def test_unsupported_caches(lib, kw):
    assert attend(lib, c=cache(**kw)) == UNSUPPORTED
    assert append(lib, c=cache(**kw)) == UNSUPPORTED


def test_a_cache_of_too_many_steps_is_refused_by_every_call(lib):
    """The page and head strides' greatest common divisor is 8: 257 steps a page, and 8 a head. The
    limit does not depend on the kernel that a call would run."""
    strides = dict(page_stride=16 * 2 * 64 + 8)
    below, above = cache(num_pages=(2 ** 31 - 1 - 16) // 257, **strides), cache(num_pages=2 ** 31 // 257 + 1, **strides)
    for total in (3, 500):
        assert attend(lib, c=above, total=total) == UNSUPPORTED
    assert append(lib, c=above) == UNSUPPORTED
    if not torch.cuda.is_available():
        assert attend(lib, c=below) == fa.FA_ERR_CUDA and append(lib, c=below) == fa.FA_ERR_CUDA


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(o=None), dict(lse=None), dict(table=None), dict(cu=None), dict(lens=None), dict(ws=None),
    dict(B=0), dict(H=0), dict(H=5), dict(total=-1), dict(pages=-1), dict(scale=0.0), dict(scale=math.nan),
    dict(mask=3), dict(mask=2, wl=-1), dict(mask=2, wr=-1),
    dict(q=AT + 8), dict(o=AT + FAR + 16), dict(lse=AT + 2 * FAR + 2), dict(cu=AT + 2), dict(table=AT + 1),
    dict(ws=AT + 6 * FAR + 16), dict(ws_bytes=1000),
    dict(o=AT), dict(lse=AT + FAR + 64), dict(o=0x200000000), dict(ws=0x300000020), dict(ws=AT + FAR),
])
def test_attention_refusals(lib, kw):
    assert attend(lib, **kw) == INVALID


def test_attention_size_limits(lib):
    assert attend(lib, pages=1 << 28) == UNSUPPORTED
    assert attend(lib, total=(1 << 29) + 1, o=1 << 50) == UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(k=FaRows(None, 0, 0, 0)), dict(v=FaRows(None, 0, 0, 0)), dict(q=FaRows(None, 0, 0, 0)),
    dict(table=None), dict(cu=None), dict(lens=None), dict(B=0), dict(total=-1), dict(lens=AT + 7 * FAR + 2),
    dict(k=FaRows(AT + 4, 0, 64, 128)), dict(y=FaRows(AT + 3 * FAR, 0, 0, 256)), dict(y=FaRows(AT + FAR, 0, 64, 256)),
    dict(k=FaRows(0x200000000, 0, 64, 128)), dict(lens=0x300000000), dict(r=rope(rotary_dim=128)),
    dict(cu=AT + 3 * FAR),                                # the batch's arrays inside q_out
])
def test_append_refusals(lib, kw):
    assert append(lib, **kw) == INVALID


def test_append_needs_keys_and_values_apart(lib):
    one = cache(v=0x200000000)
    assert one.k == one.v
    assert append(lib, c=one) == INVALID
    assert past_checks(attend(lib, c=one))


def test_no_tokens_need_no_pointers(lib):
    assert attend(lib, total=0, q=None, o=None, lse=None, ws=None) == fa.FA_OK
    none = FaRows(None, 0, 0, 0)
    assert append(lib, total=0, q=none, k=none, v=none, y=none, cu=None, lens=None) == fa.FA_OK


def test_null_descriptors(lib):
    assert lib.fa_forward_paged(AT, AT, AT, None, None, 0, None, None, 1, 1, 1, 1.0, 0, 0, 0, None, 0, None) == INVALID
    assert lib.fa_paged_append(None, None, None, None, None, None, 0, None, None, 1, 1, 1, None, None) == INVALID
    assert lib.fa_qk_norm_rope(None, None, None, None, None, None, 1, 1, 1, 1, 64, 0, None) == INVALID
    assert lib.fa_qk_norm_rope(None, None, None, None, ref(rope()), None, 1, 1, 1, 1, 64, 0, None) == INVALID


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(fa.FaError):
        fa.qk_norm_rope(x, None, fa.NormRope())
    with pytest.raises(fa.FaError):
        fa.PagedCache(x[None], x[None])
    with pytest.raises(fa.FaError):
        fa.NormRope(torch.zeros(4, dtype=torch.int64))


def test_an_integer_handle_names_the_stream_it_belongs_to(monkeypatch):
    """0 (and CUDA's other name for it, 1) is the default stream, not one of PyTorch's pool."""
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    assert binding._on(0) == "default" and binding._on(1) == "default"
    assert binding._on(0x7F0000001000) == ("external", 0x7F0000001000)


# ------------------------------------------------------------------------ rotary steps

TURN = Fraction("6.283185307179586476925286766559005768394338798750")  # 2 pi, 48 digits


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "band"])
def test_steps_are_the_frequencies_in_turns(scaling):
    freq = fa.rope_frequencies(128, 10000.0, scaling, 4.0, 4096)
    for f, s in zip(freq, fa.fa_rope_steps(freq)):
        exact = Fraction(f) / TURN * 2 ** 64
        # the product with 1 / (2 pi) in 64 bits: two roundings of 2^-53
        assert abs(s - exact) <= float(exact) * 2.0 ** -52 + 1


def test_steps_wrap_whole_turns():
    assert fa.fa_rope_steps([0.0, -0.0]) == [0, 0]
    a, b = fa.fa_rope_steps([0.25, -0.25])
    assert (a + b) % (1 << 64) == 0
    big, = fa.fa_rope_steps([7.0])
    exact = (Fraction(7) / TURN) % 1 * 2 ** 64
    assert abs(big - exact) <= 2.0 ** 64 * 2.0 ** -51


def test_steps_refusals(lib):
    f, s = (ctypes.c_double * 2)(1.0, 2.0), (ctypes.c_uint64 * 2)()
    assert lib.fa_rope_steps(None, 2, s) == INVALID
    assert lib.fa_rope_steps(f, 2, None) == INVALID
    assert lib.fa_rope_steps(f, 0, s) == INVALID
    for bad in (math.inf, math.nan, 2.0 ** 20):
        with pytest.raises(fa.FaError):
            fa.fa_rope_steps([1.0, bad])


def test_frequency_scalings():
    plain = fa.rope_frequencies(64)
    assert plain[0] == 1.0 and plain[1] == pytest.approx(10000.0 ** (-1 / 32))
    assert fa.rope_frequencies(64, scaling="linear", factor=4.0) == [x / 4.0 for x in plain]
    base = fa.rope_frequencies(64, scaling="base", factor=4.0)
    assert base[0] == 1.0 and base[-1] == pytest.approx(plain[-1] / 4.0)
    band = fa.rope_frequencies(64, scaling="band", factor=4.0, context=4096, slow=1.0, fast=32.0)
    for f, x in zip(plain, band):
        turns = 4096 * f / (2 * math.pi)
        if turns >= 32:
            assert x == f
        elif turns <= 1:
            assert x == f / 4.0
        else:
            assert f / 4.0 < x < f
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=64, scaling="other"),
                dict(rotary_dim=64, scaling="band", slow=4.0, fast=4.0), dict(rotary_dim=2, scaling="base")):
        with pytest.raises(fa.FaError):
            fa.rope_frequencies(**bad)
