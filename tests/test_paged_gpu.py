"""The paged cache: fa_paged_append and fa_forward_paged against their definitions in 64
bits. Everything that the calls must not look at (slots past a sequence's end, pages that
belong to nobody, table entries past a sequence) holds NaN or nonsense."""

import ctypes
import math
import random

import pytest
import torch

import tiled_attention_03_gb300 as fa
from tiled_attention_03_gb300 import binding

from rope_util import assert_within, attention_ref, norm_rope_ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
NAN = float("nan")


def empty_cache(pages, page, Hk, d, dtype, layout):
    """k and v (pages, page, Hk, d) full of NaN, by the memory layout's name."""
    if layout == "token":
        k, v = (torch.full((pages, page, Hk, d), NAN, dtype=dtype, device=DEV) for _ in range(2))
    elif layout == "head":
        k, v = (torch.full((pages, Hk, page, d), NAN, dtype=dtype, device=DEV).transpose(1, 2) for _ in range(2))
    else:  # K and V of a page together, the heads padded to a wider row
        both = torch.full((pages, 2, page, Hk, d + 8), NAN, dtype=dtype, device=DEV)
        k, v = both[:, 0, :, :, :d], both[:, 1, :, :, :d]
    return k, v


def paged(lens, H, Hk, d, dtype, page, layout="token", seed=0, spare=3, pad_tokens=0):
    """A serving batch: lens = [(new, keys)]. Returns q, the cache, the batch arrays and
    each sequence's (q, k, v)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV).to(dtype)  # noqa: E731
    need = [-(-n // page) for _, n in lens]
    pages = sum(need) + spare
    k, v = empty_cache(pages, page, Hk, d, dtype, layout)
    order = list(range(pages))
    random.Random(seed).shuffle(order)
    width = max(max(need), 1) + 1
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    table[:, -1] = 2 ** 30
    seqs, at, cu = [], 0, [0]
    for b, (lq, lk) in enumerate(lens):
        mine = order[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = torch.tensor(mine, dtype=torch.int32)
        kk, vv = randn(lk, Hk, d), randn(lk, Hk, d)
        for n, pg in enumerate(mine):
            part = slice(n * page, min((n + 1) * page, lk))
            k[pg, :part.stop - part.start] = kk[part]
            v[pg, :part.stop - part.start] = vv[part]
        seqs.append((randn(lq, H, d), kk, vv))
        cu.append(cu[-1] + lq)
    q = torch.cat([s[0] for s in seqs] + [randn(pad_tokens, H, d)])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return q, fa.PagedCache(k, v), table.to(DEV), i32(cu), i32([n for _, n in lens]), seqs


def run(q, cache, table, cu, lens, scale, mask, window=(0, 0), **kw):
    o = torch.full_like(q, -777.0)
    lse = torch.full(q.shape[:2], -777.0, device=DEV)
    fa.fa_forward_paged(q, o, lse, cache, table, cu, lens, scale, mask, window[0], window[1], **kw)
    st = fa.fa_sync_status()
    assert st == fa.FA_OK, fa.fa_status_string(st)
    return o, lse


def check(o, lse, seqs, scale, mask, window, dtype):
    t = 0
    for b, (q, k, v) in enumerate(seqs):
        n = q.shape[0]
        want, bound, wl, lb = attention_ref(q, k, v, scale, mask, window, dtype)
        assert_within(o[t:t + n], want, bound, f"sequence {b}: O")
        got = lse[t:t + n].double()
        none = wl == -math.inf
        assert torch.equal(got == -math.inf, none), f"sequence {b}: rows without keys"
        assert bool((o[t:t + n][none] == 0).all())
        assert_within(got[~none], wl[~none], lb[~none], f"sequence {b}: LSE")
        t += n
    assert bool((o[t:] == -777.0).all()) and bool((lse[t:] == -777.0).all()), "wrote a padded row"


LENS = {
    "steps": [(1, 1), (1, 17), (1, 128), (1, 129), (1, 1000), (0, 50), (1, 64), (1, 2), (0, 0), (1, 333)],
    "chunks": [(5, 5), (130, 300), (64, 64), (1, 700), (33, 1000), (0, 9), (200, 257)],
    "nothing": [(3, 0), (7, 3), (0, 0), (1, 0), (2, 40)],
}
MASKS = [("none", (0, 0)), ("causal", (0, 0)), ("window", (90, 3)), ("window", (0, 0))]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("mask,window", MASKS)
@pytest.mark.parametrize("lens", list(LENS))
def test_masks_and_lengths(lens, mask, window, d, dtype):
    page, layout = {32: (8, "head"), 64: (16, "token"), 128: (32, "both"), 256: (128, "head")}[d]
    b = paged(LENS[lens], 4, 2, d, dtype, page, layout, seed=d, pad_tokens=3)
    o, lse = run(*b[:5], d ** -0.5, mask, window)
    check(o, lse, b[5], d ** -0.5, mask, window, dtype)


@pytest.mark.parametrize("page", [8, 16, 64, 128, 512])
@pytest.mark.parametrize("layout", ["token", "head", "both"])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("lens", [[(1, 600), (20, 130), (1, 127), (3, 1025)], [(1, 600), (1, 7), (2, 1025)]])
def test_pages(lens, page, layout, d):
    b = paged(lens, 6, 2, d, torch.bfloat16, page, layout, seed=page)
    o, lse = run(*b[:5], d ** -0.5, "causal")
    check(o, lse, b[5], d ** -0.5, "causal", (0, 0), torch.bfloat16)


@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (8, 1), (7, 1), (6, 2), (64, 4), (40, 8), (256, 1), (130, 1)])
def test_heads(H, Hk):
    d, dtype = 64, torch.float16
    b = paged([(1, 300), (9, 140), (1, 5)], H, Hk, d, dtype, 16, seed=H)
    o, lse = run(*b[:5], d ** -0.5, "causal")
    check(o, lse, b[5], d ** -0.5, "causal", (0, 0), dtype)


@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.float16), (256, torch.bfloat16)])
@pytest.mark.parametrize("mask,window", [("causal", (0, 0)), ("window", (20000, 0))])
@pytest.mark.parametrize("new", [2, 50])
def test_long_sequences_are_cut_and_joined(new, d, dtype, mask, window):
    """A unit of some hundred tiles over all workers, with short ones around it."""
    b = paged([(1, 40), (new, 38500), (1, 2000)], 4, 1, d, dtype, 64, "head", seed=1)
    o, lse = run(*b[:5], d ** -0.5, mask, window)
    check(o, lse, b[5], d ** -0.5, mask, window, dtype)
    again = run(*b[:5], d ** -0.5, mask, window)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("new", [[0, 1, 1, 1, 2, 30], [0, 1, 1, 1, 2]])
@pytest.mark.parametrize("H,Hk", [(4, 2), (24, 1)])
def test_many_sequences(H, Hk, new):
    rng = random.Random(3)
    lens = [(rng.choice(new), rng.choice([0, 1, 50, 400])) for _ in range(700)]
    b = paged(lens, H, Hk, 64, torch.bfloat16, 16, seed=9)
    o, lse = run(*b[:5], 0.125, "causal")
    check(o, lse, b[5], 0.125, "causal", (0, 0), torch.bfloat16)


@pytest.mark.parametrize("B", [12, 300])
@pytest.mark.parametrize("kind", ["steps", "one chunk", "long steps"])
@pytest.mark.parametrize("d", [64, 256])
def test_few_tokens_per_sequence(d, kind, B):
    """A few tokens per sequence on average: every sequence some (the decode kernel), or one
    a chunk and the others one (the chunk kernel), as the device finds."""
    rng = random.Random(B)
    lens = [(rng.choice([2, 3, 4]), rng.choice([4, 100, 700])) for _ in range(B)]
    if kind == "one chunk":
        lens = [(1, n) for _, n in lens]
        lens[B // 2] = (4 * B, 4 * B + 321)
    elif kind == "long steps":
        lens[-1] = (16, 900)
    b = paged(lens, 4, 2, d, torch.bfloat16, 16, seed=B)
    o, lse = run(*b[:5], 0.1, "causal")
    check(o, lse, b[5], 0.1, "causal", (0, 0), torch.bfloat16)


@pytest.mark.parametrize("B", [40, 128, 200])
@pytest.mark.parametrize("chunks", [1, 2])
@pytest.mark.parametrize("d,H,Hk", [(32, 8, 2), (64, 4, 4), (128, 8, 1), (256, 4, 2)])
def test_a_chunk_among_empty_sequences(d, H, Hk, chunks, B):
    """No more tokens than sequences, and most sequences without any: a captured step of fixed
    size. As many single tokens as sequences beside it."""
    lens = [(0, n) for n in [0, 50] * (B // 2)]
    lens[B // 3] = (B - chunks + 1, B + 1500)
    if chunks == 2:
        lens[-1] = (1, 700)
    b = paged(lens, H, Hk, d, torch.bfloat16, 16, seed=B)
    check(*run(*b[:5], 0.1, "causal"), b[5], 0.1, "causal", (0, 0), torch.bfloat16)
    b = paged([(1, 1 + 7 * i % 500) for i in range(B)], H, Hk, d, torch.bfloat16, 16, seed=B)
    check(*run(*b[:5], 0.1, "causal"), b[5], 0.1, "causal", (0, 0), torch.bfloat16)


def test_a_workspace_passed_on():
    """One workspace, used by batches of all kinds in turn: what a call leaves there means
    nothing to the next (each is larger than the one before)."""
    ws = torch.zeros(fa.fa_forward_paged_workspace_bytes(128), dtype=torch.uint8, device=DEV)
    batches = [[(1, 4000)], [(70, 3000), (1, 900)], [(1, 2000)] * 90, [(2, 500)] * 60, [(1, 300)] * 79 + [(150, 9000)],
               [(1, 700)] * 500]
    for i, lens in enumerate(batches + batches[3:]):
        b = paged(lens, 4, 1, 128, torch.bfloat16, 64, "head", seed=i)
        o, lse = run(*b[:5], 0.1, "causal", workspace=ws)
        check(o, lse, b[5], 0.1, "causal", (0, 0), torch.bfloat16)


def test_long_prompt_chunk():
    b = paged([(1500, 4100), (1, 100)], 8, 2, 128, torch.bfloat16, 16, seed=4)
    o, lse = run(*b[:5], 128 ** -0.5, "causal")
    check(o, lse, b[5], 128 ** -0.5, "causal", (0, 0), torch.bfloat16)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_peaky_scores(d, new):
    """Scores of a few hundred: the reference maximum moves and O is rescaled."""
    dtype = torch.bfloat16
    b = paged([(1, 900), (new, 700)], 4, 4, d, dtype, 16, seed=6)
    o, lse = run(*b[:5], 3.0, "causal")
    check(o, lse, b[5], 3.0, "causal", (0, 0), dtype)


@pytest.mark.parametrize("H", [8, 80])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_window_does_not_look_at_what_it_left_behind(d, H):
    """Before the window of the only query, a page may have been given away: NaN in its
    keys and values and a nonsense page number change nothing."""
    dtype, page = torch.bfloat16, 16
    q, cache, table, cu, lens, seqs = paged([(1, 500), (1, 300)], H, 2, d, dtype, page, seed=8)
    want = run(q, cache, table, cu, lens, 0.1, "window", (100, 0))
    for b, n in ((0, 500), (1, 300)):
        first = n - 1 - 100
        for j in range(first):
            cache.k[int(table[b, j // page]), j % page] = NAN
            cache.v[int(table[b, j // page]), j % page] = NAN
        table[b, :first // page] = torch.tensor([-1, 2 ** 30, 10 ** 6] * 40, dtype=torch.int32)[:first // page]
    got = run(q, cache, table, cu, lens, 0.1, "window", (100, 0))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check(*got, seqs, 0.1, "window", (100, 0), dtype)


@pytest.mark.parametrize("H", [2, 40])
def test_nan_in_a_visible_key_is_seen(H):
    q, cache, table, cu, lens, _ = paged([(1, 200), (1, 200)], H, 1, 64, torch.float16, 16, seed=2)
    cache.k[int(table[0, 3]), 5] = NAN
    o, lse = run(q, cache, table, cu, lens, 0.125, "causal")
    assert bool(torch.isnan(o[0]).all()) and bool(torch.isnan(lse[0]).all())
    assert bool(torch.isfinite(o[1]).all()) and bool(torch.isfinite(lse[1]).all())


@pytest.mark.parametrize("H", [2, 40])
def test_page_numbers_outside_the_cache_read_as_zeros(H):
    q, cache, table, cu, lens, _ = paged([(1, 40)], H, 2, 64, torch.bfloat16, 16, seed=2)
    zero_k, zero_v = cache.k.clone(), cache.v.clone()
    zero_k[int(table[0, 1])] = 0
    zero_v[int(table[0, 1])] = 0
    want = run(q, fa.PagedCache(zero_k, zero_v), table, cu, lens, 0.125, "causal")
    for bad in (-1, cache.num_pages, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 1] = bad
        got = run(q, cache, t, cu, lens, 0.125, "causal")
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("B,T,H,Hk,width", [
    (8192, 4096, 64, 64, 128),   # units of 16 rows, sequences searched by the block
    (128, 128, 64, 64, 13000),   # units of 16 rows, sequences searched by a warp
    (8192, 4096, 64, 2, 128)])   # units of 128 rows
def test_offsets_in_no_order_write_nothing_outside(B, T, H, Hk, width):
    """Every second sequence owns all T tokens: the work of all of them passes 2^32."""
    d, page, guard = 32, 512, 64
    k, v = (torch.zeros(4, page, Hk, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cache = fa.PagedCache(k, v)
    table = torch.arange(B * width, device=DEV).remainder(4).to(torch.int32).view(B, width)
    cu = torch.tensor([0, T] * (B // 2) + [0], dtype=torch.int32, device=DEV)
    lens = torch.full((B,), width * page, dtype=torch.int32, device=DEV)
    q = torch.zeros(T, H, d, dtype=torch.bfloat16, device=DEV)
    o = torch.full((T + 2 * guard, H, d), -777.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T + 2 * guard, H), -777.0, device=DEV)
    fa.fa_forward_paged(q, o[guard:-guard], lse[guard:-guard], cache, table, cu, lens, 1.0, "none", 0, 0)
    assert fa.fa_sync_status() == fa.FA_OK
    for x in (o, lse):
        assert bool((x[:guard] == -777.0).all()) and bool((x[-guard:] == -777.0).all())
    q, cache, table, cu, lens, seqs = paged([(1, 90), (1, 700)], H, Hk, d, torch.bfloat16, 16, seed=3)
    check(*run(q, cache, table, cu, lens, d ** -0.5, "causal"), seqs, d ** -0.5, "causal", (0, 0), torch.bfloat16)


def test_lengths_are_clamped_to_the_table():
    q, cache, table, cu, lens, _ = paged([(1, 48), (1, 30)], 2, 1, 64, torch.bfloat16, 16, seed=2)
    three = table[:, :3].contiguous()
    want = run(q, cache, three, cu, lens, 0.125, "causal")
    big = lens.clone()
    big[0] = 2 ** 31 - 1
    got = run(q, cache, three, cu, big, 0.125, "causal")
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_cache_past_32_bits():
    """Pages whose elements lie past 2^31 (and bytes past 2^32) of the buffer."""
    page, Hk, d, dtype = 128, 8, 128, torch.bfloat16
    pages = (2 ** 31) // (page * Hk * d) + 40
    k, v = (torch.empty(pages, page, Hk, d, dtype=dtype, device=DEV) for _ in range(2))
    cache = fa.PagedCache(k, v)
    mine = [pages - 1, 3, pages - 7]
    table = torch.tensor([mine], dtype=torch.int32, device=DEV)
    for pg in mine:
        k[pg] = NAN
        v[pg] = NAN
    lq, lk = 300, 300
    g = torch.Generator(device=DEV).manual_seed(1)
    q, kk, vv = (torch.randn(lk, h, d, generator=g, device=DEV).to(dtype) for h in (16, Hk, Hk))
    cu = torch.tensor([0, lq], dtype=torch.int32, device=DEV)
    lens = torch.tensor([lk], dtype=torch.int32, device=DEV)
    fa.fa_paged_append(None, kk, vv, None, cache, table, cu, lens)
    o, lse = run(q, cache, table, cu, lens, d ** -0.5, "causal")
    check(o, lse, [(q, kk, vv)], d ** -0.5, "causal", (0, 0), dtype)


def rope_handle(d, r, layout, dtype, norm, seed=5):
    freq = fa.rope_frequencies(r) if r else []
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = (1 + 0.3 * torch.randn(2, d, generator=g, device=DEV)).to(dtype)
    return fa.NormRope(fa.rope_steps(r) if r else None, layout, 1.0, w[0] if norm else None,
                       w[1] if norm else None, 1e-5), freq


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d,r,layout,page,cache_layout", [
    (32, 8, "half", 8, "token"), (64, 64, "interleaved", 16, "head"), (128, 128, "half", 64, "both"),
    (256, 64, "half", 16, "token"), (128, 0, "half", 128, "head")])
@pytest.mark.parametrize("lens", ["steps", "chunks", "nothing", "many"])
def test_append(lens, d, r, layout, page, cache_layout, dtype):
    H, Hk = 5, 2
    if lens == "many":
        rng = random.Random(7)
        ls = [(rng.choice([0, 1, 1, 2, 40]), 0) for _ in range(300)]
        ls = [(n, n + rng.choice([0, 0, 3, 100])) for n, _ in ls]
    else:
        ls = LENS[lens]
    norm = d != 64
    _, cache, table, cu, lk, _ = paged(ls, H, Hk, d, dtype, page, cache_layout, seed=d)
    total = int(cu[-1])
    g = torch.Generator(device=DEV).manual_seed(11)
    qkv = torch.randn(total + 4, H + 2 * Hk, d, generator=g, device=DEV).to(dtype)  # 4 padded rows
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    rope, freq = rope_handle(d, r, layout, dtype, norm)
    before = cache.k.clone(), cache.v.clone()
    q_out = torch.full((total + 4, H, d), -777.0, dtype=dtype, device=DEV)
    fa.fa_paged_append(q, k, v, q_out, cache, table, cu, lk, rope)
    assert fa.fa_sync_status() == fa.FA_OK
    assert bool((q_out[total:] == -777.0).all()), "wrote a padded row"
    ek, ev = before
    for b, (n, keys) in enumerate(ls):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        pos = torch.arange(keys - n, keys, device=DEV)
        want, bound = norm_rope_ref(q[rows], rope.q_weight, pos, freq, layout, 1.0, 1e-5, dtype)
        assert_within(q_out[rows], want, bound, f"sequence {b}: q")
        want, bound = norm_rope_ref(k[rows], rope.k_weight, pos, freq, layout, 1.0, 1e-5, dtype)
        for i in range(n):
            if keys - n + i < 0:
                continue
            at = int(table[b, int(pos[i]) // page]), int(pos[i]) % page
            assert_within(cache.k[at], want[i], bound[i], f"sequence {b}, token {i}: k")
            ek[at] = cache.k[at]  # checked; nothing else may differ
            ev[at] = v[rows][i]
    same = lambda a, b: torch.equal(a.nan_to_num(nan=1e4), b.nan_to_num(nan=1e4))  # noqa: E731
    assert same(cache.k, ek) and same(cache.v, ev)


def test_append_without_queries_or_rope_copies():
    _, cache, table, cu, lk, _ = paged([(3, 20), (1, 33)], 2, 2, 64, torch.bfloat16, 16, seed=1)
    kv = torch.randn(4, 4, 64, device=DEV).to(torch.bfloat16)
    fa.fa_paged_append(None, kv[:, :2], kv[:, 2:], None, cache, table, cu, lk)
    for b, pos, t in ((0, 17, 0), (0, 18, 1), (0, 19, 2), (1, 32, 3)):
        at = int(table[b, pos // 16]), pos % 16
        assert torch.equal(cache.k[at], kv[t, :2]) and torch.equal(cache.v[at], kv[t, 2:])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rope", [False, True])
def test_append_without_norm_and_rotation_keeps_the_bits(rope, dtype):
    """Every 16-bit pattern, the zero below 0 and each NaN among them, with rope = NULL and with
    one that does nothing."""
    d, n, page = 64, 2 ** 16 // 256, 16
    x = torch.arange(-2 ** 15, 2 ** 15, device=DEV).to(torch.int16).view(n, 4, d).view(dtype)
    k, v = (torch.zeros(n // page, page, 4, d, dtype=dtype, device=DEV) for _ in range(2))
    table = torch.arange(n // page, dtype=torch.int32, device=DEV)[None]
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    q = torch.zeros_like(x)
    fa.fa_paged_append(x, x, x, q, fa.PagedCache(k, v), table, cu, cu[1:], fa.NormRope() if rope else None)
    assert fa.fa_sync_status() == fa.FA_OK
    for y in (q, k.view(n, 4, d), v.view(n, 4, d)):
        assert torch.equal(y.view(torch.int16), x.view(torch.int16))


@pytest.mark.parametrize("any_stride", [-8, 5, -2 ** 62])
def test_append_of_one_head_and_one_token_by_any_strides(any_stride):
    """Strides of dimensions of one entry, in the rows and in the cache, are not looked at."""
    d, page = 64, 16
    lib = binding.load_library()
    x = torch.randn(3, 1, d, device=DEV).to(torch.bfloat16)
    k, v = (torch.full((1, page, 1, d), NAN, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    c = binding.FaPagedCache(k.data_ptr(), v.data_ptr(), any_stride, d, any_stride, 1, page, 1, d, 1)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    lens = torch.tensor([7], dtype=torch.int32, device=DEV)
    q = torch.full((1, 1, d), NAN, dtype=torch.bfloat16, device=DEV)
    rows = lambda t: binding._pack_rows(t.data_ptr(), any_stride, any_stride, any_stride)  # noqa: E731
    assert lib.fa_paged_append(rows(x[0]), rows(x[1]), rows(x[2]), rows(q), ctypes.addressof(c), table.data_ptr(), 1,
                               cu.data_ptr(), lens.data_ptr(), 1, 1, 1, None, None) == fa.FA_OK
    assert fa.fa_sync_status() == fa.FA_OK
    assert torch.equal(q[0], x[0]) and torch.equal(k[0, 6], x[1]) and torch.equal(v[0, 6], x[2])
    assert int(torch.isnan(k).sum()) == int(torch.isnan(v).sum()) == (page - 1) * d


def test_append_skips_pages_outside_the_cache():
    _, cache, table, cu, lk, _ = paged([(20, 20)], 2, 2, 64, torch.bfloat16, 16, seed=1)
    kv = torch.randn(20, 2, 64, device=DEV).to(torch.bfloat16)
    before = cache.k.clone()
    for bad in (-1, cache.num_pages, 2 ** 31 - 1):
        t = table.clone()
        t[0, :2] = bad
        fa.fa_paged_append(None, kv, kv, None, cache, t, cu, lk)
        assert fa.fa_sync_status() == fa.FA_OK
    assert torch.equal(cache.k.nan_to_num(nan=1e4), before.nan_to_num(nan=1e4))


@pytest.mark.parametrize("d,layout", [(128, "half"), (64, "interleaved")])
def test_serving_loop_matches_a_whole_prompt(d, layout):
    """Prompts in chunks, then single tokens, appended and attended step by step: the rows
    of each step against attention in 64 bits over the whole rotated sequences."""
    dtype, H, Hk, page = torch.bfloat16, 8, 2, 16
    final = [45, 150, 7]
    g = torch.Generator(device=DEV).manual_seed(3)
    qkv = [torch.randn(n, H + 2 * Hk, d, generator=g, device=DEV).to(dtype) for n in final]
    rope, freq = rope_handle(d, d, layout, dtype, True)
    pages = 40
    k, v = empty_cache(pages, page, Hk, d, dtype, "token")
    cache = fa.PagedCache(k, v)
    table = torch.randperm(pages, device=DEV, generator=g)[:30].to(torch.int32).view(3, 10)
    done = [0, 0, 0]
    outs = [[] for _ in final]
    whole = [torch.empty(n, Hk, d, dtype=dtype, device=DEV) for n in final]
    rot = [torch.empty(n, H, d, dtype=dtype, device=DEV) for n in final]
    while done != final:
        n = [min(f - x, 64 if x == 0 else (30 if x < 100 else 1)) for f, x in zip(final, done)]
        cu = torch.tensor([0, n[0], n[0] + n[1], sum(n)], dtype=torch.int32, device=DEV)
        lk = torch.tensor([x + y for x, y in zip(done, n)], dtype=torch.int32, device=DEV)
        x = torch.cat([qkv[b][done[b]:done[b] + n[b]] for b in range(3)])
        q = torch.empty(sum(n), H, d, dtype=dtype, device=DEV)
        fa.fa_paged_append(x[:, :H], x[:, H:H + Hk], x[:, H + Hk:], q, cache, table, cu, lk, rope)
        o, lse = fa.forward_paged(q, cache, table, cu, lk)
        for b in range(3):
            rows = slice(int(cu[b]), int(cu[b + 1]))
            outs[b].append((o[rows], lse[rows]))
            rot[b][done[b]:done[b] + n[b]] = q[rows]
        done = [x + y for x, y in zip(done, n)]
    assert fa.fa_sync_status() == fa.FA_OK
    for b, f in enumerate(final):
        for j in range(f):
            whole[b][j] = cache.k[int(table[b, j // page]), j % page]
        pos = torch.arange(f, device=DEV)
        want, bound = norm_rope_ref(qkv[b][:, H:H + Hk], rope.k_weight, pos, freq, layout, 1.0, 1e-5, dtype)
        assert_within(whole[b], want, bound, "cached keys")
        want, bound, wl, lb = attention_ref(rot[b], whole[b], qkv[b][:, H + Hk:], d ** -0.5, "causal", (0, 0), dtype)
        assert_within(torch.cat([x for x, _ in outs[b]]), want, bound, "O")
        assert_within(torch.cat([x for _, x in outs[b]]), wl, lb, "LSE")


def test_capture_follows_the_lengths():
    """A captured step replayed as the sequences grow: the lengths are read on the device."""
    d, dtype, H, Hk, page, B = 128, torch.bfloat16, 8, 2, 16, 3
    rope, _ = rope_handle(d, d, "half", dtype, True)
    k, v = (torch.zeros(60, page, Hk, d, dtype=dtype, device=DEV) for _ in range(2))
    cache, other = fa.PagedCache(k, v), fa.PagedCache(k.clone(), v.clone())
    table = torch.randperm(60, device=DEV).to(torch.int32).view(B, 20)
    cu = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    lk = torch.tensor([3, 200, 129], dtype=torch.int32, device=DEV)
    qkv = torch.zeros(B, H + 2 * Hk, d, dtype=dtype, device=DEV)
    q, o = (torch.empty(B, H, d, dtype=dtype, device=DEV) for _ in range(2))
    lse = torch.empty(B, H, device=DEV)
    ws = torch.empty(fa.fa_forward_paged_workspace_bytes(d), dtype=torch.uint8, device=DEV)

    def step(c, stream=None):
        fa.fa_paged_append(qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], q, c, table, cu, lk, rope, stream)
        fa.fa_forward_paged(q, o, lse, c, table, cu, lk, 0.1, "causal", 0, 0, ws, stream)

    s = torch.cuda.Stream()
    step(other)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(cache, s)
    for i in range(12):
        qkv.copy_(torch.randn(qkv.shape, device=DEV))
        lk += 1
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), lse.clone()
        o.fill_(NAN)
        step(other)
        torch.cuda.synchronize()
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
        assert torch.equal(cache.k, other.k) and torch.equal(cache.v, other.v)
    assert fa.fa_sync_status() == fa.FA_OK


@pytest.mark.parametrize("d", [64, 256])
def test_capture_follows_the_tokens(d):
    """A captured step of 64 sequences and 64 tokens, replayed as the tokens move from single steps
    to a chunk of one sequence, to a few for each of some, and back."""
    B, H, Hk, page = 64, 8, 2, 16
    q, cache, table, cu, lk, _ = paged([(1, 400)] * B, H, Hk, d, torch.bfloat16, page, seed=d)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    ws = torch.empty(fa.fa_forward_paged_workspace_bytes(d), dtype=torch.uint8, device=DEV)
    step = lambda: fa.fa_forward_paged(q, o, lse, cache, table, cu, lk, 0.1, "causal", 0, 0, ws)  # noqa: E731
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rows = [torch.stack([x[table[b, j // page], j % page] for j in range(400)])
            for x in (cache.k, cache.v) for b in range(B)]
    for new in ([1] * B, [0] * 40 + [64] + [0] * 23, [4] * 16 + [0] * 48, [0] * 10 + [30, 34] + [0] * 52, [1] * B):
        cu.copy_(torch.tensor([sum(new[:b]) for b in range(B + 1)]))
        o.fill_(NAN)
        torch.cuda.synchronize()
        graph.replay()
        assert fa.fa_sync_status() == fa.FA_OK
        at = [sum(new[:b]) for b in range(B)]
        seqs = [(q[at[b]:at[b] + new[b]], rows[b], rows[B + b]) for b in range(B)]
        check(o, lse, seqs, 0.1, "causal", (0, 0), torch.bfloat16)


@pytest.mark.parametrize("new", [1, 60])
def test_two_streams_at_once(new):
    """Two calls that may overlap, without a workspace of the caller's, on streams of their
    own; many times, against the same calls one after the other."""
    bs = [paged([(new, 3000), (2, 700)], 8, 2, 128, torch.bfloat16, 16, seed=i) for i in range(2)]
    want = [run(*b[:5], 0.1, "causal") for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [(torch.empty_like(b[0]), torch.empty(b[0].shape[:2], device=DEV)) for b in bs]
        torch.cuda.synchronize()
        for b, s, (o, lse) in zip(bs, streams, got):
            fa.fa_forward_paged(b[0], o, lse, *b[1:5], 0.1, "causal", stream=s)
        torch.cuda.synchronize()
        for (o, lse), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)


def test_the_fault_hook_ends_in_a_timeout():
    """A K load that never comes: the waits run out, the call reports it, and the next
    call is right."""
    b = paged([(40, 600)], 2, 1, 128, torch.bfloat16, 16, seed=3)
    want = run(*b[:5], 0.1, "causal")
    fa.fa_set_wait_budget_ns(20_000_000)
    try:
        fa.fa_test_arm_fault(0)
        o, lse = torch.empty_like(b[0]), torch.empty(b[0].shape[:2], device=DEV)
        fa.fa_forward_paged(b[0], o, lse, *b[1:5], 0.1, "causal")
        assert fa.fa_sync_status() == fa.FA_ERR_TIMEOUT
    finally:
        fa.fa_set_wait_budget_ns(0)
    got = run(*b[:5], 0.1, "causal")
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_tokens_is_a_no_op():
    q, cache, table, cu, lk, _ = paged([(0, 20)], 2, 1, 64, torch.bfloat16, 16, seed=3)
    n = fa.fa_launch_count()
    o, lse = run(q, cache, table, cu, lk, 0.1, "causal")
    fa.fa_paged_append(None, q[:, :1], q[:, :1], None, cache, table, cu, lk)
    assert o.shape[0] == 0 and fa.fa_launch_count() == n


def test_a_strided_q_on_another_stream():
    """The copy that makes q contiguous runs on the stream of the call."""
    q, cache, table, cu, lens, _ = paged([(1, 300), (1, 40)], 8, 2, 64, torch.bfloat16, 16, seed=4)
    strided = torch.full((q.shape[0], 8, 128), NAN, dtype=q.dtype, device=DEV)[:, :, :64]
    strided.copy_(q)
    want = fa.forward_paged(q, cache, table, cu, lens)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(200_000_000)  # the current stream is busy for about 0.1 s
    got = fa.forward_paged(strided, cache, table, cu, lens, stream=s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_workspace_of_another_stream_is_not_the_current_streams():
    """Memory that the current stream has freed but still reads is no workspace of a call on
    another stream."""
    q, cache, table, cu, lens, _ = paged([(1, 30000)], 8, 2, 64, torch.bfloat16, 16, seed=4)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    size = fa.fa_forward_paged_workspace_bytes(64)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    x = torch.full((size,), 77, dtype=torch.uint8, device=DEV)
    y = torch.empty_like(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(200_000_000)
    y.copy_(x)
    del x
    fa.fa_forward_paged(q, o, lse, cache, table, cu, lens, 0.125, "causal", stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert bool((y == 77).all())


@pytest.mark.parametrize("own", [False, True])
def test_streams_given_by_their_handles(own):
    """An integer handle, the default stream's 0 among them: what the call copies and allocates
    is ordered on that stream, with another one current."""
    q, cache, table, cu, lens, _ = paged([(1, 300), (1, 40)], 8, 2, 64, torch.bfloat16, 16, seed=4)
    want = fa.forward_paged(q, cache, table, cu, lens)
    rope, _ = rope_handle(64, 64, "half", torch.bfloat16, True)
    turned = fa.qk_norm_rope(q, None, rope)[0]
    back = fa.qk_norm_rope_backward(q, None, q, None, rope)
    strided = torch.zeros((q.shape[0], 8, 128), dtype=q.dtype, device=DEV)[:, :, :64]
    s = torch.cuda.Stream() if own else torch.cuda.default_stream()
    assert own or s.cuda_stream == 0
    with binding._on(s.cuda_stream):
        assert torch.cuda.current_stream().cuda_stream == s.cuda_stream

    def step():
        return [*fa.forward_paged(strided, cache, table, cu, lens, stream=s.cuda_stream),
                fa.qk_norm_rope(strided, None, rope, stream=s.cuda_stream)[0],
                *fa.qk_norm_rope_backward(strided, None, strided, None, rope, stream=s.cuda_stream)[::2]]

    strided.copy_(q)
    for _ in range(40):  # nothing below is a first use, which would wait for the busy stream
        step()
    strided.fill_(NAN)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)  # about 0.1 s before q is there
        strided.copy_(q)
    with torch.cuda.stream(torch.cuda.Stream()):
        got = step()
    with torch.cuda.stream(s):  # the results are tensors of s
        got = [x.clone() for x in got]
    torch.cuda.synchronize()
    for a, b in zip(got, [*want, turned, back[0], back[2]]):
        assert torch.equal(a, b)


def test_append_of_long_prompts():
    """Every warp's share goes around its ring and over several tokens and sequences."""
    d, dtype, H, Hk, page = 64, torch.bfloat16, 25, 6, 32
    lens = [(4001, 4100), (0, 9), (5000, 5000), (3333, 9000)]
    _, cache, table, cu, lk, _ = paged(lens, 1, Hk, d, dtype, page, "head", seed=5)
    total = int(cu[-1])
    g = torch.Generator(device=DEV).manual_seed(12)
    qkv = torch.randn(total, H + 2 * Hk, d, generator=g, device=DEV).to(dtype)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    rope, freq = rope_handle(d, 30, "half", dtype, True)
    ek, ev = cache.k.clone(), cache.v.clone()
    q_out = torch.full((total, H, d), NAN, dtype=dtype, device=DEV)
    fa.fa_paged_append(q, k, v, q_out, cache, table, cu, lk, rope)
    assert fa.fa_sync_status() == fa.FA_OK
    for b, (n, keys) in enumerate(lens):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        pos = torch.arange(keys - n, keys, device=DEV)
        want, bound = norm_rope_ref(q[rows], rope.q_weight, pos, freq, "half", 1.0, 1e-5, dtype)
        assert_within(q_out[rows], want, bound, f"sequence {b}: q")
        at = table[b].long()[pos // page], pos % page
        want, bound = norm_rope_ref(k[rows], rope.k_weight, pos, freq, "half", 1.0, 1e-5, dtype)
        assert_within(cache.k[at], want, bound, f"sequence {b}: k")
        ek[at], ev[at] = cache.k[at], v[rows]  # the keys are checked; nothing else may differ
    same = lambda a, b: torch.equal(a.nan_to_num(nan=1e4), b.nan_to_num(nan=1e4))  # noqa: E731
    assert same(cache.k, ek) and same(cache.v, ev)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("new,H,Hk", [(1, 4, 4), (1, 16, 2), (1, 18, 2), (3, 8, 2)])
def test_steps_round_their_outputs_alone(new, H, Hk, d, dtype):
    """Units of 1, 8, 9 and 12 rows: the weights of the keys go into their product with V in two
    16-bit parts. What the second leaves is half a step of half a step of each (or 2^-25 where
    fp16 goes below its normal range), so that O is off by its own rounding, by that, and by the
    scores' products in 32 bits."""
    lens = [(new, 700), (new, 90), (1, 5000)]
    q, cache, table, cu, lk, seqs = paged(lens, H, Hk, d, dtype, 16, seed=d + H)
    o, _ = run(q, cache, table, cu, lk, d ** -0.5, "causal")
    half = torch.finfo(dtype).eps / 2
    t = 0
    for b, (qq, k, v) in enumerate(seqs):
        n = qq.shape[0]
        want = attention_ref(qq, k, v, d ** -0.5, "causal", (0, 0), dtype)[0]
        size = attention_ref(qq, k, v.abs(), d ** -0.5, "causal", (0, 0), dtype)[0]  # sums of p |v|
        scores = d ** -0.5 * d * float(qq.abs().max()) * float(k.abs().max())
        step = d * 2.0 ** -24 * scores + 2.0 ** -19
        bound = half * (1 + 2.0 ** -7) * want.abs() + (half ** 2 + 2 * step) * size
        if dtype == torch.float16:
            bound += 2.0 ** -25 * (1 + float(v.double().abs().sum(0).max()))
        assert_within(o[t:t + n], want, bound, f"sequence {b}: O")
        t += n
