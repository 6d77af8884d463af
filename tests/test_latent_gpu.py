"""The cache of latent rows: fa_latent_append and fa_forward_latent against their definitions
in 64 bits. Everything that the calls must not look at (slots past a sequence's end, pages that
belong to nobody, table entries past a sequence) holds NaN or nonsense."""

import math
import random

import pytest
import torch

import tiled_attention_03_gb300 as fa

from rope_util import assert_within, attention_ref, norm_rope_ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
NAN = float("nan")
DR = 64


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def paged(lens, H, dl, dtype, page, seed=0, spare=3, pad_tokens=0, pad_cols=0):
    """A serving batch: lens = [(new, keys)]. Returns q, the cache, the batch arrays and
    each sequence's (q, rows)."""
    d = dl + DR
    g = torch.Generator(device=DEV).manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV).to(dtype)  # noqa: E731
    need = [-(-n // page) for _, n in lens]
    pages = sum(need) + spare
    data = torch.full((pages, page, d + pad_cols), NAN, dtype=dtype, device=DEV)[..., :d]
    order = list(range(pages))
    random.Random(seed).shuffle(order)
    table = torch.full((len(lens), max(max(need), 1) + 1), -7, dtype=torch.int32)
    table[:, -1] = 2 ** 30
    seqs, at, cu = [], 0, [0]
    for b, (lq, lk) in enumerate(lens):
        mine = order[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = torch.tensor(mine, dtype=torch.int32)
        rows = randn(lk, d)
        for n, pg in enumerate(mine):
            part = slice(n * page, min((n + 1) * page, lk))
            data[pg, :part.stop - part.start] = rows[part]
        seqs.append((randn(lq, H, d), rows))
        cu.append(cu[-1] + lq)
    q = torch.cat([s[0] for s in seqs] + [randn(pad_tokens, H, d)])
    return q, fa.LatentCache(data, dl), table.to(DEV), i32(cu), i32([n for _, n in lens]), seqs


def run(q, cache, table, cu, lens, scale, mask="causal", window=(0, 0), **kw):
    o = torch.full((*q.shape[:2], cache.d_latent), -777.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:2], -777.0, device=DEV)
    fa.fa_forward_latent(q, o, lse, cache, table, cu, lens, scale, mask, window[0], window[1], **kw)
    st = fa.fa_sync_status()
    assert st == fa.FA_OK, fa.fa_status_string(st)
    return o, lse


def check(o, lse, seqs, scale, mask, window, dtype):
    t, dl = 0, o.shape[-1]
    for b, (q, rows) in enumerate(seqs):
        n = q.shape[0]
        want, bound, wl, lb = attention_ref(q, rows[:, None], rows[:, None], scale, mask, window, dtype)
        assert_within(o[t:t + n], want[..., :dl], bound[..., :dl], f"sequence {b}: O")
        got = lse[t:t + n].double()
        none = wl == -math.inf
        assert torch.equal(got == -math.inf, none), f"sequence {b}: rows without keys"
        assert bool((o[t:t + n][none] == 0).all())
        assert_within(got[~none], wl[~none], lb[~none], f"sequence {b}: LSE")
        t += n
    assert bool((o[t:] == -777.0).all()) and bool((lse[t:] == -777.0).all()), "wrote a padded row"


LENS = {
    "steps": [(1, 1), (1, 17), (1, 64), (1, 65), (1, 1000), (0, 50), (1, 63), (1, 2), (0, 0), (1, 333)],
    "chunks": [(5, 5), (70, 300), (64, 64), (1, 700), (33, 500), (0, 9), (100, 257)],
    "nothing": [(3, 0), (7, 3), (0, 0), (1, 0), (2, 40)],
}
MASKS = [("none", (0, 0)), ("causal", (0, 0)), ("window", (90, 3)), ("window", (0, 0))]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dl", [128, 256, 512])
@pytest.mark.parametrize("mask,window", MASKS)
@pytest.mark.parametrize("lens", list(LENS))
def test_masks_and_lengths(lens, mask, window, dl, dtype):
    page = {128: 8, 256: 16, 512: 128}[dl]
    b = paged(LENS[lens], 5, dl, dtype, page, seed=dl, pad_tokens=3)
    o, lse = run(*b[:5], 0.06, mask, window)
    check(o, lse, b[5], 0.06, mask, window, dtype)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 512])
@pytest.mark.parametrize("pad_cols", [0, 24])
@pytest.mark.parametrize("dl", [128, 256, 512])
def test_pages(dl, pad_cols, page):
    b = paged([(1, 600), (20, 130), (1, 127), (3, 1025)], 6, dl, torch.bfloat16, page, seed=page, pad_cols=pad_cols)
    o, lse = run(*b[:5], 0.06)
    check(o, lse, b[5], 0.06, "causal", (0, 0), torch.bfloat16)


@pytest.mark.parametrize("H", [1, 3, 12, 16, 17, 32, 33, 64, 65, 96, 128, 200])
@pytest.mark.parametrize("dl", [128, 512])
@pytest.mark.parametrize("lens", [[(1, 300), (1, 64), (1, 5), (1, 700)], [(1, 300), (2, 140), (3, 5)]])
def test_heads(lens, dl, H):
    b = paged(lens, H, dl, torch.float16, 16, seed=H)
    o, lse = run(*b[:5], 0.06)
    check(o, lse, b[5], 0.06, "causal", (0, 0), torch.float16)


@pytest.mark.parametrize("dl,dtype", [(512, torch.bfloat16), (256, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("mask,window", [("causal", (0, 0)), ("window", (9000, 0))])
@pytest.mark.parametrize("new,H", [(1, 16), (2, 64), (40, 4)])
def test_long_sequences_are_cut_and_joined(new, H, dl, dtype, mask, window):
    """A unit of some hundred tiles over all workers, with short ones around it."""
    b = paged([(1, 40), (new, 20500), (1, 2000)], H, dl, dtype, 64, seed=1)
    o, lse = run(*b[:5], 0.06, mask, window)
    check(o, lse, b[5], 0.06, mask, window, dtype)
    again = run(*b[:5], 0.06, mask, window)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("B,H,new", [(300, 4, [0, 1, 1, 2]), (600, 4, [1]), (300, 20, [1]), (100, 128, [1, 0, 1])])
def test_many_sequences(B, H, new):
    rng = random.Random(B)
    lens = [(n, n + rng.choice([0, 3, 70, 200])) for n in (rng.choice(new) for _ in range(B))]
    b = paged(lens, H, 256, torch.bfloat16, 16, seed=2)
    o, lse = run(*b[:5], 0.06)
    check(o, lse, b[5], 0.06, "causal", (0, 0), torch.bfloat16)


@pytest.mark.parametrize("dl", [128, 512])
@pytest.mark.parametrize("H", [8, 64])
def test_peaky_scores(H, dl):
    """Scores that grow along the keys: the reference moves again and again."""
    q, cache, table, cu, lens, seqs = paged([(1, 900), (3, 1500)], H, dl, torch.bfloat16, 16, seed=9)
    at = 0
    for b, (qb, rows) in enumerate(seqs):
        ramp = torch.linspace(0.1, 6.0, rows.shape[0], device=DEV)[:, None]
        rows.copy_((rows.float() * ramp).to(rows.dtype))
        for j in range(rows.shape[0]):
            cache.data[table[b, j // 16], j % 16] = rows[j]
        at += qb.shape[0]
    o, lse = run(q, cache, table, cu, lens, 0.3)
    check(o, lse, seqs, 0.3, "causal", (0, 0), torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dl", [128, 256, 512])
@pytest.mark.parametrize("H", [4, 12, 20, 25])
def test_steps_round_their_outputs_alone(H, dl, dtype):
    """Batches of up to 32 rows a sequence: the weights of the keys go into their product with the
    rows in two 16-bit parts. What the second leaves is half a step of half a step of each (or 2^-25
    where fp16 goes below its normal range).

    The scores are exact: queries are 0 on the latent columns, and what both hold on the rotary
    ones are multiples of 1/4 up to 4, so that sums of 64 products, multiples of 1/16 below
    1024, are floats. Exponents (base 2) below 32 then have two roundings of 2^-24 of themselves, so
    a weight is off by 2^-18 of itself, and 2^-21 for the exponential; so is the sum that divides it.
    The products add 16 keys at a time, each with a step of 2^-23 of the sum at most."""
    scale = 0.0625
    q, cache, table, cu, lens, seqs = paged([(1, 700), (2, 300), (1, 90), (1, 1)], H, dl, dtype, 16, seed=dl + H)
    quarter = lambda x: (x.float().clamp(-4, 4) * 4).round() / 4  # noqa: E731
    t, half = 0, torch.finfo(dtype).eps / 2
    for b, (qq, rows) in enumerate(seqs):
        qq[..., :dl], qq[..., dl:] = 0, quarter(qq[..., dl:])
        rows[:, dl:] = quarter(rows[:, dl:])
        q[t:t + qq.shape[0]] = qq
        j = torch.arange(rows.shape[0], device=DEV)
        cache.data[table[b, j // 16].long(), j % 16] = rows
        t += qq.shape[0]
    o, _ = run(q, cache, table, cu, lens, scale)
    t = 0
    for b, (qq, rows) in enumerate(seqs):
        n, L = qq.shape[0], rows.shape[0]
        x = torch.einsum("ihd,jd->ihj", qq.double(), rows.double()) * scale
        assert float(x.abs().max()) * math.log2(math.e) < 16  # and less twice that from the reference
        x.masked_fill_(~(torch.arange(L, device=DEV) <= torch.arange(L - n, L, device=DEV)[:, None])[:, None], -math.inf)
        p, v = x.softmax(-1), rows[:, :dl].double()
        want, size = p @ v, p @ v.abs()
        bound = half * want.abs() * (1 + 2.0 ** -7) + (half ** 2 + 2 * (2.0 ** -18 + 2.0 ** -21) + (L / 16 + 1) * 2.0 ** -23) * size
        if dtype == torch.float16:
            bound += 2.0 ** -25 * (1 + v.abs().sum(0))
        assert_within(o[t:t + n], want, bound, f"sequence {b}: O")
        t += n


@pytest.mark.parametrize("mask,window", [("window", (100, 0)), ("causal", (0, 0))])
def test_what_is_not_seen_is_not_looked_at(mask, window):
    """Rows before every window, and all behind a sequence's end, hold NaN."""
    q, cache, table, cu, lens, seqs = paged([(1, 900), (4, 500)], 8, 512, torch.bfloat16, 16, seed=4)
    if mask == "window":
        for b, (qb, rows) in enumerate(seqs):
            n = rows.shape[0] - qb.shape[0] - window[0]
            for j in range(n):
                cache.data[table[b, j // 16], j % 16] = NAN
            rows[:n] = 0
    o, lse = run(q, cache, table, cu, lens, 0.06, mask, window)
    check(o, lse, seqs, 0.06, mask, window, torch.bfloat16)


def test_nan_in_a_visible_row_is_seen():
    q, cache, table, cu, lens, _ = paged([(1, 300), (1, 200)], 16, 512, torch.bfloat16, 16, seed=4)
    cache.data[table[0, 7], 3, 5] = NAN
    o, lse = run(q, cache, table, cu, lens, 0.06)
    assert bool(lse[0].isnan().all()) and bool(o[0].isnan().all())
    assert bool(torch.isfinite(o[1]).all()) and bool(torch.isfinite(lse[1]).all())


def with_infinity(b, at):
    """Key `at` (all keys: None) of the first sequence gets +infinity in a rotary column; which of its
    (token, head) rows have a query of the same sign there: a score of +infinity, the others -infinity."""
    q, cache, table, _, _, seqs = b
    qq, rows = seqs[0]
    g = torch.Generator(device=DEV).manual_seed(5)
    up = torch.rand(qq.shape[:2], generator=g, device=DEV) < 0.5
    col = cache.d_latent + 8
    qq[..., col] = torch.where(up, 0.5, -0.5).to(q.dtype)
    q[:qq.shape[0]] = qq
    rows[slice(None) if at is None else at, col] = math.inf
    j = torch.arange(rows.shape[0], device=DEV)
    cache.data[table[0, j // 16].long(), j % 16] = rows
    return up


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lens,H", [([(1, 300), (1, 90)], 16), ([(1, 20000), (1, 90)], 16), ([(1, 300), (1, 90)], 32),
                                    ([(1, 700), (1, 70)], 128)])
@pytest.mark.parametrize("at", [0, 70, -1])
def test_infinite_scores(at, lens, H, dtype):
    """A score of +infinity ends in NaN, as exp(inf - inf) does; one of -infinity is a weight of 0."""
    b = paged(lens, H, 512, dtype, 16, seed=H)
    qq, rows = b[5][0]
    up = with_infinity(b, at % lens[0][1])
    o, lse = run(*b[:5], 0.06)
    assert bool(o[0][up[0]].isnan().all()) and bool(lse[0][up[0]].isnan().all())
    at %= lens[0][1]
    others = torch.cat([rows[:at], rows[at + 1:]])[:, None]
    want, bound, wl, lb = attention_ref(qq, others, others, 0.06, "none", (0, 0), dtype)
    assert_within(o[0][~up[0]], want[0][~up[0]][:, :512], bound[0][~up[0]][:, :512], "O")
    assert_within(lse[0][~up[0]], wl[0][~up[0]], lb[0][~up[0]], "LSE")
    check(o[1:], lse[1:], b[5][1:], 0.06, "causal", (0, 0), dtype)


@pytest.mark.parametrize("H", [1, 8])
@pytest.mark.parametrize("at", [240, 299])
def test_tokens_that_do_not_see_an_infinite_key_are_as_without_it(at, H):
    """In a chunk: the tokens before it. (An infinity in the rotary part: no value.)"""
    b = paged([(70, 300), (3, 40)], H, 256, torch.bfloat16, 16, seed=3)
    qq, rows = b[5][0]
    up = with_infinity(b, at)
    o, lse = run(*b[:5], 0.06)
    m = at - 230  # tokens at 230 .. at - 1
    check(o[:m], lse[:m], [(qq[:m], rows[:at])], 0.06, "causal", (0, 0), torch.bfloat16)
    assert torch.equal(lse[m:70].isnan(), up[m:])
    check(o[70:], lse[70:], b[5][1:], 0.06, "causal", (0, 0), torch.bfloat16)


@pytest.mark.parametrize("lens,H", [([(1, 300), (1, 90)], 16), ([(1, 20000), (1, 90)], 16), ([(1, 700), (1, 70)], 128),
                                    ([(70, 300), (3, 40)], 4)])
def test_rows_whose_scores_are_all_minus_infinity(lens, H):
    """They end as rows that see no key do: 0 and -infinity."""
    b = paged(lens, H, 512, torch.bfloat16, 16, seed=H)
    up = with_infinity(b, None)
    n = lens[0][0]
    o, lse = run(*b[:5], 0.06)
    assert bool((lse[:n][~up] == -math.inf).all()) and bool((o[:n][~up] == 0).all())
    assert bool(lse[:n][up].isnan().all()) and bool(o[:n][up].isnan().all())
    check(o[n:], lse[n:], b[5][1:], 0.06, "causal", (0, 0), torch.bfloat16)


@pytest.mark.parametrize("H", [8, 128])
def test_page_numbers_outside_the_cache_read_as_zeros(H):
    q, cache, table, cu, lens, seqs = paged([(1, 300), (1, 200)], H, 512, torch.bfloat16, 16, seed=4)
    for b, p, bad in ((0, 3, -1), (0, 9, cache.num_pages), (1, 0, 2 ** 31 - 1), (1, 12, -2 ** 31)):
        table[b, p] = bad
        seqs[b][1][p * 16:(p + 1) * 16] = 0
    o, lse = run(q, cache, table, cu, lens, 0.06)
    check(o, lse, seqs, 0.06, "causal", (0, 0), torch.bfloat16)


@pytest.mark.parametrize("B,T,H,width", [(8192, 4096, 64, 128), (128, 128, 64, 40000)])
def test_offsets_in_no_order_write_nothing_outside(B, T, H, width):
    """Every second sequence owns all T tokens: the work of all of them passes 2^31."""
    page, guard, dl = 512, 64, 128
    data = torch.zeros(4, page, dl + DR, dtype=torch.bfloat16, device=DEV)
    cache = fa.LatentCache(data, dl)
    table = torch.arange(B * width, device=DEV).remainder(4).to(torch.int32).view(B, width)
    cu = i32([0, T] * (B // 2) + [0])
    lens = torch.full((B,), width * page, dtype=torch.int32, device=DEV)
    q = torch.zeros(T, H, dl + DR, dtype=torch.bfloat16, device=DEV)
    o = torch.full((T + 2 * guard, H, dl), -777.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T + 2 * guard, H), -777.0, device=DEV)
    fa.fa_forward_latent(q, o[guard:-guard], lse[guard:-guard], cache, table, cu, lens, 1.0, "none", 0, 0)
    assert fa.fa_sync_status() == fa.FA_OK
    for x in (o, lse):
        assert bool((x[:guard] == -777.0).all()) and bool((x[-guard:] == -777.0).all())


def test_lengths_are_clamped_to_the_table():
    q, cache, table, cu, lens, _ = paged([(1, 48), (1, 30)], 8, 256, torch.bfloat16, 16, seed=2)
    three = table[:, :3].contiguous()
    want = run(q, cache, three, cu, lens, 0.06)
    big = lens.clone()
    big[0] = 2 ** 31 - 1
    got = run(q, cache, three, cu, big, 0.06)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_cache_past_32_bits():
    """Pages whose elements lie past 2^31 (and bytes past 2^32) of the buffer, appended and read."""
    page, dl, H, n = 128, 512, 4, 300
    d = dl + DR
    pages = 2 ** 31 // (page * d) + 40
    data = torch.empty(pages, page, d, dtype=torch.bfloat16, device=DEV)
    cache = fa.LatentCache(data, dl)
    mine = [pages - 1, 3, pages - 7]
    table = i32([mine])
    for pg in mine:
        data[pg] = NAN
    g = torch.Generator(device=DEV).manual_seed(1)
    q, rows = (torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16) for s in ((n, H, d), (n, d)))
    cu, lens = i32([0, n]), i32([n])
    fa.fa_latent_append(None, rows[:, :dl], rows[:, dl:], None, cache, table, cu, lens)
    o, lse = run(q, cache, table, cu, lens, 0.06)
    check(o, lse, [(q, rows)], 0.06, "causal", (0, 0), torch.bfloat16)


# ------------------------------------------------------------------------ append

def rope_handle(dl, r, layout, dtype, norm, magnitude=1.0, seed=5):
    freq = fa.rope_frequencies(r) if r else []
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = (1 + 0.3 * torch.randn(dl, generator=g, device=DEV)).to(dtype)
    return fa.NormRope(fa.rope_steps(r) if r else None, layout, magnitude, None, w if norm else None, 1e-5), freq, w


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dl,r,layout,norm,H", [
    (512, 64, "half", True, 16), (512, 64, "interleaved", True, 33), (256, 32, "half", False, 1),
    (256, 20, "half", True, 20), (128, 6, "interleaved", True, 3), (128, 64, "half", True, 128), (512, 0, "half", True, 5)])
@pytest.mark.parametrize("lens", ["steps", "chunks", "nothing", "many"])
def test_append(lens, dl, r, layout, norm, H, dtype):
    rng = random.Random(3)
    lens = LENS.get(lens) or [(n, n + rng.randrange(90)) for n in (rng.choice([0, 1, 1, 2, 40]) for _ in range(200))]
    page, pad = 16, 5
    g = torch.Generator(device=DEV).manual_seed(1)
    T = sum(n for n, _ in lens) + pad
    need = [-(-n // page) for _, n in lens]
    table = torch.full((len(lens), max(max(need), 1) + 1), -7, dtype=torch.int32)
    order = torch.randperm(sum(need) + 2)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    data = torch.randn(sum(need) + 2, page, dl + DR, generator=g, device=DEV).to(dtype)
    before = data.clone()
    down = torch.randn(T, dl + DR, generator=g, device=DEV).to(dtype)
    qin = torch.randn(T, H, 104 + DR, generator=g, device=DEV).to(dtype)[..., 96:96 + DR]
    full = torch.full((T, H, dl + DR), -777.0, dtype=dtype, device=DEV)
    rope, freq, w = rope_handle(dl, r, layout, dtype, norm, 1.25 if r else 1.0)
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    fa.fa_latent_append(qin, down[:, :dl], down[:, dl:], full[..., dl:], fa.LatentCache(data, dl), table.to(DEV), i32(cu),
                        i32([n for _, n in lens]), rope)
    assert fa.fa_sync_status() == fa.FA_OK
    assert bool((full[..., :dl] == -777.0).all()) and bool((full[cu[-1]:] == -777.0).all())
    touched = torch.zeros(data.shape[:2], dtype=torch.bool, device=DEV)
    for b, (lq, lk) in enumerate(lens):
        t = slice(cu[b], cu[b + 1])
        pos = torch.arange(lk - lq, lk, device=DEV)
        want, bound = norm_rope_ref(qin[t], None, pos, freq, layout, 1.25 if r else 1.0, 1e-5, dtype)
        assert_within(full[t, :, dl:], want, bound, f"sequence {b}: q")
        here = pos >= 0
        pg, sl = table.to(DEV)[b][(pos[here] // page)].long(), pos[here] % page
        touched[pg, sl] = True
        want, bound = norm_rope_ref(down[t, None, dl:], None, pos, freq, layout, 1.25 if r else 1.0, 1e-5, dtype)
        assert_within(data[pg, sl][:, dl:], want[here, 0], bound[here, 0], f"sequence {b}: rotary part")
        # the norm's sum of dl squares: at most 16 in a lane, then a tree (see norm_rope_ref)
        want, bound = norm_rope_ref(down[t, None, :dl], w if norm else None, pos, [], layout, 1.0, 1e-5, dtype)
        assert_within(data[pg, sl][:, :dl], want[here, 0], bound[here, 0], f"sequence {b}: latent")
    assert torch.equal(data[~touched], before[~touched]), "wrote another slot"


@pytest.mark.parametrize("rope", [False, True])
def test_append_without_norm_and_rotation_keeps_the_bits(rope):
    bits = torch.randint(-2 ** 15, 2 ** 15, (7, 4, 256 + DR), device=DEV).to(torch.int16)
    x = bits.view(torch.bfloat16)
    data = torch.zeros(2, 8, 256 + DR, dtype=torch.bfloat16, device=DEV)
    out = torch.zeros(7, 4, DR, dtype=torch.bfloat16, device=DEV)
    fa.fa_latent_append(x[..., 256:], x[:, 0, :256], x[:, 0, 256:], out, fa.LatentCache(data, 256), i32([[1, 0]]), i32([0, 7]),
                        i32([9]), fa.NormRope() if rope else None)
    torch.cuda.synchronize()
    got = torch.cat([data[1, 2:], data[0, :1]]).view(torch.int16)
    assert torch.equal(got, bits[:, 0]) and torch.equal(out.view(torch.int16), bits[..., 256:])


def test_append_in_place_and_without_queries():
    rope, _, _ = rope_handle(512, 64, "half", torch.bfloat16, True)
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn(9, 3, 576, generator=g, device=DEV).to(torch.bfloat16)
    down = torch.randn(9, 576, generator=g, device=DEV).to(torch.bfloat16)
    data = [torch.zeros(4, 8, 576, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    out = torch.empty(9, 3, 64, dtype=torch.bfloat16, device=DEV)
    rest = q[..., :512].clone()
    args = i32([[3, 1, 0]]), i32([0, 9]), i32([17]), rope
    fa.fa_latent_append(q[..., 512:], down[:, :512], down[:, 512:], out, fa.LatentCache(data[0], 512), *args)
    fa.fa_latent_append(q[..., 512:], down[:, :512], down[:, 512:], q[..., 512:], fa.LatentCache(data[1], 512), *args)
    fa.fa_latent_append(None, down[:, :512], down[:, 512:], None, fa.LatentCache(data[2], 512), *args)
    torch.cuda.synchronize()
    assert torch.equal(q[..., 512:], out) and torch.equal(q[..., :512], rest)
    assert torch.equal(data[0], data[1]) and torch.equal(data[0], data[2])


@pytest.mark.parametrize("first", ["queries", "latent"])
@pytest.mark.parametrize("dl,H", [(512, 5), (128, 20)])
def test_append_from_one_projection_in_place(dl, H, first):
    """[query heads | c | k_rope] of a token in one buffer, the queries rotated where they are: as with a
    buffer for each, and the other columns stay."""
    rope, _, _ = rope_handle(dl, 64, "half", torch.bfloat16, True)
    g = torch.Generator(device=DEV).manual_seed(1)
    one = torch.randn(23, 192 * H + dl + DR, generator=g, device=DEV).to(torch.bfloat16)
    cut = [192 * H, dl, DR] if first == "queries" else [dl, DR, 192 * H]
    parts = one.split(cut, 1)
    q, c, k = parts if first == "queries" else (parts[2], parts[0], parts[1])
    q = q.unflatten(1, (H, 192))
    want, out = one.clone(), torch.empty(23, H, DR, dtype=one.dtype, device=DEV)
    data = [torch.zeros(4, 8, dl + DR, dtype=one.dtype, device=DEV) for _ in range(2)]
    args = i32([[3, 1, 0, 2]]), i32([0, 23]), i32([30]), rope
    fa.fa_latent_append(q[..., 128:].contiguous(), c.contiguous(), k.contiguous(), out, fa.LatentCache(data[0], dl), *args)
    wq = want.split(cut, 1)[0 if first == "queries" else 2].unflatten(1, (H, 192))
    wq[..., 128:] = out
    fa.fa_latent_append(q[..., 128:], c, k, q[..., 128:], fa.LatentCache(data[1], dl), *args)
    assert fa.fa_sync_status() == fa.FA_OK
    assert torch.equal(one, want) and torch.equal(data[0], data[1]) and not torch.equal(out, q.new_zeros(out.shape))


def test_append_skips_pages_outside_the_cache():
    data = torch.zeros(3, 8, 192, dtype=torch.bfloat16, device=DEV)
    down = torch.ones(40, 192, dtype=torch.bfloat16, device=DEV)
    fa.fa_latent_append(None, down[:, :128], down[:, 128:], None, fa.LatentCache(data[1:2], 128),
                        i32([[0, -1, 1, 2 ** 31 - 1, -2 ** 31]]), i32([0, 40]), i32([40]))
    torch.cuda.synchronize()
    assert bool((data[1] == 1).all()) and bool((data[0] == 0).all()) and bool((data[2] == 0).all())


# ------------------------------------------------------------------------ together

@pytest.mark.parametrize("dl,H,dn", [(256, 6, 64), (512, 20, 128)])
def test_serving_loop_matches_expanded_attention(dl, H, dn):
    """Prompt and single steps through append and absorbed attention, against the expanded form of
    the whole sequence in 64 bits: keys (W_k c, k_rope), values W_v c, the latents as stored."""
    dtype, page, n, scale = torch.bfloat16, 16, 150, (dn + DR) ** -0.5
    g = torch.Generator(device=DEV).manual_seed(3)
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    wk, wv = ((randn(H, dn, dl) * dl ** -0.5).to(dtype) for _ in range(2))
    rope, freq, w = rope_handle(dl, DR, "half", dtype, True)
    down, qn, qr = randn(n, dl + DR).to(dtype), randn(n, H, dn).to(dtype), randn(n, H, DR).to(dtype)
    data = torch.full((14, page, dl + DR), NAN, dtype=dtype, device=DEV)
    cache = fa.LatentCache(data, dl)
    table = torch.randperm(14, device=DEV)[:11].to(torch.int32)[None].contiguous()
    absorbed = torch.empty(n, H, dl + DR, dtype=dtype, device=DEV)
    absorbed[..., :dl] = torch.einsum("thn,hnl->thl", qn.float(), wk.float()).to(dtype)
    outs = []
    steps = [(0, 40), (40, 41), (41, 120)] + [(t, t + 1) for t in range(120, n)]
    for a, b in steps:
        cu, lens = i32([0, b - a]), i32([b])
        q = absorbed[a:b].clone()
        fa.fa_latent_append(qr[a:b], down[a:b, :dl], down[a:b, dl:], q[..., dl:], cache, table, cu, lens, rope)
        o, _ = fa.forward_latent(q, cache, table, cu, lens, scale)
        outs.append(torch.einsum("thl,hnl->thn", o.double(), wv.double()))
        absorbed[a:b] = q
    assert fa.fa_sync_status() == fa.FA_OK
    got = torch.cat(outs)
    pos = torch.arange(n, device=DEV)
    rows = data[table[0].long()].flatten(0, 1)[:n].double()
    key = torch.cat([torch.einsum("hnl,jl->jhn", wk.double(), rows[:, :dl]), rows[:, None, dl:].expand(-1, H, -1)], -1)
    val = torch.einsum("hnl,jl->jhn", wv.double(), rows[:, :dl])
    qq = torch.cat([qn.double(), absorbed[..., dl:].double()], -1)
    x = torch.einsum("thn,jhn->htj", qq, key) * scale
    x.masked_fill_(pos[None, None] > pos[None, :, None], -math.inf)
    p = x.softmax(-1)
    want = torch.einsum("htj,jhn->thn", p, val)
    # The absorbed query is rounded to bf16 (2^-9 of each of its dl elements): the score moves by
    # at most e = 2^-9 scale sum |q_l c_l|, a weight by a factor within exp(2 e); weights are
    # rounded by 2^-9 and O by 2^-9 before its product with W_v.
    e = 2.0 ** -9 * scale * torch.einsum("thl,jl->thj", absorbed[..., :dl].double().abs(), rows[:, :dl].abs()).amax(-1)
    spread = torch.einsum("htj,jl->thl", p, rows[:, :dl].abs())
    bound = torch.einsum("thl,hnl->thn", spread, wv.double().abs()) * (2 * e[..., None].expm1().clamp(min=0) + 2.0 ** -7)
    assert_within(got, want, bound, "O")


@pytest.mark.parametrize("H", [16, 128])
def test_capture_follows_the_lengths(H):
    """A captured step replayed as the sequences grow, and as their tokens move between steps and
    chunks: everything is read on the device."""
    dl, dtype, page, B = 512, torch.bfloat16, 16, 6
    rope, _, _ = rope_handle(dl, DR, "half", dtype, True)
    data = torch.zeros(140, page, dl + DR, dtype=dtype, device=DEV)
    cache, other = fa.LatentCache(data, dl), fa.LatentCache(data.clone(), dl)
    table = torch.randperm(140, device=DEV)[:138].to(torch.int32).view(B, 23)
    cu, lk = i32(range(B + 1)), i32([3, 200, 129, 0, 64, 63])
    down, q = torch.zeros(B, dl + DR, dtype=dtype, device=DEV), torch.zeros(B, H, dl + DR, dtype=dtype, device=DEV)
    o, lse = torch.empty(B, H, dl, dtype=dtype, device=DEV), torch.empty(B, H, device=DEV)
    ws = torch.empty(fa.fa_forward_latent_workspace_bytes(dl), dtype=torch.uint8, device=DEV)

    def step(c, stream=None):
        fa.fa_latent_append(q[..., dl:], down[:, :dl], down[:, dl:], q[..., dl:], c, table, cu, lk, rope, stream)
        fa.fa_forward_latent(q, o, lse, c, table, cu, lk, 0.06, "causal", 0, 0, ws, stream)

    s = torch.cuda.Stream()
    step(other)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(cache, s)
    g = torch.Generator(device=DEV).manual_seed(1)
    for i in range(10):
        new = [[1] * B, [0, 0, 6, 0, 0, 0], [3, 0, 0, 2, 1, 0]][i % 3]
        cu.copy_(i32([sum(new[:b]) for b in range(B + 1)]))
        lk += i32(new)
        q0 = torch.randn(q.shape, generator=g, device=DEV).to(dtype)
        down.copy_(torch.randn(down.shape, generator=g, device=DEV))
        q.copy_(q0)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), lse.clone()
        o.fill_(NAN)
        q.copy_(q0)
        step(other)
        torch.cuda.synchronize()
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
        assert torch.equal(cache.data, other.data)
    assert fa.fa_sync_status() == fa.FA_OK


def test_two_streams_at_once():
    bs = [paged([(3, 3000), (2, 700)], 16, 512, torch.bfloat16, 16, seed=i) for i in range(2)]
    want = [run(*b[:5], 0.06) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [(torch.empty(*b[0].shape[:2], 512, dtype=b[0].dtype, device=DEV), torch.empty(b[0].shape[:2], device=DEV))
               for b in bs]
        torch.cuda.synchronize()
        for b, s, (o, lse) in zip(bs, streams, got):
            fa.fa_forward_latent(b[0], o, lse, *b[1:5], 0.06, stream=s)
        torch.cuda.synchronize()
        for (o, lse), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)


def test_a_strided_q_on_another_stream():
    """The copy that makes q contiguous, and what the call allocates, belong to the call's stream."""
    q, cache, table, cu, lens, _ = paged([(1, 300), (1, 40)], 8, 256, torch.bfloat16, 16, seed=4)
    strided = torch.full((*q.shape[:2], 400), NAN, dtype=q.dtype, device=DEV)[..., :320]
    strided.copy_(q)
    want = fa.forward_latent(q, cache, table, cu, lens, 0.06)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(200_000_000)  # the current stream is busy for about 0.1 s
    got = fa.forward_latent(strided, cache, table, cu, lens, 0.06, stream=s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("position,H", [(0, 16), (0, 128), (3, 128)])
def test_the_fault_hook_ends_in_a_timeout(position, H):
    """A load of keys that never comes: the waits run out, the call reports it, and the next call is
    right. (With 16 heads no CTA gets as far as a fourth tile.)"""
    b = paged([(40, 600)] * 3, H, 512, torch.bfloat16, 16, seed=3)
    want = run(*b[:5], 0.06)
    fa.fa_set_wait_budget_ns(20_000_000)
    try:
        fa.fa_test_arm_fault(position)
        o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        fa.fa_forward_latent(b[0], o, lse, *b[1:5], 0.06)
        assert fa.fa_sync_status() == fa.FA_ERR_TIMEOUT
    finally:
        fa.fa_set_wait_budget_ns(0)
    got = run(*b[:5], 0.06)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_tokens_is_a_no_op():
    q, cache, table, cu, lk, _ = paged([(0, 20)], 2, 256, torch.bfloat16, 16, seed=3)
    n = fa.fa_launch_count()
    o, _ = run(q, cache, table, cu, lk, 0.1)
    fa.fa_latent_append(None, q[:, 0, :256], q[:, 0, 256:], None, cache, table, cu, lk)
    assert o.shape[0] == 0 and fa.fa_launch_count() == n


def test_binding_refusals():
    q, cache, table, cu, lens, _ = paged([(1, 20)], 4, 256, torch.bfloat16, 16, seed=3)
    o, lse = torch.empty(1, 4, 256, dtype=q.dtype, device=DEV), torch.empty(1, 4, device=DEV)
    good = dict(q=q, o=o, lse=lse, cache=cache, block_table=table, cu_seqlens_q=cu, seqlens_k=lens, scale=0.1)
    for bad in (dict(q=q.half()), dict(q=q[..., :256]), dict(o=q), dict(lse=lse[:, :2]), dict(lse=lse.double()),
                dict(block_table=table.long()), dict(cu_seqlens_q=cu[:1]), dict(scale=0.0), dict(scale=float("nan")),
                dict(workspace=torch.empty(64, dtype=torch.uint8, device=DEV))):
        with pytest.raises(fa.FaError):
            fa.fa_forward_latent(**{**good, **bad})
    x = torch.zeros(1, 320, dtype=torch.bfloat16, device=DEV)
    for bad in ((None, x[:, :128], x[:, 256:], None), (None, x[:, :256], x[:, 256:].half(), None),
                (q[..., 256:], x[:, :256], x[:, 256:], None), (q, x[:, :256], x[:, 256:], q)):
        with pytest.raises(fa.FaError):
            fa.fa_latent_append(*bad, cache, table, cu, lens)
    with pytest.raises(fa.FaError):  # a weight of another width
        fa.fa_latent_append(None, x[:, :256], x[:, 256:], None, cache, table, cu, lens,
                            fa.NormRope(k_weight=torch.ones(128, dtype=torch.bfloat16, device=DEV)))
    assert fa.fa_sync_status() == fa.FA_OK
