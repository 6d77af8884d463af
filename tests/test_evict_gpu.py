"""Eviction from a paged cache: fa_paged_weights and fa_paged_evict against their definitions in
64 bits. Slots past a sequence's end, pages that belong to nobody and table entries past a
sequence hold NaN or nonsense."""

import math
import random

import pytest
import torch

import tiled_attention_03_gb300 as fa

from rope_util import assert_within
from test_paged_gpu import LENS, MASKS, paged

pytestmark = pytest.mark.gpu

DEV = "cuda"
NAN = float("nan")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def seen(lq, lk, mask, window):
    i = torch.arange(lq, device=DEV)[:, None] + lk - lq
    j = torch.arange(lk, device=DEV)[None]
    if mask == "causal":
        return j <= i
    if mask == "window":
        return (j >= i - window[0]) & (j <= i + window[1])
    return torch.ones(lq, lk, dtype=torch.bool, device=DEV)


def lse_of(seqs, Hk, scale, mask, window, T):
    """The LSE of every token and head, in 32 bits (-infinity: it sees nothing)."""
    out = torch.full((T, seqs[0][0].shape[1]), 5.0, device=DEV)
    at = 0
    for q, k, _ in seqs:
        n, H = q.shape[:2]
        if n:
            x = torch.einsum("ihd,jhd->hij", q.double(), k.double().repeat_interleave(H // Hk, 1)) * scale
            x.masked_fill_(~seen(n, k.shape[0], mask, window), -math.inf)
            out[at:at + n] = torch.logsumexp(x, -1).T.float() if k.shape[0] else -math.inf
        at += n
    return out


def gather_ref(q, k, lse, old, scale, mask, window):
    """Weights (L_k, H_kv) after the call and their bound, of one sequence. Each exponent is the
    sum of d products in 32 bits, scaled, less the LSE in steps of 2 to the power of: four roundings of
    numbers no larger than |score| + |LSE|; the exponential is good to 2^-21, and the running sums
    take at most one step of 2^-24 of the whole per row."""
    (n, H, d), (L, Hk) = q.shape, k.shape[:2]
    new = old.clone()
    new[max(0, L - n):] = 0
    bound = new.abs() * 2.0 ** -23
    vis = seen(n, L, mask, window)
    for h in range(H):
        kk = k[:, h // (H // Hk)].double()
        s = q[:, h].double() @ kk.T * scale
        size = q[:, h].double().abs() @ kk.abs().T * scale
        z = lse[:, h].double()[:, None]
        p = torch.where(vis & (z > -math.inf), (s - z).exp(), torch.zeros_like(s))
        rel = d * 2.0 ** -24 * size + 2.0 ** -22 * (s.abs() + z.abs().clamp(max=1e30)) + 2.0 ** -20 + n * H * 2.0 ** -24
        new[:, h // (H // Hk)] += p.sum(0)
        bound[:, h // (H // Hk)] += torch.where(p > 0, p * rel, p).sum(0)
    return new, bound


def gather(q, lse, weights, cache, table, cu, lens, scale, mask, window=(0, 0), **kw):
    fa.fa_paged_weights(q, lse, weights, cache, table, cu, lens, scale, mask, window[0], window[1], **kw)
    st = fa.fa_sync_status()
    assert st == fa.FA_OK, fa.fa_status_string(st)


def check_gather(b, scale, mask, window=(0, 0), lse=None):
    """Runs the call on weights of earlier steps (NaN in the slots of new keys and in those of nobody) and compares all
    of them."""
    q, cache, table, cu, lens, seqs = b
    Hk, page = cache.H_kv, cache.page_size
    if lse is None:
        lse = lse_of(seqs, Hk, scale, mask, window, q.shape[0])
    g = torch.Generator(device=DEV).manual_seed(11)
    weights = torch.full((cache.num_pages, Hk, page), NAN, device=DEV)
    olds = []
    for i, (qq, k, _) in enumerate(seqs):
        j = torch.arange(k.shape[0], device=DEV)
        old = torch.rand(k.shape[0], Hk, generator=g, device=DEV) * 4
        old[max(0, k.shape[0] - qq.shape[0]):] = NAN
        if qq.shape[0] == 0:
            old = torch.rand(k.shape[0], Hk, generator=g, device=DEV)
        weights[table[i, j // page].long(), :, j % page] = old
        olds.append(old)
    before = weights.clone()
    gather(q, lse, weights, cache, table, cu, lens, scale, mask, window)
    mine = torch.zeros_like(weights, dtype=torch.bool)
    at = 0
    for i, (qq, k, _) in enumerate(seqs):
        j = torch.arange(k.shape[0], device=DEV)
        n = qq.shape[0]
        pg, sl = table[i, j // page].long(), j % page
        got = weights[pg, :, sl]
        if n and k.shape[0]:
            want, bound = gather_ref(qq, k, lse[at:at + n], olds[i].double(), scale, mask, window)
            sees = seen(n, k.shape[0], mask, window).any(0)
            assert_within(got[sees], want[sees], bound[sees], f"sequence {i}")
            mine[pg[sees], :, sl[sees]] = True
        at += n
    same = (weights == before) | (weights.isnan() & before.isnan())
    assert bool(same[~mine].all()), "wrote another slot"
    return weights


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("mask,window", MASKS)
@pytest.mark.parametrize("lens", ["steps", "chunks"])
def test_masks_and_lengths(lens, mask, window, d, dtype):
    page, layout = {32: (8, "head"), 64: (16, "token"), 128: (32, "both"), 256: (128, "head")}[d]
    b = paged(LENS[lens], 4, 2, d, dtype, page, layout, seed=d, pad_tokens=3)
    check_gather(b, d ** -0.5, mask, window)


@pytest.mark.parametrize("page", [8, 16, 64, 512])
@pytest.mark.parametrize("layout", ["token", "head", "both"])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("lens", [[(1, 600), (20, 130), (1, 127), (3, 1025)], [(1, 600), (1, 7), (2, 1025)], [(200, 300)]])
def test_pages(lens, page, layout, d):
    check_gather(paged(lens, 6, 2, d, torch.bfloat16, page, layout, seed=page), d ** -0.5, "causal")


@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (8, 1), (7, 1), (6, 2), (64, 4), (40, 8), (256, 1), (130, 1), (17, 1)])
@pytest.mark.parametrize("lens", [[(1, 300), (9, 140), (1, 5)], [(1, 300), (1, 129)], [(70, 300)]])
def test_heads(lens, H, Hk):
    check_gather(paged(lens, H, Hk, 64, torch.float16, 16, seed=H), 0.125, "causal")


@pytest.mark.parametrize("lens", [[(1, 33000), (1, 50)], [(1500, 4000), (1, 700)], [(2, 9000), (30, 30)]])
def test_long_sequences(lens):
    check_gather(paged(lens, 8, 2, 128, torch.bfloat16, 64, "head", seed=1), 128 ** -0.5, "causal")
    check_gather(paged(lens, 8, 2, 128, torch.bfloat16, 64, "head", seed=1), 128 ** -0.5, "window", (777, 0))


@pytest.mark.parametrize("B", [100, 300])
def test_many_sequences(B):
    rng = random.Random(B)
    lens = [(n, n + rng.choice([0, 3, 70, 300])) for n in (rng.choice([0, 1, 1, 2, 30]) for _ in range(B))]
    check_gather(paged(lens, 4, 2, 64, torch.bfloat16, 16, seed=2), 0.125, "causal")


@pytest.mark.parametrize("H,Hk,d", [(64, 2, 64), (48, 1, 128), (32, 1, 256), (5, 1, 32)])
@pytest.mark.parametrize("most", [2, 3, 7])
def test_units_of_different_numbers_of_rows(H, Hk, d, most):
    """Tiles of keys that one, two, three and more tiles of rows see, in all orders: the warps that share a
    unit's rows and those that have one to themselves stay in step."""
    lens = [(1 + i * i % most, 700 + 61 * i) for i in range(24)]
    check_gather(paged(lens, H, Hk, d, torch.bfloat16, 64, seed=most), d ** -0.5, "causal")


def test_rows_without_keys_add_nothing():
    """A position before 0 under a mask leaves LSE = -infinity; its scores may be anything."""
    b = paged([(7, 3), (2, 40)], 4, 2, 64, torch.bfloat16, 16, seed=2)
    check_gather(b, 0.125, "causal")
    lse = lse_of(b[5], 2, 0.125, "causal", (0, 0), b[0].shape[0])
    lse[8] = -math.inf  # by hand: as if that token had seen nothing
    check_gather(b, 0.125, "causal", lse=lse)


@pytest.mark.parametrize("bad", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("lens,H,Hk", [([(1, 300), (2, 140), (1, 40)], 8, 2), ([(20, 300), (20, 200)], 4, 2),
                                       ([(70, 300), (40, 60)], 4, 2), ([(300, 900)], 8, 2)])
def test_rows_of_lse_minus_infinity_add_nothing_whatever_they_hold(lens, H, Hk, d, bad):
    """Queries of NaN and infinities whose LSE is -infinity, in tiles that every row sees and in others."""
    b = paged(lens, H, Hk, d, torch.bfloat16, 16, seed=6)
    q, seqs = b[0], b[5]
    lse = lse_of(seqs, Hk, 0.1, "causal", (0, 0), q.shape[0])
    g = torch.Generator(device=DEV).manual_seed(3)
    hit = torch.rand(lse.shape, generator=g, device=DEV) < 0.2
    hit[0, 0] = True
    lse[hit] = -math.inf
    q[hit] = bad
    t = 0
    for qq, _, _ in seqs:
        qq.copy_(q[t:t + qq.shape[0]])
        t += qq.shape[0]
    check_gather(b, 0.1, "causal", lse=lse)


@pytest.mark.parametrize("lens", [[(1, 300), (1, 40)], [(300, 900)]])
def test_infinite_scores(lens):
    """A key of +infinity in one column: for a finite LSE its weight is infinite if a query of its group
    has the same sign there, else it adds 0; for an LSE of +infinity it is NaN, and other keys get 0."""
    H, Hk, d = 8, 2, 64
    b = paged(lens, H, Hk, d, torch.bfloat16, 16, seed=8)
    q, cache, table, cu, seq_k, seqs = b
    lse = lse_of(seqs, Hk, 0.1, "causal", (0, 0), q.shape[0])
    q[..., 3] = -0.5
    q[0, :4, 3] = 0.5  # the first K/V head's: a score of +infinity for the first token
    L, at = lens[0][1], 100
    cache.k[table[0, at // 16], at % 16, :, 3] = math.inf
    weights = torch.zeros(cache.num_pages, Hk, 16, device=DEV)
    gather(q, lse, weights, cache, table, cu, seq_k, 0.1, "causal")
    got = weights[table[0, torch.arange(L, device=DEV) // 16].long(), :, torch.arange(L, device=DEV) % 16]
    assert float(got[at, 0]) == math.inf and float(got[at, 1]) == 0
    got[at] = 1
    assert bool(torch.isfinite(got).all()) and bool((got > 0).all())
    n = lens[0][0]
    lse[:n, :4] = math.inf
    weights.zero_()
    gather(q, lse, weights, cache, table, cu, seq_k, 0.1, "causal")
    got = weights[table[0, torch.arange(L, device=DEV) // 16].long(), :, torch.arange(L, device=DEV) % 16]
    assert bool(got[at, 0].isnan()) and float(got[at, 1]) == 0
    got[at, 0] = 0
    assert bool((got[:, 0] == 0).all())


def test_nan_of_another_sequence_and_of_a_key_stay_there():
    q, cache, table, cu, lens, seqs = paged([(1, 90), (1, 100), (3, 70)], 4, 2, 64, torch.bfloat16, 16, seed=2)
    scale = 0.125
    lse = lse_of(seqs, 2, scale, "causal", (0, 0), q.shape[0])
    clean = torch.zeros(cache.num_pages, 2, 16, device=DEV)
    gather(q, lse, clean, cache, table, cu, lens, scale, "causal")
    bad, weights = q.clone(), torch.zeros_like(clean)
    bad[1] = NAN
    gather(bad, lse, weights, cache, table, cu, lens, scale, "causal")
    for i, n in ((0, 90), (2, 70)):
        pg = table[i, :-(-n // 16)].long()
        assert torch.equal(weights[pg], clean[pg])
    cache.k[table[0, 2], 5, 1] = NAN
    weights = torch.zeros_like(clean)
    gather(q, lse, weights, cache, table, cu, lens, scale, "causal")
    assert bool(weights[table[0, 2], 1, 5].isnan()) and int(weights.isnan().sum()) == 1


def test_page_numbers_outside_the_cache_are_not_written():
    q, cache, table, cu, lens, seqs = paged([(1, 300), (1, 200)], 4, 2, 64, torch.bfloat16, 16, seed=4)
    lse = lse_of(seqs, 2, 0.125, "causal", (0, 0), q.shape[0])
    want, got = (torch.zeros(cache.num_pages + 4, 2, 16, device=DEV) for _ in range(2))
    gather(q, lse, want[2:-2], cache, table, cu, lens, 0.125, "causal")
    lost = []
    for b, p, bad in ((0, 3, -1), (0, 9, cache.num_pages), (1, 0, 2 ** 31 - 1), (1, 12, -2 ** 31)):
        lost.append(int(table[b, p]))
        table[b, p] = bad
    gather(q, lse, got[2:-2], cache, table, cu, lens, 0.125, "causal")
    want[2:-2][lost] = 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("B,T", [(2, 1), (40, 30), (70, 3)])
def test_offsets_in_no_order_give_a_token_to_the_first_sequence(B, T):
    """Every second sequence claims all tokens: the others of them add nothing."""
    q, cache, table, cu, lens, seqs = paged([(T, 300)] + [(0, 300)] * (B - 1), 8, 2, 64, torch.bfloat16, 16, seed=4)
    lse = lse_of(seqs, 2, 0.125, "causal", (0, 0), T)
    want = torch.ones(cache.num_pages, 2, 16, device=DEV)
    got = want.clone()
    gather(q, lse, want, cache, table, cu, lens, 0.125, "causal")
    gather(q, lse, got, cache, table, i32(([0, T] * B)[:B + 1]), lens, 0.125, "causal")
    assert torch.equal(got, want) and not bool((want == 1).all())
    gather(q, lse, got, cache, table, i32([-5, 0] + [T + 9, -1] * B)[:B + 1].contiguous(), lens, 0.125, "causal")


@pytest.mark.parametrize("H,Hk,d", [(4, 2, 64), (64, 2, 64), (8, 1, 256)])
@pytest.mark.parametrize("cu,lens", [
    ([0, 5, 3, 8], [90, 40, 70]),               # the last sequence keeps its tokens 5 to 7
    ([5, 0, 8], [30, 90]),                      # an empty first one, far along
    ([8, 8, 0, 4, 8], [30, 30, 20, 90]),
    ([5, 8, 0, 6], [90, 30, 70]),               # behind the first one's end: nothing left
    ([0, 6, 2, 9, 4, 12], [50, 9, 300, 11, 77]),
    ([-5, 3, -1, 7, 2, 40], [4, 60, 200, 8, 90]),  # clamped to the tokens
    ([-5, 0, 21, -1, 21], [30, 90, 40, 60]),
    ([0, 12, 0, 12, 0, 12], [200, 1, 300, 2, 10]),
])
def test_offsets_in_no_order_against_the_definition(cu, lens, H, Hk, d):
    """Each sequence's tokens before the furthest end so far are left out; the others, its last
    ones, stand where they stood. Nothing outside the array is written."""
    T, page, scale, guard = 12, 16, 0.1, 3
    q, cache, table, _, seq_k, seqs = paged([(0, n) for n in lens], H, Hk, d, torch.bfloat16, page, seed=len(cu))
    g = torch.Generator(device=DEV).manual_seed(7)
    q = torch.randn(T, H, d, generator=g, device=DEV).to(torch.bfloat16)
    lse = torch.rand(T, H, generator=g, device=DEV) + 1  # any will do
    whole = torch.full((cache.num_pages + 2 * guard, Hk, page), -777.0, device=DEV)
    weights = whole[guard:-guard]
    weights.copy_(torch.rand(weights.shape, generator=g, device=DEV))
    before, rest = weights.clone(), torch.ones(weights.shape, dtype=torch.bool, device=DEV)
    gather(q, lse, weights, cache, table, i32(cu), seq_k, scale, "causal")
    end = 0
    for b, (_, k, _) in enumerate(seqs):
        first = min(max(cu[b], 0), T)
        stop = min(max(cu[b + 1], first), T)
        skip = min(max(end - first, 0), stop - first)
        if stop > first:
            end = max(end, stop)
        n, L = stop - first - skip, lens[b]
        if n == 0:
            continue
        j = torch.arange(L, device=DEV)
        pg, sl = table[b, j // page].long(), j % page
        old = before[pg, :, sl].double()
        old[max(0, L - (stop - first)):] = 0  # the call's own keys, those of tokens left out among them
        # gather_ref clears the keys of the tokens it is given, which are the last of these
        want, bound = gather_ref(q[first + skip:stop], k, lse[first + skip:stop], old, scale, "causal", (0, 0))
        assert_within(weights[pg, :, sl], want, bound, f"sequence {b}")
        rest[pg, :, sl] = False
    assert torch.equal(weights[rest], before[rest]), "wrote another slot"
    assert bool((whole[:guard] == -777.0).all()) and bool((whole[-guard:] == -777.0).all())


@pytest.mark.parametrize("new", [1, 40])
def test_a_shared_page_gets_every_sequences_share(new):
    """Two sequences over the same pages but for their own tokens': both add to the shared ones."""
    page, Hk, H, d, n = 16, 2, 4, 64, 160
    g = torch.Generator(device=DEV).manual_seed(1)
    k = torch.randn(30, page, Hk, d, generator=g, device=DEV).to(torch.bfloat16)
    cache = fa.PagedCache(k, k.clone())
    table = i32([list(range(10)) + [10, 11, 12], list(range(10)) + [13, 14, 15]])
    q = torch.randn(2 * new, H, d, generator=g, device=DEV).to(torch.bfloat16)
    cu, lens = i32([0, new, 2 * new]), i32([n + new] * 2)
    seqs = [(q[i * new:(i + 1) * new], k[table[i].long()].flatten(0, 1)[:n + new], None) for i in range(2)]
    lse = lse_of(seqs, Hk, 0.125, "causal", (0, 0), 2 * new)
    weights = torch.full((30, Hk, page), 1.0, device=DEV)
    gather(q, lse, weights, cache, table, cu, lens, 0.125, "causal")
    want, bound = torch.ones(n, Hk, dtype=torch.float64, device=DEV), 0
    for i, (qq, kk, _) in enumerate(seqs):
        one, b = gather_ref(qq, kk, lse[i * new:(i + 1) * new], torch.zeros(n + new, Hk, dtype=torch.float64, device=DEV), 0.125,
                            "causal", (0, 0))
        want, bound = want + one[:n], bound + b[:n]
    assert_within(weights[:10].transpose(1, 2).reshape(n, Hk), want, bound + 2.0 ** -22 * want, "shared")


def test_weights_past_32_bits():
    """Keys whose elements lie past 2^31 of the cache."""
    page, Hk, d, n = 128, 8, 128, 300
    pages = 2 ** 31 // (page * Hk * d) + 40
    k = torch.empty(pages, page, Hk, d, dtype=torch.bfloat16, device=DEV)
    cache = fa.PagedCache(k, k)
    mine = [pages - 1, 3, pages - 7]
    g = torch.Generator(device=DEV).manual_seed(1)
    for pg in mine:
        k[pg] = torch.randn(page, Hk, d, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn(2, 16, d, generator=g, device=DEV).to(torch.bfloat16)
    kk = k[mine].flatten(0, 1)[:n]
    seqs = [(q, kk, None)]
    lse = lse_of(seqs, Hk, 0.09, "causal", (0, 0), 2)
    weights = torch.zeros(pages, Hk, page, device=DEV)
    gather(q, lse, weights, cache, i32([mine]), i32([0, 2]), i32([n]), 0.09, "causal")
    want, bound = gather_ref(q, kk, lse, torch.zeros(n, Hk, dtype=torch.float64, device=DEV), 0.09, "causal", (0, 0))
    assert_within(weights[mine].transpose(1, 2).reshape(-1, Hk)[:n], want, bound, "weights")


def test_weights_are_the_same_every_time_and_captured():
    b = paged([(1, 5000), (40, 700), (0, 30), (1, 17)], 8, 2, 128, torch.bfloat16, 16, seed=5)
    q, cache, table, cu, lens, seqs = b
    lse = lse_of(seqs, 2, 0.09, "causal", (0, 0), q.shape[0])
    start = torch.rand(cache.num_pages, 2, 16, device=DEV)
    outs = []
    for _ in range(4):
        w = start.clone()
        for _ in range(3):
            gather(q, lse, w, cache, table, cu, lens, 0.09, "causal")
        outs.append(w)
    w, s = start.clone(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        fa.fa_paged_weights(q, lse, w, cache, table, cu, lens, 0.09, "causal", stream=s)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for x in (*outs[1:], w):
        assert torch.equal(x, outs[0])


def test_weights_on_two_streams_at_once():
    bs = [paged(lens, 8, 2, 128, torch.bfloat16, 64, seed=9 + i)
          for i, lens in enumerate([[(1, 9000)] * 6, [(700, 3000), (1, 50)]])]
    lses = [lse_of(b[5], 2, 0.1, "causal", (0, 0), b[0].shape[0]) for b in bs]
    blank = [torch.zeros(b[1].num_pages, 2, 64, device=DEV) for b in bs]
    want = [w.clone() for w in blank]
    for b, lse, w in zip(bs, lses, want):
        gather(b[0], lse, w, *b[1:5], 0.1, "causal")
    streams = [torch.cuda.Stream() for _ in bs]
    got = [[w.clone() for w in blank] for _ in range(20)]
    torch.cuda.synchronize()
    for one in got:
        for b, lse, w, s in zip(bs, lses, one, streams):
            fa.fa_paged_weights(b[0], lse, w, *b[1:5], 0.1, stream=s)
    torch.cuda.synchronize()
    assert fa.fa_sync_status() == fa.FA_OK
    assert all(torch.equal(g, w) for one in got for g, w in zip(one, want))


def test_the_fault_hook_ends_in_a_timeout():
    b = paged([(40, 600)], 2, 1, 128, torch.bfloat16, 16, seed=3)
    want = check_gather(b, 0.1, "causal")
    lse = lse_of(b[5], 1, 0.1, "causal", (0, 0), 40)
    fa.fa_set_wait_budget_ns(20_000_000)
    try:
        fa.fa_test_arm_fault(0)
        fa.fa_paged_weights(b[0], lse, torch.zeros_like(want), *b[1:5], 0.1, "causal")
        assert fa.fa_sync_status() == fa.FA_ERR_TIMEOUT
    finally:
        fa.fa_set_wait_budget_ns(0)
    again = check_gather(b, 0.1, "causal")
    assert torch.equal(again.nan_to_num(), want.nan_to_num())


# ------------------------------------------------------------------------ eviction

def filled(lens, Hk, d, dtype, page, layout, kind, seed=0):
    """A cache whose sequences have `lens` keys, and weights of a kind."""
    _, cache, table, _, seq_k, _ = paged([(0, n) for n in lens], Hk, Hk, d, dtype, page, layout, seed=seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = torch.randn(cache.num_pages, Hk, page, generator=g, device=DEV)
    if kind == "ties":
        w = (w * 2).round() / 2
    elif kind == "equal":
        w = torch.zeros_like(w)
    elif kind == "signed zeros":
        w = torch.where(w > 0, torch.zeros_like(w), -torch.zeros_like(w))
    elif kind == "near":  # neighbouring numbers, told apart by the last bits only
        w = (torch.randint(0, 5, w.shape, generator=g, device=DEV, dtype=torch.int32) + 0x3f800000).view(torch.float32)
    elif kind == "odd":
        pick = torch.randint(0, 8, w.shape, generator=g, device=DEV)
        for i, x in enumerate((NAN, math.inf, -math.inf, -0.0, 0.0, 1e-45)):
            w[pick == i] = x
    elif kind == "skewed":
        w = (w * 6).exp()
    return cache, w.contiguous(), table, seq_k


def keep(w, budget, first, recent):
    """The places that a head with weights w keeps: by the definition, in Python."""
    n = len(w)
    w = [-math.inf if x != x else x for x in w]
    mid = sorted(range(first, n - recent), key=lambda j: (-w[j], j))[:budget - first - recent]
    return list(range(first)) + sorted(mid) + list(range(n - recent, n))


def check_evict(cache, w, table, seq_k, budget, first=0, recent=0, **kw):
    page, Hk = cache.page_size, cache.H_kv
    k, v, weights = cache.k.clone(), cache.v.clone(), w.clone()
    lens = seq_k.tolist()
    for b, n in enumerate(lens):
        if n <= budget:
            continue
        j = torch.arange(n, device=DEV)
        pg, sl = table[b, j // page].long(), j % page
        for h in range(Hk):
            src = torch.tensor(keep(w[pg, h, sl].tolist(), budget, first, recent), dtype=torch.long, device=DEV)
            m = len(src)
            assert m == budget
            k[pg[:m], sl[:m], h] = cache.k[pg[src], sl[src], h]
            v[pg[:m], sl[:m], h] = cache.v[pg[src], sl[src], h]
            weights[pg[:m], h, sl[:m]] = w[pg[src], h, sl[src]]
    out = torch.full_like(seq_k, -9)
    fa.fa_paged_evict(cache, w, table, seq_k, out, budget, first, recent, **kw)
    assert fa.fa_sync_status() == fa.FA_OK
    assert out.tolist() == [min(n, budget) for n in lens]
    for got, want, what in ((cache.k, k, "keys"), (cache.v, v, "values")):
        assert torch.equal(got.contiguous().view(torch.int16), want.contiguous().view(torch.int16)), what
    assert torch.equal(w.view(torch.int32), weights.view(torch.int32)), "weights"
    return out


KINDS = ["plain", "ties", "equal", "signed zeros", "near", "odd", "skewed"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("budget,first,recent", [(100, 0, 0), (100, 4, 30), (1, 0, 0), (1, 1, 0), (60, 10, 50), (0, 0, 0), (299, 0, 7)])
def test_evict_kinds_of_weights(kind, budget, first, recent):
    check_evict(*filled([300, 100, 99, 101, 0, 1, 2, 700, 60, 1300], 2, 64, torch.bfloat16, 16, "token", kind),
                budget, first, recent)


@pytest.mark.parametrize("layout", ["token", "head", "both"])
@pytest.mark.parametrize("page", [8, 16, 128, 1024])
@pytest.mark.parametrize("d,dtype", [(32, torch.float16), (64, torch.bfloat16), (128, torch.bfloat16), (256, torch.float16)])
def test_evict_layouts(d, dtype, page, layout):
    check_evict(*filled([900, 2500, 400, 401], 3, d, dtype, page, layout, "ties", seed=page), 400, 4, 100)


@pytest.mark.parametrize("B,Hk,n", [(1, 1, 5000), (1, 8, 30000), (40, 1, 700), (300, 2, 90), (3, 1, 70000)])
@pytest.mark.parametrize("share", [0.1, 0.5, 0.95])
def test_evict_sizes(B, Hk, n, share):
    """Few and many sequences, up to more keys than stay in shared memory."""
    rng = random.Random(B)
    lens = [n] + [rng.randrange(n // 3, n + 1) for _ in range(B - 1)]
    check_evict(*filled(lens, Hk, 32 if n > 40000 else 64, torch.bfloat16, 16, "token", "skewed", seed=B), int(n * share), 2,
                int(n * share) // 3)


def test_evict_twice_and_at_a_budget_past_every_length():
    cache, w, table, seq_k = filled([500, 900, 30], 2, 128, torch.bfloat16, 16, "head", "ties")
    out = check_evict(cache, w, table, seq_k, 2 ** 40)
    assert torch.equal(out, seq_k)
    out = check_evict(cache, w, table, out, 300, 4, 50)
    out = check_evict(cache, w, table, out, 299, 4, 50)
    out = check_evict(cache, w, table, out, 20, 4, 16)
    assert out.tolist() == [20, 20, 20]


def test_evict_does_not_follow_pages_outside_the_cache():
    """They count as weight 0 and rows of zeros, and are not written."""
    cache, w, table, seq_k = filled([200], 1, 64, torch.bfloat16, 16, "token", "plain")
    whole = [torch.full((cache.num_pages + 4, 16, 1, 64), -777.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for t, x in zip(whole, (cache.k, cache.v)):
        t[2:-2] = x
    inner = fa.PagedCache(*(t[2:-2] for t in whole))
    wide = torch.full((cache.num_pages + 4, 1, 16), -777.0, device=DEV)
    wide[2:-2] = w
    j = torch.arange(200, device=DEV)
    pg, sl = table[0, j // 16].long().clone(), j % 16
    for p, bad in ((2, -1), (7, cache.num_pages), (11, -2 ** 31)):
        table[0, p] = bad
    there = ~torch.isin(j // 16, torch.tensor([2, 7, 11], device=DEV))
    rows = [torch.where(there[:, None], x[pg, sl, 0], torch.zeros((), dtype=x.dtype, device=DEV)) for x in (cache.k, cache.v)]
    ws = torch.where(there, w[pg, 0, sl], torch.zeros((), device=DEV))
    src = torch.tensor(keep(ws.tolist(), 120, 3, 20), device=DEV)
    want = [t.clone() for t in whole]
    want_w = wide.clone()
    for x, y in enumerate(src.tolist()):
        if bool(there[x]):
            for t, r in zip(want, rows):
                t[2 + pg[x], sl[x], 0] = r[y]
            want_w[2 + pg[x], 0, sl[x]] = ws[y]
    out = torch.empty_like(seq_k)
    fa.fa_paged_evict(inner, wide[2:-2], table, seq_k, out, 120, 3, 20)
    assert fa.fa_sync_status() == fa.FA_OK
    for got, x in zip(whole, want):
        assert torch.equal(got.view(torch.int16), x.view(torch.int16))
    assert torch.equal(wide, want_w)


def test_evict_lengths_are_clamped_to_the_table():
    cache, w, table, seq_k = filled([48, 30], 2, 64, torch.bfloat16, 16, "token", "plain")
    three = table[:, :3].contiguous()
    out = torch.empty_like(seq_k)
    fa.fa_paged_evict(cache, w, three, i32([2 ** 31 - 1, -5]), out, 40, 0, 0)
    assert fa.fa_sync_status() == fa.FA_OK and out.tolist() == [40, 0]


def test_evict_past_32_bits():
    page, Hk, d = 128, 8, 128
    pages = 2 ** 31 // (page * Hk * d) + 40
    k, v = (torch.zeros(pages, page, Hk, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    mine = [pages - 1, 3, pages - 7]
    g = torch.Generator(device=DEV).manual_seed(1)
    for pg in mine:
        for x in (k, v):
            x[pg] = torch.randn(page, Hk, d, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.rand(pages, Hk, page, generator=g, device=DEV)
    kk, vv, ww = k[mine].flatten(0, 1)[:300], v[mine].flatten(0, 1)[:300], w[mine].transpose(1, 2).reshape(-1, Hk)[:300]
    out = torch.empty(1, dtype=torch.int32, device=DEV)
    fa.fa_paged_evict(fa.PagedCache(k, v), w, i32([mine]), i32([300]), out, 150, 1, 20)
    assert fa.fa_sync_status() == fa.FA_OK
    for h in range(Hk):
        src = torch.tensor(keep(ww[:, h].tolist(), 150, 1, 20), device=DEV)
        assert torch.equal(k[mine].flatten(0, 1)[:150, h], kk[src, h])
        assert torch.equal(v[mine].flatten(0, 1)[:150, h], vv[src, h])
        assert torch.equal(w[mine].transpose(1, 2).reshape(-1, Hk)[:150, h], ww[src, h])


# ------------------------------------------------------------------------ together

@pytest.mark.parametrize("d,layout", [(128, "half"), (64, "interleaved")])
def test_a_serving_loop_that_evicts(d, layout):
    """Prompt and single steps with weights gathered; at a length the cache is cut back, and later
    tokens, rotated for their true positions, attend to what is left. Against a model of it in 64 bits
    on the rows as stored."""
    dtype, page, H, Hk, scale = torch.bfloat16, 16, 8, 2, d ** -0.5
    budget, most, first, recent, n = 48, 64, 2, 16, 110
    g = torch.Generator(device=DEV).manual_seed(d)
    qkv = torch.randn(n, H + 2 * Hk, d, generator=g, device=DEV).to(dtype)
    rope = fa.NormRope(fa.rope_steps(d), layout)
    k, v = (torch.full((9, page, Hk, d), NAN, dtype=dtype, device=DEV) for _ in range(2))
    weights = torch.full((9, Hk, page), NAN, device=DEV)
    cache, table = fa.PagedCache(k, v), torch.randperm(9, device=DEV)[:6].to(torch.int32)[None].contiguous()
    held = [[torch.zeros(0, d, device=DEV, dtype=dtype)] * 2 for _ in range(Hk)]  # rows as stored
    gathered = [torch.zeros(0, dtype=torch.float64, device=DEV) for _ in range(Hk)]
    lens = i32([0])
    cuts = 0
    for a, b in [(0, 40)] + [(t, t + 1) for t in range(40, n)]:
        new = b - a
        x = qkv[a:b]
        q, kk = fa.qk_norm_rope(x[:, :H], x[:, H:H + Hk], rope, torch.arange(a, b, dtype=torch.int32, device=DEV))
        lens = lens + new
        cu = i32([0, new])
        fa.fa_paged_append(None, kk, x[:, H + Hk:], None, cache, table, cu, lens)
        o, lse = fa.forward_paged(q, cache, table, cu, lens)
        fa.fa_paged_weights(q, lse, weights, cache, table, cu, lens, scale)
        length = int(lens)
        pos = torch.arange(length, device=DEV)
        for h in range(Hk):
            held[h] = [torch.cat([held[h][0], kk[:, h]]), torch.cat([held[h][1], x[:, H + Hk + h]])]
            s = torch.einsum("igd,jd->gij", q[:, h * 4:h * 4 + 4].double(), held[h][0].double()) * scale
            s.masked_fill_(pos[None, None] > pos[None, length - new:, None], -math.inf)
            p = s.softmax(-1)
            want = torch.einsum("gij,jd->igd", p, held[h][1].double())
            spread = torch.einsum("gij,jd->igd", p, held[h][1].double().abs())
            # weights and outputs rounded to bf16, scores of order 10 in 32 bits
            assert_within(o[:, h * 4:h * 4 + 4], want, 2.0 ** -8 * (spread + want.abs()) + 2.0 ** -15 * spread, f"tokens {a}")
            gathered[h] = torch.cat([gathered[h], torch.zeros(new, dtype=torch.float64, device=DEV)]) + p.sum((0, 1))
        got = weights[table[0, pos // page].long(), :, pos % page]
        want = torch.stack(gathered, 1)
        # each of at most n sums: 2^-16 of itself for the scores and LSE, and its rounding
        assert_within(got, want, want * 2.0 ** -15, f"weights after {a}")
        if length > most:
            cuts += 1
            lens2 = torch.empty_like(lens)
            # what is kept is decided by the 32-bit weights
            keeps = [keep(got[:, h].tolist(), budget, first, recent) for h in range(Hk)]
            fa.fa_paged_evict(cache, weights, table, lens, lens2, budget, first, recent)
            lens = lens2
            for h in range(Hk):
                src = torch.tensor(keeps[h], device=DEV)
                held[h] = [r[src] for r in held[h]]
                gathered[h] = gathered[h][src]
    assert cuts >= 3 and fa.fa_sync_status() == fa.FA_OK


def test_evict_captured_and_on_another_stream():
    a = filled([500, 900, 30, 1500], 2, 128, torch.bfloat16, 16, "head", "ties")
    cache, w, table, seq_k = a
    other = fa.PagedCache(cache.k.clone(), cache.v.clone())
    w2, out, out2 = w.clone(), torch.empty_like(seq_k), torch.empty_like(seq_k)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        fa.fa_paged_evict(cache, w, table, seq_k, out, 300, 4, 50, stream=s)
    for lens in ([500, 900, 30, 1500], [300, 300, 30, 301], [10, 299, 900, 1500]):
        seq_k.copy_(i32(lens))
        torch.cuda.synchronize()
        graph.replay()
        fa.fa_paged_evict(other, w2, table, seq_k, out2, 300, 4, 50)
        torch.cuda.synchronize()
        assert torch.equal(out, out2) and torch.equal(w, w2)
        for x, y in ((cache.k, other.k), (cache.v, other.v)):
            assert torch.equal(x.contiguous().view(torch.int16), y.contiguous().view(torch.int16))


def test_binding_refusals():
    q, cache, table, cu, lens, _ = paged([(1, 20)], 4, 2, 64, torch.bfloat16, 16, seed=3)
    lse, w, out = torch.zeros(1, 4, device=DEV), torch.zeros(cache.num_pages, 2, 16, device=DEV), torch.empty_like(lens)
    good = dict(q=q, lse=lse, weights=w, cache=cache, block_table=table, cu_seqlens_q=cu, seqlens_k=lens, scale=0.1)
    for bad in (dict(q=q.half()), dict(lse=lse[:, :2]), dict(lse=lse.double()), dict(weights=w.double()),
                dict(weights=w.transpose(1, 2)), dict(weights=w[1:]), dict(block_table=table.long()), dict(scale=-1.0)):
        with pytest.raises(fa.FaError):
            fa.fa_paged_weights(**{**good, **bad})
    good = dict(cache=cache, weights=w, block_table=table, seqlens_k=lens, seqlens_out=out, budget=10)
    for bad in (dict(weights=w.half()), dict(weights=w[:, :1]), dict(seqlens_out=lens), dict(seqlens_out=out.long()),
                dict(seqlens_k=i32([1, 2])), dict(budget=-1), dict(first=11), dict(recent=11), dict(first=6, recent=6)):
        with pytest.raises(fa.FaError):
            fa.fa_paged_evict(**{**good, **bad})
    assert fa.fa_sync_status() == fa.FA_OK
