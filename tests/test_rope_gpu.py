"""fa_qk_norm_rope, its backward and the rotary steps, against their formulas in 64 bits."""

import math

import pytest
import torch

import tiled_attention_03_gb300 as fa
from tiled_attention_03_gb300 import binding

from rope_util import assert_within, norm_rope_bwd_ref, norm_rope_ref, rotate

pytestmark = pytest.mark.gpu

DEV = "cuda"
EPS = 1e-5


def make(shape, dtype, seed, spread=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * spread).to(dtype)


def handle(d, r, layout, dtype, norm_q=True, norm_k=True, scaling="none", magnitude=1.0, seed=5):
    freq = fa.rope_frequencies(r, 10000.0, scaling, 8.0, 2048) if r else []
    wq, wk = 1 + 0.3 * make((2, d), torch.float32, seed)
    wq, wk = (w.to(dtype) if on else None for w, on in ((wq, norm_q), (wk, norm_k)))
    steps = fa.rope_steps(r, 10000.0, scaling, 8.0, 2048) if r else None
    return fa.NormRope(steps, layout, magnitude, wq, wk, EPS), freq


def tok(x):
    """(B, H, N, d) -> B tensors (N, H, d); (tokens, H, d) as one."""
    return list(x.transpose(1, 2)) if x.dim() == 4 else [x]


def check_forward(x, y, w, rope_freq, pos, layout, magnitude, dtype, what):
    n = x.shape[2] if x.dim() == 4 else x.shape[0]
    for b, (xi, yi) in enumerate(zip(tok(x), tok(y))):
        p = torch.arange(n, device=DEV) if pos is None else pos.view(-1, n)[b]
        want, bound = norm_rope_ref(xi, w, p, rope_freq, layout, magnitude, EPS, dtype)
        assert_within(yi, want, bound, what)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,r", [(32, 32), (32, 8), (64, 64), (64, 30), (128, 128), (128, 32), (128, 2),
                                 (256, 256), (256, 64), (128, 0)])
def test_forward(d, r, layout, dtype):
    B, H, Hk, N = 2, 5, 2, 37
    rope, freq = handle(d, r, layout, dtype, magnitude=1.25, scaling="band" if r > 2 else "none")
    qkv = make((B, N, H + 2 * Hk, d), dtype, 1)
    q, k = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hk].transpose(1, 2)
    y, z = fa.qk_norm_rope(q, k, rope)
    assert fa.fa_sync_status() == fa.FA_OK
    assert y.is_contiguous() and z.is_contiguous()
    check_forward(q, y, rope.q_weight, freq, None, layout, 1.25, dtype, "q")
    check_forward(k, z, rope.k_weight, freq, None, layout, 1.25, dtype, "k")


@pytest.mark.parametrize("tokens,H,Hk", [(1, 1, 1), (1, 64, 8), (3, 7, 1), (129, 40, 8), (2000, 3, 3), (4096, 1, 0),
                                         (5, 0, 3)])
@pytest.mark.parametrize("norm_q,norm_k", [(True, False), (False, True), (False, False)])
def test_packed_positions_and_head_counts(tokens, H, Hk, norm_q, norm_k):
    dtype, d = torch.bfloat16, 64
    rope, freq = handle(d, d, "half", dtype, norm_q, norm_k)
    x = make((tokens, H + Hk, d), dtype, 2)
    q, k = (x[:, :H] if H else None), (x[:, H:] if Hk else None)
    g = torch.Generator().manual_seed(tokens)
    pos = torch.randint(-1000, 1 << 20, (tokens,), generator=g, dtype=torch.int32).to(DEV)
    y, z = fa.qk_norm_rope(q, k, rope, pos)
    if H:
        check_forward(q, y, rope.q_weight, freq, pos, "half", 1.0, dtype, "q")
    if Hk:
        check_forward(k, z, rope.k_weight, freq, pos, "half", 1.0, dtype, "k")


def test_in_place_and_into_a_fused_buffer():
    dtype, d, N, H = torch.float16, 128, 50, 6
    rope, freq = handle(d, 64, "interleaved", dtype)
    x = make((N, 2 * H, d), dtype, 3)
    want = fa.qk_norm_rope(x[:, :H], x[:, H:], rope)
    y = x.clone()
    fa.fa_qk_norm_rope(y[:, :H], y[:, H:], y[:, :H], y[:, H:], rope)
    assert torch.equal(y[:, :H], want[0]) and torch.equal(y[:, H:], want[1])
    wide = torch.full((N, 2 * H + 3, d), -777.0, dtype=dtype, device=DEV)
    fa.fa_qk_norm_rope(x[:, :H], x[:, H:], wide[:, :H], wide[:, H + 1:2 * H + 1], rope)
    assert torch.equal(wide[:, :H], want[0]) and torch.equal(wide[:, H + 1:2 * H + 1], want[1])
    assert bool((wide[:, H] == -777.0).all()) and bool((wide[:, 2 * H + 1:] == -777.0).all())


@pytest.mark.parametrize("any_stride", [-8, 5, -2 ** 62])
@pytest.mark.parametrize("B,H,Hk,N", [(2, 1, 3, 37), (2, 3, 1, 37), (1, 1, 1, 1), (1, 5, 2, 40), (3, 4, 1, 1)])
def test_strides_of_single_entries_do_not_matter(B, H, Hk, N, any_stride):
    """Through the C ABI (PyTorch makes no such strides): the same bits as with strides of 0."""
    dtype, d = torch.bfloat16, 128
    rope, _ = handle(d, d, "half", dtype)
    lib = binding.load_library()

    def step(single):
        x, g = ([make((B, h, N, d), dtype, 40 + 2 * i + j) for j, h in enumerate((H, Hk))] for i in range(2))
        y, dx = ([torch.full_like(t, math.nan) for t in x] for _ in range(2))
        dw = [torch.full((d,), math.nan, device=DEV) for _ in range(2)]
        ws = torch.empty(fa.fa_qk_norm_rope_backward_workspace_bytes(d), dtype=torch.uint8, device=DEV)

        def rows(t):
            s = [st if n > 1 else single for st, n in zip(t.stride()[:3], t.shape)]
            return binding._pack_rows(t.data_ptr(), *s)

        assert lib.fa_qk_norm_rope(*map(rows, x + y), rope.address, None, B, H, Hk, N, d, 1, None) == fa.FA_OK
        assert lib.fa_qk_norm_rope_backward(
            *map(rows, x + g + dx), dw[0].data_ptr(), dw[1].data_ptr(), rope.address, None, B, H, Hk, N, d, 1,
            ws.data_ptr(), ws.numel(), None) == fa.FA_OK
        assert fa.fa_sync_status() == fa.FA_OK
        return y + dx + dw

    for a, b in zip(step(any_stride), step(0)):
        assert bool(torch.isfinite(b).all()) and torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("r", [0, 32])
def test_elements_without_norm_and_rotation_stay(r, layout, dtype):
    """Every 16-bit value, the zero below 0 among them; a NaN stays one."""
    d = 64
    x = torch.arange(-2 ** 15, 2 ** 15, device=DEV).flip(0).to(torch.int16).view(-1, 4, d).view(dtype)
    assert bool((x[..., 32:].view(torch.int16) == -2 ** 15).any())
    rope, _ = handle(d, r, layout, dtype, True, False)
    for y in (*fa.qk_norm_rope(x, x, rope)[1:], fa.qk_norm_rope(None, x, rope)[1],
              fa.qk_norm_rope_backward(None, None, None, x, rope)[1]):
        x0, y0 = x[..., r:], y[..., r:]
        nan = torch.isnan(x0)
        assert bool(torch.isnan(y0[nan]).all())
        assert torch.equal(y0.contiguous().view(torch.int16)[~nan], x0.contiguous().view(torch.int16)[~nan])


def test_far_positions_keep_their_phase():
    """The whole range of int32 positions: a frequency of 1 wraps 340 million times."""
    d, dtype = 64, torch.float16
    rope, freq = handle(d, d, "half", dtype, False, False)
    pos = torch.tensor([0, 1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, -1, 1_000_003, 123_456_789],
                       dtype=torch.int32, device=DEV)
    x = make((8, 2, d), dtype, 4)
    y, _ = fa.qk_norm_rope(x, None, rope, pos)
    want, bound = norm_rope_ref(x, None, pos, freq, "half", 1.0, EPS, dtype)
    # the reference's own angles, p f in 64 bits, are off by 2^-53 p f <= 2^-22 radians, the
    # steps' (a product and a constant in 64 bits) by twice that
    _, size = rotate(x.double(), pos, freq, "half", 1.0)
    assert_within(y, want, bound + 2.0 ** -20 * size)


def test_infinities_stay_where_they_are():
    dtype, d = torch.bfloat16, 64
    rope, _ = handle(d, 32, "interleaved", dtype, False, False)
    x = make((4, 1, d), dtype, 6)
    x[2, 0, 50] = math.inf
    y, _ = fa.qk_norm_rope(x, None, rope)
    assert torch.isinf(y).sum() == 1 and bool(torch.isinf(y[2, 0, 50])) and not bool(torch.isnan(y).any())
    x[1, 0, 3] = math.nan
    y, _ = fa.qk_norm_rope(x, None, rope)
    assert torch.isnan(y).sum() == 2 and bool(torch.isnan(y[1, 0, 2:4]).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,r", [(32, 32), (32, 8), (64, 64), (128, 128), (128, 30), (256, 256), (256, 64), (64, 0)])
def test_backward(d, r, layout, dtype):
    B, H, Hk, N = 2, 6, 2, 45
    rope, freq = handle(d, r, layout, dtype, magnitude=0.75)
    qkv = make((B, N, H + 2 * Hk, d), dtype, 7, 1.5)
    q, k = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hk].transpose(1, 2)
    dy, dz = make((B, H, N, d), dtype, 8), make((B, Hk, N, d), dtype, 9)
    grad = torch.full_like(qkv, -777.0)
    dq, dk = grad[:, :, :H].transpose(1, 2), grad[:, :, H:H + Hk].transpose(1, 2)
    dwq, dwk = torch.empty(2, d, device=DEV)
    fa.fa_qk_norm_rope_backward(q, k, dy, dz, dq, dk, dwq, dwk, rope)
    assert fa.fa_sync_status() == fa.FA_OK
    assert bool((grad[:, :, H + Hk:] == -777.0).all()), "wrote the values' slice"
    pos = torch.arange(N, device=DEV)
    for x, g, dx, w, dw in ((q, dy, dq, rope.q_weight, dwq), (k, dz, dk, rope.k_weight, dwk)):
        sums, bounds = 0, 0
        for xi, gi, di in zip(tok(x), tok(g), tok(dx)):
            want, bound, s, sb = norm_rope_bwd_ref(xi, gi, w, pos, freq, layout, 0.75, EPS, dtype)
            assert_within(di, want, bound, "dx")
            sums, bounds = sums + s, bounds + sb
        assert_within(dw, sums, bounds, "dw")


@pytest.mark.parametrize("tokens,H,Hk", [(1, 1, 1), (1, 40, 8), (700, 9, 3), (3001, 2, 2), (40, 0, 2)])
@pytest.mark.parametrize("norm_q,norm_k", [(True, True), (True, False), (False, False)])
def test_backward_sizes(tokens, H, Hk, norm_q, norm_k):
    dtype, d = torch.bfloat16, 128
    rope, freq = handle(d, d, "half", dtype, norm_q, norm_k)
    x, dy = make((tokens, H + Hk, d), dtype, 10), make((tokens, H + Hk, d), dtype, 11)
    pos = torch.randperm(tokens, device=DEV).to(torch.int32)
    q, dq_out = (x[:, :H], dy[:, :H]) if H else (None, None)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(q, x[:, H:], dq_out, dy[:, H:], rope, pos)
    again = fa.qk_norm_rope_backward(q, x[:, H:], dq_out, dy[:, H:], rope, pos)
    for part, dx, w, dw in ((slice(0, H), dq, rope.q_weight, dwq), (slice(H, H + Hk), dk, rope.k_weight, dwk)):
        if dx is None:
            continue
        want, bound, s, sb = norm_rope_bwd_ref(x[:, part], dy[:, part], w, pos, freq, "half", 1.0, EPS, dtype)
        assert_within(dx, want, bound, "dx")
        assert (dw is None) == (w is None)
        if w is not None:
            assert_within(dw, s, sb, "dw")
    for a, b in zip((dq, dk, dwq, dwk), again):
        assert (a is None and b is None) or torch.equal(a, b), "not the same twice"


def test_backward_in_place():
    dtype, d, N, H = torch.bfloat16, 64, 33, 4
    rope, _ = handle(d, 32, "half", dtype)
    x, dy = make((N, 2 * H, d), dtype, 12), make((N, 2 * H, d), dtype, 13)
    want = fa.qk_norm_rope_backward(x[:, :H], x[:, H:], dy[:, :H], dy[:, H:], rope)
    g, dw = dy.clone(), torch.empty(2, d, device=DEV)
    fa.fa_qk_norm_rope_backward(x[:, :H], x[:, H:], g[:, :H], g[:, H:], g[:, :H], g[:, H:], dw[0], dw[1], rope)
    for a, b in zip((g[:, :H], g[:, H:], dw[0], dw[1]), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_against_differences(layout):
    """Central differences of the 64-bit forward reference along random directions: the
    differences' own error is of the order h^2 = 1e-8 of the function's size, so the 16-bit
    rounding of the gradients (half a step each, summed as random signs would not be:
    at most half a step of sum |dx| |direction|) is the bound."""
    dtype, d, N, H = torch.float16, 64, 9, 2
    rope, freq = handle(d, 48, layout, dtype)
    x, dy = make((N, H, d), dtype, 14), make((N, H, d), dtype, 15)
    pos = torch.arange(N, device=DEV)
    dx, _, dw, _ = fa.qk_norm_rope_backward(x, None, dy, None, rope)

    def f(xx, w):
        n = xx / (xx.square().mean(-1, keepdim=True) + EPS).sqrt() * w
        return (rotate(n, pos, freq, layout, 1.0)[0] * dy.double()).sum()

    h = 1e-4
    w = rope.q_weight.double()
    for seed in range(4):
        g = torch.Generator(device=DEV).manual_seed(seed)
        e = torch.randn(x.shape, generator=g, device=DEV, dtype=torch.float64)
        num = (f(x.double() + h * e, w) - f(x.double() - h * e, w)) / (2 * h)
        tol = 2.0 ** -11 * (dx.double() * e).abs().sum() + 1e-5 * dy.double().abs().sum()
        assert abs(num - (dx.double() * e).sum()) <= tol
        ew = torch.randn(d, generator=g, device=DEV, dtype=torch.float64)
        num = (f(x.double(), w + h * ew) - f(x.double(), w - h * ew)) / (2 * h)
        assert abs(num - (dw.double() * ew).sum()) <= 1e-5 * dy.double().abs().sum()


def test_capture_and_streams():
    """Captured and replayed on new inputs, and on a stream of its own, the same bits as a
    direct call; two captured graphs with a workspace each run at once."""
    dtype, d, N, H = torch.bfloat16, 128, 300, 8
    rope, _ = handle(d, d, "half", dtype)
    xs = [make((N, H, d), dtype, 20 + i) for i in range(4)]
    x = [torch.empty_like(xs[0]) for _ in range(2)]
    y = [torch.empty_like(xs[0]) for _ in range(2)]
    dx = [torch.empty_like(xs[0]) for _ in range(2)]
    dw = [torch.empty(d, device=DEV) for _ in range(2)]
    ws = [torch.empty(fa.fa_qk_norm_rope_backward_workspace_bytes(d), dtype=torch.uint8, device=DEV)
          for _ in range(2)]

    def step(i, stream=None):
        fa.fa_qk_norm_rope(x[i], None, y[i], None, rope, None, stream)
        fa.fa_qk_norm_rope_backward(x[i], None, y[i], None, dx[i], None, dw[i], None, rope, None, ws[i], stream)

    for i in range(2):
        x[i].copy_(xs[i])
        step(i)
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            step(i, streams[i])
    for i in range(2):
        x[i].copy_(xs[2 + i])
    torch.cuda.synchronize()
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            graphs[i].replay()
    torch.cuda.synchronize()
    got = [(y[i].clone(), dx[i].clone(), dw[i].clone()) for i in range(2)]
    for i in range(2):
        step(i)
        torch.cuda.synchronize()
        for a, b in zip(got[i], (y[i], dx[i], dw[i])):
            assert torch.equal(a, b)


def test_before_attention_and_back():
    """A training step's run of calls: norm and rotation into fa_forward, fa_backward, and
    back through the norm; against the same run in 64 bits with autograd. The bound of
    each gradient is what 16-bit roundings on the way (four of them, two steps each on
    sums that random signs shrink) leave of its norm."""
    dtype, B, H, Hk, N, d = torch.bfloat16, 1, 4, 2, 200, 64
    rope, freq = handle(d, d, "half", dtype)
    qkv = make((B, N, H + 2 * Hk, d), dtype, 30)
    q0, k0, v0 = qkv[:, :, :H], qkv[:, :, H:H + Hk], qkv[:, :, H + Hk:]
    q, k = fa.qk_norm_rope(q0.transpose(1, 2), k0.transpose(1, 2), rope)
    v = v0.transpose(1, 2).contiguous()
    o, lse = fa.forward(q, k, v, mask="causal")
    do = make(o.shape, dtype, 31)
    dq1, dk1, dv = fa.backward(q, k, v, o, lse, do, mask="causal")
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(q0.transpose(1, 2), k0.transpose(1, 2), dq1, dk1, rope)
    assert fa.fa_sync_status() == fa.FA_OK

    x = [t.double().detach().requires_grad_() for t in (q0, k0, v0, rope.q_weight, rope.k_weight)]
    pos = torch.arange(N, device=DEV)

    def nr(t, w):
        n = t / (t.square().mean(-1, keepdim=True) + EPS).sqrt() * w
        f = torch.tensor(freq, dtype=torch.float64, device=DEV)
        ang = pos.double()[:, None, None] * f
        a, b = n[..., :d // 2], n[..., d // 2:]
        return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)

    qq, kk = nr(x[0], x[3]).transpose(1, 2), nr(x[1], x[4]).transpose(1, 2)
    kk, vv = (t.repeat_interleave(H // Hk, 1) for t in (kk, x[2].transpose(1, 2)))
    s = (qq @ kk.transpose(2, 3) * d ** -0.5).masked_fill(
        torch.ones(N, N, dtype=torch.bool, device=DEV).triu(1), -math.inf)
    (s.softmax(-1) @ vv).backward(do.double())
    for got, want in ((dq.transpose(1, 2), x[0].grad), (dk.transpose(1, 2), x[1].grad),
                      (dv.transpose(1, 2), x[2].grad), (dwq, x[3].grad), (dwk, x[4].grad)):
        assert (got.double() - want).norm() <= 8 * 2.0 ** -8 * want.norm()


# How a launch is cut (the library's rule): tokens x stages of 256 / d heads (twice as many in
# the forward) over 8 warps a block, of as many blocks as the GPU holds at once, or, forward,
# more, a multiple of those, where each warp still gets 28 stages.
RESIDENT, LONG = 2, 28


def per_warp(tokens, H, Hk, d, rows):
    per = rows * 256 // d
    stages = tokens * (-(-H // per) + -(-Hk // per))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    blocks = RESIDENT * sms
    if rows == 2:
        blocks *= max(1, stages // (8 * LONG * blocks))
    return stages / (8 * blocks)


@pytest.mark.parametrize("dtype", [torch.bfloat16])
@pytest.mark.parametrize("layout,part", [("half", 1.0), ("half", 0.4), ("interleaved", 0.5)])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
def test_many_stages_per_warp(d, layout, part, dtype):
    """Training sizes: a warp's share takes its ring around several times, runs on from queries to
    keys, from token to token and from one batch entry into the next, and ends anywhere."""
    B, N, H, Hk = 3, 4001, 33, 5
    r = int(d * part) // 2 * 2
    assert (layout == "interleaved") or (r % 16 == 0) == (part == 1.0)  # partners: beside, in a lane, anywhere
    assert per_warp(B * N, H, Hk, d, 2) > 16 and per_warp(B * N, H, Hk, d, 1) > 28
    rope, freq = handle(d, r, layout, dtype)
    qkv = make((B, N, H + Hk, d), dtype, 50)
    q, k = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:].transpose(1, 2)
    y, z = fa.qk_norm_rope(q, k, rope)
    assert fa.fa_sync_status() == fa.FA_OK
    check_forward(q, y, rope.q_weight, freq, None, layout, 1.0, dtype, "q")
    check_forward(k, z, rope.k_weight, freq, None, layout, 1.0, dtype, "k")
    same = qkv.clone()
    qs, ks = same[:, :, :H].transpose(1, 2), same[:, :, H:].transpose(1, 2)
    fa.fa_qk_norm_rope(qs, ks, qs, ks, rope)
    assert torch.equal(qs, y) and torch.equal(ks, z), "in place"

    dqkv = make((B, N, H + Hk, d), dtype, 51)
    dy, dz = dqkv[:, :, :H].transpose(1, 2), dqkv[:, :, H:].transpose(1, 2)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(q, k, dy, dz, rope)
    assert fa.fa_sync_status() == fa.FA_OK
    # dw: 2^-18 of each term; a lane's running sum, then 64 rows of a block, a tenth of the
    # blocks and five halvings: that many steps of 2^-24 of the terms' sizes (sb is 2^-17 of them)
    more = 0.5 + (per_warp(B * N, H, Hk, d, 1) + 80) / 128
    pos = torch.arange(N, device=DEV)
    for x, g, dx, w, dw in ((q, dy, dq, rope.q_weight, dwq), (k, dz, dk, rope.k_weight, dwk)):
        sums, bounds = 0, 0
        for xi, gi, di in zip(tok(x), tok(g), tok(dx)):
            want, bound, s, sb = norm_rope_bwd_ref(xi, gi, w, pos, freq, layout, 1.0, EPS, dtype)
            assert_within(di, want, bound, "dx")
            sums, bounds = sums + s, bounds + more * sb
        assert_within(dw, sums, bounds, "dw")
    again = fa.qk_norm_rope_backward(q, k, dy, dz, rope)
    assert all(torch.equal(a, b) for a, b in zip(again, (dq, dk, dwq, dwk))), "not the same twice"


@pytest.mark.parametrize("more", [-1, 0, 1, 2000])
def test_around_the_switch_to_more_blocks(more):
    """The last sizes of resident blocks alone and the first of more."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    d, dtype = 128, torch.bfloat16
    tokens = 8 * LONG * 2 * RESIDENT * sms + more  # a stage each: 3 of its 4 heads there
    assert (per_warp(tokens, 3, 0, d, 2) * 8 * RESIDENT * sms >= tokens) == (more < 0)
    rope, freq = handle(d, d, "half", dtype)
    x = make((tokens, 3, d), dtype, 52)
    y, _ = fa.qk_norm_rope(x, None, rope)
    check_forward(x, y, rope.q_weight, freq, None, "half", 1.0, dtype, "q")
