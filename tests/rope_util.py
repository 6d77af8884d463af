"""64-bit references of the norm-and-rotation and paged-cache operators, from their
formulas, with elementwise bounds on what 32-bit arithmetic and one final rounding may
add. Everything runs on the inputs' device."""

import math

import torch


def half_step(dtype):
    """Relative error of rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Absolute error of rounding below the normal range (fp16)."""
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


def pairs(rotary_dim, layout, device):
    j = torch.arange(rotary_dim // 2, device=device)
    return (j, j + rotary_dim // 2) if layout == "half" else (2 * j, 2 * j + 1)


def rotate(x, pos, freq, layout, magnitude, transpose=False):
    """x (..., tokens, heads, d) float64, pos (tokens,) -> rotated, and |a| + |b| per element."""
    n = len(freq)
    f = torch.tensor(freq, dtype=torch.float64, device=x.device)
    ang = pos.double()[:, None, None] * f
    c, s = ang.cos() * magnitude, ang.sin() * magnitude
    if transpose:
        s = -s
    a, b = pairs(2 * n, layout, x.device)
    y, size = x.clone(), x.abs()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = (x[..., a].abs() + x[..., b].abs()) * abs(magnitude)
    return y, size


def norm_rope_ref(x, w, pos, freq, layout, magnitude, eps, dtype):
    """y and its bound for x (tokens, heads, d). In 32 bits: the mean and its root (d + 3
    roundings of positive terms), the products with the weight and the rotation (a few
    more), and the angle (2^-24 turns of a half): under 64 steps of 2^-24 for d = 256 with
    the sum split over lanes, so 2^-18 of |a| + |b|; then one rounding of y."""
    n = x.double()
    if w is not None:
        n = n / (n.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    y, size = rotate(n, pos, freq, layout, magnitude)
    return y, half_step(dtype) * y.abs() * (1 + 2 ** -8) + 2.0 ** -18 * size + tiny(dtype)


def norm_rope_bwd_ref(x, dy, w, pos, freq, layout, magnitude, eps, dtype):
    """(dx, bound, dw, bound) for x, dy (tokens, heads, d). dx as above, with the size of
    both terms of its difference; dw: each term off by 2^-18 of itself and the running
    sums (at most 64 terms in a lane, then trees) by 64 steps of 2^-24 of the terms' sizes."""
    u, size = rotate(dy.double(), pos, freq, layout, magnitude, transpose=True)
    if w is None:
        return u, half_step(dtype) * u.abs() * (1 + 2 ** -8) + 2.0 ** -18 * size + tiny(dtype), None, None
    x, w = x.double(), w.double()
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    z = x * r
    dx = r * (u * w - z * (u * w * z).mean(-1, keepdim=True))
    big = r * (size * w.abs() + z.abs() * (size * w.abs() * z.abs()).mean(-1, keepdim=True))
    dw = (u * z).sum((0, 1))
    return (dx, half_step(dtype) * dx.abs() * (1 + 2 ** -8) + 2.0 ** -17 * big + tiny(dtype), dw,
            2.0 ** -17 * (size * z.abs()).sum((0, 1)))


def assert_within(got, want, bound, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - bound
    assert bool((over <= 0).all()), f"{what}: off by {(got - want).abs().max():.3g}, over its bound by {over.max():.3g}"


def attention_ref(q, k, v, scale, mask, window, dtype):
    """One sequence: q (L_q, H, d), k, v (L_k, H_kv, d) in 16 bits. (O, bound, LSE, bound):
    a token at position i + L_k - L_q; rows that see no key give 0 and -inf.
    P is rounded to 16 bits (half a step of each p, or 2^-25 where fp16 goes below its
    normal range, over l >= 1), O once more; scores have d products summed in 32 bits."""
    Lq, H, d = q.shape
    Lk, Hk = k.shape[:2]
    dev = q.device
    i = torch.arange(Lq, device=dev)[:, None] + Lk - Lq
    j = torch.arange(Lk, device=dev)[None]
    see = torch.ones(Lq, Lk, dtype=torch.bool, device=dev)
    if mask == "causal":
        see = j <= i
    if mask == "window":
        see = (j >= i - window[0]) & (j <= i + window[1])
    o = torch.zeros(Lq, H, d, dtype=torch.float64, device=dev)
    ob = torch.zeros_like(o)
    lse = torch.full((Lq, H), -math.inf, dtype=torch.float64, device=dev)
    lb = torch.zeros_like(lse)
    some = see.any(1)
    g = H // Hk
    for h in range(H):
        if not bool(some.any()):
            break
        kk, vv = k[:, h // g].double(), v[:, h // g].double()
        # keys that this row does not see count for nothing, whatever they hold
        seen = see.any(0)
        kk = torch.where(seen[:, None], kk, torch.zeros_like(kk))
        vv = torch.where(seen[:, None], vv, torch.zeros_like(vv))
        x = (q[:, h].double() @ kk.T * scale).masked_fill(~see, -math.inf)
        size = ((q[:, h].double().abs() @ kk.abs().T) * scale).masked_fill(~see, 0).amax(1)
        top = x.amax(1, keepdim=True).clamp(min=-1e300)
        e = (x - top).exp()
        total = e.sum(1, keepdim=True)
        p = e / total.clamp(min=1e-300)
        lse[:, h] = torch.where(some, (top + total.log())[:, 0], lse[:, h])
        o[:, h] = p @ vv
        a = p @ vv.abs()
        step = d * 2.0 ** -24 * size + 2.0 ** -19
        ob[:, h] = half_step(dtype) * (a + o[:, h].abs()) * (1 + 2 ** -7) + 2 * step[:, None] * a + tiny(dtype) * (
            1 + vv.abs().sum(0)[None])
        lb[:, h] = step + 2.0 ** -20 * (lse[:, h].abs().clamp(max=1e30))
    return o, ob, lse, lb
