"""Cases of the operators that keep a serving cache small: a paged cache of one latent row a
token (its append, and the attention of new tokens over it in the absorbed form), and the
eviction of keys from a paged K/V cache by the attention weight they have gathered (its
accumulation, and the choice and move of what is kept). For each: the plain form in
elementary torch operations, the library's call, and the definition in 64 bits.

A sequence of a serving batch is (new, past): `new` tokens processed by this call and
`past` tokens that its pages already hold; the new tokens stand at positions past ..
past + new - 1. Lengths follow from the case alone; the seed orders them.
"""

import math
import random

import torch

own = False

DEV = "cuda"
BASE = 10000.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------------ cases

def _latent(op, name, dtype, batch, new_lo, new_hi, past_lo, past_hi, heads, d_latent, d_rope, page, **more):
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "past_lo": past_lo,
            "past_hi": past_hi, "heads": heads, "d_latent": d_latent, "d_rope": d_rope, "page": page, **more}


def _keys(op, name, dtype, batch, new_lo, new_hi, past_lo, past_hi, heads, kv_heads, head_dim, page, cache, **more):
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "past_lo": past_lo,
            "past_hi": past_hi, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "cache": cache, **more}


def listed():
    return [
        # one decode step: 64 sequences store one latent row each, launch latency
        _latent("latent_append", "latent_append_step", "bf16", 64, 1, 1, 1, 4000, 32, 512, 64, 64, norm=True, layout="interleaved"),
        # prompts of many lengths written to fresh and to half-filled pages, narrow rows that are stored as they come
        _latent("latent_append", "latent_append_prompts_d256", "fp16", 24, 1, 2000, 0, 500, 12, 256, 64, 16, norm=False, layout="half"),
        # one decode step of a few short conversations: latency
        _latent("latent_attention", "latent_step_short", "bf16", 4, 1, 1, 60, 1000, 16, 512, 64, 16, mask="causal", window=0),
        # one decode step over long caches
        _latent("latent_attention", "latent_step_long", "bf16", 8, 1, 1, 32767, 32767, 32, 512, 64, 64, mask="causal", window=0),
        # many sequences of all lengths with many heads: as much to compute as to read
        _latent("latent_attention", "latent_step_wide", "bf16", 40, 1, 1, 0, 16000, 128, 512, 64, 32, mask="causal", window=0),
        # few heads in odd number, one to three tokens at once, a sliding window, narrow rows
        _latent("latent_attention", "latent_ragged_d256", "fp16", 96, 1, 3, 0, 12000, 12, 256, 64, 16, mask="window", window=4096),
        # a chunk of a long prompt
        _latent("latent_attention", "latent_chunk", "bf16", 1, 1000, 1000, 14000, 14000, 16, 512, 64, 64, mask="causal", window=0),
        # the weights of one decode step over long caches, the benchmark's decode sizes in pages
        _keys("weights", "weights_step_long", "bf16", 8, 1, 1, 32767, 32767, 32, 8, 128, 64, "token", mask="causal", window=0),
        # many sequences of all lengths, small heads, one or two tokens at once
        _keys("weights", "weights_ragged_d64", "fp16", 100, 1, 2, 0, 12000, 16, 4, 64, 16, "head", mask="causal", window=0),
        # a chunk of a prompt: every key's weight over all of its queries
        _keys("weights", "weights_chunk", "bf16", 1, 2048, 2048, 6000, 6000, 32, 8, 128, 16, "token", mask="causal", window=0),
        # caches cut back to a budget, as when memory runs short
        _keys("evict", "evict_long", "bf16", 16, 0, 0, 5000, 20000, 32, 8, 128, 64, "token", budget=8192, first=4, recent=512),
        # a few short conversations, some of them within their budget: latency
        _keys("evict", "evict_short_d64", "fp16", 6, 0, 0, 200, 1500, 16, 4, 64, 16, "head", budget=500, first=0, recent=64),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["latent_append", "latent_attention", "latent_attention", "weights", "weights", "evict"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    page = rng.choice([8, 16, 32, 64, 128])
    mask = rng.choice(["causal", "causal", "window", "none"])
    window = _log(rng, 30, 5000) if mask == "window" else 0
    if op.startswith("latent"):
        heads = rng.choice([1, 4, 8, 12, 16, 20, 32, 64, 128])
        d_latent = rng.choice([128, 256, 512, 512])
        if op == "latent_append":
            batch = _log(rng, 1, 128)
            hi = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, 12000 // batch))
            c = _latent(op, "", dtype, batch, 1, hi, 0, _log(rng, 1, 4000), heads, d_latent, 64, page,
                        norm=rng.random() < 0.7, layout=rng.choice(["half", "interleaved"]))
        elif rng.random() < 0.6:  # decode, or a few tokens at once
            batch = _log(rng, 1, 128)
            c = _latent(op, "", dtype, batch, 1, rng.choice([1, 1, 1, 4]), 0, _log(rng, 100, max(200, min(32000, 300000 // batch))),
                        heads, d_latent, 64, page, mask=mask, window=window)
        else:  # chunks of prompts
            batch = _log(rng, 1, 12)
            c = _latent(op, "", dtype, batch, 1, _log(rng, 8, 1000 // batch + 8), 0, _log(rng, 8, 14000 // batch + 8),
                        heads, d_latent, 64, page, mask=mask, window=window)
        most_bytes, most_flops = 4.2e8, 5.0e11
    else:
        kv = rng.choice([1, 2, 4, 8])
        heads, d, cache = kv * rng.choice([1, 2, 3, 4, 7, 8]), rng.choice([32, 64, 128, 128, 256]), rng.choice(["token", "head"])
        if op == "evict":
            batch = _log(rng, 1, 64)
            n = _log(rng, 64, max(128, min(30000, 200000 // batch)))
            budget = max(1, int(n * rng.uniform(0.2, 0.95)))
            first = rng.choice([0, 0, 1, 4])
            recent = min(rng.choice([0, 16, 100, budget // 4, budget // 2]), budget)
            first = min(first, budget - recent)
            c = _keys(op, "", dtype, batch, 0, 0, max(1, n // 4), n, heads, kv, d, page, cache, budget=budget, first=first, recent=recent)
        elif rng.random() < 0.6:
            batch = _log(rng, 1, 128)
            c = _keys(op, "", dtype, batch, 1, rng.choice([1, 1, 1, 4]), 0, _log(rng, 100, max(200, min(32000, 300000 // batch))),
                      heads, kv, d, page, cache, mask=mask, window=window)
        else:
            batch = _log(rng, 1, 12)
            c = _keys(op, "", dtype, batch, 1, _log(rng, 8, 2000 // batch + 8), 0, _log(rng, 8, 8000 // batch + 8),
                      heads, kv, d, page, cache, mask=mask, window=window)
        most_bytes, most_flops = 6e8, 1.2e11
    while op != "evict" and (work(c)["flops"] > most_flops or work(c)["bytes"] > most_bytes):  # no more than the largest listed case
        c["new_hi"], c["past_hi"] = -(-c["new_hi"] * 3 // 4), c["past_hi"] // 2
    while op == "evict" and work(c)["bytes"] > most_bytes:
        c["batch"] = -(-c["batch"] // 2)
        if c["batch"] == 1:
            break
    c.pop("name")
    return c


def lengths(case):
    """[(new, past)]: the longest of each first, the others spread over the logarithm."""
    rng = random.Random("%(batch)d %(new_lo)d %(new_hi)d %(past_lo)d %(past_hi)d" % case)
    out = [(case["new_hi"], case["past_hi"])]
    while len(out) < case["batch"]:
        new = 0 if case["new_hi"] == 0 else _log(rng, case["new_lo"], case["new_hi"])
        out.append((new, _log(rng, max(1, case["past_lo"]), max(1, case["past_hi"])) - (case["past_lo"] == 0)))
    return out


def work(case):
    h, lens = case["heads"], lengths(case)
    new = sum(n for n, _ in lens)
    pages = sum(-(-(n + p) // case["page"]) for n, p in lens)
    plan = 4 * (pages + 2 * case["batch"] + 1)
    if case["op"] == "latent_append":
        dl, dr = case["d_latent"], case["d_rope"]
        return {"bytes": new * (dl + dr + h * dr) * 4 + plan, "flops": new * (dl * (4 if case["norm"] else 0) + (1 + h) * dr * 3)}
    if case["op"] == "evict":
        # every weight is read; kept rows behind the first one that goes (about as far in as is protected) are read and written
        over = [p for _, p in lens if p > case["budget"]]
        moved = len(over) * (case["budget"] - case["first"])
        kv, d = case["kv_heads"], case["head_dim"]
        return {"bytes": sum(over) * kv * 4 + moved * kv * 2 * (4 * d + 4) + plan, "flops": sum(over) * kv}
    keys = pairs = 0
    for n, p in lens:
        first = max(0, p - case["window"]) if case["mask"] == "window" else 0
        keys += n + p - first
        if case["mask"] == "none":
            pairs += n * (n + p)
        else:
            reach = case["window"] if case["mask"] == "window" else n + p
            pairs += sum(min(p + i, reach) + 1 for i in range(n))
    if case["op"] == "weights":
        kv, d = case["kv_heads"], case["head_dim"]
        return {"bytes": keys * kv * (2 * d + 8) + new * h * (2 * d + 4) + plan, "flops": 2 * pairs * h * d}
    dl, dr = case["d_latent"], case["d_rope"]
    return {"bytes": keys * (dl + dr) * 2 + new * h * (4 * dl + 2 * dr + 4) + plan, "flops": 2 * pairs * h * (2 * dl + dr)}


# ------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt, h, page = DTYPES[case["dtype"]], case["heads"], case["page"]
    randn = lambda *shape: torch.randn(shape, generator=g, device=DEV).to(dt)  # noqa: E731
    s = {"case": case, "op": case["op"]}
    lens = lengths(case)
    random.Random(seed).shuffle(lens)
    b = len(lens)
    total = [n + p for n, p in lens]
    need = [-(-t // page) for t in total]
    pages = sum(need) + 5
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).cpu()
    table, at = torch.full((b, max(need) + 1), -1, dtype=torch.int32), 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    s["table"] = table.to(DEV)
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    s["seq_k"] = torch.tensor(total, dtype=torch.int32, device=DEV)
    s["max_new"], s["max_k"] = max(n for n, _ in lens), max(total)

    if case["op"].startswith("latent"):
        dl, dr = case["d_latent"], case["d_rope"]
        s["data"] = randn(pages, page, dl + dr)
        if own:
            import tiled_attention_03_gb300 as fa
            s["cache"] = fa.LatentCache(s["data"], dl)
        if case["op"] == "latent_append":
            freq = [BASE ** (-2.0 * i / dr) for i in range(dr // 2)]
            s["freq"] = torch.tensor(freq, dtype=torch.float64, device=DEV)
            s["weight"] = (1 + 0.2 * torch.randn(dl, generator=g, device=DEV)).to(dt) if case["norm"] else None
            if own:
                s["rope"] = fa.NormRope(fa.rope_steps(dr, BASE), layout=case["layout"], k_weight=s["weight"], eps=EPS)
            # one projection per token gives latent and key part, another the queries' heads, their rotary part last
            down = randn(cu[-1], dl + dr)
            s["c"], s["k_rope"] = down[:, :dl], down[:, dl:]
            s["q_rope"] = randn(cu[-1], h, 128 + dr)[..., 128:]
            # the other columns of the absorbed queries come from their product with the up-projection
            s["q"] = randn(cu[-1], h, dl + dr)
            s["q_out"] = s["q"][..., dl:]
        else:
            s["q"] = randn(cu[-1], h, dl + dr)
            s["o"] = torch.empty(cu[-1], h, dl, dtype=dt, device=DEV)
            s["lse"] = torch.empty(cu[-1], h, dtype=torch.float32, device=DEV)
            s["scale"] = (dl + dr) ** -0.5
            if own:
                s["workspace"] = torch.empty(fa.fa_forward_latent_workspace_bytes(dl), dtype=torch.uint8, device=DEV)
        return s

    kv, d = case["kv_heads"], case["head_dim"]
    shape = (pages, page, kv, d) if case["cache"] == "token" else (pages, kv, page, d)
    caches = [randn(*shape) for _ in range(2 if case["op"] == "evict" else 1)]
    if case["cache"] == "head":
        caches = [c.transpose(1, 2) for c in caches]
    s["k_cache"], s["v_cache"] = caches[0], caches[-1]  # pages x page x heads x d, in memory token- or head-major
    if own:
        import tiled_attention_03_gb300 as fa
        s["cache"] = fa.PagedCache(s["k_cache"], s["v_cache"])
    # what earlier steps have gathered: a few keys have most of it
    s["weights"] = torch.randn(pages, kv, page, generator=g, device=DEV).mul_(2).exp_()
    if case["op"] == "evict":
        # keys that nothing looked at, and keys that were looked at alike
        s["weights"][s["weights"] < 0.25] = 0
        coarse = torch.rand(pages, kv, page, generator=g, device=DEV) < 0.5
        s["weights"] = torch.where(coarse, (s["weights"] * 16).floor() / 16, s["weights"])
        s["seq_out"] = torch.empty_like(s["seq_k"])
    else:
        s["q"] = randn(cu[-1], h, d)
        s["scale"] = d ** -0.5
        # the step's own sums, as its attention left them
        x = scores(s)
        s["lse"] = by_row(s, torch.logsumexp(x, -1))
        s["weights"] *= cu[-1] * h / kv / max(1, sum(total))
    return s


# ------------------------------------------------------------------------ one pass

def run(s):
    if not own:
        return {"latent_append": plain_latent_append, "latent_attention": plain_latent_attention, "weights": plain_weights,
                "evict": plain_evict}[s["op"]](s)
    import tiled_attention_03_gb300 as fa
    case = s["case"]
    if s["op"] == "latent_append":
        fa.fa_latent_append(s["q_rope"], s["c"], s["k_rope"], s["q_out"], s["cache"], s["table"], s["cu"], s["seq_k"], s["rope"])
        return {"q": s["q"], "data": s["data"]}
    if s["op"] == "latent_attention":
        fa.fa_forward_latent(s["q"], s["o"], s["lse"], s["cache"], s["table"], s["cu"], s["seq_k"], s["scale"], case["mask"], case["window"], 0, s["workspace"])
        return {"o": s["o"], "lse": s["lse"]}
    if s["op"] == "weights":
        fa.fa_paged_weights(s["q"], s["lse"], s["weights"], s["cache"], s["table"], s["cu"], s["seq_k"], s["scale"], case["mask"], case["window"], 0)
        return {"weights": s["weights"]}
    fa.fa_paged_evict(s["cache"], s["weights"], s["table"], s["seq_k"], s["seq_out"], case["budget"], case["first"], case["recent"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weights": s["weights"], "lengths": s["seq_out"]}


def rotate(x, cos, sin, layout):
    """The pairs of x's columns, rotated."""
    y, n = torch.empty_like(x), x.shape[-1]
    if layout == "half":
        a, b = x[..., :n // 2], x[..., n // 2:]
        y[..., :n // 2], y[..., n // 2:] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0::2], x[..., 1::2]
        y[..., 0::2], y[..., 1::2] = a * cos - b * sin, b * cos + a * sin
    return y


def places(s):
    """For each new token: its sequence and its position there."""
    new, n = (s["cu"][1:] - s["cu"][:-1]).long(), s["q"].shape[0]
    seq = torch.repeat_interleave(torch.arange(len(new), device=DEV), new, output_size=n)
    return seq, torch.arange(n, device=DEV) - s["cu"][seq] + s["seq_k"][seq] - new[seq]


def plain_latent_append(s):
    case, dl = s["case"], s["case"]["d_latent"]
    seq, pos = places(s)
    angle = pos.double()[:, None] * s["freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    c = s["c"].float()
    if s["weight"] is not None:
        c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    at = s["table"][seq, pos // case["page"]].long(), pos % case["page"]
    row = torch.cat([c, rotate(s["k_rope"].float(), cos, sin, case["layout"])], -1)
    s["data"][at] = row.to(s["data"].dtype)
    s["q_out"].copy_(rotate(s["q_rope"].float(), cos[:, None], sin[:, None], case["layout"]))
    assert s["data"].shape[-1] == dl + case["d_rope"]
    return {"q": s["q"], "data": s["data"]}


def rows_of(s, cache):
    """Each sequence's rows of the cache (batch x max_k x ...), in 32 bits."""
    pages = s["table"][:, :-(-s["max_k"] // s["case"]["page"])].clamp(min=0).long()
    return cache[pages].flatten(1, 2)[:, :s["max_k"]].float()


def scores(s):
    """The scaled scores, batch x kv heads x queries of each x new x keys; -inf where a key is not seen or no token is."""
    case, new = s["case"], (s["cu"][1:] - s["cu"][:-1]).long()
    b, nq, nk, h = len(new), s["max_new"], s["max_k"], case["heads"]
    k = rows_of(s, s["data"])[:, :, None] if "data" in s else rows_of(s, s["k_cache"])  # b x nk x kv x d
    i = torch.arange(nq, device=DEV)
    token = (s["cu"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"][token].float().reshape(b, nq, k.shape[2], h // k.shape[2], k.shape[3])
    x = torch.einsum("bikgd,bjkd->bkgij", q, k) * s["scale"]
    pos = i[None, :, None] + (s["seq_k"] - new)[:, None, None]  # b x nq x 1
    j = torch.arange(nk, device=DEV)[None, None, :]
    seen = (j < s["seq_k"][:, None, None]) & (i[None, :, None] < new[:, None, None])
    if case["mask"] != "none":
        seen = seen & (j <= pos)
    if case["mask"] == "window":
        seen = seen & (j >= pos - case["window"])
    return x.masked_fill_(~seen[:, None, None], -math.inf)


def by_row(s, x):
    """batch x kv x queries x new (x ...) as tokens x heads (x ...)."""
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    there = torch.arange(s["max_new"], device=DEV)[None] < new[:, None]
    return x.movedim(3, 1).flatten(2, 3)[there]


def plain_latent_attention(s):
    x = scores(s)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.einsum("bkgij,bjd->bkgid", x, rows_of(s, s["data"])[..., :s["case"]["d_latent"]]) / total.clamp(min=1e-30)
    s["o"].copy_(by_row(s, o))
    s["lse"].copy_(by_row(s, (top + total.log()).squeeze(-1)))
    return {"o": s["o"], "lse": s["lse"]}


def slots(s, n):
    """Where keys 0 .. n-1 of each sequence lie: their pages and the tokens there (batch x n)."""
    j = torch.arange(n, device=DEV)
    return s["table"][:, j // s["case"]["page"]].long(), (j % s["case"]["page"]).expand(len(s["seq_k"]), n)


def plain_weights(s):
    case, new = s["case"], (s["cu"][1:] - s["cu"][:-1]).long()
    b, nq, h, kv = len(new), s["max_new"], case["heads"], case["kv_heads"]
    token = (s["cu"][:-1, None] + torch.arange(nq, device=DEV)).clamp(max=s["q"].shape[0] - 1).long()
    lse = s["lse"][token].reshape(b, nq, kv, h // kv).permute(0, 2, 3, 1)[..., None]
    lse = torch.where(lse == -math.inf, torch.zeros_like(lse), lse)
    got = scores(s).sub_(lse).exp_().sum((2, 3))  # b x kv x nk
    page, slot = slots(s, s["max_k"])
    j = torch.arange(s["max_k"], device=DEV)[None]
    past, there = j < (s["seq_k"] - new)[:, None], j < s["seq_k"][:, None]
    old = torch.where(past[..., None], s["weights"][page.clamp(min=0), :, slot], torch.zeros((), device=DEV))
    s["weights"][page[there], :, slot[there]] = (old + got.transpose(1, 2))[there]
    return {"weights": s["weights"]}


def plain_evict(s):
    case, n = s["case"], s["max_k"]
    budget, kv = case["budget"], case["kv_heads"]
    s["seq_out"].copy_(s["seq_k"].clamp(max=budget))
    if n <= budget:
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weights": s["weights"], "lengths": s["seq_out"]}
    page, slot = slots(s, n)
    length, j = s["seq_k"][:, None, None].long(), torch.arange(n, device=DEV)
    w = s["weights"][page.clamp(min=0), :, slot].transpose(1, 2)  # b x kv x n
    w = torch.where(w.isnan(), torch.full_like(w, -math.inf), w)
    # classes: protected, others, none; within a class by weight, ties by place
    group = ((j < case["first"]) | (j >= length - case["recent"])).long() - 2 * (j >= length).long()
    order = w.sort(dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, group.expand_as(order).gather(-1, order).sort(dim=-1, descending=True, stable=True).indices)
    src = order[..., :budget].sort(-1).values  # b x kv x budget, in their order
    over = (s["seq_k"] > budget).nonzero()[:, 0]
    src, head = src[over], torch.arange(kv, device=DEV)[None, :, None]
    from_page, from_slot = page[over][:, None].expand(-1, kv, -1).gather(-1, src), src % case["page"]
    to_page, to_slot = page[over][:, None, :budget], slot[over][:, None, :budget]
    for cache in (s["k_cache"], s["v_cache"]):
        cache[to_page, to_slot, head] = cache[from_page, from_slot, head]
    s["weights"][to_page, head, to_slot] = s["weights"][from_page, head, from_slot]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weights": s["weights"], "lengths": s["seq_out"]}


# ------------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    global own
    keep, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    page = case["page"]
    cu, seq_k, table = s["cu"].tolist(), s["seq_k"].tolist(), s["table"].tolist()
    if case["op"] == "evict":
        k, v, weights, out = s["k_cache"].clone(), s["v_cache"].clone(), s["weights"].clone(), []
        for b, n in enumerate(seq_k):
            out.append(min(n, case["budget"]))
            if n <= case["budget"]:
                continue
            pg = torch.tensor(table[b], device=DEV)[torch.arange(n, device=DEV) // page].long()
            sl = torch.arange(n, device=DEV) % page
            mid = range(case["first"], n - case["recent"])
            for x in range(case["kv_heads"]):
                w = s["weights"][pg, x, sl].double().tolist()
                best = sorted(mid, key=lambda j: (-w[j], j))[:case["budget"] - case["first"] - case["recent"]]
                kept = list(range(case["first"])) + sorted(best) + list(range(n - case["recent"], n))
                at = torch.tensor(kept, device=DEV)
                m = len(kept)
                k[pg[:m], sl[:m], x] = s["k_cache"][pg[at], sl[at], x]
                v[pg[:m], sl[:m], x] = s["v_cache"][pg[at], sl[at], x]
                weights[pg[:m], x, sl[:m]] = s["weights"][pg[at], x, sl[at]]
        return {"k_cache": k.double(), "v_cache": v.double(), "weights": weights.double(), "lengths": None}
    if work(case)["flops"] > 4e12:
        return None
    h = case["heads"]
    if case["op"] == "latent_append":
        dl, dr = case["d_latent"], case["d_rope"]
        data, q = s["data"].double(), s["q"].double()
        for b, n in enumerate(seq_k):
            t = slice(cu[b], cu[b + 1])
            pos = torch.arange(n - (cu[b + 1] - cu[b]), n, device=DEV)
            turn = torch.exp(1j * pos.double()[:, None] * s["freq"])

            def spin(x, w):
                z = torch.complex(x[..., :dr // 2], x[..., dr // 2:]) if case["layout"] == "half" else torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous())
                z = z * w
                return torch.cat([z.real, z.imag], -1) if case["layout"] == "half" else torch.view_as_real(z).flatten(-2)

            c = s["c"][t].double()
            if s["weight"] is not None:
                c = c / ((c * c).sum(-1, keepdim=True) / dl + EPS).sqrt() * s["weight"].double()
            at = torch.tensor(table[b], device=DEV)[pos // page].long(), pos % page
            data[at] = torch.cat([c, spin(s["k_rope"][t].double(), turn)], -1)
            q[t, :, dl:] = spin(s["q_rope"][t].double(), turn[:, None])
        return {"q": q, "data": data}
    kv = case.get("kv_heads", 1)
    cache = s["data"][:, :, None] if "data" in s else s["k_cache"]
    o = torch.zeros(cu[-1], h, case.get("d_latent", 1), dtype=torch.float64, device=DEV)
    lse = torch.full((cu[-1], h), -math.inf, dtype=torch.float64, device=DEV)
    weights = s["weights"].double() if "weights" in s else None
    for b, n in enumerate(seq_k):
        j = torch.arange(n, device=DEV)
        pg, sl = torch.tensor(table[b], device=DEV)[j // page].long(), j % page
        past = n - (cu[b + 1] - cu[b])
        if weights is not None:
            weights[pg[past:], :, sl[past:]] = 0
        for x in range(kv):
            rows = cache[pg, sl, x].double()
            heads = slice(x * (h // kv), (x + 1) * (h // kv))
            for t0 in range(cu[b], cu[b + 1], 64):
                t1 = min(t0 + 64, cu[b + 1])
                y = s["q"][t0:t1, heads].double().flatten(0, 1) @ rows.T * s["scale"]
                at = (torch.arange(t0, t1, device=DEV) - cu[b] + past).repeat_interleave(h // kv)[:, None]
                hidden = torch.zeros_like(y, dtype=torch.bool)
                if case["mask"] != "none":
                    hidden |= j[None] > at
                if case["mask"] == "window":
                    hidden |= j[None] < at - case["window"]
                y[hidden] = -math.inf
                if weights is not None:
                    weights[pg, x, sl] += torch.exp(y - s["lse"][t0:t1, heads].double().flatten()[:, None]).sum(0)
                else:
                    z = torch.logsumexp(y, -1)
                    lse[t0:t1, heads] = z.reshape(t1 - t0, -1)
                    o[t0:t1, heads] = (torch.exp(y - z[:, None]) @ rows[:, :case["d_latent"]]).reshape(t1 - t0, h // kv, -1)
    return {"weights": weights} if weights is not None else {"o": o, "lse": lse}
