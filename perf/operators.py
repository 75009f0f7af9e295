"""The attention side of a decode layer, next to the library's projections and FFN: what its
operators compute, as a user calls them, with their plain forms.

  norm       sum = x + residual; y = sum * rsqrt(mean(sum^2) + eps) * weight, in bf16 or in E4M3
             with one scale per token and 128 columns
  append     rotary positions on q and k, then k and v quantised into a paged E4M3 cache with one
             power-of-two scale per page and head (a page's scale grows when a larger token comes)
  read       the same tokens read back from the cache as bf16
  attention  q over that cache, causal at the end of each sequence, with an optional sliding window
             and first tokens that stay visible

A cache is k_codes and v_codes [pages, kv_heads, page, head_dim] and k_scales and v_scales
[pages, kv_heads]; a batch is q_start [batch + 1] (which tokens belong to which sequence), kv_len
[batch] (each sequence's length, its new tokens included) and page_table [batch, pages of a
sequence].
"""
import math

import torch

own = False

DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn
EPS = 1e-6


# ------------------------------------------------------------------------------ cases

def _norm(name, rows, width, kind, residual):
    return dict(name=name, op="norm", rows=rows, width=width, kind=kind, residual=residual)


def _append(name, batch, new, kv_lo, kv_hi, heads, kv_heads, dim, page, rot, interleaved):
    return dict(name=name, op="append", batch=batch, new=new, kv_lo=kv_lo, kv_hi=kv_hi,
                heads=heads, kv_heads=kv_heads, dim=dim, page=page, rot=rot,
                interleaved=interleaved)


def _read(name, batch, kv_lo, kv_hi, kv_heads, dim, page):
    return dict(name=name, op="read", batch=batch, kv_lo=kv_lo, kv_hi=kv_hi, kv_heads=kv_heads,
                dim=dim, page=page)


def _attention(name, batch, new, kv_lo, kv_hi, heads, kv_heads, dim, page, window, sinks):
    return dict(name=name, op="attention", batch=batch, new=new, kv_lo=kv_lo, kv_hi=kv_hi,
                heads=heads, kv_heads=kv_heads, dim=dim, page=page, window=window, sinks=sinks)


def listed():
    return [
        # the norm before a projection or the FFN of one decoded token (H = 5120 layers)
        _norm("norm_token", 1, 5120, "bf16", True),
        # a prompt's rows (H = 5376 layers), normalised into 8 bits for an FP8 product
        _norm("norm_prompt_e4m3", 4096, 5376, "e4m3", True),
        # one decoded token of one conversation goes into the cache
        _append("append_token", 1, 1, 1000, 1000, 40, 8, 128, 64, 128, False),
        # a full serving batch, one token each; rotation of half of the head, pairs interleaved
        _append("append_batch", 64, 1, 200, 9000, 64, 8, 128, 32, 64, True),
        # prompts of unequal lengths, behind earlier turns that end inside a page
        _append("append_prompts", 5, 3001, 3001, 8111, 32, 16, 128, 64, 128, False),
        # short sequences handed to another consumer
        _read("read_short", 5, 37, 901, 8, 128, 16),
        # long contexts brought back to bf16
        _read("read_long", 2, 30011, 65500, 8, 128, 64),
        # one decoded token, a short conversation: latency
        _attention("attention_token", 1, 1, 1000, 1000, 40, 8, 128, 64, 0, 0),
        # a serving batch of unequal contexts, one token each: the cache's bytes
        _attention("attention_batch", 32, 1, 1001, 16003, 64, 8, 128, 64, 0, 0),
        # one token over a very long context: split along the cache
        _attention("attention_long", 1, 1, 131071, 131071, 64, 8, 128, 128, 0, 0),
        # drafts of 4 tokens verified in a layer with a sliding window and visible first tokens
        _attention("attention_window", 16, 4, 700, 20000, 32, 16, 128, 32, 1024, 4),
        # the last 64 rows of a prompt over what came before: the products' rate
        _attention("attention_chunk", 1, 64, 32805, 32805, 64, 8, 128, 64, 0, 0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(rng):
    op = rng.choice(("norm", "append", "append", "read", "attention", "attention", "attention"))
    if op == "norm":
        return _norm("", _log(rng, 1, 4096), 16 * _log(rng, 16, 1344), rng.choice(("bf16", "e4m3")),
                     rng.random() < 0.7)
    dim = rng.choice((64, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8, 16))
    page = rng.choice((16, 32, 64, 128))
    batch = _log(rng, 1, 64)
    if op == "read":
        hi = _log(rng, 1, 65500)
        return _read("", batch, _log(rng, 1, hi), hi, kv_heads, dim, page)
    heads = kv_heads * rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 16))
    if op == "append":
        new = _log(rng, 1, 3001)
        hi = _log(rng, new, 40000)
        return _append("", batch, new, _log(rng, new, hi), hi, heads, kv_heads, dim, page,
                       rng.choice((0, dim // 2, dim)), rng.random() < 0.5)
    new = rng.choice((1, 1, _log(rng, 2, 64)))
    hi = _log(rng, max(new, 20), 131071)
    window = rng.choice((0, 0, _log(rng, 16, 4096)))
    return _attention("", batch, new, _log(rng, new, hi), hi, heads, kv_heads, dim, page, window,
                      rng.choice((0, 1, 4, 37)) if window else 0)


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        case = _drawn(rng)
        del case["name"]
        if _cost(case) > most:
            continue
        if case["op"] != "norm":  # the plain forms pad every sequence to the longest
            padded = case["batch"] * case["kv_hi"] * case["kv_heads"] * case["dim"]
            scores = (case["batch"] * case["new"] * case["heads"] * case["kv_hi"]
                      if case["op"] == "attention" else 0)
            if max(padded, scores) > 1 << 29:
                continue
        return case


def _kv_lens(case):
    """The sequences' lengths: spread evenly over the logarithm from kv_lo to kv_hi."""
    n, lo, hi = case["batch"], case["kv_lo"], case["kv_hi"]
    return [int(round(lo * (hi / lo) ** (b / max(1, n - 1)))) for b in range(n)]


def _q_lens(case):
    """Each sequence's new tokens: from 1 to `new`, the first has `new`."""
    if case["op"] == "read":
        return _kv_lens(case)
    new = case["new"]
    return [new - (b * 5) % new for b in range(case["batch"])]


def _visible(case, kv, q):
    """(query-key pairs, distinct keys) that one sequence's new tokens see."""
    w, s = case["window"], case["sinks"]
    first = kv - q
    pairs = 0
    for p in range(first, kv):
        n = p + 1
        pairs += n if not w else min(n, w) + max(0, min(s, n - w))
    keys = kv if not w else kv - max(0, first + 1 - w) + max(0, min(s, first + 1 - w))
    return pairs, keys


def work(case):
    if case["op"] == "norm":
        n, groups = case["rows"] * case["width"], case["rows"] * (-(-case["width"] // 128))
        out = 2 * n if case["kind"] == "bf16" else n + 4 * groups
        return {"bytes": n * (6 if case["residual"] else 2) + out + 2 * case["width"],
                "flops": 6 * n}
    kv, q = _kv_lens(case), _q_lens(case)
    t, row = sum(q), case["kv_heads"] * case["dim"]
    pages = sum(-(-k // case["page"]) - (k - n) // case["page"] for k, n in zip(kv, q))
    tables = 4 * (2 * case["batch"] + 1) + 4 * pages
    if case["op"] == "read":
        return {"bytes": 6 * t * row + 8 * pages * case["kv_heads"] + tables, "flops": 2 * t * row}
    if case["op"] == "append":
        turn = case["heads"] * case["dim"]
        return {"bytes": 6 * t * row + 4 * t * turn + 4 * t * case["rot"] + tables
                + 8 * pages * case["kv_heads"],
                "flops": t * (3 * case["rot"] * (case["heads"] + case["kv_heads"]) + 4 * row)}
    pairs = keys = 0
    for k, n in zip(kv, q):
        a, b = _visible(case, k, n)
        pairs, keys = pairs + a, keys + b
    seen = -(-keys // case["page"])
    return {"bytes": 2 * keys * row + 8 * seen * case["kv_heads"] + 4 * seen
            + 4 * t * case["heads"] * case["dim"] + 4 * t * case["heads"]
            + 4 * (2 * case["batch"] + 1),
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ------------------------------------------------------------------------------ inputs

def _codes(gen, shape):
    """E4M3 bytes of a page's tokens: normal values that reach the top of the range."""
    return (torch.randn(shape, generator=gen, device=DEV) * 100).clamp(-448, 448).to(E4M3).view(
        torch.uint8)


def _rotation(positions, rot, factor=4.0, base=500000.0):
    """cos and sin [positions, rot / 2, 2]: frequencies slowed by `factor` for a longer context."""
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    angle = (torch.arange(positions, device=DEV, dtype=torch.float64)[:, None]
             * (base ** (-2 * i / rot) / factor))
    return torch.stack((angle.cos(), angle.sin()), -1).float().contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "norm":
        shape = (case["rows"], case["width"])
        s["x"] = torch.randn(shape, generator=gen, device=DEV).bfloat16()
        s["residual"] = ((torch.randn(shape, generator=gen, device=DEV) * 3).bfloat16()
                         if case["residual"] else None)
        s["weight"] = (1 + 0.2 * torch.randn(case["width"], generator=gen, device=DEV)).bfloat16()
        s["sum"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["out"] = torch.empty_like(s["x"])
        s["codes"] = torch.empty(shape, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty((shape[0], -(-shape[1] // 128)), device=DEV)
        return s
    kv, q = _kv_lens(case), _q_lens(case)
    batch, page, dim, kv_heads = case["batch"], case["page"], case["dim"], case["kv_heads"]
    need = [-(-k // page) for k in kv]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).int()
    host = [sum(need[:b]) for b in range(batch)]
    at = (torch.tensor(host, device=DEV)[:, None] + torch.arange(max(need), device=DEV)[None])
    s["page_table"] = order[at.clamp(max=pages - 1)].contiguous()
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    s["q_start"] = torch.tensor([sum(q[:b]) for b in range(batch + 1)], dtype=torch.int32,
                                device=DEV)
    s["max_kv"], s["max_q"], t = max(kv), max(q), sum(q)
    for name in ("k", "v"):
        s[name + "_codes"] = _codes(gen, (pages, kv_heads, page, dim))
        s[name + "_scales"] = torch.exp2(torch.randint(-8, -4, (pages, kv_heads), generator=gen,
                                                       device=DEV).float())
    # the sequence of each new token, and its place in it
    s["owner"] = torch.repeat_interleave(torch.arange(batch, device=DEV),
                                         torch.tensor(q, device=DEV))
    s["place"] = torch.arange(t, device=DEV) - s["q_start"].long()[s["owner"]]
    if case["op"] == "read":
        s["k_out"] = torch.empty((t, kv_heads, dim), dtype=torch.bfloat16, device=DEV)
        s["v_out"] = torch.empty_like(s["k_out"])
    else:
        # one row of the fused projection of a token: its query, key and value heads
        heads = case["heads"]
        row = torch.randn((t, heads + 2 * kv_heads, dim), generator=gen, device=DEV)
        row = (row * torch.exp(0.3 * torch.randn((t, 1, 1), generator=gen, device=DEV))).bfloat16()
        s["q"], s["k"], s["v"] = row.split((heads, kv_heads, kv_heads), 1)
        s["out"] = torch.empty((t, heads, dim), dtype=torch.bfloat16, device=DEV)
    if case["op"] == "append":
        s["rope"] = _rotation(max(kv), case["rot"]) if case["rot"] else None
        # the pages that the new tokens touch
        first = [(k - n) // page for k, n in zip(kv, q)]
        touched = torch.cat([s["page_table"][b, first[b]:need[b]] for b in range(batch)])
        s["touched"] = touched.long()
    if case["op"] == "attention":
        s["lse"] = torch.empty((t, case["heads"]), device=DEV)
        s["softmax_scale"] = 2.0 / math.sqrt(dim)
    if own:
        from nvfp4_weight_only_gb300 import ffi
        s["cache"] = ffi.Kv8Cache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
        s["batch_of"] = ffi.Kv8Batch(s["q_start"], s["kv_len"], s["page_table"])
        if case["op"] == "attention":
            s["ws"] = ffi.workspace(ffi.kv8_attention_workspace_bytes(
                s["cache"], s["batch_of"], t, case["heads"]), DEV)
    return s


# ------------------------------------------------------------------------------ one pass

def run(s):
    return {"norm": _run_norm, "append": _run_append, "read": _run_read,
            "attention": _run_attention}[s["op"]](s)


def _run_norm(s):
    if own:
        from nvfp4_weight_only_gb300 import ffi
        if s["kind"] == "bf16":
            ffi.add_rmsnorm_bf16(s["x"], s["weight"], EPS, residual=s["residual"],
                                 sum_out=s["sum"], out=s["out"])
            return {"sum": s["sum"], "out": s["out"]}
        ffi.add_rmsnorm_e4m3(s["x"], s["weight"], EPS, residual=s["residual"], sum_out=s["sum"],
                             codes=s["codes"], scales=s["scales"])
        return {"sum": s["sum"], "codes": s["codes"].view(E4M3), "scales": s["scales"]}
    total = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
    y = total * torch.rsqrt((total * total).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    summed = None if s["residual"] is None else total.bfloat16()
    if s["kind"] == "bf16":
        return {"sum": summed, "out": y.bfloat16()}
    rows, width = y.shape
    groups = -(-width // 128)
    y = torch.nn.functional.pad(y, (0, groups * 128 - width)).view(rows, groups, 128)
    amax = y.abs().amax(-1)
    scales = torch.where(amax == 0, 1.0, (amax / 448).clamp(min=2.0 ** -126))
    codes = (y / scales[..., None]).clamp(-448, 448).to(E4M3)
    codes = codes.view(rows, groups * 128)[:, :width].contiguous()
    return {"sum": summed, "codes": codes, "scales": scales}


def _turned(x, rope, positions, interleaved):
    """Rotary positions on the first 2 * rope.shape[1] values of each head, in 32 bits."""
    x = x.float()
    half = rope.shape[1]
    cos, sin = rope[positions][:, None].unbind(-1)
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = head[..., :half], head[..., half:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1)


def _power_scale(amax):
    """The smallest 2^e with amax <= 448 * 2^e, e in -60..119."""
    m, e = torch.frexp(amax.clamp(min=2.0 ** -60))
    e = (e - 9 + (m > 0.875)).clamp(-60, 119)
    return ((e + 127) << 23).int().view(torch.float32)


def _store(s, x, codes, scales, pages, rows):
    """Quantises the new tokens x [tokens, kv_heads, dim] into their pages."""
    size, touched = codes.shape[2], s["touched"]
    amax = torch.zeros_like(scales).scatter_reduce_(
        0, pages[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")[touched]
    old_rows = torch.full((scales.shape[0],), size, device=x.device).scatter_reduce_(
        0, pages, rows, "amin")[touched]
    before = scales[touched]
    after = _power_scale(amax)
    after = torch.where((old_rows > 0)[:, None], torch.maximum(after, before), after)
    was = codes[touched]
    moved = was.view(E4M3).float() * (before / after)[..., None, None]
    moved = moved.clamp(-448, 448).to(E4M3).view(torch.uint8)
    kept = torch.arange(size, device=x.device) < old_rows[:, None]
    codes[touched] = torch.where(kept[:, None, :, None], moved, was)
    scales[touched] = after
    scaled = x / scales[pages][..., None]
    codes[pages, :, rows] = scaled.clamp(-448, 448).to(E4M3).view(torch.uint8)


def _run_append(s):
    if own:
        from nvfp4_weight_only_gb300 import ffi
        ffi.kv8_append(s["cache"], s["batch_of"], s["k"], s["v"], q=s["q"], q_out=s["out"],
                       rope=s["rope"], interleaved=s["interleaved"])
        q = s["out"]
    else:
        positions, pages, rows = _places(s)
        q, k = s["q"].float(), s["k"].float()
        if s["rope"] is not None:
            q = _turned(q, s["rope"], positions, s["interleaved"])
            k = _turned(k, s["rope"], positions, s["interleaved"])
        q = q.bfloat16()
        _store(s, k, s["k_codes"], s["k_scales"], pages, rows)
        _store(s, s["v"].float(), s["v_codes"], s["v_scales"], pages, rows)
    return {"q": q, "k_codes": s["k_codes"].view(E4M3), "v_codes": s["v_codes"].view(E4M3),
            "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _places(s):
    """Position, page and row of each new token."""
    lens = s["q_start"].long().diff()
    positions = (s["kv_len"].long() - lens)[s["owner"]] + s["place"]
    pages = s["page_table"].long()[s["owner"], positions // s["page"]]
    return positions, pages, positions % s["page"]


def _run_read(s):
    if own:
        from nvfp4_weight_only_gb300 import ffi
        ffi.kv8_read(s["cache"], s["batch_of"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    _, pages, rows = _places(s)
    k = s["k_codes"][pages, :, rows].view(E4M3).float() * s["k_scales"][pages][..., None]
    v = s["v_codes"][pages, :, rows].view(E4M3).float() * s["v_scales"][pages][..., None]
    return {"k": k.bfloat16(), "v": v.bfloat16()}


def _run_attention(s):
    if own:
        from nvfp4_weight_only_gb300 import ffi
        ffi.kv8_attention(s["q"], s["cache"], s["batch_of"], s["softmax_scale"],
                          window=s["window"], sinks=s["sinks"], ws=s["ws"], out=s["out"],
                          lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    batch, kv_heads, dim = s["batch"], s["kv_heads"], s["dim"]
    at = torch.arange(s["max_kv"], device=s["q"].device)
    pages, rows = s["page_table"].long()[:, at // s["page"]], at % s["page"]

    def padded(codes, scales):  # [batch, kv_heads, keys, dim]
        x = codes.transpose(1, 2)[pages, rows].view(E4M3).float() * scales[pages][..., None]
        return x.transpose(1, 2)

    q = torch.zeros((batch, s["max_q"], s["heads"], dim), device=s["q"].device)
    q[s["owner"], s["place"]] = s["q"].float()
    q = q.view(batch, s["max_q"], kv_heads, -1, dim).permute(0, 2, 1, 3, 4).flatten(2, 3)
    scores = q @ padded(s["k_codes"], s["k_scales"]).transpose(2, 3) * s["softmax_scale"]
    lens = s["q_start"].long().diff()
    p = (s["kv_len"].long() - lens)[:, None] + torch.arange(s["max_q"], device=q.device)
    seen = at <= p[..., None]
    if s["window"]:
        seen &= (at > p[..., None] - s["window"]) | (at < s["sinks"])
    group = s["heads"] // kv_heads
    scores.masked_fill_(~seen.repeat_interleave(group, 1)[:, None], -torch.inf)
    top = scores.amax(-1, keepdim=True)
    weights = torch.exp(scores - top)
    total = weights.sum(-1, keepdim=True)
    out = weights @ padded(s["v_codes"], s["v_scales"]) / total
    lse = top + torch.log(total)

    def ragged(x):  # [batch, kv_heads, max_q * group, n] -> [tokens, heads, n]
        x = x.view(batch, kv_heads, s["max_q"], group, -1).permute(0, 2, 1, 3, 4).flatten(2, 3)
        return x[s["owner"], s["place"]]

    return {"out": ragged(out).bfloat16(), "lse": ragged(lse).squeeze(-1)}


# ------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "read": _exact_read,
            "attention": _exact_attention}[s["op"]](s)


def _exact_norm(s):
    r = s["x"].double()
    if s["residual"] is not None:
        r = r + s["residual"].double()
    y = r / (r.pow(2).sum(1) / r.shape[1] + EPS).sqrt()[:, None] * s["weight"].double()
    summed = None if s["residual"] is None else r
    if s["kind"] == "bf16":
        return {"sum": summed, "out": y}
    codes, scales = [], []
    for g in range(0, y.shape[1], 128):
        part = y[:, g:g + 128]
        top = part.abs().max(1).values / 448
        top = torch.where(top == 0, torch.ones_like(top), top)
        codes.append(_round_e4m3(part / top[:, None]))
        scales.append(top)
    return {"sum": summed, "codes": torch.cat(codes, 1), "scales": torch.stack(scales, 1)}


def _two_to(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(x):
    """The nearest E4M3 value (ties to even), saturated, from 64 bits."""
    x = x.clamp(-448, 448)
    step = _two_to(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 4)
    return torch.round(x / step) * step


def _exact_append(s):
    size, half = s["page"], s["rot"] // 2
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    new = {n: (s[n + "_codes"].view(E4M3).double(), s[n + "_scales"].double()) for n in "kv"}
    for b, n in enumerate(lens):
        t0, t1 = starts[b], starts[b + 1]
        first = n - (t1 - t0)
        if half:
            c, d = s["rope"][first:n].double().unbind(-1)
            i = torch.arange(half, device=c.device)
            i0, i1 = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
            for x in (q, k):
                a, e = x[t0:t1, :, i0], x[t0:t1, :, i1]
                x[t0:t1, :, i0] = a * c[:, None] - e * d[:, None]
                x[t0:t1, :, i1] = e * c[:, None] + a * d[:, None]
        row = s["page_table"][b].tolist()
        for j in range(first // size, -(-n // size)):
            lo, hi = max(first, j * size), min(n, (j + 1) * size)
            for name, x in (("k", k), ("v", v)):
                codes, scales = new[name]
                part = x[t0 + lo - first:t0 + hi - first].transpose(0, 1)
                top = part.abs().amax((1, 2))
                part_of_one, e = torch.frexp(top.clamp(min=2.0 ** -60) / 448)
                scale = _two_to((e - (part_of_one == 0.5).int()).clamp(-60, 119))
                if lo > j * size:
                    scale = torch.maximum(scale, scales[row[j]])
                    r = slice(0, lo - j * size)
                    old = codes[row[j], :, r] * (scales[row[j]] / scale)[:, None, None]
                    codes[row[j], :, r] = _round_e4m3(old)
                codes[row[j], :, lo - j * size:hi - j * size] = _round_e4m3(
                    part / scale[:, None, None])
                scales[row[j]] = scale
    return {"q": q, "k_codes": new["k"][0], "v_codes": new["v"][0], "k_scales": new["k"][1],
            "v_scales": new["v"][1]}


def _sequence(s, name, b, n):
    """The first n tokens [kv_heads, n, dim] of sequence b in 64 bits."""
    rows = s["page_table"][b, :-(-n // s["page"])].long()
    x = s[name + "_codes"][rows].view(E4M3).double() * s[name + "_scales"][rows].double()[
        ..., None, None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_read(s):
    out = {n: [_sequence(s, n, b, m).transpose(0, 1) for b, m in enumerate(s["kv_len"].tolist())]
           for n in "kv"}
    return {n: torch.cat(x) for n, x in out.items()}


def _exact_attention(s):
    starts, outs, lses = s["q_start"].tolist(), [], []
    for b, n in enumerate(s["kv_len"].tolist()):
        q = s["q"][starts[b]:starts[b + 1]].double()
        new = q.shape[0]
        keys, values = _sequence(s, "k", b, n), _sequence(s, "v", b, n)
        at = torch.arange(n, device=q.device)
        p = torch.arange(n - new, n, device=q.device)[:, None]
        hidden = at > p
        if s["window"]:
            hidden = hidden | ((at <= p - s["window"]) & (at >= s["sinks"]))
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64,
                                                    device=q.device)
        group = s["heads"] // s["kv_heads"]
        for h in range(s["heads"]):
            x = (q[:, h] @ keys[h // group].T) * s["softmax_scale"]
            x = x.masked_fill(hidden, -math.inf)
            lse[:, h] = torch.logsumexp(x, 1)
            out[:, h] = torch.exp(x - lse[:, h:h + 1]) @ values[h // group]
        outs.append(out)
        lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
