"""Plain 64-bit statements of the attention-side operators, for the tests: norm, rotation,
quantisation into pages of E4M3, and attention over them.  CPU tensors, loops where they are
clearest, nothing shared with the library."""
import math

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


def e4m3_value(codes):
    return codes.view(E4M3).to(torch.float32).double()


def round_e4m3(x):
    """E4M3 bytes of fp64 values: nearest, ties to even, saturated, NaN kept (own arithmetic)."""
    x = x.double()
    a = x.abs().clamp(max=448.0).numpy()
    step = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    r = np.rint(a / step) * step
    r = torch.from_numpy(np.asarray(r))
    # every value is now on the grid, so the conversion below is exact
    codes = r.float().to(E4M3).view(torch.uint8)
    codes = codes | torch.signbit(x).to(torch.uint8) * 128
    return torch.where(torch.isnan(x), codes | 127, codes)


def rounds_to(out, want, e):
    """Where a bf16 `out` is the rounding of some fp32 value within e of `want` (fp64): rounding is
    monotone, so between the roundings of both ends."""
    out = out.cpu().double()
    lo, hi = (want - e).float().bfloat16().double(), (want + e).float().bfloat16().double()
    return (out >= lo) & (out <= hi)


def norm(x, residual, weight, eps, weight_bias=0.0):
    """(r, y) in fp64."""
    r = x.double() if residual is None else x.double() + residual.double()
    y = r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * (weight.double() + weight_bias)
    return r, y


def rope_frequencies(rot, base, scaling=0, factor=1.0, context=1.0, slow=1.0, fast=32.0):
    f = []
    for i in range(rot // 2):
        if scaling == 2:
            b = base * factor ** (rot / (rot - 2))
            f.append(b ** (-2 * i / rot))
            continue
        x = base ** (-2 * i / rot)
        if scaling == 1:
            x /= factor
        if scaling == 3:
            turns = context * x / (2 * math.pi)
            g = min(max((turns - slow) / (fast - slow), 0.0), 1.0)
            x = x * g + x * (1 - g) / factor
        f.append(x)
    return f


def rotate(x, table, positions, interleaved):
    """x [tokens, heads, dim] -> fp64, turned by table [positions, rot/2, 2]."""
    x = x.double().clone()
    half = table.shape[1]
    for t, p in enumerate(positions):
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = float(table[p, i, 0]), float(table[p, i, 1])
            u, w = x[t, :, a].clone(), x[t, :, b].clone()
            x[t, :, a] = u * c - w * s
            x[t, :, b] = w * c + u * s
    return x


def power_scale(amax):
    """The smallest 2^e >= amax / 448, e in -60..119."""
    if amax == 0:
        return 2.0 ** -60
    if math.isinf(amax):
        return 2.0 ** 119
    m, e = math.frexp(amax / 448.0)  # m in [0.5, 1)
    return 2.0 ** min(max(e - 1 if m == 0.5 else e, -60), 119)


def append(codes, scales, page, x, q_lens, kv_lens, table):
    """Quantises x [tokens, kv_heads, dim] (fp64) into codes [pages, kv_heads, page, dim] and
    scales [pages, kv_heads], in place."""
    t0 = 0
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        first = kv - n
        for j in range(first // page, -(-kv // page)):
            lo, hi = max(first, j * page), min(kv, (j + 1) * page)
            if lo >= hi:
                continue
            p = int(table[b, j])
            for h in range(x.shape[1]):
                part = x[t0 + lo - first:t0 + hi - first, h]
                known = part[~torch.isnan(part)].abs()
                scale = power_scale(float(known.max()) if known.numel() else 0.0)
                old = lo - j * page
                if old > 0:
                    before = float(scales[p, h])
                    scale = max(scale, before)
                    if scale != before:
                        codes[p, h, :old] = round_e4m3(e4m3_value(codes[p, h, :old])
                                                       * (before / scale))
                scales[p, h] = scale
                codes[p, h, old:old + hi - lo] = round_e4m3(part / scale)
        t0 += n


def dequantise(codes, scales):
    return e4m3_value(codes) * scales.double()[..., None, None]


def sequence(values, page, table_row, n):
    """The first n tokens [n, kv_heads, dim] of dequantised pages."""
    rows = [values[int(table_row[j // page]), :, j % page] for j in range(n)]
    return torch.stack(rows) if rows else values.new_zeros((0,) + values[0, :, 0].shape)


def attention(q, k_values, v_values, page, table, q_lens, kv_lens, scale, window=0, sinks=0):
    """(out, lse, weight, reach) in fp64: weight = sum_j softmax_j |v_j| and reach = the largest
    sum of |q_d k_d| * scale over the visible keys, which the error bounds are made of."""
    T, heads, dim = q.shape
    kv_heads = k_values.shape[1]
    group = heads // kv_heads
    out = torch.zeros((T, heads, dim), dtype=torch.float64)
    weight = torch.zeros_like(out)
    lse = torch.full((T, heads), -math.inf, dtype=torch.float64)
    reach = torch.zeros((T, heads), dtype=torch.float64)
    t = 0
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        if n == 0:
            continue
        keys = sequence(k_values, page, table[b], kv)
        values = sequence(v_values, page, table[b], kv)
        for i in range(n):
            p = kv - n + i
            at = torch.arange(kv)
            seen = at <= p
            if window:
                seen &= (at > p - window) | (at < sinks)
            js = seen.nonzero().flatten()
            if js.numel():
                for h in range(heads):
                    x = q[t, h].double()
                    k, v = keys[js, h // group], values[js, h // group]
                    s = (k * x).sum(1) * scale
                    lse[t, h] = torch.logsumexp(s, 0)
                    w = torch.exp(s - lse[t, h])
                    out[t, h] = w @ v
                    weight[t, h] = w @ v.abs()
                    reach[t, h] = ((k * x).abs().sum(1) * abs(scale)).max()
            t += 1
    return out, lse, weight, reach
