"""The operators on 4-bit activations in 64 bits, from their definitions: what the tests of the
w4a4 and experts calls compare with.  Works on the device of its inputs."""
import math

import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# magnitudes from 0 to 448, bytes 0x00..0x7e
E4M3 = tuple((b & 7) * 2.0 ** -9 if b < 8 else (1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 7)
             for b in range(0x7f))


def nearest(v, values):
    """Index of the nearest of ascending `values` to each v >= 0; ties to the even index, beyond
    the largest the largest."""
    t = torch.tensor(values, dtype=torch.float64, device=v.device)
    up = torch.searchsorted(t, v.contiguous()).clamp(max=len(values) - 1)
    down = (up - 1).clamp(min=0)
    far_up, far_down = t[up] - v, v - t[down]
    take_up = (far_up < far_down) | ((far_up == far_down) & (up % 2 == 0))
    return torch.where(take_up, up, down)


def power(e):
    """2^e from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def quantize(x):
    """x [M, K] (bf16 values) -> (codes as values, E4M3 scales as values [M, K/16], r [M]), with
    r NaN for rows that are not finite."""
    v = x.double()
    fine = torch.isfinite(v).all(1)
    v = torch.where(fine[:, None], v, torch.zeros_like(v))
    top = v.abs().amax(1)
    _, e = torch.frexp(top)
    e = torch.where(top > 2688 * power(e - 12), e - 11, e - 12)
    r = torch.where(top > 0, power(e.clamp(-100, 117)), torch.ones_like(top))
    blocks = (v / r[:, None]).view(v.shape[0], -1, 16)
    # a quotient by 6 that is a tie would not survive a product with 1/6
    six = torch.full((), 6.0, dtype=torch.float64, device=x.device)
    code = nearest(blocks.abs().amax(2) / six, E4M3)
    s = torch.tensor(E4M3, dtype=torch.float64, device=x.device)[code]
    q = torch.where(s[..., None] > 0, blocks / s.clamp(min=2.0 ** -9)[..., None], 0.0)
    c = torch.tensor(E2M1, dtype=torch.float64, device=x.device)[nearest(q.abs(), E2M1)]
    c = (c * torch.sign(q)).view(v.shape)
    return c, s, torch.where(fine, r, torch.full_like(r, math.nan))


def values(x):
    """The values that quantised rows stand for, in 64 bits."""
    c, s, r = quantize(x)
    return c * s.repeat_interleave(16, 1) * r[:, None]


def weight(codes, scales, scale2):
    """NVFP4 codes [N, K/2] and scales [N, K/16] in 64 bits."""
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    s = torch.tensor(E4M3, dtype=torch.float64, device=codes.device)[scales.long()]
    return table[nib] * s.repeat_interleave(16, 1) * scale2


def act(kind, g):
    """0: SiLU, 1: GeLU (tanh form)."""
    y = g if kind == 0 else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    return g * torch.sigmoid(y)


def product(x, w):
    """(x values [M, K] times w [N, K], how far fp32 sums may be off): K products, each sum off by
    half a step of what has been added up so far, 2^-24 of it."""
    return x @ w.T, x.shape[1] * 2.0 ** -24 * (x.abs() @ w.abs().T)


def order(ids, experts):
    """(start, source, place) of a routed batch, by Python's own lists."""
    T, k = ids.shape
    rows = [[] for _ in range(experts)]
    for t, row in enumerate(ids.tolist()):
        for j, e in enumerate(row):
            if 0 <= e < experts:
                rows[e].append((t, j))
    start, source = [0], []
    place = torch.full((T, k), -1, dtype=torch.int32)
    for mine in rows:
        for t, j in mine:
            place[t, j] = len(source)
            source.append(t)
        start.append(len(source))
    source += [-1] * (T * k - len(source))
    return (torch.tensor(start, dtype=torch.int32), torch.tensor(source, dtype=torch.int32), place)
