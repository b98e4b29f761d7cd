"""MXFP4 and attention from their definitions, in binary64 (torch, any device)."""
from __future__ import annotations

import math

import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
MIDS = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)


def pow2(e):
    """2^e in binary64 for whole e in -1022..1023, from its bits: torch.pow on
    the GPU is off by an ulp for some."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def encode(x):
    """[..., 32 b] -> (element codes uint8 [..., 32 b], scale codes uint8 [..., b]).

    The block's scale is 2^(floor(log2 max) - 2), not below 2^-127; an element
    is the nearest grid value, the one with the even code at a midpoint."""
    b = x.double().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    exp = torch.frexp(torch.where(bad, 0.0, amax)).exponent.to(torch.int64) - 1  # floor(log2) for amax > 0
    e = torch.where(amax > 0, exp - 2 + 127, 0).clamp(min=0)
    y = b.abs() * pow2(127 - e).unsqueeze(-1)
    y = torch.where(bad.unsqueeze(-1), 0.0, y)
    mids = MIDS.to(x.device)
    up = torch.bucketize(y, mids, right=False)   # midpoints below y
    at = torch.bucketize(y, mids, right=True)    # midpoints up to y
    code = torch.where(up == at, up, up + (up & 1))  # on a midpoint: the even one of up, up + 1
    code = code + 8 * torch.signbit(b)
    code = torch.where(bad.unsqueeze(-1), 0, code)
    return code.to(torch.uint8).flatten(-2), torch.where(bad, 255, e).to(torch.uint8)


def decode(code, scale):
    """Element codes and scale codes -> float64 values (NaN under scale 255)."""
    c = code.long()
    v = GRID.to(code.device)[c & 7] * torch.where(c >= 8, -1.0, 1.0)
    s = pow2(scale.long() - 127)
    s = torch.where(scale == 255, math.nan, s)
    return (v.unflatten(-1, (-1, 32)) * s.unsqueeze(-1)).flatten(-2)


def pad_cols(x):
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % 128))


def values(x):
    """What MXFP4 holds of the rows of x, float64."""
    cols = x.shape[-1]
    return decode(*encode(torch.nn.functional.pad(x.double(), (0, -cols % 32))))[..., :cols]


def unpack(q):
    return torch.stack((q & 15, q >> 4), -1).flatten(-2)


def tile_scales(scales, rows, cols):
    """Tiled scale bytes of a [rows, cols] matrix -> [rows, padded cols / 32]."""
    groups = -(-cols // 128)
    panels = -(-rows // 128)
    t = scales[:panels * groups * 512].reshape(panels, groups, 32, 4, 4)  # row % 32, row / 32, column
    return t.permute(0, 3, 2, 1, 4).reshape(panels * 128, groups * 4)[:rows]


def attention(q, k, v, table, lens, q_starts, page, scale, causal=True, window=0, sinks=0):
    """q [total, hq, d] float64; k, v [pages, hkv, page, d] float64 (the cache's
    values).  Returns (out, lse, sum of p |v|), computed key by key so that what a
    query does not see never enters."""
    total, hq, d = q.shape
    hkv = k.shape[1]
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((total, hq), -math.inf, dtype=torch.float64, device=q.device)
    for b, length in enumerate(lens):
        q0, n = q_starts[b], q_starts[b + 1] - q_starts[b]
        if n == 0 or length <= 0:
            continue
        pages = table[b, :-(-length // page)].long()
        kk = k[pages].transpose(1, 2).flatten(0, 1)[:length]
        vv = v[pages].transpose(1, 2).flatten(0, 1)[:length]
        p = torch.arange(length - n, length, device=q.device).unsqueeze(1)
        j = torch.arange(length, device=q.device)
        seen = (j <= p) if causal else torch.ones_like(j <= p)
        if window:
            seen = seen & ((j > p - window) | (j < sinks))
        for h in range(hq):
            s = q[q0:q0 + n, h] @ kk[:, h // (hq // hkv)].T * scale
            s = torch.where(seen, s, -math.inf)
            top = s.amax(1, keepdim=True)
            w = torch.where(seen, torch.exp(s - torch.where(top == -math.inf, 0.0, top)), 0.0)
            tot = w.sum(1, keepdim=True)
            vh = vv[:, h // (hq // hkv)]
            # 0 * NaN of an unseen key must not enter: products with zero weights are left out
            bad = ~torch.isfinite(vh)
            num = w @ torch.where(bad, 0.0, vh)
            num = torch.where((w > 0).double() @ bad.double() > 0, math.nan, num)
            live = (tot > 0) | torch.isnan(tot)
            out[q0:q0 + n, h] = torch.where(live, num / tot, 0.0)
            mag[q0:q0 + n, h] = torch.where(live, (w @ torch.where(bad, 0.0, vh).abs()) / tot, 0.0)
            lse[q0:q0 + n, h] = torch.where(live, top + torch.log(tot), -math.inf)[:, 0]
    return out, lse, mag
