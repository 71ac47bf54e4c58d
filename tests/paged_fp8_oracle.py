"""64-bit references of the quantised paged cache, written from its definitions in include/ffpa.h, with
the error bounds the GPU tests use."""
from __future__ import annotations

import math

import torch

from tests import paged_oracle as po

E4M3 = torch.float8_e4m3fn


def nearest_e4m3(y):
    """The e4m3 value nearest to each of y (64 bits; ties to even; at most 448 in size)."""
    _, e = torch.frexp(y)                                       # |y| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(y), e.clamp(min=-5) - 4)  # 2^-9 below 2^-6
    return (torch.round(y / step) * step).clamp(-448, 448)


def quantise(y):
    """(codes, scales) of rows [..., D] by the definition, in 64 bits."""
    top = y.double().abs().amax(-1)
    scale = torch.where(top == 0, torch.ones_like(top), top / 448)
    return nearest_e4m3(y.double() / scale[..., None]), scale


def make_cache(g, lens, Hkv, D, page, spare=3, layout="psh", spread=0.0):
    """As paged_oracle.make_cache: codes, scales [pages, Hkv, page], table, lengths (CPU).  Rows that no request
    owns hold NaN codes and NaN scales.  spread: scales vary by 2 ** (+- spread) from row to row."""
    k16, v16, table, n = po.make_cache(g, lens, Hkv, D, page, torch.float32, spare, layout)
    out = []
    for x in (k16, v16):
        codes, scale = quantise(torch.nan_to_num(x))
        codes = codes.float().to(E4M3)
        scale = scale.float()
        if spread:
            scale = scale * torch.exp2(spread * (2 * torch.rand(scale.shape, generator=g) - 1))
        unused = torch.isnan(x[..., 0])
        scale = scale.masked_fill(unused, math.nan)
        codes.view(torch.uint8)[unused] = 0x7f
        if layout == "phs":                                     # as the 16-bit caches: heads outside the slots
            codes = codes.transpose(1, 2).contiguous().transpose(1, 2)
        out += [codes, scale.transpose(1, 2).contiguous()]
    kc, ks, vc, vs = out
    return kc, vc, ks, vs, table, n


def widened(codes, scale):
    """The values that a cache stands for, 64 bits."""
    return codes.to(torch.float32).double() * scale.transpose(1, 2).double()[..., None]


def decode(q, kc, vc, ks, vs, table, lens, scale=None):
    """(o, lse, bound on |o's error|, bound on |lse's error|) in 64 bits.

    o is rounded once (u |o|).  A weight times its value's scale enters the sum as two fp16 values, off by
    2^-21 of it, or (bf16) as one, off by half a step of fp16, 2^-11; and below the normal range by half
    of 2^-24, which is 2^-40 of the largest such product (2^15), times the code (at most 448).  A score is a sum of
    at most 64 steps of 16 products, each step off by 2^-23 of partial sums below `size` (the sum of
    the products' sizes, here at most a few times 8): 2^-17 of `size`; the units and scales it is
    multiplied by add 2^-21 of it, and bf16 queries' small columns less.  Exponentials and the other fp32
    steps are off by less than 2^-18 of the weight in all."""
    B, Hq, D = q.shape
    page, Hkv = kc.shape[1], kc.shape[2]
    u = po.half_step(q.dtype)
    weight = 2.0 ** -21 if q.dtype == torch.float16 else 2.0 ** -11
    scale = D ** -0.5 if scale is None else scale
    o = torch.zeros(B, Hq, D, dtype=torch.float64)
    bound = torch.zeros_like(o)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    lbound = torch.zeros_like(lse)
    kd, vd = widened(kc, ks), widened(vc, vs)
    for b, n in enumerate(lens.tolist()):
        if n == 0:
            continue
        at = torch.arange(n)
        rows = table[b].long()[at // page]
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            kk, vv, sv = kd[rows, at % page, hk], vd[rows, at % page, hk], vs[rows, hk, at % page].double()
            x = scale * (kk @ q[b, h].double())
            size = abs(scale) * (kk.abs() @ q[b, h].double().abs())
            off = (2.0 ** -17 + 2.0 ** -21) * size + 2.0 ** -18           # of each weight
            lse[b, h] = torch.logsumexp(x, 0)
            p = torch.exp(x - lse[b, h])
            o[b, h] = p @ vv
            # a weight off by a factor 1 + off moves numerator and sum
            bound[b, h] = u * o[b, h].abs() + ((p * (off + weight)) @ vv.abs()) + (p @ off) * o[b, h].abs()
            bound[b, h] += 2.0 ** -39 * (p * sv).max() * 448 * n
            if q.dtype == torch.float16:
                bound[b, h] += 2.0 ** -25                               # half the smallest fp16
            lbound[b, h] = off.max() + 2.0 ** -22 * lse[b, h].abs()
    return o, lse, bound, lbound


def check_codes(codes, scale, y, off):
    """Stored rows against rows y (64 bits) whose fp32 values may be off by `off`: the scale by that and two
    roundings, and each code the nearest one to some value within reach."""
    top = y.abs().amax(-1)
    want = torch.where(top == 0, torch.ones_like(top), top / 448)
    far = off.amax(-1) / 448 + 2.0 ** -22 * want
    s = scale.double()
    assert ((s - want).abs() <= far).all(), ((s - want).abs() / far).max()
    c = codes.to(torch.float32).double()
    q, d = y / want[..., None], off / want[..., None]
    # the quotient: its numerator off by `off`, its denominator by far / want, and three roundings
    d = d + q.abs() * (far / want)[..., None] + 2.0 ** -22 * q.abs()
    lo, hi = nearest_e4m3((q - d).clamp(-448, 448)), nearest_e4m3((q + d).clamp(-448, 448))
    assert ((c >= lo) & (c <= hi)).all(), "a code is not the nearest"


def read(cache, scale, table, lens, dtype):
    """Packed rows [sum(lens), Hkv, D] of one cache in 64 bits, and the bound of one rounding (two in fp32
    arithmetic: the product, then the type)."""
    x = widened(cache, scale) if scale is not None else cache.double()
    page = cache.shape[1]
    rows = []
    for b, n in enumerate(lens.tolist()):
        at = torch.arange(n)
        rows.append(x[table[b].long()[at // page], at % page])
    y = torch.cat(rows) if rows else x[:0, 0]
    tiny = torch.finfo(dtype).tiny * po.half_step(dtype)
    return y, po.half_step(dtype) * (1 + 2.0 ** -10) * y.abs() + tiny
