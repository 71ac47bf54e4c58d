"""64-bit references of the paged-cache operators and of the head norm with rotation, written from
their definitions in include/ffpa.h, with the error bounds the GPU tests use."""
from __future__ import annotations

import math

import torch


def half_step(dtype):
    """Relative error of one rounding to `dtype`."""
    return torch.finfo(dtype).eps / 2


# ---------------------------------------------------------------------------------- inputs
def make_cache(g, lens, Hkv, D, page, dtype, spare=3, layout="psh"):
    """A cache of randomly placed pages, its block table and lengths (CPU).  Slots and pages that no
    request owns hold NaN: a kernel that reads one shows it.  layout "phs" keeps the heads outside
    the slots of a page."""
    held = [-(-n // page) for n in lens]
    pool = sum(held) + spare
    order = torch.randperm(pool, generator=g)
    table = torch.full((len(lens), max(held + [1]) + 2), -1, dtype=torch.int32)
    shape = (pool, page, Hkv, D) if layout == "psh" else (pool, Hkv, page, D)
    k, v = (torch.full(shape, math.nan, dtype=dtype) for _ in range(2))
    if layout == "phs":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    at = 0
    for b, n in enumerate(lens):
        for j in range(held[b]):
            p = int(order[at])
            at += 1
            table[b, j] = p
            m = min(page, n - j * page)
            k[p, :m] = torch.randn(m, Hkv, D, generator=g).to(dtype)
            v[p, :m] = torch.randn(m, Hkv, D, generator=g).to(dtype)
    return k, v, table, torch.tensor(lens, dtype=torch.int32)


# ---------------------------------------------------------------------------------- decode
def decode(q, k_cache, v_cache, table, lens, scale=None):
    """(o, lse, bound on |o's error|, bound on |lse's error|) in 64 bits.

    With u the half step of the type: o is rounded once (u |o|) and every p once before its product
    (u sum p |v| / l; in fp16 also 2^-25 below the normal range).  Scores are summed in fp32 over at
    most 64 steps of 16 products, each step off by 2^-23 of partial sums that stay below 8 for these
    inputs (2^-14 in all, as a relative error of p); exponentials, sums and the scale are off by less."""
    B, Hq, D = q.shape
    page, Hkv = k_cache.shape[1], k_cache.shape[2]
    u = half_step(q.dtype)
    scale = D ** -0.5 if scale is None else scale
    o = torch.zeros(B, Hq, D, dtype=torch.float64)
    bound = torch.zeros_like(o)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    for b, n in enumerate(lens.tolist()):
        if n == 0:
            continue
        at = torch.arange(n)
        rows = table[b].long()[at // page]
        for h in range(Hq):
            kk = k_cache[rows, at % page, h // (Hq // Hkv)].double()
            vv = v_cache[rows, at % page, h // (Hq // Hkv)].double()
            x = scale * (kk @ q[b, h].double())
            lse[b, h] = torch.logsumexp(x, 0)
            p = torch.exp(x - lse[b, h])
            o[b, h] = p @ vv
            bound[b, h] = u * o[b, h].abs() + (u + 2.0 ** -14) * (p @ vv.abs())
            if q.dtype == torch.float16:
                top = torch.exp(x.max() - lse[b, h])       # p in the kernel is relative to the largest
                bound[b, h] += 2.0 ** -24 * top * vv.abs().sum(0)
    return o, lse, bound, 2.0 ** -14 + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)


# ------------------------------------------------------------------------------------ rope
def rope(x, positions, inv_freq, w, eps=1e-6, interleaved=False, rope_scale=1.0):
    """One tensor [..., H, D] with positions [...] (x and w 64-bit for gradients)."""
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w
    if inv_freq is None:
        return x
    rot = 2 * inv_freq.numel()
    t = (positions.double()[..., None] * inv_freq)[..., None, :]
    c, s = rope_scale * torch.cos(t), rope_scale * torch.sin(t)
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., rot:]), -1)


def rope_bound(x, positions, inv_freq, w, eps=1e-6, interleaved=False, rope_scale=1.0):
    """(reference, bound on the error) of `rope` rounded once to x's type.

    fp32 inside: the norm is off by a few 2^-24 (row sums of at most 1024 squares in a tree of some
    40 steps: 2^-19 of r), cosines and sines by 2^-20 (2^-21 of the function, 2^-22 of the angle's
    rounding and 2^-31 turns of its fixed point); both act on |a| and |b| of the pair: 2^-18 in all."""
    xd = x.double()
    wd = None if w is None else w.double()
    y = rope(xd, positions, inv_freq, wd, eps, interleaved, rope_scale)
    m = rope(xd, positions, None, wd, eps).abs()
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        if interleaved:
            pair = (m[..., 0:rot:2] + m[..., 1:rot:2]).repeat_interleave(2, -1)
        else:
            pair = (m[..., :rot // 2] + m[..., rot // 2:rot]).repeat(*[1] * (m.dim() - 1), 2)
        m = torch.cat((pair * abs(rope_scale), m[..., rot:]), -1)
    tiny = torch.finfo(x.dtype).tiny * half_step(x.dtype)     # half a step below the normal range
    return y, half_step(x.dtype) * y.abs() + 2.0 ** -18 * m + tiny


def rope_grads(g, x, positions, inv_freq, w, eps=1e-6, interleaved=False, rope_scale=1.0):
    """(dx, dw, bounds of both) by differentiating the 64-bit definition.

    dx is rounded once; inside, with g' the rotated gradient, its terms r w g' and r xn mean(w g' xn)
    are off by 2^-17 of their sizes.  dw sums fp32 values in chains of at most some 300 and trees
    after that: 2^-15 of sum |g' xn| bounds it, and one rounding to the weight's type."""
    xd = x.double().requires_grad_()
    wd = None if w is None else w.double().requires_grad_()
    y = rope(xd, positions, inv_freq, wd, eps, interleaved, rope_scale)
    grads = torch.autograd.grad(y, [xd] + ([] if wd is None else [wd]), g.double())
    dx, dw = grads[0], None if wd is None else grads[1]
    # |g'| <= |scale| (|g_a| + |g_b|) on the pair
    gm = g.double().abs()
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        if interleaved:
            pair = (gm[..., 0:rot:2] + gm[..., 1:rot:2]).repeat_interleave(2, -1)
        else:
            pair = (gm[..., :rot // 2] + gm[..., rot // 2:rot]).repeat(*[1] * (gm.dim() - 1), 2)
        gm = torch.cat((pair * abs(rope_scale), gm[..., rot:]), -1)
    tiny = torch.finfo(x.dtype).tiny * half_step(x.dtype)
    u = half_step(x.dtype)
    if w is None:
        return dx, None, u * dx.abs() + 2.0 ** -18 * gm + tiny, None
    xv, wv = x.double(), w.double()
    r = torch.rsqrt(xv.square().mean(-1, keepdim=True) + eps)
    xn = (xv * r).abs()
    t = wv.abs() * gm
    size = r * (t + xn * (t * xn).mean(-1, keepdim=True))
    flat = (gm * xn).flatten(0, -2).sum(0)
    return dx, dw, u * dx.abs() + 2.0 ** -17 * size + tiny, half_step(w.dtype) * dw.abs() + 2.0 ** -15 * flat


# ------------------------------------------------------------------------------------ plan
def page_plan(table, seq_lens, new_lens, free_pages, free_count, page, tokens):
    """The plan request by request, page by page, in plain Python.  Returns the new table, slots,
    positions, cu_seqlens, seq_lens, free_count and whether the call is to be reported."""
    table = table.clone()
    cap = table.shape[1] * page
    bad = not 0 <= free_count <= len(free_pages)
    count = min(max(free_count, 0), len(free_pages))
    slots, positions, cu, out = [], [], [0], []
    for b, (old, new) in enumerate(zip(seq_lens, new_lens)):
        bad |= old < 0 or new < 0 or old > cap
        old, new = min(max(old, 0), cap), max(new, 0)
        held = -(-old // page)
        bad |= old + new > cap
        got = old
        for pos in range(old, old + new):
            j = pos // page
            if j >= table.shape[1]:
                p = -1
            elif j < held:
                p = int(table[b, j])
            else:
                if pos % page == 0:
                    if count > 0:
                        count -= 1
                        table[b, j] = free_pages[count]
                    else:
                        table[b, j] = -1
                        bad = True
                p = int(table[b, j])
            slots.append(-1 if p < 0 else p * page + pos % page)
            positions.append(pos)
            if p >= 0 or j < held:
                got = pos + 1
        out.append(got)
        cu.append(cu[-1] + new)
    bad |= len(slots) > tokens
    slots = (slots + [-1] * tokens)[:tokens]
    positions = (positions + [0] * tokens)[:tokens]
    return table, slots, positions, [min(c, tokens) for c in cu], out, count, bad
