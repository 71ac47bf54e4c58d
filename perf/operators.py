"""The operators around a paged key/value cache: cases, inputs, plain forms and floors.

One generation step of a served model makes four calls, and a training step makes the second and
its gradient before its attention:

  plan     new tokens of each request -> pages taken from the free list, block table, slot of every
           token, positions, cumulative lengths
  rope     RMS norm of every query and key head and the rotation by position, in one pass
  rope_bwd the gradients of `rope` (queries, keys, both norm weights)
  append   `rope` for a step that serves: keys and values go to their slots of the paged cache
  decode   attention of one new token per request over the paged cache

Every case is one call.  `run` computes it in elementary torch operations where `own` is false and
through the framework's entry points where it is true.
"""
import math
import random

import torch

own = False
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # The shortest call: one conversation of a few hundred tokens, grouped heads, wide heads.
        dict(name="decode_b1_d512", kind="decode", B=1, Hq=16, Hkv=4, D=512, lo=777, hi=777, page=16, dtype="bf16",
             spare=40, lens=1),
        # An ordinary batch in service: ragged contexts, group of 4, D = 512.
        dict(name="decode_b32_d512", kind="decode", B=32, Hq=32, Hkv=8, D=512, lo=512, hi=4096, page=32, dtype="bf16",
             spare=100, lens=2),
        # Two long documents under one shared key head: only the split over the length fills the card.
        dict(name="decode_long_mqa_d256", kind="decode", B=2, Hq=16, Hkv=1, D=256, lo=260000, hi=393216, page=64,
             dtype="fp16", spare=64, lens=3),
        # Many requests of any age, as many key heads as query heads, small pages.
        dict(name="decode_b128_mha_d128", kind="decode", B=128, Hq=16, Hkv=16, D=128, lo=1, hi=2048, page=16,
             dtype="bf16", spare=200, lens=4),
        # A packed training or prefill batch: every head normed, whole head rotated, halves layout.
        dict(name="rope_t8192_d512", kind="rope", T=8192, Hq=32, Hkv=8, D=512, rot=512, inter=False, norm=True,
             wdtype="bf16", dtype="bf16", far=8192, factor=1.0),
        # A short prompt with far positions: part of the head, interleaved pairs, no norm.
        dict(name="rope_t515_part_d128", kind="rope", T=515, Hq=16, Hkv=16, D=128, rot=64, inter=True, norm=False,
             wdtype="fp32", dtype="fp16", far=1 << 20, factor=4.0),
        # The gradient of a training batch, weights kept in 32 bits.
        dict(name="rope_bwd_t8192_d512", kind="rope_bwd", T=8192, Hq=16, Hkv=4, D=512, rot=512, inter=False, norm=True,
             wdtype="fp32", dtype="bf16", far=8192, factor=1.0),
        # The gradient of one short sequence, part of the head rotated.
        dict(name="rope_bwd_t333_d320", kind="rope_bwd", T=333, Hq=8, Hkv=8, D=320, rot=160, inter=True, norm=True,
             wdtype="bf16", dtype="bf16", far=32768, factor=1.0),
        # One token of each of 32 requests.
        dict(name="append_t32_d512", kind="append", T=32, Hq=32, Hkv=8, D=512, rot=512, inter=False, norm=True,
             wdtype="bf16", dtype="bf16", far=4096, factor=1.0, page=32, pages=3000),
        # A prompt of 16k tokens going into the cache, with some padding tokens.
        dict(name="append_t16384_d256", kind="append", T=16384, Hq=16, Hkv=4, D=256, rot=128, inter=False, norm=True,
             wdtype="fp32", dtype="fp16", far=131072, factor=8.0, page=16, pages=1500),
        # The plan of one generation step.
        dict(name="plan_b64", kind="plan", B=64, old=4096, new=1, idle=0.1, page=16, lens=5),
        # The plan of a step that mixes prompts and single tokens.
        dict(name="plan_b512_prompts", kind="plan", B=512, old=8192, new=700, idle=0.2, page=32, lens=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "rope", "rope_bwd", "append", "plan"])
    D = 8 * rng.randint(8, 128) if rng.random() < 0.4 else rng.choice([64, 128, 256, 320, 512, 768, 1024])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8, 16])
    if kind == "plan":
        return dict(kind=kind, B=_log(rng, 1, 512), old=_log(rng, 1, 8192), new=_log(rng, 1, 700), idle=rng.choice([0.0, 0.2]),
                    page=rng.choice([1, 8, 16, 32, 64, 100]), lens=rng.randrange(1 << 30))
    if kind == "decode":
        Hq = min(Hq, 64) // Hkv * Hkv or Hkv
        most = (1 << 28) // (Hkv * D)  # keys in all: at most 1 GB of keys and values
        B = _log(rng, 1, 128)
        hi = max(1, min(393216, most // B))
        hi = _log(rng, max(1, hi // 64), hi)
        return dict(kind=kind, B=B, Hq=Hq, Hkv=Hkv, D=D, lo=rng.choice([0, 1, hi]), hi=hi, page=rng.choice([1, 8, 16, 16, 32, 64, 100]),
                    dtype=dtype, spare=rng.randint(1, 50), lens=rng.randrange(1 << 30))
    norm = rng.random() < 0.75
    rot = 8 * rng.randint(1, D // 8) if rng.random() < 0.4 else D
    T = _log(rng, 1, max(1, min(16384, (1 << 27) // ((Hq + Hkv) * D))))
    case = dict(kind=kind, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, inter=rng.random() < 0.5, norm=norm,
                wdtype=rng.choice(["fp32", dtype]), dtype=dtype, far=_log(rng, 16, 1 << 20), factor=rng.choice([1.0, 4.0]))
    if kind == "append":
        page = rng.choice([1, 8, 16, 32, 100])
        case.update(page=page, pages=-(-T // page) + rng.randint(1, 40))
    return case


def _lengths(c):
    """Cached tokens of each request."""
    r = random.Random(c["lens"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]


def _growth(c):
    """(cached tokens, new tokens) of each request; an idle request adds none."""
    r = random.Random(c["lens"])
    old = [r.randint(0, c["old"]) for _ in range(c["B"])]
    new = [0 if r.random() < c["idle"] else r.randint(1, c["new"]) for _ in range(c["B"])]
    return old, new


# ------------------------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def prepare(case, seed):
    return {"decode": _prepare_decode, "plan": _prepare_plan}.get(case["kind"], _prepare_rope)(case, seed)


def _prepare_decode(c, seed):
    g, dt, page = _generator(seed), TYPES[c["dtype"]], c["page"]
    lens = _lengths(c)
    held = [-(-n // page) for n in lens]
    pool = sum(held) + c["spare"]
    order = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    width = max(max(held), 1)
    # The table holds the pages of each request in order and -1 behind them.
    n = torch.tensor(held, device=DEV)
    first = torch.cumsum(n, 0) - n
    j = torch.arange(width, device=DEV)
    at = (first[:, None] + j[None]).clamp(max=pool - 1)
    table = torch.where(j[None] < n[:, None], order[at], torch.full_like(order[at], -1))
    shape = (pool, page, c["Hkv"], c["D"])
    return dict(c=c, kind="decode", q=torch.randn(c["B"], c["Hq"], c["D"], generator=g, device=DEV).to(dt),
                k_cache=torch.randn(shape, generator=g, device=DEV, dtype=dt),
                v_cache=torch.randn(shape, generator=g, device=DEV, dtype=dt),
                table=table, lens=torch.tensor(lens, dtype=torch.int32, device=DEV))


def _prepare_rope(c, seed):
    g, dt = _generator(seed), TYPES[c["dtype"]]
    T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
    s = dict(c=c, kind=c["kind"])
    # One projection makes queries, keys and values: the three are slices of its rows.
    heads = Hq + 2 * Hkv
    qkv = torch.randn(T, heads, D, generator=g, device=DEV, dtype=dt) * 1.5
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    start = int(torch.randint(0, max(1, c["far"] - T), (1,), generator=g, device=DEV).item())
    s["positions"] = torch.arange(start, start + T, device=DEV, dtype=torch.int32)
    half = c["rot"] // 2
    i = torch.arange(half, device=DEV, dtype=torch.float64)
    s["inv_freq"] = 10000.0 ** (-i / half) / c["factor"]
    s["rope_scale"] = 1.0 if c["factor"] == 1.0 else 0.1 * math.log(c["factor"]) + 1.0
    s["qw"] = s["kw"] = None
    if c["norm"]:
        w = 1.0 + 0.2 * torch.randn(2, D, generator=g, device=DEV)
        s["qw"], s["kw"] = w[0].to(TYPES[c["wdtype"]]), w[1].to(TYPES[c["wdtype"]])
    if c["kind"] == "rope_bwd":
        s["dq"] = torch.randn(T, Hq, D, generator=g, device=DEV, dtype=dt)
        s["dk"] = torch.randn(T, Hkv, D, generator=g, device=DEV, dtype=dt)
    if c["kind"] == "append":
        shape = (c["pages"], c["page"], Hkv, D)
        s["k_cache"] = torch.randn(shape, generator=g, device=DEV, dtype=dt)
        s["v_cache"] = torch.randn(shape, generator=g, device=DEV, dtype=dt)
        slots = torch.randperm(c["pages"] * c["page"], generator=g, device=DEV)[:T]
        pad = torch.rand(T, generator=g, device=DEV) < 0.03
        s["slots"] = torch.where(pad, torch.full_like(slots, -1), slots)
    return s


def _prepare_plan(c, seed):
    g, page = _generator(seed), c["page"]
    old, new = _growth(c)
    total = sum(-(-(a + b) // page) for a, b in zip(old, new))
    pool = total + 7
    order = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    held = torch.tensor([-(-n // page) for n in old], device=DEV)
    first = torch.cumsum(held, 0) - held
    width = max(-(-(a + b) // page) for a, b in zip(old, new)) + 2
    j = torch.arange(width, device=DEV)
    at = (first[:, None] + j[None]).clamp(max=pool - 1)
    table = torch.where(j[None] < held[:, None], order[at], torch.full_like(order[at], -1))
    used = int(held.sum().item())
    free = order.clone()
    free[:pool - used] = order[used:]
    return dict(c=c, kind="plan", table=table, lens=torch.tensor(old, dtype=torch.int32, device=DEV),
                new=torch.tensor(new, dtype=torch.int32, device=DEV), free=free,
                count=torch.tensor([pool - used], dtype=torch.int32, device=DEV), tokens=sum(new) + 5)


# ----------------------------------------------------------------------------------- the pass
def run(state):
    s, c = state, state["c"]
    if own:
        import exact_headdim_attention_gb300 as ffpa

        rope = dict(positions=s.get("positions"), inv_freq=s.get("inv_freq"), q_weight=s.get("qw"), k_weight=s.get("kw"))
        how = dict(interleaved=c.get("inter", False), rope_scale=s.get("rope_scale", 1.0))
        if s["kind"] == "decode":
            return ffpa.ffpa_decode_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], enable_gqa=True,
                                          return_lse=True)
        if s["kind"] == "rope":
            return ffpa.ffpa_qk_norm_rope(s["q"], s["k"], **rope, **how)
        if s["kind"] == "rope_bwd":
            return [t for t in ffpa.ffpa_qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], **rope, **how) if t is not None]
        if s["kind"] == "append":
            q = ffpa.ffpa_kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], **rope, **how)
            return q, s["k_cache"], s["v_cache"]
        return (s["table"],) + tuple(ffpa.ffpa_page_plan(s["table"], s["lens"], s["new"], s["free"], s["count"], c["page"],
                                                         s["tokens"]))
    if s["kind"] == "decode":
        return _plain_decode(s)
    if s["kind"] == "plan":
        return _plain_plan(s)
    if s["kind"] == "rope_bwd":
        return _plain_rope_bwd(s)
    q, k = _plain_rope(s, s["q"], s["qw"]), _plain_rope(s, s["k"], s["kw"])
    if s["kind"] == "rope":
        return q, k
    kept = s["slots"] >= 0
    at = s["slots"][kept]
    s["k_cache"].view(-1, *k.shape[1:])[at] = k[kept]
    s["v_cache"].view(-1, *k.shape[1:])[at] = s["v"][kept]
    return q, s["k_cache"], s["v_cache"]


def _plain_decode(s):
    q, kc, table, lens = s["q"], s["k_cache"], s["table"], s["lens"].long()
    B, Hq, D = q.shape
    page, Hkv = kc.shape[1], kc.shape[2]
    N = table.shape[1] * page
    pages = table.clamp(min=0).long()
    seen = torch.arange(N, device=q.device)[None] < lens[:, None]                     # [B, N]
    k = kc[pages].reshape(B, N, Hkv, D).permute(0, 2, 3, 1).float()                   # [B, Hkv, D, N]
    x = torch.matmul(q.float().reshape(B, Hkv, Hq // Hkv, D), k) / math.sqrt(D)
    del k
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    lse = torch.log(total) + torch.where(torch.isinf(m), torch.zeros_like(m), m)
    v = s["v_cache"][pages].reshape(B, N, Hkv, D).permute(0, 2, 1, 3).float()
    v = v.masked_fill(~seen[:, None, :, None], 0.0)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.reshape(B, Hq, D).to(q.dtype), lse.reshape(B, Hq)


def _angles(s):
    """cos and sin [T, 1, rot/2] in 32 bits, from angles in 64: far positions turn many times."""
    a = s["positions"].double()[:, None] * s["inv_freq"][None]
    return (torch.cos(a) * s["rope_scale"]).float()[:, None], (torch.sin(a) * s["rope_scale"]).float()[:, None]


def _turn(s, x, back=False):
    """The rotated copy of x (fp32); back: by the opposite angle."""
    rot = s["c"]["rot"]
    cos, sin = _angles(s)
    if back:
        sin = -sin
    h = x[..., :rot]
    if s["c"]["inter"]:
        a, b = h[..., 0::2], h[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = h[..., :rot // 2], h[..., rot // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_rope(s, x, w):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    return _turn(s, y).to(x.dtype)


def _plain_norm_back(s, dy, x, w):
    dy = _turn(s, dy.float(), back=True)
    if w is None:
        return dy.to(x.dtype), None
    x32 = x.float()
    r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + 1e-6)
    xn = x32 * r
    dw = (dy * xn).sum((0, 1), dtype=torch.float64).to(w.dtype)
    t = dy * w.float()
    dx = r * (t - xn * (t * xn).mean(-1, keepdim=True))
    return dx.to(x.dtype), dw


def _plain_rope_bwd(s):
    dq, dqw = _plain_norm_back(s, s["dq"], s["q"], s["qw"])
    dk, dkw = _plain_norm_back(s, s["dk"], s["k"], s["kw"])
    return [t for t in (dq, dk, dqw, dkw) if t is not None]


def _plain_plan(s):
    page, table, T = s["c"]["page"], s["table"], s["tokens"]
    old, new = s["lens"].long(), s["new"].long()
    after = old + new
    before, held = (old + page - 1) // page, (after + page - 1) // page
    need = held - before
    taken = torch.cumsum(need, 0)
    # New pages come off the end of the free list in the order of requests, then of their pages.
    j = torch.arange(table.shape[1], device=table.device)[None]
    nth = (taken - need)[:, None] + j - before[:, None]
    at = (s["count"].long() - 1 - nth).clamp(0, s["free"].numel() - 1)
    fresh = (j >= before[:, None]) & (j < held[:, None])
    table.copy_(torch.where(fresh, s["free"][at], table))
    cu = torch.zeros(new.numel() + 1, dtype=torch.int64, device=table.device)
    cu[1:] = torch.cumsum(new, 0)
    t = torch.arange(T, device=table.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    real = t < cu[-1]
    b = torch.where(real, b, torch.zeros_like(b)).clamp(0, new.numel() - 1)
    pos = torch.where(real, old[b] + t - cu[b], torch.zeros_like(t))
    slots = table[b, pos // page].long() * page + pos % page
    slots = torch.where(real, slots, torch.full_like(slots, -1))
    return (table, slots, pos.int(), cu.int(), after.int(), (s["count"].long() - taken[-1:]).int())


# ------------------------------------------------------------------------------------ floors
def work(case):
    """Bytes that a pass reads and writes once, and its operations."""
    c = case
    if c["kind"] == "plan":
        old, new = _growth(c)
        fresh = sum(-(-(a + b) // c["page"]) - -(-a // c["page"]) for a, b in zip(old, new))
        # lengths read and written, cumulative lengths, new pages read and written, 12 bytes a token,
        # the page that each growing request goes on filling
        return {"bytes": c["B"] * 16 + fresh * 8 + (sum(new) + 5) * 12 + 8, "flops": 0}
    if c["kind"] == "decode":
        lens = _lengths(c)
        n = sum(lens)
        pages = sum(-(-x // c["page"]) for x in lens)
        io = c["B"] * c["Hq"] * (4 * c["D"] + 4) + c["B"] * 4 + pages * 4
        return {"bytes": 4 * n * c["Hkv"] * c["D"] + io, "flops": 4 * n * c["Hq"] * c["D"]}
    T, D = c["T"], c["D"]
    rows = T * (c["Hq"] + c["Hkv"])
    small = T * 4 + c["rot"] * 4 + (2 * D * (4 if c["wdtype"] == "fp32" else 2) if c["norm"] else 0)
    if c["kind"] == "rope_bwd":
        # without a norm the inputs themselves are not needed
        return {"bytes": rows * D * 2 * (3 if c["norm"] else 2) + small * (2 if c["norm"] else 1), "flops": rows * D * (16 if c["norm"] else 3)}
    extra = T * c["Hkv"] * D * 4 + T * 8 if c["kind"] == "append" else 0
    return {"bytes": rows * D * 4 + small + extra, "flops": rows * D * (7 if c["norm"] else 3)}


# ------------------------------------------------------------------------- 64-bit definitions
def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "plan":
        return None
    if case["kind"] == "decode":
        return _exact_decode(s)
    if case["kind"] == "rope_bwd":
        return _exact_gradients(s)
    qw, kw = s["qw"], s["kw"]
    q = _exact_rope(s, s["q"].double(), None if qw is None else qw.double())
    if case["kind"] == "rope":
        return q, _exact_rope(s, s["k"].double(), None if kw is None else kw.double())
    k = _exact_rope(s, s["k"].double(), None if kw is None else kw.double())
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    page = kc.shape[1]
    rows = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][rows]
    kc[at // page, at % page] = k[rows]
    vc[at // page, at % page] = s["v"].double()[rows]
    return q, kc, vc


def _exact_decode(s):
    """Request by request: the softmax of its scores over its own pages."""
    q, page = s["q"].double(), s["k_cache"].shape[1]
    B, Hq, D = q.shape
    Hkv = s["k_cache"].shape[2]
    o = torch.zeros(B, Hq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        ids = s["table"][b, : -(-n // page)].long()
        for h in range(Hkv):
            rows = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            k = s["k_cache"][ids, :, h].double().flatten(0, 1)[:n]
            v = s["v_cache"][ids, :, h].double().flatten(0, 1)[:n]
            x = (q[b, rows] @ k.T) * D ** -0.5
            lse[b, rows] = torch.logsumexp(x, -1)
            o[b, rows] = torch.softmax(x, -1) @ v
    return o, lse


def _exact_rope(s, x, w):
    """As complex numbers: each pair times exp(i * angle)."""
    rot = s["c"]["rot"]
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * w
    a = torch.outer(s["positions"].double(), s["inv_freq"])
    z = torch.polar(torch.full_like(a, s["rope_scale"]), a)[:, None]
    if s["c"]["inter"]:
        y = torch.view_as_real(torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
    else:
        y = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * z
        y = torch.cat((y.real, y.imag), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _exact_gradients(s):
    """By differentiating the 64-bit definition."""
    ins, outs, grads = [], [], []
    weights = []
    for x, w, dy in ((s["q"], s["qw"], s["dq"]), (s["k"], s["kw"], s["dk"])):
        x = x.double().requires_grad_()
        w = None if w is None else w.double().requires_grad_()
        with torch.enable_grad():
            outs.append(_exact_rope(s, x, w))
        ins.append(x)
        weights += [] if w is None else [w]
        grads.append(dy.double())
    return list(torch.autograd.grad(outs, ins + weights, grads))
