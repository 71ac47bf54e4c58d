"""A quantised paged cache, and attention of a batch with a shared prefix: cases, inputs, plain forms and floors.

A service that holds many or long conversations keeps its keys and values in 8 bits:

  append8  head norm and rotation of a step's rows, keys and values to their slots as e4m3 codes with
           a scale for each token and head
  decode8  attention of one new token per request over that cache
  read     the cached rows of each request as packed 16-bit rows (from codes, or from 16-bit pages),
           for a prompt's attention over what is cached before it

and requests that begin with the same tokens (instructions, a document) share the pages of those:

  shared   attention of one new token per request over a 16-bit cache, the shared pages read and
           multiplied once for all requests

Every case is one call.  `run` computes it in elementary torch operations where `own` is false and
through the framework's entry points where it is true.
"""
import math
import random

import torch

own = False
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # The shortest call: one conversation of a few hundred tokens, wide heads.
        dict(name="decode8_b1_d512", kind="decode8", B=1, Hq=16, Hkv=4, D=512, lo=777, hi=777, page=16, dtype="bf16",
             spare=40, lens=1),
        # An ordinary batch in service, contexts of all lengths, group of 4.
        dict(name="decode8_b32_d512", kind="decode8", B=32, Hq=32, Hkv=8, D=512, lo=512, hi=8192, page=32, dtype="bf16",
             spare=100, lens=2),
        # Many requests of any age, as many key heads as query heads, narrow heads, small pages.
        dict(name="decode8_b128_mha_d128", kind="decode8", B=128, Hq=16, Hkv=16, D=128, lo=1, hi=2048, page=16,
             dtype="fp16", spare=200, lens=4),
        # One token of each of 32 requests goes into the cache.
        dict(name="append8_t32_d512", kind="append8", T=32, Hq=32, Hkv=8, D=512, rot=512, inter=False, norm=True,
             wdtype="bf16", dtype="bf16", far=4096, factor=1.0, page=32, pages=40),
        # A prompt of some 16k tokens, part of each head rotated, some padding tokens.
        dict(name="append8_t16001_d256", kind="append8", T=16001, Hq=16, Hkv=4, D=256, rot=128, inter=False, norm=True,
             wdtype="fp32", dtype="fp16", far=131072, factor=8.0, page=16, pages=1100),
        # A prompt's rows as they are: no norm, no rotation of the keys, as many key heads as query heads.
        dict(name="append8_t5000_mha_d128", kind="append8", T=5000, Hq=32, Hkv=32, D=128, rot=0, inter=False, norm=False,
             wdtype="bf16", dtype="bf16", far=8192, factor=1.0, page=64, pages=90),
        # A few hundred cached tokens of three short conversations, before their next prompts.
        dict(name="read_b3_d512", kind="read", B=3, Hkv=4, D=512, lo=1, hi=400, page=16, dtype="bf16", bits=8, spare=20,
             lens=7),
        # The contexts of a batch of long conversations.
        dict(name="read_b24_d512", kind="read", B=24, Hkv=8, D=512, lo=100, hi=8192, page=32, dtype="bf16", bits=8,
             spare=50, lens=8),
        # The same from a 16-bit cache of narrow heads.
        dict(name="read16_b40_d128", kind="read", B=40, Hkv=16, D=128, lo=0, hi=3000, page=16, dtype="fp16", bits=16,
             spare=50, lens=9),
        # A few requests that share instructions of about a thousand tokens.
        dict(name="shared_b16_d128", kind="shared", B=16, Hq=16, Hkv=4, D=128, S=1010, lo=1, hi=100, page=16, dtype="bf16",
             spare=20, lens=10),
        # A batch that asks about one document, group of 4, wide heads.
        dict(name="shared_b64_d512", kind="shared", B=64, Hq=32, Hkv=8, D=512, S=16384, lo=1, hi=512, page=32,
             dtype="bf16", spare=50, lens=11),
        # A large batch behind long shared instructions with examples.
        dict(name="shared_b128_d128", kind="shared", B=128, Hq=32, Hkv=8, D=128, S=32768, lo=0, hi=1024, page=64,
             dtype="fp16", spare=50, lens=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode8", "decode8", "append8", "read", "shared", "shared"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    if kind == "shared":
        D = rng.choice([64, 128, 128, 192, 256, 320, 512, 768, 1024])
        g = rng.choice([1, 2, 3, 4, 5, 8])
        B = _log(rng, 2, 160)
        # operations: at most 4 D Hq B S = 2^36; bytes of the pages: at most 2 GB in all
        S = min(65536, (1 << 36) // (4 * D * Hkv * g * B), (1 << 28) // (Hkv * D))
        S = _log(rng, max(1, S // 64), max(2, S))
        own_most = max(2, min(2048, (1 << 28) // (Hkv * D * B)))
        return dict(kind=kind, B=B, Hq=Hkv * g, Hkv=Hkv, D=D, S=S, lo=rng.choice([0, 1]), hi=_log(rng, 1, own_most),
                    page=rng.choice([8, 16, 16, 32, 64, 128]), dtype=dtype, spare=rng.randint(1, 50),
                    lens=rng.randrange(1 << 30))
    D = 16 * rng.randint(4, 64) if rng.random() < 0.4 else rng.choice([64, 128, 256, 320, 512, 768, 1024])
    page = rng.choice([1, 8, 16, 16, 32, 64, 100])
    if kind in ("decode8", "read"):
        most = (1 << 29) // (Hkv * D)  # keys in all: at most 1 GB of codes
        if kind == "read":
            most //= 2
        B = _log(rng, 1, 128)
        hi = max(1, min(393216, most // B))
        hi = _log(rng, max(1, hi // 64), hi)
        case = dict(kind=kind, B=B, Hkv=Hkv, D=D, lo=rng.choice([0, 1, hi]), hi=hi, page=page, dtype=dtype,
                    spare=rng.randint(1, 50), lens=rng.randrange(1 << 30))
        if kind == "read":
            case.update(bits=rng.choice([8, 8, 16]))
        else:
            case.update(Hq=min(Hkv * rng.choice([1, 2, 3, 4, 5, 8, 16]), 64) // Hkv * Hkv or Hkv)
        return case
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8])
    rot = 8 * rng.randint(0, D // 8) if rng.random() < 0.4 else D
    T = _log(rng, 1, max(1, min(16384, (1 << 26) // ((Hq + Hkv) * D))))
    return dict(kind=kind, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rot, inter=rng.random() < 0.5, norm=rng.random() < 0.75,
                wdtype=rng.choice(["fp32", dtype]), dtype=dtype, far=_log(rng, 16, 1 << 20), factor=rng.choice([1.0, 4.0]),
                page=page, pages=-(-T // page) + rng.randint(1, 40))


def _lengths(c):
    """Cached tokens of each request (behind the shared ones)."""
    r = random.Random(c["lens"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]


# ------------------------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _amax_scale(y):
    """(factor before the rounding, scale) of rows [..., D] in 32 bits; a row of zeros has scale 1."""
    top = y.abs().amax(-1)
    whole = torch.full_like(top, 448.0)
    zero = top == 0
    return (torch.where(zero, torch.ones_like(top), torch.div(whole, top)),
            torch.where(zero, torch.ones_like(top), torch.div(top, whole)))


def _codes(y):
    """e4m3 codes and scales of rows [..., D] (32 bits)."""
    f, scale = _amax_scale(y)
    return (y * f[..., None]).clamp(-448, 448).to(E4M3), scale


def _paged(g, lens, page, spare, first=0):
    """Pages in use and spare, the pages of each request in order (-1 behind them and in the first `first` columns)."""
    held = [-(-n // page) for n in lens]
    pool = sum(held) + spare
    order = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    width = max(max(held), 1) + first
    n = torch.tensor(held, device=DEV)
    begin = torch.cumsum(n, 0) - n
    j = torch.arange(width, device=DEV) - first
    at = (begin[:, None] + j[None]).clamp(0, pool - 1)
    used = (j[None] >= 0) & (j[None] < n[:, None])
    return pool, order, torch.where(used, order[at], torch.full_like(order[at], -1))


def _filled8(g, pool, page, Hkv, D):
    """A cache as append8 leaves it: codes [pool, page, Hkv, D] and scales [pool, Hkv, page]."""
    codes = torch.empty(pool, page, Hkv, D, dtype=E4M3, device=DEV)
    scale = torch.empty(pool, Hkv, page, device=DEV)
    step = max(1, (1 << 27) // (page * Hkv * D))
    for a in range(0, pool, step):
        n = min(step, pool - a)
        c, s = _codes(torch.randn(n, page, Hkv, D, generator=g, device=DEV))
        codes[a:a + n] = c
        scale[a:a + n] = s.transpose(1, 2)
    return codes, scale


def prepare(case, seed):
    return {"append8": _prepare_append, "shared": _prepare_shared}.get(case["kind"], _prepare_cache)(case, seed)


def _prepare_cache(c, seed):
    g, dt = _generator(seed), TYPES[c["dtype"]]
    lens = _lengths(c)
    pool, _, table = _paged(g, lens, c["page"], c["spare"])
    s = dict(c=c, kind=c["kind"], table=table, lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    if c["kind"] == "read" and c["bits"] == 16:
        shape = (pool, c["page"], c["Hkv"], c["D"])
        s["k_cache"], s["v_cache"] = (torch.randn(shape, generator=g, device=DEV, dtype=dt) for _ in range(2))
        s["k_scale"] = s["v_scale"] = None
    else:
        s["k_cache"], s["k_scale"] = _filled8(g, pool, c["page"], c["Hkv"], c["D"])
        s["v_cache"], s["v_scale"] = _filled8(g, pool, c["page"], c["Hkv"], c["D"])
    if c["kind"] == "read":
        s["tokens"] = sum(lens)
        cu = torch.zeros(c["B"] + 1, dtype=torch.int32, device=DEV)
        cu[1:] = torch.cumsum(s["lens"], 0)
        s["cu"] = cu
    else:
        s["q"] = torch.randn(c["B"], c["Hq"], c["D"], generator=g, device=DEV).to(dt)
    return s


def _prepare_append(c, seed):
    g, dt = _generator(seed), TYPES[c["dtype"]]
    T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
    s = dict(c=c, kind=c["kind"])
    # One projection makes queries, keys and values: the three are slices of its rows.
    heads = Hq + 2 * Hkv
    qkv = torch.randn(T, heads, D, generator=g, device=DEV, dtype=dt) * 1.5
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    s["positions"] = s["inv_freq"] = s["qw"] = s["kw"] = None
    s["rope_scale"] = 1.0
    if c["rot"]:
        start = int(torch.randint(0, max(1, c["far"] - T), (1,), generator=g, device=DEV).item())
        s["positions"] = torch.arange(start, start + T, device=DEV, dtype=torch.int32)
        half = c["rot"] // 2
        s["inv_freq"] = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half) / c["factor"]
        s["rope_scale"] = 1.0 if c["factor"] == 1.0 else 0.1 * math.log(c["factor"]) + 1.0
    if c["norm"]:
        w = 1.0 + 0.2 * torch.randn(2, D, generator=g, device=DEV)
        s["qw"], s["kw"] = w[0].to(TYPES[c["wdtype"]]), w[1].to(TYPES[c["wdtype"]])
    s["k_cache"], s["k_scale"] = _filled8(g, c["pages"], c["page"], Hkv, D)
    s["v_cache"], s["v_scale"] = _filled8(g, c["pages"], c["page"], Hkv, D)
    slots = torch.randperm(c["pages"] * c["page"], generator=g, device=DEV)[:T]
    pad = torch.rand(T, generator=g, device=DEV) < 0.03
    s["slots"] = torch.where(pad, torch.full_like(slots, -1), slots)
    return s


def _prepare_shared(c, seed):
    g, dt, page = _generator(seed), TYPES[c["dtype"]], c["page"]
    lens = _lengths(c)
    # Whole pages of the shared tokens are shared; each request has the rest of them in pages of its own.
    shared = c["S"] // page
    more = c["S"] - shared * page
    pool, order, table = _paged(g, [n + more for n in lens], page, c["spare"] + shared, first=shared)
    shape = (pool, page, c["Hkv"], c["D"])
    s = dict(c=c, kind="shared", table=table, q=torch.randn(c["B"], c["Hq"], c["D"], generator=g, device=DEV).to(dt),
             k_cache=torch.randn(shape, generator=g, device=DEV, dtype=dt),
             v_cache=torch.randn(shape, generator=g, device=DEV, dtype=dt),
             lens=torch.tensor([n + c["S"] for n in lens], dtype=torch.int32, device=DEV),
             shared_len=torch.tensor([c["S"]], dtype=torch.int32, device=DEV),
             shared_pages=order[pool - c["spare"] - shared: pool - c["spare"]].contiguous())
    return s


# ----------------------------------------------------------------------------------- the pass
def run(state):
    s, c = state, state["c"]
    if own:
        import exact_headdim_attention_gb300 as ffpa

        if s["kind"] == "decode8":
            return ffpa.ffpa_decode_paged_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                              s["lens"], enable_gqa=True, return_lse=True)
        if s["kind"] == "read":
            return ffpa.ffpa_kv_read(s["k_cache"], s["v_cache"], s["table"], s["cu"], s["tokens"], k_scale=s["k_scale"],
                                     v_scale=s["v_scale"], dtype=TYPES[c["dtype"]])
        if s["kind"] == "shared":
            return ffpa.ffpa_decode_shared(s["q"], s["k_cache"], s["v_cache"], s["shared_pages"], s["shared_len"],
                                           s["table"], s["lens"], enable_gqa=True, return_lse=True)
        q = ffpa.ffpa_kv_append_fp8(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                    s["slots"], positions=s["positions"], inv_freq=s["inv_freq"], q_weight=s["qw"],
                                    k_weight=s["kw"], interleaved=c["inter"], rope_scale=s["rope_scale"])
        return q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    return {"decode8": _plain_decode, "read": _plain_read, "shared": _plain_shared, "append8": _plain_append}[s["kind"]](s)


def _widened(s, name, pages):
    """Rows of the pages [..., page, Hkv, D] in 32 bits."""
    x = s[name + "_cache"][pages].float()
    if s.get(name + "_scale") is not None:
        x *= s[name + "_scale"][pages].transpose(-1, -2)[..., None]
    return x


def _softmax_sums(x):
    """(weights, their sum, log-sum-exp) over the last dimension, a row without keys among them."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    return p, torch.where(total > 0, total, torch.ones_like(total)), torch.log(total) + m


def _own_scores(s, q, table, lens):
    """Scores [B, Hkv, g, N] of the keys in each request's table, and the values [B, Hkv, N, D]."""
    B, Hq, D = q.shape
    page, Hkv = s["k_cache"].shape[1], s["k_cache"].shape[2]
    N = table.shape[1] * page
    pages = table.clamp(min=0).long()
    seen = torch.arange(N, device=q.device)[None] < lens[:, None]                     # [B, N]
    k = _widened(s, "k", pages).reshape(B, N, Hkv, D).permute(0, 2, 3, 1)
    x = torch.matmul(q.float().reshape(B, Hkv, Hq // Hkv, D), k) / math.sqrt(D)
    del k
    v = _widened(s, "v", pages).reshape(B, N, Hkv, D).permute(0, 2, 1, 3)
    return x.masked_fill(~seen[:, None, None], -math.inf), v.masked_fill(~seen[:, None, :, None], 0.0)


def _plain_decode(s):
    q = s["q"]
    B, Hq, D = q.shape
    x, v = _own_scores(s, q, s["table"], s["lens"].long())
    p, total, lse = _softmax_sums(x)
    return (torch.matmul(p, v) / total).reshape(B, Hq, D).to(q.dtype), lse.reshape(B, Hq)


def _plain_shared(s):
    q, page = s["q"], s["k_cache"].shape[1]
    B, Hq, D = q.shape
    Hkv = s["k_cache"].shape[2]
    n = s["shared_pages"].numel() * page
    pages = s["shared_pages"].long()
    k = _widened(s, "k", pages).reshape(n, Hkv, D).permute(1, 2, 0)                    # [Hkv, D, n]
    rows = q.float().reshape(B, Hkv, Hq // Hkv, D)
    x = torch.matmul(rows.transpose(0, 1).reshape(Hkv, -1, D), k) / math.sqrt(D)       # [Hkv, B g, n]
    x = x.reshape(Hkv, B, Hq // Hkv, n).transpose(0, 1)
    x2, v2 = _own_scores(s, q, s["table"][:, s["shared_pages"].numel():], s["lens"].long() - n)
    p, total, lse = _softmax_sums(torch.cat((x, x2), -1))
    v = _widened(s, "v", pages).reshape(n, Hkv, D).permute(1, 0, 2)
    o = torch.matmul(p[..., :n].transpose(0, 1).reshape(Hkv, -1, n), v).reshape(Hkv, B, Hq // Hkv, D).transpose(0, 1)
    o = (o + torch.matmul(p[..., n:], v2)) / total
    return o.reshape(B, Hq, D).to(q.dtype), lse.reshape(B, Hq)


def _plain_read(s):
    c, page = s["c"], s["k_cache"].shape[1]
    t = torch.arange(s["tokens"], device=DEV)
    b = torch.searchsorted(s["cu"].long(), t, right=True) - 1
    at = t - s["cu"].long()[b]
    p, i = s["table"][b, at // page].long(), at % page
    out = []
    for name in ("k", "v"):
        x = s[name + "_cache"][p, i].float()
        if s[name + "_scale"] is not None:
            x *= s[name + "_scale"][p, :, i][..., None]
        out.append(x.to(TYPES[c["dtype"]]))
    return out


def _turned(s, x):
    """The rotated copy of x (fp32); angles in 64 bits: far positions turn many times."""
    rot = s["c"]["rot"]
    if not rot:
        return x
    a = s["positions"].double()[:, None] * s["inv_freq"][None]
    cos, sin = (torch.cos(a) * s["rope_scale"]).float()[:, None], (torch.sin(a) * s["rope_scale"]).float()[:, None]
    h = x[..., :rot]
    if s["c"]["inter"]:
        a, b = h[..., 0::2], h[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = h[..., :rot // 2], h[..., rot // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_rows(s, x, w):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    return _turned(s, y)


def _plain_append(s):
    page, Hkv = s["c"]["page"], s["c"]["Hkv"]
    kept = s["slots"] >= 0
    at = s["slots"][kept]
    for name, rows in (("k", _plain_rows(s, s["k"], s["kw"])), ("v", s["v"].float())):
        codes, scale = _codes(rows[kept])
        s[name + "_cache"].view(torch.uint8).view(-1, Hkv, s["c"]["D"])[at] = codes.view(torch.uint8)
        s[name + "_scale"][at // page, :, at % page] = scale
    return _plain_rows(s, s["q"], s["qw"]).to(s["q"].dtype), s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


# ------------------------------------------------------------------------------------ floors
def work(case):
    """Bytes that a pass reads and writes once, and its operations."""
    c = case
    D, Hkv = c["D"], c["Hkv"]
    if c["kind"] == "append8":
        T = c["T"]
        small = T * 12 + c["rot"] * 4 + (2 * D * (4 if c["wdtype"] == "fp32" else 2) if c["norm"] else 0)
        return {"bytes": T * c["Hq"] * D * 4 + T * Hkv * (D * 6 + 8) + small,
                "flops": T * (c["Hq"] + 2 * Hkv) * D * (7 if c["norm"] else 3)}
    lens = _lengths(c)
    n = sum(lens)
    if c["kind"] == "read":
        row = 2 * D if c["bits"] == 16 else D + 4
        return {"bytes": 2 * n * Hkv * (row + 2 * D) + sum(-(-x // c["page"]) for x in lens) * 4 + c["B"] * 4,
                "flops": 2 * n * Hkv * D}
    io = c["B"] * c["Hq"] * (4 * D + 4) + c["B"] * 4
    if c["kind"] == "decode8":
        pages = sum(-(-x // c["page"]) for x in lens)
        return {"bytes": 2 * n * Hkv * (D + 4) + io + pages * 4, "flops": 4 * n * c["Hq"] * D}
    S = c["S"] // c["page"] * c["page"]
    n += (c["S"] - S) * c["B"]
    return {"bytes": 4 * (S + n) * Hkv * D + io + (S + n) // c["page"] * 4, "flops": 4 * D * c["Hq"] * (c["B"] * S + n)}


# ------------------------------------------------------------------------- 64-bit definitions
def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "append8":
        return _exact_append(s)
    if case["kind"] == "read":
        return _exact_read(s)
    return _exact_decode(s)


def _rows_of(s, name, ids, h, n):
    """The first n rows of head h in the pages `ids`, in 64 bits."""
    x = s[name + "_cache"][ids, :, h].double()
    if s.get(name + "_scale") is not None:
        x = x * s[name + "_scale"][ids, h].double()[..., None]
    return x.flatten(0, 1)[:n]


def _exact_decode(s):
    """Request by request: the softmax of its scores over all its pages, shared or its own."""
    q, page = s["q"].double(), s["k_cache"].shape[1]
    B, Hq, D = q.shape
    Hkv = s["k_cache"].shape[2]
    first = s.get("shared_pages", s["table"][0, :0]).long()
    o = torch.zeros(B, Hq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    m = first.numel() * page
    for h in range(Hkv):
        rows = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
        kf, vf = _rows_of(s, "k", first, h, m), _rows_of(s, "v", first, h, m)
        for b, n in enumerate(s["lens"].tolist()):
            ids = s["table"][b, first.numel(): -(-n // page)].long()
            k, v = torch.cat((kf, _rows_of(s, "k", ids, h, n - m))), torch.cat((vf, _rows_of(s, "v", ids, h, n - m)))
            if n:
                x = (q[b, rows] @ k.T) * D ** -0.5
                lse[b, rows] = torch.logsumexp(x, -1)
                o[b, rows] = torch.softmax(x, -1) @ v
    return o, lse


def _exact_read(s):
    page, out = s["k_cache"].shape[1], []
    for name in ("k", "v"):
        parts = []
        for b, n in enumerate(s["lens"].tolist()):
            ids = s["table"][b, : -(-n // page)].long()
            parts.append(torch.stack([_rows_of(s, name, ids, h, n) for h in range(s["c"]["Hkv"])], 1))
        out.append(torch.cat(parts))
    return out


def _exact_rows(s, x, w):
    """As complex numbers: each pair times exp(i * angle)."""
    rot = s["c"]["rot"]
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * w.double()
    if not rot:
        return x
    a = torch.outer(s["positions"].double(), s["inv_freq"])
    z = torch.polar(torch.full_like(a, s["rope_scale"]), a)[:, None]
    if s["c"]["inter"]:
        y = torch.view_as_real(torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
    else:
        y = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * z
        y = torch.cat((y.real, y.imag), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _nearest_e4m3(y):
    """The e4m3 value nearest to each of y (64 bits, |y| <= 448; ties to even)."""
    _, e = torch.frexp(y)                                      # |y| in [2^(e-1), 2^e)
    step = torch.ldexp(torch.ones_like(y), e.clamp(min=-5) - 4)
    return torch.round(y / step) * step


def _exact_append(s):
    page = s["c"]["page"]
    outs = [_exact_rows(s, s["q"].double(), s["qw"])]
    keep = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][keep]
    caches, scales = [], []
    for name, rows in (("k", _exact_rows(s, s["k"].double(), s["kw"])), ("v", s["v"].double())):
        y = rows[keep]
        top = y.abs().amax(-1)
        scale = torch.where(top == 0, torch.ones_like(top), top / 448)
        cache, old = s[name + "_cache"].double(), s[name + "_scale"].double()
        cache[at // page, at % page] = _nearest_e4m3(y / scale[..., None])
        old[at // page, :, at % page] = scale
        caches.append(cache)
        scales.append(old)
    return (*outs, *caches, *scales)
