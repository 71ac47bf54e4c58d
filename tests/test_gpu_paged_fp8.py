"""The paged cache of 8 bits a value on the GPU: append, decode and read back against 64-bit references;
the bounds are derived in paged_fp8_oracle.py."""
import math

import pytest
import torch

import exact_headdim_attention_gb300 as pkg
from tests import paged_fp8_oracle as p8
from tests import paged_oracle as po
from tests.gpu_util import device_ok
from tests.test_gpu_paged import close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, HF = torch.bfloat16, torch.float16
E4M3 = torch.float8_e4m3fn


def word_():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def dev(t):      # keeps the strides, unlike .to() of a transposed view
    return t.to(DEV) if t.is_contiguous() else t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)


def decode_case(lens, Hq, Hkv, D, page, dtype, seed=0, layout="psh", scale=None, spread=0.0, q_size=1.0):
    g = torch.Generator().manual_seed(seed)
    cache = p8.make_cache(g, lens, Hkv, D, page, layout=layout, spread=spread)
    q = (q_size * torch.randn(len(lens), Hq, D, generator=g)).to(dtype)
    return [q.to(DEV)] + [dev(t) for t in cache], p8.decode(q, *cache, scale)


def check_decode(args, ref, what="", scale=None, **kw):
    word = word_()
    o, lse = pkg.ffpa_decode_paged_fp8(*args, scale=scale, enable_gqa=True, return_lse=True, status=word, **kw)
    torch.cuda.synchronize()
    assert word.item() == pkg.FFPA_OK
    close(o, ref[0], ref[2], f"{what} O")
    close(lse, ref[1], ref[3], f"{what} LSE")
    return o, lse


# ------------------------------------------------------------------------------------ decode
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 80, 112, 128, 144, 192, 256, 272, 320, 384, 448, 512, 528, 640, 768, 912, 960, 1008, 1024])
def test_decode_head_dims(D, dtype):
    args, ref = decode_case([1, 0, 333, 17], 8, 2, D, 16, dtype, seed=D)
    check_decode(args, ref, f"D={D}")


@pytest.mark.parametrize("D", [64, 128, 320, 512, 768])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 6), (3, 1), (16, 2), (9, 1), (32, 2), (17, 1), (40, 1)])
def test_decode_groups(Hq, Hkv, D):
    args, ref = decode_case([5, 130, 64], Hq, Hkv, D, 32, BF, seed=Hq * 7 + D)
    check_decode(args, ref, f"Hq={Hq} Hkv={Hkv}")


@pytest.mark.parametrize("page", [1, 3, 8, 9, 16, 20, 60, 100, 130, 256, 999])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(4, 2, 64, HF), (4, 2, 512, BF), (2, 2, 208, BF), (40, 2, 128, HF), (8, 2, 1008, BF)])
def test_decode_page_sizes_and_lengths(page, Hq, Hkv, D, dtype):
    """Lengths around pages and tiles, empty requests at both ends of the batch."""
    lens = [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 255, 257, 0, page, page + 1, 3 * page + 7, 2 * page - 1, 0]
    args, ref = decode_case([min(n, 700) for n in lens], Hq, Hkv, D, page, dtype, seed=page + D)
    check_decode(args, ref, f"page={page}")


@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [1], [20000], [0, 9000, 1, 0, 700], [3000] * 5])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 256), (2, 2, 512), (12, 1, 64)])
def test_decode_splits(lens, Hq, Hkv, D):
    args, ref = decode_case(lens, Hq, Hkv, D, 64, HF, seed=len(lens) + lens[0])
    check_decode(args, ref, f"lens={lens}")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("page", [16, 20, 3])
def test_decode_scales_of_any_size(page, dtype):
    """Rows' scales that differ by 2^40: every one is weighed as it is."""
    args, ref = decode_case([700, 40, 3], 8, 2, 128, page, dtype, seed=page, spread=20.0, q_size=2.0 ** -12)
    if dtype == HF:   # outputs in fp16's range
        args[4].mul_(2.0 ** -12)
        ref = p8.decode(*[t.cpu() for t in args])
    check_decode(args, ref)


@pytest.mark.parametrize("size", [2.0 ** -60, 1.0, 2.0 ** 60])
def test_decode_bf16_queries_of_any_size(size):
    """Queries outside fp16's range, against keys whose scales bring the scores back."""
    args, _ = decode_case([300, 77], 4, 2, 256, 16, BF, seed=5, q_size=size)
    args[3].div_(size)
    check_decode(args, p8.decode(*[t.cpu() for t in args]))


def test_decode_queries_with_columns_of_many_sizes():
    args, _ = decode_case([300, 77], 4, 2, 512, 16, BF, seed=6)
    args[0].mul_(torch.exp2(-30 * torch.rand(512, device=DEV)).to(BF))
    check_decode(args, p8.decode(*[t.cpu() for t in args]))


@pytest.mark.parametrize("scale", [0.0, 0.5, -0.1])
def test_decode_softmax_scale(scale):
    args, ref = decode_case([100, 1, 300], 4, 2, 64, 16, BF, seed=12, scale=scale)
    check_decode(args, ref, scale=scale)


def test_decode_layouts():
    """Heads outside the slots, strided queries and outputs, a wider table, scales cut from a wider buffer."""
    args, ref = decode_case([40, 0, 700], 8, 2, 128, 16, BF, layout="phs", seed=9)
    q, kc, vc, ks, vs, table, n = args
    assert not kc.is_contiguous()
    wide = torch.full((3, 12, 128), math.nan, dtype=BF, device=DEV)
    wide[:, 2:10] = q
    out = torch.full((3, 16, 128), 7.0, dtype=BF, device=DEV)
    t2 = torch.full((3, 2 * table.shape[1] + 3), -9, dtype=torch.int32, device=DEV)
    t2[:, :table.shape[1]] = table
    both = torch.full((ks.shape[0], 5, 21), math.nan, device=DEV)
    both[:, :2, 3:19], both[:, 3:, 3:19] = ks, vs
    check_decode((wide[:, 2:10], kc, vc, both[:, :2, 3:19], both[:, 3:, 3:19], t2[:, :table.shape[1]], n), ref, "strided",
                 out=out[:, 4:12])
    assert (out[:, :4] == 7).all() and (out[:, 12:] == 7).all()


def test_decode_nothing_cached_and_empty_batch():
    q = torch.randn(2, 4, 64, device=DEV).to(BF)
    kc, ks = torch.empty(0, 16, 2, 64, dtype=E4M3, device=DEV), torch.empty(0, 2, 16, device=DEV)
    table, n = torch.zeros(2, 0, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    o, lse = pkg.ffpa_decode_paged_fp8(q, kc, kc, ks, ks, table, n, enable_gqa=True, return_lse=True)
    assert (o == 0).all() and (lse == -math.inf).all()
    assert pkg.ffpa_decode_paged_fp8(q[:0], kc, kc, ks, ks, table[:0], n[:0], enable_gqa=True).shape == (0, 4, 64)
    device_ok()


@pytest.mark.parametrize("page,D", [(16, 64), (16, 512), (100, 512), (20, 1008), (3, 128)])
def test_decode_bad_pages_are_reported_and_count_as_zeros(page, D):
    args, _ = decode_case([3 * page + 7, page, 2 * page - 1], 4, 2, D, page, BF, seed=D)
    q, kc, vc, ks, vs, table, n = args
    for b, bad in [(0, -1), (2, kc.shape[0]), (1, 2**31 - 1)]:
        t2, word = table.clone(), word_()
        t2[b, 0] = bad
        o = pkg.ffpa_decode_paged_fp8(q, kc, vc, ks, vs, t2, n, enable_gqa=True, status=word)
        assert word.item() == pkg.FFPA_ERR_INVALID
        zero = lambda x: torch.cat((x.view(torch.uint8) if x.dtype == E4M3 else x,     # noqa: E731
                                    torch.zeros_like(x[:1].view(torch.uint8) if x.dtype == E4M3 else x[:1])))
        t2[b, 0] = kc.shape[0]
        want = pkg.ffpa_decode_paged_fp8(q, zero(kc).view(E4M3), zero(vc).view(E4M3), zero(ks), zero(vs), t2, n, enable_gqa=True)
        assert torch.equal(o, want)
    word = word_()
    n2 = torch.tensor([-3, page, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    t2 = torch.where(table < 0, torch.zeros_like(table), table)
    k0 = torch.nan_to_num(kc.float()).to(E4M3)
    v0 = torch.nan_to_num(vc.float()).to(E4M3)
    o = pkg.ffpa_decode_paged_fp8(q, k0, v0, torch.nan_to_num(ks), torch.nan_to_num(vs), t2, n2, enable_gqa=True, status=word)
    assert word.item() == pkg.FFPA_ERR_INVALID and (o[0] == 0).all() and torch.isfinite(o).all()
    device_ok()


@pytest.mark.parametrize("D,page", [(64, 3), (512, 16), (512, 100), (1008, 20), (208, 16)])
def test_decode_ends_when_a_wait_runs_out(D, page):
    args, ref = decode_case([300, 20, 0, 900], 4, 2, D, page, BF, seed=D + page)
    word = word_()
    pkg.ffpa_decode_paged_fp8(*args, enable_gqa=True, status=word, wait_timeout_ns=3_000_000, test_drop_first_copy=True)
    torch.cuda.synchronize()
    assert word.item() == pkg.FFPA_ERR_DEVICE_TIMEOUT
    check_decode(args, ref)
    device_ok()


def test_decode_twice_is_the_same_and_captured_lengths_may_change():
    args, ref = decode_case([900, 3, 0, 2000, 411], 8, 2, 256, 16, BF, seed=3)
    a, la = check_decode(args, ref)
    b, lb = check_decode(args, ref)
    assert torch.equal(a, b) and torch.equal(la, lb)
    n, side = args[6].clone(), torch.cuda.Stream()
    lens = args[6].clone()
    with torch.cuda.stream(side):
        pkg.ffpa_decode_paged_fp8(*args[:6], lens, enable_gqa=True)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            o = pkg.ffpa_decode_paged_fp8(*args[:6], lens, enable_gqa=True)
        graph.replay()
        side.synchronize()
        assert torch.equal(o, a)
        lens.copy_(torch.tensor([1, 0, 0, 77, 411], dtype=torch.int32))
        graph.replay()
        side.synchronize()
    assert torch.equal(o, pkg.ffpa_decode_paged_fp8(*args[:6], lens, enable_gqa=True))
    assert torch.equal(o[4], a[4]) or (o[4] - a[4]).abs().max() < 0.01
    assert torch.equal(n, args[6])


# ------------------------------------------------------------------------------------ append
def append_case(T, Hq, Hkv, D, page, pages, dtype, rot, norm, seed, wdtype=torch.float32, layout="psh"):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pos = torch.randint(0, 1 << 18, (T,), generator=g)
    inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2)) if rot else None
    w = (1 + 0.2 * torch.randn(2, D, generator=g)).to(wdtype) if norm else (None, None)
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[torch.rand(T, generator=g) < 0.1] = -1
    return q, k, v, pos, inv, w, slots


def run_append(case, page, pages, q_too=True, layout="psh", **kw):
    q, k, v, pos, inv, w, slots = case
    Hkv, D = k.shape[1], k.shape[2]
    shape = (pages, page, Hkv, D) if layout == "psh" else (pages, Hkv, page, D)
    kc, vc = (torch.full(shape, 0x7f, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2))
    if layout == "phs":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    ks, vs = torch.full((2, pages, Hkv, page), -7.0, device=DEV)
    word = word_()
    d = lambda t: None if t is None else t.to(DEV)   # noqa: E731
    qkv = torch.cat((q, k, v), 1).to(DEV)
    Hq = q.shape[1]
    out = pkg.ffpa_kv_append_fp8(qkv[:, :Hq] if q_too else None, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], kc, vc, ks, vs, d(slots),
                                 d(pos) if inv is not None else None, d(inv), d(w[0]) if q_too else None, d(w[1]), status=word,
                                 **kw)
    torch.cuda.synchronize()
    return out, kc, vc, ks, vs, word.item()


def check_append(case, got, interleaved=False, rope_scale=1.0):
    q, k, v, pos, inv, w, slots = case
    out, kc, vc, ks, vs, word = got
    assert word == pkg.FFPA_OK
    if out is not None:
        y, bound = po.rope_bound(q, pos, inv, w[0], interleaved=interleaved, rope_scale=rope_scale)
        close(out, y, bound, "queries")
    page, kept = kc.shape[1], slots >= 0
    at = slots[kept]
    yk, kb = po.rope_bound(k, pos, inv, w[1], interleaved=interleaved, rope_scale=rope_scale)
    off = (kb - po.half_step(k.dtype) * yk.abs()).clamp(min=0)          # without the rounding to 16 bits
    if inv is None and w[1] is None:
        off = torch.zeros_like(off)
    for cache, scale, y, far in ((kc, ks, yk, off), (vc, vs, v.double(), torch.zeros(v.shape, dtype=torch.float64))):
        rows = cache.cpu().view(torch.uint8)[at // page, at % page].view(E4M3)
        p8.check_codes(rows, scale.cpu()[at // page, :, at % page], y[kept], far[kept])
        left = torch.ones(cache.shape[:2], dtype=torch.bool)
        left[at // page, at % page] = False
        assert (cache.cpu().view(torch.uint8)[left] == 0x7f).all() and (scale.cpu().transpose(1, 2)[left] == -7).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,rot", [(64, 64), (80, 40), (112, 112), (128, 64), (144, 0), (208, 104), (256, 256), (320, 160),
                                   (512, 512), (528, 8), (640, 640), (768, 256), (1008, 1008), (1024, 1024)])
def test_append_head_dims(D, rot, dtype):
    case = append_case(37, 3, 2, D, 16, 5, dtype, rot, True, D)
    for inter in (False, True):
        check_append(case, run_append(case, 16, 5, interleaved=inter), inter)


@pytest.mark.parametrize("T,Hq,Hkv,page,pages", [(1, 1, 1, 1, 3), (2, 40, 5, 3, 4), (600, 8, 8, 32, 20), (33, 32, 1, 100, 1)])
@pytest.mark.parametrize("norm", [True, False])
def test_append_shapes(T, Hq, Hkv, page, pages, norm):
    case = append_case(T, Hq, Hkv, 128, page, pages, BF, 64, norm, T, wdtype=BF)
    check_append(case, run_append(case, page, pages, rope_scale=1.25), rope_scale=1.25)
    check_append(case, run_append(case, page, pages, q_too=False, layout="phs"))


@pytest.mark.parametrize("dtype", [BF, HF])
def test_append_rows_as_they_are(dtype):
    """Without norm and rotation the codes are those of the rows themselves; zeros, tiny and large rows among them."""
    case = append_case(50, 2, 3, 192, 16, 4, dtype, 0, False, 11)
    k, v = case[1], case[2]
    k[3], v[4, 1], k[5, 0] = 0.0, 0.0, -0.0
    k[6] *= 2.0 ** -14
    v[7] *= 2.0 ** 11
    if dtype == BF:
        k[8] *= 2.0 ** -100
        v[9] *= 2.0 ** 100
    k[10, 0, :] = 0.0
    k[10, 0, 7] = 1.5
    v[11, 0] = 3.0
    got = run_append(case, 16, 4)
    check_append(case, got)
    assert torch.isfinite(got[1].float()[got[3].transpose(1, 2) != -7]).all()


def test_append_smallest_rows():
    """Rows below 2^-117 keep a normal scale and finite codes."""
    case = append_case(4, 1, 1, 64, 16, 1, BF, 0, False, 12)
    case[1][:] = torch.randn(4, 1, 64).to(BF) * 2.0 ** -125
    case[6][:] = torch.arange(4)
    out, kc, vc, ks, vs, word = run_append(case, 16, 1)
    y = kc[0, :4].float().cpu().double() * ks[0, :, :4].t().cpu().double()[..., None]
    assert ((y - case[1].double()).abs() <= 2.0 ** -10 * 2.0 ** -117 / 448 * 1.01 + 2.0 ** -4 * case[1].double().abs()).all()
    assert (ks[0, :, :4] > 0).all() and word == pkg.FFPA_OK


def test_append_slots_beyond_the_cache_are_reported():
    case = append_case(20, 2, 2, 64, 16, 2, BF, 64, True, 13)
    case[6][:] = torch.arange(20)
    case[6][3], case[6][4], case[6][5] = 32, 2 ** 62, -2 ** 63
    out, kc, vc, ks, vs, word = run_append(case, 16, 2)
    assert word == pkg.FFPA_ERR_INVALID
    ok = tuple(t if i != 6 else torch.where((t < 0) | (t >= 32), torch.full_like(t, -1), t) for i, t in enumerate(case))
    check_append(ok, (out, kc, vc, ks, vs, pkg.FFPA_OK))
    device_ok()


def test_append_into_strided_scales():
    """Scales cut from a wider buffer, keys' and values' halves of one."""
    case = append_case(40, 2, 2, 128, 16, 4, BF, 64, True, 15)
    q, k, v, pos, inv, w, slots = case
    d = lambda t: t.to(DEV)   # noqa: E731
    both = torch.full((4, 2, 3, 19), -7.0, device=DEV)
    ks, vs = both[:, 0, :2, 1:17], both[:, 1, 1:, 3:]
    cache = torch.full((4, 16, 2, 2, 128), 0x7f, dtype=torch.uint8, device=DEV).view(E4M3)
    kc, vc = cache[:, :, 0], cache[:, :, 1]
    word = word_()
    out = pkg.ffpa_kv_append_fp8(d(q), d(k), d(v), kc, vc, ks, vs, d(slots), d(pos), d(inv), d(w[0]), d(w[1]), status=word)
    torch.cuda.synchronize()
    check_append(case, (out, kc, vc, ks, vs, word.item()))
    assert (both[:, 0, 2] == -7).all() and (both[:, 1, 0] == -7).all() and (both[..., 0] == -7).all() and (both[:, 0, :, 17:] == -7).all()


def test_append_agrees_with_the_16_bit_append():
    """The same rows in a 16-bit cache: queries equal bit for bit, keys within half a step of e4m3 and of bf16."""
    case = append_case(60, 4, 2, 512, 16, 6, BF, 512, True, 14)
    out, kc, vc, ks, vs, _ = run_append(case, 16, 6)
    q, k, v, pos, inv, w, slots = case
    d = lambda t: t.to(DEV)   # noqa: E731
    k16, v16 = torch.zeros(2, 6, 16, 2, 512, dtype=BF, device=DEV)
    q16 = pkg.ffpa_kv_append(d(q), d(k), d(v), k16, v16, d(slots), d(pos), d(inv), d(w[0]), d(w[1]))
    assert torch.equal(out, q16)
    at = d(slots[slots >= 0])
    for c, s, x in ((kc, ks, k16), (vc, vs, v16)):
        y = c.view(torch.uint8)[at // 16, at % 16].view(E4M3).float() * s[at // 16, :, at % 16][..., None]
        ref = x[at // 16, at % 16].float()
        far = 2.0 ** -4 * ref.abs() * (1 + 2.0 ** -7) + 2.0 ** -10 * s[at // 16, :, at % 16][..., None] + 2.0 ** -8 * ref.abs()
        assert ((y - ref).abs() <= far).all()


# -------------------------------------------------------------------------------------- read
def read_case(lens, Hkv, D, page, seed, codes=True, dtype=BF, layout="psh"):
    g = torch.Generator().manual_seed(seed)
    if codes:
        kc, vc, ks, vs, table, n = p8.make_cache(g, lens, Hkv, D, page, layout=layout)
    else:
        kc, vc, table, n = po.make_cache(g, lens, Hkv, D, page, dtype, layout=layout)
        ks = vs = None
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(n, 0)
    return kc, vc, ks, vs, table, n, cu


def check_read(case, dtype, spare=0, **kw):
    kc, vc, ks, vs, table, n, cu = case
    T = int(cu[-1]) + spare
    k, v = torch.full((2, T, *kc.shape[2:]), 9.0, dtype=dtype, device=DEV)
    word = word_()
    d = lambda t: None if t is None else t.to(DEV)   # noqa: E731
    got = pkg.ffpa_kv_read(dev(kc), dev(vc), table.to(DEV), cu.to(DEV), T, k_scale=d(ks), v_scale=d(vs), dtype=dtype, k_out=k,
                           v_out=v, status=word, **kw)
    torch.cuda.synchronize()
    assert word.item() == pkg.FFPA_OK and got[0] is k and got[1] is v
    for out, c, s in ((k, kc, ks), (v, vc, vs)):
        y, bound = p8.read(c, s, table, n, dtype)
        if s is None:
            assert torch.equal(out[:T - spare].cpu().double(), y)
        else:
            close(out[:T - spare], y, bound, "rows")
        assert (out[T - spare:] == 9).all()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("codes", [True, False])
@pytest.mark.parametrize("D", [64, 80, 128, 320, 512, 1008, 1024])
def test_read_head_dims(D, codes, dtype):
    check_read(read_case([5, 0, 77, 16, 1], 3, D, 16, D, codes, dtype), dtype, spare=3)


@pytest.mark.parametrize("page", [1, 3, 16, 100])
@pytest.mark.parametrize("lens", [[1], [0, 0, 7, 0], [700] * 3, [0, 1, 0, 0, 5000, 2], list(range(60))])
@pytest.mark.parametrize("Hkv,D,codes", [(1, 64, True), (8, 128, True), (2, 72, False)])
def test_read_lengths_and_pages(lens, page, Hkv, D, codes):
    check_read(read_case(lens, Hkv, D, page, page + len(lens), codes, HF, layout="phs" if page == 16 else "psh"), HF, spare=page % 2)


def test_read_into_strided_rows():
    """Outputs as slices of one buffer of keys and values."""
    kc, vc, ks, vs, table, n, cu = read_case([20, 0, 33], 2, 128, 16, 5)
    both = torch.full((60, 5, 128), 9.0, dtype=BF, device=DEV)
    k, v = both[:53, :2], both[:53, 3:]
    d = [t.to(DEV) for t in (kc, vc, table, cu, ks, vs)]
    pkg.ffpa_kv_read(*d[:4], 53, k_scale=d[4], v_scale=d[5], k_out=k, v_out=v)
    device_ok()
    close(k, *p8.read(kc, ks, table, n, BF), "k")
    close(v, *p8.read(vc, vs, table, n, BF), "v")
    assert (both[:, 2] == 9).all() and (both[53:] == 9).all()


def test_read_defaults_and_nothing():
    kc, vc, ks, vs, table, n, cu = read_case([9, 30], 2, 128, 16, 3)
    d = [t.to(DEV) for t in (kc, vc, table, cu, ks, vs)]
    k, v = pkg.ffpa_kv_read(*d[:4], 39, k_scale=d[4], v_scale=d[5])
    assert k.dtype == BF and k.shape == (39, 2, 128)
    assert pkg.ffpa_kv_read(*d[:4], 0, k_scale=d[4], v_scale=d[5])[0].shape == (0, 2, 128)
    close(k, *p8.read(kc, ks, table, n, BF), "k")
    device_ok()


def test_read_reports_what_is_out_of_range():
    kc, vc, ks, vs, table, n, cu = read_case([20, 30, 40], 2, 64, 16, 4)
    kc, ks = torch.nan_to_num(kc.float()).to(E4M3), torch.nan_to_num(ks)

    def run(table, cu, T=90):
        word = word_()
        k, v = torch.full((2, T, 2, 64), 9.0, dtype=BF, device=DEV)
        pkg.ffpa_kv_read(kc.to(DEV), kc.to(DEV), table.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV), T, k_scale=ks.to(DEV),
                         v_scale=ks.to(DEV), k_out=k, v_out=v, status=word)
        torch.cuda.synchronize()
        return word.item(), k

    good, rows = run(table, [0, 20, 50, 90])
    assert good == pkg.FFPA_OK
    for bad in (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31):
        t2 = table.clone()
        t2[1, 1] = bad
        word, k = run(t2, [0, 20, 50, 90])
        assert word == pkg.FFPA_ERR_INVALID
        assert torch.equal(k[:36], rows[:36]) and (k[36:50] == 0).all() and torch.equal(k[50:], rows[50:])
    for cu in ([0, 20, 50, 91], [0, 20, 10, 90], [0, -5, 50, 90], [-3, 20, 50, 90], [-2 ** 31, 2 ** 31 - 1, 50, 90]):
        assert run(torch.where(table < 0, 0, table), cu)[0] == pkg.FFPA_ERR_INVALID
    word, k = run(table[:, :2].contiguous(), [0, 20, 50, 90])                # 40 rows, two pages
    assert word == pkg.FFPA_ERR_INVALID and torch.equal(k[:82], rows[:82]) and (k[82:] == 9).all()
    word, k = run(torch.zeros(3, 0, dtype=torch.int32), [0, 0, 0, 0])
    assert word == pkg.FFPA_OK and (k == 9).all()
    device_ok()


# ---------------------------------------------------------------------------------- together
@pytest.mark.parametrize("dtype", [BF, HF])
def test_generation_steps_with_a_quantised_cache(dtype):
    """Prompts, then single tokens: plan, append, the prompt's attention over what is read back, decode.  Every
    result is that of 64-bit attention over the values that the cache holds."""
    g = torch.Generator().manual_seed(21)
    Hq, Hkv, D, page, pool = 4, 2, 128, 16, 40
    kc, vc = torch.zeros(2, pool, page, Hkv, D, device=DEV).to(E4M3)
    ks, vs = torch.ones(2, pool, Hkv, page, device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)   # noqa: E731
    table, lens = torch.full((3, 9), -1, dtype=torch.int32, device=DEV), i32([0, 0, 0])
    free, left = torch.randperm(pool, generator=g).to(torch.int32).to(DEV), i32([pool])
    inv, scale = pkg.rope_inv_freq(D, device="cuda")
    for new in ([37, 0, 90], [1, 1, 0], [20, 1, 1], [1, 1, 1]):
        T = sum(new)
        slots, pos, cu, lens, left = pkg.ffpa_page_plan(table, lens, i32(new), free, left, page, T)
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dtype).to(DEV)
        q = pkg.ffpa_kv_append_fp8(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], kc, vc, ks, vs, slots, pos, inv)
        held = lens.tolist()
        cu_k = i32([0] + torch.cumsum(lens, 0).tolist())
        k, v = pkg.ffpa_kv_read(kc, vc, table, cu_k, sum(held), k_scale=ks, v_scale=vs, dtype=dtype)
        o = pkg.ffpa_attn_varlen_func(q, k, v, cu, cu_k, max(new), max(held), causal=True, enable_gqa=True)
        last = (cu[1:] - 1).clamp(min=0)
        od, lse = pkg.ffpa_decode_paged_fp8(q[last], kc, vc, ks, vs, table, lens, enable_gqa=True, return_lse=True)
        cache = [t.cpu() for t in (kc, vc, ks, vs, table, lens)]
        ref = p8.decode(q[last].cpu(), *cache)
        close(od, ref[0], ref[2], "decode")
        for b, n in enumerate(new):
            if n:   # the last row of a prompt's attention: the rows were rounded once more, and its weights
                err = (o[last[b]].double().cpu() - ref[0][b]).abs()
                assert err.max() <= 2e-2 and err.mean() <= 2e-3
    device_ok()


def test_torch_operators():
    args, ref = decode_case([40, 0, 130], 8, 2, 128, 16, BF, seed=31)
    o, lse = pkg.ffpa_attn_decode_fp8_func(*args, enable_gqa=True, return_lse=True)
    close(o, ref[0], ref[2], "O")
    q, kc, vc, ks, vs, table, n = args
    cu = torch.tensor([0, 40, 40, 170], dtype=torch.int32, device=DEV)
    k, v = pkg.ffpa_kv_read_func(kc, vc, table, cu, 170, k_scale=ks, v_scale=vs, dtype=HF)
    k2, v2 = pkg.ffpa_kv_read(kc, vc, table, cu, 170, k_scale=ks, v_scale=vs, dtype=HF)
    assert torch.equal(k, k2) and torch.equal(v, v2) and k.dtype == HF
    rows = torch.randn(3, 2, 128, device=DEV).to(BF)
    slots = torch.tensor([0, -1, 5], device=DEV)
    a, b = [t.clone() for t in (kc, vc, ks, vs)], [t.clone() for t in (kc, vc, ks, vs)]
    assert pkg.ffpa_kv_append_fp8_func(None, rows, rows, *a, slots) is None
    assert pkg.ffpa_kv_append_fp8(None, rows, rows, *b, slots) is None
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    step = torch.compile(lambda q: pkg.ffpa_attn_decode_fp8_func(q * 1, kc, vc, ks, vs, table, n, enable_gqa=True), backend="eager",
                         fullgraph=True)
    assert torch.equal(step(q), o)
    device_ok()


def test_calls_on_a_stream_of_the_callers():
    args, ref = decode_case([3000, 1, 0, 800], 8, 2, 256, 16, BF, seed=18)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = pkg.ffpa_decode_paged_fp8(*args, enable_gqa=True, stream=side)
    q, kc, vc, ks, vs, table, n = args
    cu = torch.tensor([0, 3000, 3001, 3001, 3801], dtype=torch.int32, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    k, v = pkg.ffpa_kv_read(kc, vc, table, cu, 3801, k_scale=ks, v_scale=vs, stream=side)
    side.synchronize()
    close(o, ref[0], ref[2], "O")
    assert torch.equal(k, pkg.ffpa_kv_read(kc, vc, table, cu, 3801, k_scale=ks, v_scale=vs)[0])
    device_ok()
