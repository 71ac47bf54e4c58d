"""Decode attention over a paged cache, cache append and page plan on the GPU against 64-bit (or
plain integer) references; the error bounds are derived in paged_oracle.py."""
import math
import threading

import pytest
import torch

import exact_headdim_attention_gb300 as pkg
from tests import paged_oracle as po
from tests.gpu_util import device_ok

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, HF = torch.bfloat16, torch.float16


def status_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def close(got, want, bound, what):
    got, want, bound = got.double().cpu(), want.cpu(), bound.cpu()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"{what}: finite values differ"
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine].nan_to_num(nan=7.0), want[~fine].nan_to_num(nan=7.0)), what
    over = ((got - want).abs() - bound)[fine]
    assert over.numel() == 0 or over.max() <= 0, f"{what}: {over.max().item():.3e} beyond the bound"


def decode_case(lens, Hq, Hkv, D, page, dtype, seed=0, layout="psh", scale=None):
    g = torch.Generator().manual_seed(seed)
    kc, vc, table, n = po.make_cache(g, lens, Hkv, D, page, dtype, layout=layout)
    q = torch.randn(len(lens), Hq, D, generator=g).to(dtype)
    ref = po.decode(q, kc, vc, table, n, scale)

    def dev(t):      # keeps the strides, unlike .to() of a transposed view
        return t.to(DEV) if t.is_contiguous() else t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)

    return (q.to(DEV), dev(kc), dev(vc), table.to(DEV), n.to(DEV)), ref


def check_decode(args, ref, what="", scale=None, **kw):
    word = status_word()
    o, lse = pkg.ffpa_decode_paged(*args, scale=scale, enable_gqa=True, return_lse=True, status=word, **kw)
    torch.cuda.synchronize()
    assert word.item() == pkg.FFPA_OK
    close(o, ref[0], ref[2], f"{what} O")
    close(lse, ref[1], ref[3], f"{what} LSE")
    return o, lse


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 72, 120, 128, 192, 256, 320, 384, 448, 512, 520, 576, 640, 704, 768, 832, 896, 960, 1016, 1024])
def test_decode_head_dims(D, dtype):
    args, ref = decode_case([1, 0, 333, 17], 8, 2, D, 16, dtype, seed=D)
    check_decode(args, ref, f"D={D}")


@pytest.mark.parametrize("D", [64, 128, 320, 512, 768])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 6), (3, 1), (16, 2), (9, 1), (32, 2), (17, 1), (40, 1), (66, 2)])
def test_decode_groups(Hq, Hkv, D):
    args, ref = decode_case([5, 130, 64], Hq, Hkv, D, 32, BF, seed=Hq * 7 + D)
    check_decode(args, ref, f"Hq={Hq} Hkv={Hkv}")


@pytest.mark.parametrize("page", [9, 20, 60, 130, 250, 999])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (2, 2, 200), (6, 1, 320), (40, 2, 512), (8, 2, 1000)])
def test_decode_tiles_that_end_with_their_page(page, Hq, Hkv, D):
    """Page sizes that are no multiple of 8: smaller than half a tile, than a tile, and of several."""
    lens = [page - 1, page, page + 1, 0, 3 * page + 7, 1, 2 * page - 1, 1111, 5 * page]
    args, ref = decode_case(lens, Hq, Hkv, D, page, HF if D == 320 else BF, seed=page + D)
    check_decode(args, ref, f"page={page} D={D}")


@pytest.mark.parametrize("page", [1, 3, 8, 16, 100, 256])
@pytest.mark.parametrize("D", [64, 512])
def test_decode_page_sizes_and_lengths(page, D):
    """Lengths around pages and tiles, and empty requests at both ends of the batch."""
    lens = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 255, 256, 257, 0, page, page + 1, 2 * page, 511, 0]
    args, ref = decode_case(lens, 4, 2, D, page, BF, seed=page)
    check_decode(args, ref, f"page={page}")


@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [1], [20000], [0, 9000, 1, 0, 700], [3000] * 5])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 1, 256), (2, 2, 512)])
def test_decode_splits(lens, Hq, Hkv, D):
    """Requests shared by many CTAs, CTAs shared by many requests, batches with nothing to do."""
    args, ref = decode_case(lens, Hq, Hkv, D, 64, HF, seed=len(lens) + lens[0])
    check_decode(args, ref, f"lens={lens}")


def test_decode_many_requests():
    """More requests than threads in a block, most of them empty or short."""
    g = torch.Generator().manual_seed(3)
    lens = [int(x) if x > 0 else 0 for x in torch.randint(-20, 40, (900,), generator=g)]
    args, ref = decode_case(lens, 2, 1, 64, 8, BF, seed=4)
    check_decode(args, ref)


def test_decode_layouts():
    """Heads outside the slots, queries cut from a projection, a strided output, a wider table."""
    args, ref = decode_case([40, 0, 700], 8, 2, 128, 16, BF, layout="phs", seed=9)
    q, kc, vc, table, n = args
    assert not kc.is_contiguous()
    wide = torch.full((3, 12, 128), math.nan, dtype=BF, device=DEV)
    wide[:, 2:10] = q
    out = torch.full((3, 16, 128), 7.0, dtype=BF, device=DEV)
    t2 = torch.full((3, 2 * table.shape[1] + 3), -9, dtype=torch.int32, device=DEV)
    t2[:, :table.shape[1]] = table
    check_decode((wide[:, 2:10], kc, vc, t2[:, :table.shape[1]], n), ref, "strided", out=out[:, 4:12])
    assert (out[:, :4] == 7).all() and (out[:, 12:] == 7).all()
    # keys and values as two halves of one buffer with different strides
    both = torch.empty(kc.shape[0], 2, *kc.shape[1:], dtype=BF, device=DEV)
    both[:, 0], both[:, 1] = kc, vc
    check_decode((q, both[:, 0], vc, table, n), ref, "mixed strides")
    check_decode((q, both[:, 0], both[:, 1], table, n), ref, "halves")


@pytest.mark.parametrize("scale", [0.0, 0.5, -0.1])
def test_decode_scales(scale):
    args, ref = decode_case([100, 1, 300], 4, 2, 64, 16, BF, seed=12, scale=scale)
    check_decode(args, ref, scale=scale)


def test_decode_default_arguments():
    args, ref = decode_case([50, 90], 4, 4, 128, 16, BF, seed=13)
    o = pkg.ffpa_decode_paged(*args)
    device_ok()
    close(o, ref[0], ref[2], "O")
    ws = torch.empty(pkg.decode_paged_workspace_bytes(4, 4, 128), dtype=torch.uint8, device=DEV)
    lse = torch.full((2, 4), 3.0, device=DEV)
    o2, l2 = pkg.ffpa_decode_paged(*args, workspace=ws, lse=lse, return_lse=True)
    assert torch.equal(o, o2) and l2 is lse
    close(l2, ref[1], ref[3], "LSE")
    empty = pkg.ffpa_decode_paged(args[0][:0], *args[1:3], args[3][:0], args[4][:0])
    assert empty.shape == (0, 4, 128)


def test_decode_nothing_cached_at_all():
    q = torch.randn(2, 4, 64, device=DEV).to(BF)
    kc = torch.empty(0, 16, 2, 64, dtype=BF, device=DEV)
    table, n = torch.zeros(2, 0, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    o, lse = pkg.ffpa_decode_paged(q, kc, kc, table, n, enable_gqa=True, return_lse=True)
    assert (o == 0).all() and (lse == -math.inf).all()
    device_ok()


def test_decode_infinities_and_nan():
    """An infinite key gives what the formula gives (NaN for its rows), a NaN value its column;
    scores of -inf alone leave the row empty, as the library's other kernels do."""
    args, ref = decode_case([40, 40, 40], 2, 1, 64, 16, BF, seed=14)
    q, kc, vc, table, n = args
    q[0, :, 0] = 1.0
    kc[table[0, 1].item(), 3, 0, 0] = math.inf
    vc[table[1, 0].item(), 2, 0, 5] = math.nan
    q[2, :, 0] = 1.0
    for j in range(3):
        kc[table[2, j].item(), :, 0, 0] = -math.inf
    o, lse = pkg.ffpa_decode_paged(q, kc, vc, table, n, enable_gqa=True, return_lse=True)
    assert torch.isnan(o[0]).all()
    assert torch.isnan(o[1, :, 5]).all() and torch.isfinite(o[1, :, :5]).all() and torch.isfinite(o[1, :, 6:]).all()
    assert (o[2] == 0).all() and (lse[2] == -math.inf).all()


def test_decode_bad_pages_and_lengths_are_reported_and_not_followed():
    args, _ = decode_case([40, 40, 50], 2, 1, 64, 16, BF, seed=15)
    q, kc, vc, table, n = args
    kc, vc = torch.nan_to_num(kc), torch.nan_to_num(vc)
    good = pkg.ffpa_decode_paged(q, kc, vc, table, n, enable_gqa=True)
    for bad in (kc.shape[0], -1, -2 ** 31, 2 ** 31 - 1):
        t2, word = table.clone(), status_word()
        t2[1, 1] = bad
        o = pkg.ffpa_decode_paged(q, kc, vc, t2, n, enable_gqa=True, status=word)
        assert word.item() == pkg.FFPA_ERR_INVALID
        assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
        # its 16 keys count as zeros
        k0, v0 = torch.cat((kc, torch.zeros_like(kc[:1]))), torch.cat((vc, torch.zeros_like(vc[:1])))
        t2[1, 1] = kc.shape[0]
        assert torch.equal(o, pkg.ffpa_decode_paged(q, k0, v0, t2, n, enable_gqa=True))
    assert pkg.ffpa_last_device_error() == pkg.FFPA_OK
    n2 = torch.tensor([-3, 40, 50], dtype=torch.int32, device=DEV)
    o = pkg.ffpa_decode_paged(q, kc, vc, table, n2, enable_gqa=True)       # no word: the device's fallback word
    assert pkg.ffpa_last_device_error() == pkg.FFPA_ERR_INVALID
    assert (o[0] == 0).all() and torch.equal(o[1:], good[1:])
    narrow = table[:, :3].contiguous()
    word = status_word()
    o = pkg.ffpa_decode_paged(q, kc, vc, narrow, torch.tensor([40, 40, 1000], dtype=torch.int32, device=DEV), enable_gqa=True, status=word)
    assert word.item() == pkg.FFPA_ERR_INVALID
    want = pkg.ffpa_decode_paged(q, kc, vc, narrow, torch.tensor([40, 40, 48], dtype=torch.int32, device=DEV), enable_gqa=True)
    assert torch.equal(o, want)
    device_ok()


@pytest.mark.parametrize("page,D", [(100, 512), (20, 1000), (100, 64)])
def test_decode_bad_pages_of_any_size(page, D):
    """A page that does not exist counts as keys and values of zeros, and is reported."""
    args, _ = decode_case([3 * page + 7, page, 2 * page - 1], 4, 2, D, page, BF, seed=D)
    q, kc, vc, table, n = args
    for b, bad in [(0, -1), (2, kc.shape[0]), (1, 2**31 - 1)]:
        word = status_word()
        broken, k0, v0 = table.clone(), kc.clone(), vc.clone()
        broken[b, 0] = bad
        k0[table[b, 0]] = 0
        v0[table[b, 0]] = 0
        got = pkg.ffpa_decode_paged(q, kc, vc, broken, n, enable_gqa=True, status=word)
        assert word.item() == pkg.FFPA_ERR_INVALID
        assert torch.equal(got, pkg.ffpa_decode_paged(q, k0, v0, table, n, enable_gqa=True))


@pytest.mark.parametrize("page", [16, 100])
@pytest.mark.parametrize("D", [200, 512])
def test_decode_strides_of_single_entries_are_free(page, D):
    """One key head, and one page: their strides are never used and may be anything."""
    args, ref = decode_case([page - 3], 4, 1, D, page, BF, seed=D + page)
    q, kc, vc, table, n = args
    kc, vc = (x[:1].contiguous() for x in (kc[table[0, 0]:], vc[table[0, 0]:]))
    odd = [x.as_strided(x.shape, (5, D, 3, 1)) for x in (kc, vc)]
    check_decode((q, *odd, torch.zeros_like(table), n), ref, f"page={page} D={D}")


def test_decode_pages_beyond_32_bit_offsets():
    """A cache of 2^31 + elements whose used pages lie at its end."""
    Hkv, D, page = 2, 512, 16
    pool = (1 << 31) // (page * Hkv * D) + 64
    kc, vc = (torch.empty(pool, page, Hkv, D, dtype=BF, device=DEV) for _ in range(2))
    g = torch.Generator().manual_seed(17)
    k, v, table, n = po.make_cache(g, [700, 33], Hkv, D, page, BF)
    q = torch.randn(2, 4, D, generator=g).to(BF)
    ref = po.decode(q, k, v, table, n)
    base = pool - k.shape[0]
    kc[base:], vc[base:] = k.to(DEV), v.to(DEV)
    t = torch.where(table >= 0, table + base, table).to(DEV)
    check_decode((q.to(DEV), kc, vc, t, n.to(DEV)), ref, "far pages")


def test_decode_is_repeatable_on_streams_and_in_graphs():
    """The same bits from call to call, on a side stream, from two threads, and from two captured
    graphs whose lengths change between replays."""
    args, ref = decode_case([3000, 1, 0, 800], 8, 2, 256, 16, BF, seed=18)
    q, kc, vc, table, n = args
    first = check_decode(args, ref)
    assert all(torch.equal(a, b) for a, b in zip(first, check_decode(args, ref)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pkg.ffpa_decode_paged(*args, enable_gqa=True, stream=side)
    side.synchronize()
    assert torch.equal(got, first[0])
    outs, errors = [None] * 4, []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    outs[i] = pkg.ffpa_decode_paged(*args, enable_gqa=True)
            s.synchronize()
        except Exception as e:      # reported below: a thread's exception would be lost
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors and all(torch.equal(o, first[0]) for o in outs)
    lens = n.clone()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, l = pkg.ffpa_decode_paged(q, kc, vc, table, lens, enable_gqa=True, return_lse=True)
        graphs.append((graph, o, l))
    for new in ([3000, 1, 0, 800], [17, 0, 0, 1], [0, 0, 0, 0], [2999, 1, 0, 799]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        for graph, o, l in graphs:
            o.fill_(math.nan)
            graph.replay()
        want = pkg.ffpa_decode_paged(q, kc, vc, table, lens, enable_gqa=True, return_lse=True)
        for _, o, l in graphs:
            assert torch.equal(o, want[0]) and torch.equal(l, want[1]), new
    device_ok()


def test_decode_reports_a_wait_that_runs_out():
    """A copy that never starts: the call ends after its limit with the timeout status, and the next
    call is whole."""
    for D in (64, 512, 1024):
        args, ref = decode_case([300, 20], 4, 2, D, 16, BF, seed=19)
        word = status_word()
        pkg.ffpa_decode_paged(*args, enable_gqa=True, status=word, wait_timeout_ns=3_000_000, test_drop_first_copy=True)
        torch.cuda.synchronize()
        assert word.item() == pkg.FFPA_ERR_DEVICE_TIMEOUT
        check_decode(args, ref)
    device_ok()


# ------------------------------------------------------------------------------------ append
def append_case(T, Hq, Hkv, D, rot, page, dtype, wdtype, norm, seed=0, far=4000):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dtype)
    pages = -(-T // page) + 3
    kc, vc = (torch.randn(pages, page, Hkv, D, generator=g).to(dtype) for _ in range(2))
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[torch.rand(T, generator=g) < 0.1] = -1
    pos = torch.randint(0, far, (T,), generator=g, dtype=torch.int32)
    inv = pkg.rope_inv_freq(rot)[0] if rot else None
    qw, kw = ((1 + 0.2 * torch.randn(2, D, generator=g)).to(wdtype) if norm else (None, None))
    return qkv, kc, vc, slots, pos, inv, qw, kw


def to_dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,page,dtype,wdtype,norm,inter", [
    (1, 4, 1, 64, 64, 16, BF, BF, True, False), (37, 8, 2, 512, 512, 16, BF, torch.float32, True, False),
    (300, 4, 4, 128, 64, 1, HF, HF, True, True), (65, 6, 3, 120, 120, 7, HF, torch.float32, True, False),
    (50, 2, 2, 1024, 512, 32, BF, BF, False, True), (129, 4, 2, 1016, 72, 16, BF, BF, True, True),
    (40, 3, 1, 256, 0, 16, BF, BF, True, False), (40, 2, 1, 320, 0, 16, HF, BF, False, False)])
def test_append(T, Hq, Hkv, D, rot, page, dtype, wdtype, norm, inter):
    qkv, kc, vc, slots, pos, inv, qw, kw = append_case(T, Hq, Hkv, D, rot, page, dtype, wdtype, norm, seed=T)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    dq, dk, dvv = (t for t in (qkv.to(DEV)[:, :Hq], qkv.to(DEV)[:, Hq:Hq + Hkv], qkv.to(DEV)[:, Hq + Hkv:]))
    dkc, dvc, ds, dp, di, dqw, dkw = to_dev(kc, vc, slots, pos, inv, qw, kw)
    word = status_word()
    out = pkg.ffpa_kv_append(dq, dk, dvv, dkc, dvc, ds, dp, di, dqw, dkw, interleaved=inter, rope_scale=1.1, status=word)
    torch.cuda.synchronize()
    assert word.item() == pkg.FFPA_OK
    close(out, *po.rope_bound(q, pos, inv, qw, interleaved=inter, rope_scale=1.1), "q")
    want, bound = po.rope_bound(k, pos, inv, kw, interleaved=inter, rope_scale=1.1)
    full, fb, vfull = kc.double(), torch.zeros(kc.shape, dtype=torch.float64), vc.clone()
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            full[s // page, s % page], fb[s // page, s % page], vfull[s // page, s % page] = want[t], bound[t], v[t]
    close(dkc, full, fb, "k cache")              # slots that are not written keep their bits (bound 0)
    assert torch.equal(dvc.cpu(), vfull)


def test_append_without_queries_bad_slots_and_a_strided_cache():
    qkv, kc, vc, slots, pos, inv, qw, kw = append_case(20, 2, 2, 64, 64, 4, BF, BF, True, seed=3)
    k, v = qkv[:, 2:4].to(DEV), qkv[:, 4:].to(DEV)
    slots = torch.arange(20)
    slots[3], slots[7], slots[8] = kc.shape[0] * 4, 2 ** 40, -2 ** 62
    dkc = kc.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)          # heads outside the slots
    dvc = vc.to(DEV)
    word = status_word()
    assert pkg.ffpa_kv_append(None, k, v, dkc, dvc, slots.to(DEV), status=word) is None
    torch.cuda.synchronize()
    assert word.item() == pkg.FFPA_ERR_INVALID
    for t in range(20):
        hit = t not in (3, 7, 8)
        assert torch.equal(dkc[t // 4, t % 4].cpu(), qkv[t, 2:4] if hit else kc[t // 4, t % 4])
        assert torch.equal(dvc[t // 4, t % 4].cpu(), qkv[t, 4:] if hit else vc[t // 4, t % 4])
    # in place, no token, int64 positions
    q = qkv[:, :2].to(DEV)
    want = pkg.ffpa_kv_append(q, k, v, dkc, dvc, torch.full((20,), -1, device=DEV), pos.to(DEV), inv.to(DEV), qw.to(DEV), kw.to(DEV))
    same = pkg.ffpa_kv_append(q, k, v, dkc, dvc, torch.full((20,), -1, device=DEV), pos.long().to(DEV), inv.to(DEV), qw.to(DEV),
                              kw.to(DEV), q_out=q)
    assert same is q and torch.equal(q, want)
    assert pkg.ffpa_kv_append(q[:0], k[:0], v[:0], dkc, dvc, torch.empty(0, dtype=torch.int64, device=DEV)).shape == (0, 2, 64)
    device_ok()


# -------------------------------------------------------------------------------------- plan
def run_plan(table, old, new, free, count, page, tokens):
    word = status_word()
    t, o, w, f, c = to_dev(table, torch.tensor(old, dtype=torch.int32), torch.tensor(new, dtype=torch.int32),
                           torch.tensor(free, dtype=torch.int32), torch.tensor([count], dtype=torch.int32))
    got = pkg.ffpa_page_plan(t, o, w, f, c, page, tokens, status=word)
    again = t.clone()
    twice = pkg.ffpa_page_plan(again, o, w, f, c, page, tokens, status=status_word())
    assert torch.equal(again, t) and all(torch.equal(a, b) for a, b in zip(got, twice))
    ref = po.page_plan(table, old, new, free, count, page, tokens)
    return t, got, word.item(), ref


def check_plan(*a):
    t, (slots, pos, cu, lens, left), word, ref = run_plan(*a)
    assert torch.equal(t.cpu(), ref[0])
    assert slots.tolist() == ref[1] and pos.tolist() == ref[2] and cu.tolist() == ref[3]
    assert lens.tolist() == ref[4] and left.tolist() == [ref[5]]
    assert word == (pkg.FFPA_ERR_INVALID if ref[6] else pkg.FFPA_OK)


def table_of(old, page, width, seed):
    g = torch.Generator().manual_seed(seed)
    pool = torch.randperm(4096, generator=g).tolist()
    t = torch.full((len(old), width), -1, dtype=torch.int32)
    for b, n in enumerate(old):
        for j in range(min(width, max(0, -(-n // page)))):
            t[b, j] = pool.pop()
    return t, pool


@pytest.mark.parametrize("page", [1, 5, 16, 64])
@pytest.mark.parametrize("B,old,new", [(1, 0, 1), (1, 100, 5000), (3, 7, 40), (9, 50, 3), (64, 200, 1), (300, 30, 2), (40, 0, 300)])
def test_plan(B, old, new, page):
    g = torch.Generator().manual_seed(B * 31 + page)
    olds = torch.randint(0, old + 1, (B,), generator=g).tolist()
    news = torch.randint(0, new + 1, (B,), generator=g).tolist()
    if B == 1:
        news = [new]
    width = max(-(-(a + b) // page) for a, b in zip(olds, news)) + 1
    g2 = torch.Generator().manual_seed(1)
    free = torch.randperm(20000, generator=g2).tolist()
    table, _ = table_of(olds, page, width, 2) if sum(-(-n // page) for n in olds) < 4000 else (torch.randint(0, 9999, (B, width), dtype=torch.int32), None)
    check_plan(table, olds, news, free, 19990, page, sum(news) + 3)


@pytest.mark.parametrize("old,new,free,count,width,tokens", [
    ([5, 0, 9], [20, 30, 1], 4, 4, 10, 60),        # the list runs out inside a request
    ([5, 0, 9], [20, 30, 1], 3, 0, 10, 60),        # nothing to give
    ([5, 0, 9], [20, 30, 1], 20, 25, 10, 60),      # a count beyond the list
    ([5, 0, 9], [20, 30, 1], 20, -2, 10, 60),
    ([5, 0, 9], [20, 90, 1], 40, 40, 4, 200),      # a request outgrows its row
    ([5, 99, 9], [2, 3, 1], 40, 40, 4, 200),       # ... or did before
    ([5, -4, 9], [2, 3, -7], 40, 40, 4, 200),      # negative lengths
    ([5, 0, 9], [20, 30, 1], 20, 20, 10, 33),      # more tokens than rows
    ([5, 0, 9], [0, 0, 0], 20, 20, 10, 4), ([5, 0, 9], [0, 0, 0], 0, 0, 10, 0)])
def test_plan_at_its_limits(old, new, free, count, width, tokens):
    table, pool = table_of(old, 8, width, 5)
    check_plan(table, old, new, pool[:free], count, 8, tokens)


def test_plan_strided_table_and_graph():
    old, new = [5, 0, 17, 30], [1, 12, 0, 3]
    table, pool = table_of(old, 8, 6, 6)
    wide = torch.full((4, 11), 77, dtype=torch.int32, device=DEV)
    wide[:, :6] = table.to(DEV)
    o, w, f, c = to_dev(*(torch.tensor(x, dtype=torch.int32) for x in (old, new, pool[:9], [9])))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = pkg.ffpa_page_plan(wide[:, :6], o, w, f, c, 8, 20)
    for news in (new, [0, 1, 1, 1], [8, 0, 0, 0]):
        wide[:, :6] = table.to(DEV)
        w.copy_(torch.tensor(news, dtype=torch.int32))
        graph.replay()
        ref = po.page_plan(table, old, news, pool[:9], 9, 8, 20)
        assert torch.equal(wide[:, :6].cpu(), ref[0]) and (wide[:, 6:] == 77).all()
        assert [t.tolist() for t in got] == [ref[1], ref[2], ref[3], ref[4], [ref[5]]]
    device_ok()


# ---------------------------------------------------------------------------------- together
@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", [(8, 2, 512, 16, BF), (4, 4, 128, 5, HF)])
def test_generation_matches_attention_of_the_whole_sequences(Hq, Hkv, D, page, dtype):
    """Prompts, then single tokens, through plan, append and decode; each step's output against the
    64-bit attention of the rows appended so far, as they were stored."""
    g = torch.Generator().manual_seed(21)
    B, width, pages = 4, 40, 120
    inv, scale = pkg.rope_inv_freq(D, scaling="by_parts", factor=4.0, original_length=64)
    inv = inv.to(DEV)
    qw, kw = (1 + 0.2 * torch.randn(2, D, generator=g)).to(dtype).to(DEV)
    kc, vc = (torch.full((pages, page, Hkv, D), math.nan, dtype=dtype, device=DEV) for _ in range(2))
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    free = torch.randperm(pages, generator=g).to(torch.int32).to(DEV)
    count = torch.tensor([pages], dtype=torch.int32, device=DEV)
    held = [([], []) for _ in range(B)]
    word = status_word()
    for step, new in enumerate(([33, 0, 1, 70], [1, 1, 1, 1], [1, 0, 1, 1], [0, 20, 0, 1], [1, 1, 1, 1])):
        T = sum(new) + 2
        qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dtype).to(DEV)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        nt = torch.tensor(new, dtype=torch.int32, device=DEV)
        slots, pos, cu, lens, count = pkg.ffpa_page_plan(table, lens, nt, free, count, page, T, status=word)
        rope = dict(positions=pos, inv_freq=inv, q_weight=qw, k_weight=kw, rope_scale=scale)
        qr, kr = pkg.ffpa_qk_norm_rope(q, k, **rope)
        q2 = pkg.ffpa_kv_append(q, k, v, kc, vc, slots, **rope, status=word)
        assert torch.equal(qr, q2)                                   # the same rows from both
        cuh = cu.tolist()
        for b in range(B):
            held[b][0].extend(kr[cuh[b]:cuh[b + 1]].cpu().unbind(0))
            held[b][1].extend(v[cuh[b]:cuh[b + 1]].cpu().unbind(0))
        last = [cuh[b + 1] - 1 if new[b] else 0 for b in range(B)]    # the last new token of each request
        qd = q2[last]
        o, lse = pkg.ffpa_decode_paged(qd, kc, vc, table, lens, enable_gqa=True, return_lse=True, status=word)
        n = [len(h[0]) for h in held]
        assert lens.tolist() == n and word.item() == pkg.FFPA_OK
        top = max(n)
        kd, vd = (torch.zeros(B, top, Hkv, D, dtype=dtype) for _ in range(2))
        for b in range(B):
            if n[b]:
                kd[b, :n[b]], vd[b, :n[b]] = torch.stack(held[b][0]), torch.stack(held[b][1])
        flat = torch.arange(B, dtype=torch.int32)[:, None]
        ref = po.decode(qd.cpu(), kd, vd, flat, torch.tensor(n))     # a dense cache: one page a request
        close(o, ref[0], ref[2], f"step {step} O")
        close(lse, ref[1], ref[3], f"step {step} LSE")
    device_ok()
