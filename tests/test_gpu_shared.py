"""Decode attention of a batch with a shared prefix on the GPU, against the 64-bit reference of decode
attention over the same keys (paged_oracle.py, whose bound counts one rounding of a weight)."""
import functools
import math

import pytest
import torch

import exact_headdim_attention_gb300 as pkg
from tests import paged_oracle as po
from tests.gpu_util import device_ok
from tests.test_gpu_paged import close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, HF = torch.bfloat16, torch.float16


def word_():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def make(own, shared, Hq, Hkv, D, page, dtype, seed=0, layout="psh", scale=None, lens=None):
    """(arguments on the GPU, reference).  own: keys of each request behind `shared` ones, of which whole pages
    are shared; lens: lengths in place of shared + own (shorter requests see fewer of the shared keys)."""
    g = torch.Generator().manual_seed(seed)
    whole = shared // page
    rest = shared - whole * page
    full = [whole * page] + [n + rest for n in own]                  # the shared keys as a request of their own
    kc, vc, table, _ = po.make_cache(g, full, Hkv, D, page, dtype, layout=layout)
    pages = table[0, :whole].clone()
    B = len(own)
    n = torch.tensor([shared + x for x in own] if lens is None else lens, dtype=torch.int32)
    mine = torch.full((B, whole + table.shape[1]), -7, dtype=torch.int32)
    mine[:, whole:] = table[1:]
    both = mine.clone()
    both[:, :whole] = pages
    q = torch.randn(B, Hq, D, generator=g).to(dtype)
    ref = po.decode(q, kc, vc, both, n, scale)

    def dev(t):
        return t.to(DEV) if t.is_contiguous() else t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)

    return [q.to(DEV), dev(kc), dev(vc), pages.to(DEV), torch.tensor([shared], dtype=torch.int32, device=DEV), mine.to(DEV),
            n.to(DEV)], ref


def check(args, ref, what="", scale=None, **kw):
    """In one pass, by the call's own choice, and with the shared keys apart (whose result is returned)."""
    for kernel in ("single", None, "split"):
        word = word_()
        o, lse = pkg.ffpa_decode_shared(*args, scale=scale, enable_gqa=True, return_lse=True, status=word, kernel=kernel, **kw)
        torch.cuda.synchronize()
        assert word.item() == pkg.FFPA_OK
        close(o, ref[0], ref[2], f"{what} {kernel} O")
        close(lse, ref[1], ref[3], f"{what} {kernel} LSE")
    return o, lse


def split(*args, **kw):
    return pkg.ffpa_decode_shared(*args, kernel="split", **kw)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128, 192, 256, 320, 384, 448, 512, 576, 640, 704, 768, 832, 896, 960, 1024])
def test_head_dims(D, dtype):
    args, ref = make([1, 0, 40, 17, 200], 333, 8, 2, D, 16, dtype, seed=D)
    check(args, ref, f"D={D}")


@pytest.mark.parametrize("B", [1, 2, 33, 70])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (3, 1), (10, 2), (16, 1), (40, 1), (128, 1)])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_groups_and_batches(Hq, Hkv, D, B):
    """Groups that do and do not divide a query tile, one tile and several, pairs of tiles with an empty second."""
    if B * Hq > 1200:
        pytest.skip("the reference would take long")
    args, ref = make([(7 * b) % 31 for b in range(B)], 150, Hq, Hkv, D, 16, BF, seed=Hq + B)
    check(args, ref, f"Hq={Hq} Hkv={Hkv} B={B}")


@pytest.mark.parametrize("page", [8, 16, 24, 40, 64, 128, 256, 384])
@pytest.mark.parametrize("shared", [0, 7, 8, 129, 640, 1111])
@pytest.mark.parametrize("D,dtype", [(64, HF), (128, BF), (192, BF), (512, HF), (768, BF)])
def test_pages_and_shared_lengths(page, shared, D, dtype):
    """Whole pages of any number, none, and ends inside a page; pages that end inside a tile."""
    args, ref = make([5, 0, 66], shared, 4, 2, D, page, dtype, seed=page + shared)
    if shared + 0 == 0:
        assert ref[1][1].isinf().all()
    check(args, ref, f"page={page} shared={shared}")


@pytest.mark.parametrize("D", [128, 256, 512, 1024])
def test_long_prefix(D):
    """Many tiles a part, some parts, more than one step of the running maximum."""
    args, ref = make([3, 100], 9000, 6, 2, D, 32, BF, seed=D)
    check(args, ref, f"D={D}")


@pytest.mark.parametrize("D", [64, 128, 256, 320, 1024])
def test_requests_shorter_than_the_prefix(D):
    """Requests that see none, one, some and all of the shared keys."""
    lens = [0, 1, 100, 129, 256, 300, 320, 0, 127]
    args, ref = make([0] * 9, 320, 4, 2, D, 16, BF, seed=D, lens=lens)
    check(args, ref, f"D={D}")
    o, lse = split(*args, enable_gqa=True, return_lse=True)
    assert (o[0] == 0).all() and (o[7] == 0).all() and (lse[[0, 7]] == -math.inf).all()


@pytest.mark.parametrize("D", [64, 128, 256, 320, 1024])
def test_shared_pages_may_hold_anything_behind_the_last_key(D):
    """Where no request is as long as the shared keys, infinities and NaN behind the longest."""
    lens = [0, 1, 100, 129, 256, 300, 0, 127]
    args, ref = make([0] * 8, 320, 4, 2, D, 16, BF, seed=D, lens=lens)
    q, kc, vc, pages = args[:4]
    for i, p in enumerate(pages.tolist()):
        seen = max(0, min(16, 300 - 16 * i))
        kc[p, seen:], vc[p, seen:] = math.nan, math.inf
    check(args, ref, f"D={D}")


@pytest.mark.parametrize("scale", [0.0, 0.5, -0.1])
@pytest.mark.parametrize("D", [128, 256, 512])
def test_softmax_scale(D, scale):
    args, ref = make([40, 3], 300, 4, 2, D, 16, BF, seed=12, scale=scale)
    check(args, ref, scale=scale)


@pytest.mark.parametrize("D", [64, 256, 512])
def test_layouts(D):
    args, ref = make([40, 0, 70], 200, 8, 2, D, 16, BF, layout="phs", seed=9)
    q, kc, vc, pages, sl, table, n = args
    assert not kc.is_contiguous()
    wide = torch.full((3, 12, D), math.nan, dtype=BF, device=DEV)
    wide[:, 2:10] = q
    out = torch.full((3, 16, D), 7.0, dtype=BF, device=DEV)
    t2 = torch.full((3, 2 * table.shape[1] + 3), -9, dtype=torch.int32, device=DEV)
    t2[:, :table.shape[1]] = table
    check((wide[:, 2:10], kc, vc, pages, sl, t2[:, :table.shape[1]], n), ref, "strided", out=out[:, 4:12])
    assert (out[:, :4] == 7).all() and (out[:, 12:] == 7).all()


@pytest.mark.parametrize("D,dtype", [(64, HF), (128, HF), (256, HF), (512, HF), (1024, BF)])
def test_scores_that_grow_along_the_prefix(D, dtype):
    """The running maximum moves by more than 2^8 several times, in the parts and between them."""
    args, _ = make([30, 1], 1000, 4, 1, D, 8, dtype, seed=D)
    q, kc, vc, pages, sl, table, n = args
    q[:, :, 0] = 4.0
    kc[:, :, :, 0] = 0
    for i, p in enumerate(pages.tolist()):
        kc[p, :, :, 0] = float(i) * 0.25 * D ** 0.5 / 2
    both = table.cpu().clone()
    both[:, :pages.numel()] = pages.cpu()
    ref = po.decode(q.cpu(), kc.cpu(), vc.cpu(), both, n.cpu())
    # Partial sums of a score are as large as the score here (63 D^0.5 / 2 D^-0.5 ... up to 62 in units of the
    # exponent, in at most 64 fp32 steps of 2^-24 each): 62 * 64 * 2^-24 = 2^-12 of each weight.
    more = 2.0 ** -12 * vc.cpu().double().nan_to_num().abs().max()
    o, lse = split(*args, enable_gqa=True, return_lse=True)
    device_ok()
    close(o, ref[0], ref[2] + more, "O")
    close(lse, ref[1], ref[3] + 2.0 ** -12, "LSE")


def test_agrees_with_decode_and_repeats():
    args, ref = make([40, 0, 300, 9], 2000, 16, 4, 512, 32, BF, seed=3)
    a, la = check(args, ref)
    b, lb = check(args, ref)
    assert torch.equal(a, b) and torch.equal(la, lb)
    q, kc, vc, pages, sl, table, n = args
    both = table.clone()
    both[:, :pages.numel()] = pages
    o, lse = pkg.ffpa_decode_paged(q, kc, vc, both, n, enable_gqa=True, return_lse=True)
    one = pkg.ffpa_decode_shared(*args, enable_gqa=True, return_lse=True, kernel="single")
    assert torch.equal(one[0], o) and torch.equal(one[1], lse)
    assert (lse - la).abs().max() < 1e-4 and (o.float() - a.float()).abs().max() < 2e-2
    ws = torch.empty(pkg.decode_shared_workspace_bytes(4, 16, 4, 512), dtype=torch.uint8, device=DEV).fill_(255)
    c = split(*args, enable_gqa=True, workspace=ws)
    assert torch.equal(a, c)


@pytest.mark.parametrize("kernel", ["split", "single"])
def test_captured_lengths_may_change(kernel):
    split = functools.partial(pkg.ffpa_decode_shared, kernel=kernel)
    args, _ = make([40, 0, 300, 9], 700, 8, 2, 256, 16, BF, seed=4)
    q, kc, vc, pages, sl, table, n = args
    sl, n = sl.clone(), n.clone()
    table[:, :pages.numel()] = pages             # so that any shared length is right
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        split(q, kc, vc, pages, sl, table, n, enable_gqa=True)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            o = split(q, kc, vc, pages, sl, table, n, enable_gqa=True)
    full = n.tolist()
    for shared, lens in ((700, full), (0, full), (16, [5, 700, 0, 300]), (10 ** 6, [1, 2, 704, 33]), (350, full)):
        with torch.cuda.stream(side):
            sl.fill_(shared)
            n.copy_(torch.tensor(lens, dtype=torch.int32))
            graph.replay()
            side.synchronize()
        both = table.cpu()
        ref = po.decode(q.cpu(), kc.cpu(), vc.cpu(), both, n.cpu())
        close(o, ref[0], ref[2], f"shared={shared}")
    device_ok()


@pytest.mark.parametrize("kernel", ["split", "single", None])
def test_nothing_shared_and_nothing_cached(kernel):
    split = functools.partial(pkg.ffpa_decode_shared, kernel=kernel)
    args, ref = make([40, 3], 0, 4, 2, 128, 16, BF, seed=5)
    assert args[3].numel() == 0
    check(args, ref)
    q = torch.randn(2, 4, 64, device=DEV).to(BF)
    kc = torch.empty(0, 16, 2, 64, dtype=BF, device=DEV)
    table, n = torch.zeros(2, 0, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    none, zero = torch.empty(0, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = split(q, kc, kc, none, zero, table, n, enable_gqa=True, return_lse=True)
    assert (o == 0).all() and (lse == -math.inf).all()
    assert split(q[:0], kc, kc, none, zero, table[:0], n[:0], enable_gqa=True).shape == (0, 4, 64)
    device_ok()


@pytest.mark.parametrize("kernel", ["split", "single"])
@pytest.mark.parametrize("D", [64, 256, 512, 768])
def test_bad_pages_and_lengths_are_reported(D, kernel):
    """A shared page that does not exist counts as keys and values of zeros; a negative shared length as none."""
    split = functools.partial(pkg.ffpa_decode_shared, kernel=kernel)
    args, _ = make([40, 0, 70], 200, 4, 2, D, 16, BF, seed=15)
    q, kc, vc, pages, sl, table, n = args
    kc, vc = torch.nan_to_num(kc), torch.nan_to_num(vc)
    k0, v0 = torch.cat((kc, torch.zeros_like(kc[:1]))), torch.cat((vc, torch.zeros_like(vc[:1])))
    for bad in (kc.shape[0], -1, -2 ** 31, 2 ** 31 - 1):
        p2, word = pages.clone(), word_()
        p2[5] = bad
        o = split(q, kc, vc, p2, sl, table, n, enable_gqa=True, status=word)
        assert word.item() == pkg.FFPA_ERR_INVALID
        p2[5] = kc.shape[0]
        assert torch.equal(o, split(q, k0, v0, p2, sl, table, n, enable_gqa=True))
    word = word_()
    table[:, :pages.numel()] = pages
    o = split(q, kc, vc, pages, torch.full_like(sl, -5), table, n, enable_gqa=True, status=word)
    assert word.item() == pkg.FFPA_ERR_INVALID
    assert torch.equal(o, split(q, kc, vc, pages, torch.zeros_like(sl), table, n, enable_gqa=True))
    n2, word = torch.tensor([-1, 200, 2 ** 31 - 1], dtype=torch.int32, device=DEV), word_()
    t2 = table.clamp(min=0)
    o = split(q, kc, vc, pages, sl, t2, n2, enable_gqa=True, status=word)
    assert word.item() == pkg.FFPA_ERR_INVALID and (o[0] == 0).all() and torch.isfinite(o).all()
    device_ok()


@pytest.mark.parametrize("D,B", [(64, 9), (128, 70), (192, 3), (256, 9), (512, 9), (768, 9), (1024, 9)])
def test_ends_when_a_wait_runs_out(D, B):
    args, ref = make([3] * B, 500, 8, 2, D, 16, BF, seed=D)
    word = word_()
    for kernel in ("split", "single"):
        word.zero_()
        pkg.ffpa_decode_shared(*args, enable_gqa=True, status=word, kernel=kernel, wait_timeout_ns=3_000_000, test_drop_first_copy=True)
        torch.cuda.synchronize()
        assert word.item() == pkg.FFPA_ERR_DEVICE_TIMEOUT
    check(args, ref)
    device_ok()


def test_torch_operator_and_streams():
    args, ref = make([40, 0, 130], 300, 8, 2, 128, 16, BF, seed=31)
    o, lse = pkg.ffpa_attn_decode_shared_func(*args, enable_gqa=True, return_lse=True)
    close(o, ref[0], ref[2], "O")
    step = torch.compile(lambda q: pkg.ffpa_attn_decode_shared_func(q * 1, *args[1:], enable_gqa=True), backend="eager", fullgraph=True)
    assert torch.equal(step(args[0]), o)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2 = pkg.ffpa_decode_shared(*args, enable_gqa=True, stream=side)
    side.synchronize()
    assert torch.equal(o, o2)
    side.wait_stream(torch.cuda.current_stream())
    o3 = split(*args, enable_gqa=True, stream=side)
    side.synchronize()
    close(o3, ref[0], ref[2], "O")
    device_ok()
