"""Rows at the ends of the range going into the paged cache of 8 bits a value, on the GPU: the smallest
normed rows against the 64-bit definition, rows with NaN and infinities against the 16-bit append."""
import pytest
import torch

import exact_headdim_attention_gb300 as pkg
from tests import paged_fp8_oracle as p8
from tests import paged_oracle as po
from tests.test_gpu_paged_fp8 import run_append

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
E4M3 = torch.float8_e4m3fn
LEAST = 2.0 ** -117 / 448          # the smallest scale


def rows_case(k, v, rot, norm, dtype, seed, w_size=1.0):
    """The arguments of run_append for rows k, v [T, Hkv, D] in slots 0, 1, ...; a query head of ordinary values."""
    g = torch.Generator().manual_seed(seed)
    T, D = k.shape[0], k.shape[2]
    inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2)) if rot else None
    w = w_size * (1 + 0.2 * torch.randn(2, D, generator=g)) if norm else (None, None)
    return (torch.randn(T, 1, D, generator=g).to(dtype), k, v, torch.randint(0, 1 << 18, (T,), generator=g), inv, w,
            torch.arange(T))


def stored(cache, scale, T):
    """(codes, scales) of slots 0 .. T - 1 (CPU)."""
    page = cache.shape[1]
    at = torch.arange(T)
    return cache.cpu().view(torch.uint8)[at // page, at % page].view(E4M3), scale.cpu()[at // page, :, at % page]


def check_small(case, got, eps=1e-6):
    q, k, v, pos, inv, w, slots = case
    out, kc, vc, ks, vs, word = got
    assert word == pkg.FFPA_OK
    # Off in fp32 by 2^-18 of the pair's sizes (rope_bound, without its rounding to 16 bits), and below the normal range
    # by half of 2^-149 in each of two steps before the norm's factor r and one behind it.
    y, bound = po.rope_bound(k, pos, inv, w[1], eps=eps)
    tiny = torch.finfo(k.dtype).tiny * po.half_step(k.dtype)
    off = (bound - po.half_step(k.dtype) * y.abs() - tiny).clamp(min=0)
    r = torch.ones(()) if w[1] is None else torch.rsqrt(k.double().square().mean(-1, keepdim=True) + eps)
    off = off + 2.0 ** -149 * r + 2.0 ** -150
    codes, scale = stored(kc, ks, k.shape[0])
    assert torch.isfinite(codes.float()).all() and (scale >= LEAST * (1 - 2.0 ** -22)).all()
    # every row: half a step of e4m3, of the row's scale, which is LEAST at the least
    top = y.abs().amax(-1, keepdim=True)
    half = 2.0 ** -4 * y.abs() + 2.0 ** -10 * (top / 448).clamp(min=LEAST)
    err = (codes.double() * scale.double()[..., None] - y).abs()
    assert (err <= half * (1 + 2.0 ** -18) + 2 * off).all(), (err / (half + 2 * off)).max()
    # rows whose scale is not the smallest: the nearest codes
    large = top[..., 0] > 2.0 ** -117 * (1 + 2.0 ** -10)
    assert large.any()
    p8.check_codes(codes.view(torch.uint8)[large].view(E4M3), scale[large], y[large], off[large])
    assert (codes.float()[(k == 0).all(-1)] == 0).all() and (scale[(k == 0).all(-1)] == 1).all()


@pytest.mark.parametrize("D,rot", [(64, 0), (64, 64), (80, 40), (112, 0), (256, 128), (512, 512), (1008, 0), (1024, 1024)])
@pytest.mark.parametrize("eps", [1e-6, 1e-20])
def test_smallest_normed_rows(D, rot, eps):
    """Normed rows of 2^-108 to 2^-132, whose norm's factor is 1 / sqrt(eps): exact zeros stay zeros, the others
    are the codes of the normed row."""
    g = torch.Generator().manual_seed(D + rot)
    size = torch.exp2(-torch.arange(108.0, 133.0, dtype=torch.float64))[:, None, None]
    k = (size * torch.randn(25, 2, D, generator=g).double()).to(BF)
    k[..., ::5] = 0.0
    k[-1, 0] = 0.0
    case = rows_case(k, k.clone(), rot, True, BF, D)
    check_small(case, run_append(case, 16, 2, eps=eps), eps)


@pytest.mark.parametrize("D,rot", [(64, 64), (80, 0), (512, 128)])
def test_smallest_weighted_rows(D, rot):
    """fp16 rows times weights of 2^-100 (the norm's factor at its largest and near 1)."""
    g = torch.Generator().manual_seed(D)
    size = torch.exp2(-torch.arange(0.0, 24.0))[:, None, None]
    k = (size * torch.randn(24, 2, D, generator=g)).to(HF)
    k[..., 1::7] = 0.0
    case = rows_case(k, k.clone(), rot, True, HF, D, w_size=2.0 ** -100)
    check_small(case, run_append(case, 16, 2))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,rot", [(64, 0), (80, 40), (128, 128), (512, 256), (1024, 0)])
@pytest.mark.parametrize("norm", [True, False])
def test_rows_with_nan_and_infinities(norm, D, rot, dtype):
    """Codes are NaN where the 16-bit append's row is not finite, and there alone.  The scale of a row with a NaN is
    NaN with the norm; of one with an infinity 1 with the norm (it leaves zeros) and infinite without."""
    g = torch.Generator().manual_seed(D)
    k = torch.randn(7, 2, D, generator=g).to(dtype)
    k[1, 0, 3] = torch.nan
    k[2, 1, D - 1] = torch.inf
    k[3, 0, 5], k[3, 0, 0] = -torch.inf, torch.inf
    k[4, 1, 2], k[4, 1, 9] = torch.nan, torch.inf
    k[5] = torch.nan
    case = rows_case(k, k.clone(), rot, norm, dtype, D)
    _, kc, vc, ks, vs, word = run_append(case, 16, 1)
    assert word == pkg.FFPA_OK
    q, _, v, pos, inv, w, slots = case
    d = lambda t: None if t is None else t.to("cuda:0")   # noqa: E731
    x16 = torch.zeros(2, 1, 16, 2, D, dtype=dtype, device="cuda:0")
    pkg.ffpa_kv_append(d(q), d(k), d(v), x16[0], x16[1], d(slots), d(pos) if rot else None, d(inv), d(w[0]), d(w[1]))
    torch.cuda.synchronize()
    for cache, scale, x, normed in ((kc, ks, x16[0], norm), (vc, vs, x16[1], False)):
        codes, scale = stored(cache, scale, 7)
        codes, x = codes.float(), x[0, :7].float().cpu()
        bad = ~torch.isfinite(x)
        assert torch.equal(torch.isnan(codes), bad)
        nan, endless = torch.isnan(k).any(-1), torch.isinf(k).any(-1)
        some = nan | endless
        if normed:
            assert torch.isnan(scale[nan]).all() and (scale[endless & ~nan] == 1).all()
            assert (codes[some.unsqueeze(-1) & ~bad] == 0).all()
        else:
            assert torch.isinf(scale[torch.isinf(x).any(-1)]).all()
            assert (codes[torch.isinf(x).any(-1, keepdim=True) & ~bad] == 0).all()
            assert (scale[bad.all(-1) & nan & ~endless] == 1).all()
        assert torch.isfinite(scale[~some]).all() and (scale[~some] > 0).all()
