"""Decode attention over a paged cache: every weight of the softmax reaches the output, however small
and however rounded.  Bounds are derived below; references in paged_oracle.py."""
import math

import pytest
import torch

import exact_headdim_attention_gb300 as pkg
from tests import paged_oracle as po
from tests.gpu_util import device_ok
from tests.test_gpu_paged import close, decode_case

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, HF = torch.bfloat16, torch.float16


def weighed(q, kc, vc, table, n):
    """sum p |v| of every output in 64 bits."""
    return po.decode(q, kc, vc.abs(), table, n)[0]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (16, 1), (20, 1)])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 3), (200, 100), (256, 32), (512, 16), (1024, 16)])
def test_weights_are_not_rounded_to_the_inputs_type(D, page, Hq, Hkv, dtype):
    """o is rounded once, to its type.  Inside: a weight takes two values of the type, 2^-16 of it at
    most apart from it; scores (at most 64 steps of 16 products of partial sums below 8, each step off
    by 2^-23) 2^-14; at most 2 * 2500 / 16 products of 16 keys on an accumulator, each off by 2^-23
    of sums below sum p |v|: 2^-14.  2^-13 + 2^-16 in all, of sum p |v|."""
    args, ref = decode_case([300, 40, 2, 2500, 0, 17], Hq, Hkv, D, page, dtype, seed=D + Hq)
    o, lse = pkg.ffpa_decode_paged(*args, enable_gqa=True, return_lse=True)
    device_ok()
    size = weighed(*(t.cpu() for t in args))
    close(o, ref[0], po.half_step(dtype) * ref[0].abs() + (2.0 ** -13 + 2.0 ** -16) * size + 2.0 ** -25, "O")
    close(lse, ref[1], ref[3], "LSE")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n,D,Hq,page", [(20000, 64, 2, 16), (393217, 64, 1, 64), (30000, 512, 16, 16), (5000, 128, 4, 3)])
def test_many_small_weights_are_not_lost(n, D, Hq, page, dtype):
    """One key, and many that lie 17.375 below it in the exponent (2.8e-8 of its weight, under half of the
    smallest fp16 number): the output is made of the small ones alone.  Their scores are exact; the
    exponentials (2^-22, and 2^-20 of the exponent's own rounding), the pairs of 16-bit values (2^-16) and
    the fp32 sums (chains of at most 2 * 393217 / 16 steps of 2^-24 over 152 blocks at least: 2^-15) stay
    below 2^-13 of the result, which is rounded once."""
    g = torch.Generator().manual_seed(n)
    pages = -(-n // page)
    kc = torch.zeros(pages, page, 1, D, dtype=dtype)
    kc.view(-1, D)[1:, 0] = -17.375
    vc = (0.5 + torch.rand(pages, page, 1, D, generator=g)).to(dtype)
    vc.view(-1, D)[0] = 0.0
    q = torch.zeros(1, Hq, D, dtype=dtype)
    q[..., 0] = 1.0
    table = torch.randperm(pages, generator=g).to(torch.int32)
    kp, vp = torch.empty_like(kc), torch.empty_like(vc)
    kp[table.long()], vp[table.long()] = kc, vc
    w = math.exp(-17.375)
    total = 1.0 + w * (n - 1)
    want = (w * vc.view(-1, D)[:n].double().sum(0) / total).expand(1, Hq, D)
    o, lse = pkg.ffpa_decode_paged(q.to(DEV), kp.to(DEV), vp.to(DEV), table[None].to(DEV),
                                   torch.tensor([n], dtype=torch.int32, device=DEV), scale=1.0, enable_gqa=True, return_lse=True)
    device_ok()
    tiny = torch.finfo(dtype).tiny * po.half_step(dtype)
    close(o, want, (po.half_step(dtype) + 2.0 ** -13) * want + tiny, "O")
    close(lse, torch.full((1, Hq), math.log(total), dtype=torch.float64), torch.full((1, Hq), 2.0 ** -18), "LSE")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,Hq", [(64, 2), (512, 16), (1024, 4)])
def test_infinite_values_give_infinities(D, Hq, dtype):
    """An infinite value whose weight is not zero makes its column infinite, of its sign; two of both signs NaN."""
    args, _ = decode_case([40, 700], Hq, 1, D, 16, dtype, seed=D)
    q, kc, vc, table, n = args
    for b in range(2):
        vc[table[b, 1].item(), 3, 0, 5] = math.inf
        vc[table[b, 0].item(), 0, 0, 6] = -math.inf
        vc[table[b, 0].item(), 7, 0, 7], vc[table[b, 1].item(), 7, 0, 7] = math.inf, -math.inf
    q[:, 0] = 0                      # equal weights, of which each is a number of 16 bits
    o = pkg.ffpa_decode_paged(q, kc, vc, table, n, enable_gqa=True)
    device_ok()
    assert (o[..., 5] == math.inf).all() and (o[..., 6] == -math.inf).all() and torch.isnan(o[..., 7]).all()
    assert torch.isfinite(o[..., :5]).all() and torch.isfinite(o[..., 8:]).all()
