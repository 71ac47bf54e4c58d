"""bf16 queries whose columns differ widely in size, over a cache of codes: the bound that include/ffpa.h gives."""
import pytest
import torch

import exact_headdim_attention_gb300 as pkg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16
E4M3 = torch.float8_e4m3fn


@pytest.mark.parametrize("D", [64, 128, 256, 512, 1024])
@pytest.mark.parametrize("large", [1.0, 1.9921875, 2.0 ** 100])
def test_small_columns(D, large):
    """One key a request, so that the LSE is the score.  The largest column meets a zero of the key; the others are
    2^-20 to 2^-38 of it, in a few columns or in all.  q enters to 2^-39 of the largest of its row, and the sums of
    at most 64 steps and the factors behind them are off by 2^-16 of the products' sizes."""
    g = torch.Generator().manual_seed(D)
    B, Hq = 19, 2
    q = torch.randn(B, Hq, D, generator=g).to(BF) * torch.exp2(-torch.arange(20.0, 39.0))[:, None, None].to(BF) * large
    q[:, 1, : D // 2] = 0.0                                      # (far from the largest column too)
    q[:, :, 0] = large
    k = (100 * torch.randn(B, 1, 1, D, generator=g)).clamp(-448, 448)
    k[..., 0] = 0.0
    codes = k.to(E4M3)
    ones = torch.ones(B, 1, 1, device=DEV)
    i32 = lambda t: t.to(dtype=torch.int32, device=DEV)          # noqa: E731
    scale = 2.0 ** 26 / large
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    _, lse = pkg.ffpa_decode_paged_fp8(q.to(DEV), codes.to(DEV), codes.to(DEV), ones, ones, i32(torch.arange(B)[:, None]),
                                       i32(torch.ones(B)), scale=scale, enable_gqa=True, return_lse=True, status=word)
    torch.cuda.synchronize()
    assert word.item() == pkg.FFPA_OK
    kd, qd = codes.float().double()[:, 0], q.double()            # [B,1,D], [B,Hq,D]
    x = scale * (qd * kd).sum(-1)
    size = abs(scale) * (qd * kd).abs().sum(-1)
    off = abs(scale) * 2.0 ** -39 * qd.abs().amax(-1) * kd.abs().sum(-1) + 2.0 ** -16 * size + 2.0 ** -22 * x.abs()
    err = (lse.cpu().double() - x).abs()
    assert (err <= off).all(), (err / off).max()
    # (columns that the largest one's unit does not hold lose bits: more than fp32 sums would)
    assert (err > 2.0 ** -12 * size).any()
