"""The rotation's cosines and sines to 2^-22 of themselves: rows whose pairs have one member, so that each output is one
product and a small one keeps its leading bits."""
import math

import pytest
import torch

import exact_headdim_attention_gb300 as pkg
from tests import paged_oracle as po
from tests.gpu_util import device_ok
from tests.test_gpu_paged import close, to_dev

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


def positions():
    """Small, ordinary and far positions; those below 10^6 whose cosine or sine at 1 radian a position is smallest."""
    p = torch.arange(1000000, dtype=torch.float64)
    near = torch.cat((torch.cos(p).abs().argsort()[:24], torch.sin(p).abs().argsort()[1:25]))
    return torch.cat((torch.tensor([0, 1, 2, 3, 7, 100, 5003, 70001, 1 << 20, -1, -2, -4099]), near))


def frequencies(rot):
    """Plain ones, slower ones to 1e-9 radians, and quarters of a turn, whose cosines and sines are 0 and 1."""
    inv = 10.0 ** torch.linspace(0, -9, rot // 2, dtype=torch.float64)
    inv[1], inv[2], inv[3] = math.pi / 2, math.pi / 4, -1.0
    return inv


def halves(x, rot, inter, keep):
    """x with zeros for one member of each pair."""
    x = x.clone()
    drop = slice(1 - keep, rot, 2) if inter else slice((1 - keep) * rot // 2, (2 - keep) * rot // 2)
    x[..., drop] = 0
    return x


def bound(y, size, angle, dtype):
    """y is rounded once.  Cosine and sine are off by 2^-22 of themselves, two products by 2^-24 each: 2^-21 of
    y.  The angle is off by 2^-33 turns (2^-30 radians) and 2^-52 of its size, the reference's by 2^-52 of it too."""
    slack = 2.0 ** -51 * angle.abs() + 2.0 ** -30
    return po.half_step(dtype) * y.abs() + 2.0 ** -21 * y.abs() + slack * size + torch.finfo(dtype).tiny * po.half_step(dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,rot", [(64, 64), (512, 512), (120, 40), (1016, 1016)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("keep", [0, 1])
@pytest.mark.parametrize("scale", [1.0, 1.25])
def test_one_member_pairs(D, rot, inter, keep, dtype, scale):
    pos, inv = positions(), frequencies(rot)
    g = torch.Generator().manual_seed(D + keep)
    T = pos.numel()
    x = halves(torch.randn(T, 1, D, generator=g).to(dtype), rot, inter, keep)
    angle = torch.outer(pos.double(), inv)
    size = torch.zeros(T, 1, D, dtype=torch.float64)
    full = torch.zeros(T, 1, D, dtype=torch.float64)
    both = x.double().abs()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    for part in (a, b):
        size[..., part] = (both[..., a] + both[..., b]) * scale
        full[..., part] = angle[:, None]
    how = dict(interleaved=inter, rope_scale=scale)
    dev = to_dev(x, x, pos, inv)
    out, _ = pkg.ffpa_qk_norm_rope(*dev, **how)
    back, _, _, _ = pkg.ffpa_qk_norm_rope_bwd(dev[0], dev[0], *dev, **how)       # the opposite rotation of x
    device_ok()
    want = po.rope(x.double(), pos, inv, None, **how)
    close(out, want, bound(want, size, full, dtype), "rotated")
    want = po.rope(x.double(), -pos, inv, None, **how)
    close(back, want, bound(want, size, full, dtype), "rotated back")
