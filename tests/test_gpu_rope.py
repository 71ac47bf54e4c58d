"""Head norm with rotation and its gradients on the GPU against 64-bit references; the error bounds
are derived in paged_oracle.py."""
import math

import pytest
import torch

import exact_headdim_attention_gb300 as pkg
from tests import paged_oracle as po
from tests.gpu_util import device_ok
from tests.test_gpu_paged import close, to_dev

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32

CASES = [  # T, Hq, Hkv, D, rot, dtype, weight type (None: no norm), interleaved
    (1, 1, 1, 64, 64, BF, BF, False), (3, 4, 2, 64, 32, HF, F32, True), (130, 8, 2, 128, 128, BF, F32, False),
    (65, 6, 3, 120, 120, HF, HF, False), (65, 2, 1, 120, 40, BF, BF, True), (20, 5, 5, 192, 64, BF, None, False),
    (33, 16, 4, 256, 256, HF, F32, True), (40, 3, 1, 264, 24, BF, F32, False), (17, 8, 2, 320, 160, BF, BF, True),
    (200, 4, 4, 512, 512, BF, F32, False), (31, 2, 2, 520, 520, BF, F32, True), (50, 4, 2, 768, 384, HF, None, True),
    (9, 20, 4, 1016, 1016, BF, BF, False), (77, 2, 1, 1024, 1024, BF, F32, False), (77, 2, 1, 1024, 64, HF, F32, True),
    (60, 4, 2, 512, 0, BF, BF, False), (60, 4, 2, 72, 0, BF, None, False), (3000, 4, 1, 64, 64, BF, F32, False)]


def make(T, Hq, Hkv, D, rot, dtype, wdtype, seed=0, far=100000):
    g = torch.Generator().manual_seed(seed)
    q, k = torch.randn(T, Hq, D, generator=g).to(dtype), torch.randn(T, Hkv, D, generator=g).to(dtype)
    pos = torch.randint(0, far, (T,), generator=g)
    inv = pkg.rope_inv_freq(rot)[0] if rot else None
    qw, kw = (None, None) if wdtype is None else (1 + 0.3 * torch.randn(2, D, generator=g)).to(wdtype)
    up = torch.randn(T, Hq, D, generator=g).to(dtype), torch.randn(T, Hkv, D, generator=g).to(dtype)
    return q, k, pos, inv, qw, kw, up


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,dtype,wdtype,inter", CASES)
def test_forward(T, Hq, Hkv, D, rot, dtype, wdtype, inter):
    q, k, pos, inv, qw, kw, _ = make(T, Hq, Hkv, D, rot, dtype, wdtype, seed=D + T)
    how = dict(interleaved=inter, rope_scale=0.8, eps=1e-5)
    qo, ko = pkg.ffpa_qk_norm_rope(*to_dev(q, k, pos, inv, qw, kw), **how)
    device_ok()
    close(qo, *po.rope_bound(q, pos, inv, qw, **how), "q")
    close(ko, *po.rope_bound(k, pos, inv, kw, **how), "k")


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,dtype,wdtype,inter", CASES)
def test_backward(T, Hq, Hkv, D, rot, dtype, wdtype, inter):
    q, k, pos, inv, qw, kw, (gq, gk) = make(T, Hq, Hkv, D, rot, dtype, wdtype, seed=D + T)
    how = dict(interleaved=inter, rope_scale=0.8, eps=1e-5)
    dev = to_dev(gq, gk, q, k, pos.int(), inv, qw, kw)
    dq, dk, dqw, dkw = pkg.ffpa_qk_norm_rope_bwd(*dev, **how)
    again = pkg.ffpa_qk_norm_rope_bwd(*dev, **how)
    device_ok()
    for got, other, x, w, g, name in ((dq, again[0], q, qw, gq, "q"), (dk, again[1], k, kw, gk, "k")):
        dx, _, bx, _ = po.rope_grads(g, x, pos, inv, w, **how)
        close(got, dx, bx, f"d{name}")
        assert torch.equal(got, other)
    for got, other, x, w, g, name in ((dqw, again[2], q, qw, gq, "q"), (dkw, again[3], k, kw, gk, "k")):
        if w is None:
            assert got is None
            continue
        _, dw, _, bw = po.rope_grads(g, x, pos, inv, w, **how)
        close(got, dw, bw, f"d{name}_weight")
        assert torch.equal(got, other)


def test_one_weight_only_and_dense_layout():
    """[B,H,N,D] rows, positions for all sequences or for each, queries normed and keys not."""
    g = torch.Generator().manual_seed(2)
    B, Hq, Hkv, N, D = 3, 4, 2, 37, 128
    q, k = torch.randn(B, Hq, N, D, generator=g).to(BF), torch.randn(B, Hkv, N, D, generator=g).to(BF)
    w, inv = (1 + 0.3 * torch.randn(D, generator=g)), pkg.rope_inv_freq(64)[0]
    for pos in (torch.arange(N), torch.randint(0, 999, (1, N), generator=g), torch.randint(0, 999, (B, N), generator=g).int()):
        dq, dk, dp, di, dw = to_dev(q, k, pos, inv, w)
        # rows stored as [B,N,H,D]
        sq, sk = dq.transpose(1, 2).contiguous().transpose(1, 2), dk.transpose(1, 2).contiguous().transpose(1, 2)
        qo, ko = torch.empty_like(sq), torch.empty_like(dk)
        pkg.ffpa_qk_norm_rope(sq, sk, dp, di, dw, q_out=qo, k_out=ko)
        at = (pos if pos.dim() == 2 else pos[None]).expand(B, N)
        want, bound = po.rope_bound(q.transpose(1, 2), at, inv, w)
        close(qo.transpose(1, 2), want, bound, "q")
        want, bound = po.rope_bound(k.transpose(1, 2), at, inv, None)
        close(ko.transpose(1, 2), want, bound, "k")
        grads = pkg.ffpa_qk_norm_rope_bwd(dq, dk, sq, sk, dp, di, dw)
        dx, dwr, bx, bw = po.rope_grads(q.transpose(1, 2), q.transpose(1, 2), at, inv, w)
        close(grads[0].transpose(1, 2), dx, bx, "dq")
        close(grads[2], dwr, bw, "dw")
        assert grads[3] is None
    device_ok()


def test_far_negative_and_wide_positions():
    """Angles stay exact: positions to 2^31 (and beyond, int64), negative ones, a frequency of many turns."""
    g = torch.Generator().manual_seed(6)
    pos = torch.tensor([0, 1, -1, -70000, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31, 2 ** 40 + 12345])
    x = torch.randn(8, 2, 64, generator=g).to(BF)
    inv = pkg.rope_inv_freq(64)[0]
    inv[3], inv[4], inv[5] = 40.0, -0.7, math.pi
    qo, _ = pkg.ffpa_qk_norm_rope(*to_dev(x, x, pos, inv))
    # The reference multiplies in integers: the angle in turns of 2^-96, exactly, modulo whole turns.
    y = torch.empty(8, 2, 64, dtype=torch.float64)
    from fractions import Fraction
    pi2 = 2 * Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    for t, p in enumerate(pos.tolist()):
        for i, f in enumerate(inv.tolist()):
            turns = Fraction(f) / pi2 * p
            a = 2 * math.pi * float(turns - math.floor(turns))
            u, v = x[t, :, i].double(), x[t, :, 32 + i].double()
            y[t, :, i], y[t, :, 32 + i] = u * math.cos(a) - v * math.sin(a), v * math.cos(a) + u * math.sin(a)
    # The frequency in turns is a double: 1 / (2 pi) is off by 2^-54 of itself and the product by
    # 2^-53, so the angle p f by 1.5 * 2^-53 |p f| radians (40 * 2^40 of them at the far end: 7e-3).
    m = (x[..., :32].double().abs() + x[..., 32:].double().abs()).repeat(1, 1, 2)
    slack = 2.0 ** -18 + 1.5 * 2.0 ** -53 * (pos.double()[:, None] * inv).abs().repeat(1, 2)[:, None]
    close(qo, y, po.half_step(BF) * y.abs() + slack * m, "q")
    small = pos[:7]
    a, _ = pkg.ffpa_qk_norm_rope(*to_dev(x[:7], x[:7], small, inv))
    b, _ = pkg.ffpa_qk_norm_rope(*to_dev(x[:7], x[:7], small.int(), inv))
    assert torch.equal(a, b)
    device_ok()


def test_slices_in_place_and_rows_that_are_zero():
    q, k, pos, inv, qw, kw, _ = make(50, 8, 2, 256, 256, BF, F32, seed=8)
    qkv = torch.cat((q, k, torch.full_like(k, math.nan)), 1).to(DEV)
    qkv[4, 0] = 0.0
    a, b = qkv[:, :8], qkv[:, 8:10]
    dp, di, dqw, dkw = to_dev(pos, inv, qw, kw)
    want = pkg.ffpa_qk_norm_rope(a, b, dp, di, dqw, dkw)
    assert (want[0][4, 0] == 0).all()
    got = pkg.ffpa_qk_norm_rope(a, b, dp, di, dqw, dkw, q_out=a, k_out=b)
    assert got[0] is a and torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert torch.isnan(qkv[:, 10:]).all()
    # nothing to do
    e = pkg.ffpa_qk_norm_rope(a[:0], b[:0], dp[:0], di, dqw, dkw)
    assert e[0].shape == (0, 8, 256)
    z = pkg.ffpa_qk_norm_rope_bwd(a[:0], b[:0], a[:0], b[:0], dp[:0], di, dqw, dkw)
    assert z[0].shape == (0, 8, 256) and (z[2] == 0).all() and (z[3] == 0).all()
    device_ok()


def test_infinite_and_nan_rows_stay_in_their_rows():
    q, k, pos, inv, qw, kw, (gq, gk) = make(20, 2, 1, 128, 64, BF, F32, seed=9)
    q[3, 1, 5], q[7, 0, 100] = math.inf, math.nan
    dev = to_dev(q, k, pos, inv, qw, kw)
    qo, ko = pkg.ffpa_qk_norm_rope(*dev)
    bad = torch.zeros(20, 2, dtype=torch.bool)
    bad[3, 1] = bad[7, 0] = True
    assert torch.isfinite(qo.cpu()[~bad]).all() and not torch.isfinite(qo.cpu()[bad]).all(-1).any()
    assert torch.isfinite(ko).all()
    dq, _, dqw, dkw = pkg.ffpa_qk_norm_rope_bwd(*to_dev(gq, gk), *dev)
    assert torch.isfinite(dq.cpu()[~bad]).all() and torch.isfinite(dkw).all()
    assert torch.isnan(dqw).any()


def test_streams_and_graphs():
    q, k, pos, inv, qw, kw, (gq, gk) = make(300, 8, 2, 512, 512, BF, F32, seed=10)
    dev = to_dev(q, k, pos, inv, qw, kw)
    g = to_dev(gq, gk)
    want = pkg.ffpa_qk_norm_rope(*dev) + pkg.ffpa_qk_norm_rope_bwd(*g, *dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pkg.ffpa_qk_norm_rope(*dev, stream=side) + pkg.ffpa_qk_norm_rope_bwd(*g, *dev, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = pkg.ffpa_qk_norm_rope(*dev) + pkg.ffpa_qk_norm_rope_bwd(*g, *dev)
        graphs.append((graph, out))
    for graph, out in graphs + graphs:
        [t.fill_(math.nan) for t in out]
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, out))
    device_ok()
