"""The paged-cache operators and the head norm with rotation, without a GPU: refusals of the C ABI
and of the binding, frequencies, and the 64-bit gradients against differences."""
import ctypes
import math

import pytest
import torch

import exact_headdim_attention_gb300 as pkg
from exact_headdim_attention_gb300 import build as bld
from exact_headdim_attention_gb300._binding import Rope
from tests import paged_oracle as po

FAKE = 0x7F0000000000          # aligned, never dereferenced by host checks
DTYPE, INVALID, UNSUPPORTED = pkg.FFPA_ERR_DTYPE, pkg.FFPA_ERR_INVALID, pkg.FFPA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    bld.build()
    return pkg.load_library()


def arr(*v):
    return (ctypes.c_int64 * len(v))(*v)


def decode_call(lib, dt=0, B=2, Hq=4, Hkv=2, D=128, pages=8, page=16, width=4, q=FAKE, k=FAKE, v=FAKE, o=FAKE,
                lse=None, table=FAKE, table_str=4, lens=FAKE, qs=None, ks=None, scale=None, gqa=1, ws=FAKE, ws_bytes=None,
                options=None):
    qs = qs or arr(Hq * D, D, 1)
    ks = ks or arr(page * Hkv * D, Hkv * D, D, 1)
    sc = None if scale is None else ctypes.byref(ctypes.c_float(scale))
    if ws_bytes is None:
        ws_bytes = 1 << 30
    return lib.ffpa_decode_paged(q, k, v, o, lse, dt, B, Hq, Hkv, D, pages, page, width, qs, ks, ks, qs, table,
                                 table_str, lens, sc, gqa, ws, ws_bytes, None, options)


def rope_arg(**kw):
    r = Rope(positions=FAKE, position_str_b=0, position_str_n=1, position_bits=32, rot_dim=64, inv_freq=FAKE,
             rope_scale=1.0, q_weight=FAKE, k_weight=FAKE, eps=1e-6)
    for n, x in kw.items():
        setattr(r, n, x)
    return r


def rope_call(lib, dt=0, B=2, Hq=4, Hkv=2, N=16, D=128, q=FAKE, qs=None, out=FAKE, rope=None):
    a, b = arr(Hq * N * D, N * D, D, 1), arr(Hkv * N * D, N * D, D, 1)
    return lib.ffpa_qk_norm_rope(q, FAKE, out, FAKE, dt, B, Hq, Hkv, N, D, qs or a, b, a, b, rope or rope_arg(), None)


def bwd_call(lib, dt=0, B=2, Hq=4, Hkv=2, N=16, D=128, dqw=FAKE, dkw=FAKE, ws=FAKE, ws_bytes=1 << 30, rope=None):
    a, b = arr(Hq * N * D, N * D, D, 1), arr(Hkv * N * D, N * D, D, 1)
    return lib.ffpa_qk_norm_rope_bwd(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, dqw, dkw, dt, B, Hq, Hkv, N, D, a, b, a, b, a, b,
                                     rope or rope_arg(), ws, ws_bytes, None)


def append_call(lib, dt=0, T=16, Hq=4, Hkv=2, D=128, pages=8, page=16, q=FAKE, qo=FAKE, k=FAKE, slots=FAKE, ks=None,
                cs=None, rope=None):
    a, b = arr(Hq * D, D, 1), arr(Hkv * D, D, 1)
    cs = cs or arr(page * Hkv * D, Hkv * D, D, 1)
    return lib.ffpa_kv_append(q, k, FAKE, qo, FAKE, FAKE, dt, T, Hq, Hkv, D, pages, page, a, ks or b, b, a, cs, cs, slots,
                              rope or rope_arg(), None, None)


def plan_call(lib, B=4, width=8, table=FAKE, table_str=8, lens=FAKE, new=FAKE + 64, free=FAKE, n_free=5, count=FAKE,
              page=16, tokens=10, slots=FAKE, pos=FAKE, cu=FAKE, lens_out=FAKE + 128, count_out=FAKE + 256):
    return lib.ffpa_page_plan(table, table_str, B, width, lens, new, free, n_free, count, page, tokens, slots, pos, cu,
                              lens_out, count_out, None, None)


def test_decode_refusals(lib):
    for kw, want in ((dict(dt=2), DTYPE), (dict(D=56), UNSUPPORTED), (dict(D=1032), UNSUPPORTED), (dict(D=100), UNSUPPORTED),
                     (dict(B=-1), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=5), INVALID), (dict(gqa=0), INVALID),
                     (dict(page=0), INVALID), (dict(width=-1), INVALID), (dict(pages=-1), INVALID),
                     (dict(width=1 << 20, page=1 << 12), INVALID), (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID),
                     (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(k=None), INVALID), (dict(table=None), INVALID),
                     (dict(lens=None), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=1000), INVALID), (dict(ws=FAKE + 16), INVALID),
                     (dict(q=FAKE + 8), INVALID), (dict(k=FAKE + 2), INVALID), (dict(lse=FAKE + 2), INVALID), (dict(table=FAKE + 2), INVALID),
                     (dict(qs=arr(512, 128, 2)), INVALID), (dict(qs=arr(512, 132, 1)), INVALID), (dict(qs=arr(512, 0, 1)), INVALID),
                     (dict(ks=arr(4096, 256, -128, 1)), INVALID), (dict(ks=arr(4100, 256, 128, 1)), INVALID), (dict(table_str=3), INVALID)):
        assert decode_call(lib, **kw) == want, kw
    assert decode_call(lib, B=0) == pkg.FFPA_OK
    assert decode_call(lib, dt=7, D=3, q=None) == DTYPE          # the type first, then the head dim
    assert decode_call(lib, D=48, q=None) == UNSUPPORTED


def test_decode_workspace_size(lib):
    need = pkg.decode_paged_workspace_bytes(32, 8, 512)
    assert need > 0 and pkg.decode_paged_workspace_bytes(32, 8, 100) == 0 and pkg.decode_paged_workspace_bytes(3, 2, 128) == 0
    ok = decode_call(lib, Hq=32, Hkv=8, D=512, ws_bytes=need)
    assert ok in (pkg.FFPA_ERR_CUDA, INVALID)                    # past the size check: FAKE is no device memory
    assert decode_call(lib, Hq=32, Hkv=8, D=512, ws_bytes=need - 1) == INVALID


def test_rope_refusals(lib):
    for kw, want in ((dict(dt=3), DTYPE), (dict(D=40), UNSUPPORTED), (dict(D=68), UNSUPPORTED), (dict(B=-1), INVALID), (dict(N=-1), INVALID),
                     (dict(Hkv=0), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(q=FAKE + 8), INVALID),
                     (dict(qs=arr(8192, 2048, 128, 2)), INVALID), (dict(qs=arr(8192, 2048, 132, 1)), INVALID),
                     (dict(rope=rope_arg(rot_dim=136)), INVALID), (dict(rope=rope_arg(rot_dim=12)), INVALID), (dict(rope=rope_arg(rot_dim=-8)), INVALID),
                     (dict(rope=rope_arg(inv_freq=None)), INVALID), (dict(rope=rope_arg(positions=None)), INVALID),
                     (dict(rope=rope_arg(position_bits=16)), INVALID), (dict(rope=rope_arg(positions=FAKE + 2)), INVALID),
                     (dict(rope=rope_arg(eps=-1.0)), INVALID), (dict(rope=rope_arg(eps=math.nan)), INVALID),
                     (dict(rope=rope_arg(rope_scale=math.inf)), INVALID), (dict(rope=rope_arg(q_weight=FAKE + 1)), INVALID),
                     (dict(rope=rope_arg(weight_f32=1, k_weight=FAKE + 2)), INVALID)):
        assert rope_call(lib, **kw) == want, kw
    assert rope_call(lib, N=0) == pkg.FFPA_OK and rope_call(lib, B=0, q=None) == pkg.FFPA_OK
    assert rope_call(lib, N=0, rope=rope_arg(positions=None)) == pkg.FFPA_OK


def test_rope_backward_refusals(lib):
    for kw, want in ((dict(dt=3), DTYPE), (dict(D=40), UNSUPPORTED), (dict(dqw=None), INVALID), (dict(dkw=None), INVALID),
                     (dict(rope=rope_arg(q_weight=None)), INVALID), (dict(dqw=FAKE + 1), INVALID), (dict(ws=None), INVALID),
                     (dict(ws_bytes=pkg.qk_norm_rope_bwd_workspace_bytes(128) - 1), INVALID), (dict(ws=FAKE + 8), INVALID),
                     (dict(rope=rope_arg(rot_dim=12)), INVALID)):
        assert bwd_call(lib, **kw) == want, kw
    none = rope_arg(q_weight=None, k_weight=None)
    assert bwd_call(lib, rope=none, dqw=None, dkw=None, N=0) == pkg.FFPA_OK
    assert bwd_call(lib, rope=none, dqw=None, dkw=None, ws=None, ws_bytes=0) in (pkg.FFPA_ERR_CUDA, INVALID)
    assert pkg.qk_norm_rope_bwd_workspace_bytes(65) == 0


def test_append_refusals(lib):
    for kw, want in ((dict(dt=3), DTYPE), (dict(D=40), UNSUPPORTED), (dict(T=-1), INVALID), (dict(pages=0), INVALID), (dict(page=0), INVALID),
                     (dict(qo=None), INVALID), (dict(k=None), INVALID), (dict(slots=None), INVALID), (dict(slots=FAKE + 4), INVALID),
                     (dict(ks=arr(256, 132, 1)), INVALID), (dict(cs=arr(4096, 256, 128, 2)), INVALID), (dict(cs=arr(4096, 0, 128, 1)), INVALID),
                     (dict(q=FAKE + 4), INVALID), (dict(rope=rope_arg(rot_dim=20)), INVALID)):
        assert append_call(lib, **kw) == want, kw
    assert append_call(lib, T=0) == pkg.FFPA_OK


def test_plan_refusals(lib):
    for kw in (dict(B=0), dict(width=0), dict(n_free=-1), dict(page=0), dict(tokens=-1), dict(width=1 << 20, page=1 << 12, table_str=1 << 20),
               dict(table_str=7), dict(table=None), dict(lens=None), dict(new=None), dict(free=None), dict(count=None), dict(slots=None),
               dict(pos=None), dict(cu=None), dict(lens_out=None), dict(count_out=None), dict(lens_out=FAKE), dict(lens_out=FAKE + 64),
               dict(count_out=FAKE), dict(slots=FAKE + 4), dict(table=FAKE + 2)):
        assert plan_call(lib, **kw) == INVALID, kw


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_valid_calls_without_gpu_report_a_cuda_error(lib):
    for call in (decode_call, rope_call, bwd_call, append_call, plan_call):
        assert call(lib) == pkg.FFPA_ERR_CUDA, call.__name__


def test_binding_refusals(lib):
    q, kc = torch.zeros(2, 4, 128, dtype=torch.bfloat16), torch.zeros(3, 16, 2, 128, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    bad = [(dict(q=q[0]), ValueError), (dict(q=q.half()), TypeError), (dict(v_cache=kc[:2]), ValueError), (dict(k_cache=kc[..., :64]), ValueError),
           (dict(block_table=table.long()), TypeError), (dict(block_table=table[:1]), ValueError), (dict(block_table=table.t()), ValueError),
           (dict(seq_lens=lens.long()), TypeError), (dict(seq_lens=lens[:1]), ValueError), (dict(out=q[:1]), ValueError),
           (dict(workspace=torch.zeros(8)), ValueError), (dict(enable_gqa=False), ValueError), (dict(status=torch.zeros(2, dtype=torch.int32)), ValueError)]
    for kw, want in bad:
        a = dict(q=q, k_cache=kc, v_cache=kc, block_table=table, seq_lens=lens, enable_gqa=True)
        a.update(kw)
        with pytest.raises(want):
            pkg.ffpa_decode_paged(**a)
    k = torch.zeros(2, 2, 128, dtype=torch.bfloat16)
    pos, inv, w = torch.zeros(2, dtype=torch.int32), torch.ones(32, dtype=torch.float64), torch.ones(128)
    for kw, want in ((dict(k=k[:1]), ValueError), (dict(k=k.half()), TypeError), (dict(positions=None), ValueError), (dict(positions=pos.float()), TypeError),
                     (dict(positions=pos[:1]), ValueError), (dict(inv_freq=inv.float()), TypeError), (dict(inv_freq=torch.ones(80, dtype=torch.float64)), ValueError),
                     (dict(inv_freq=inv[:30]), ValueError), (dict(q_weight=w.half()), TypeError), (dict(q_weight=w[:64]), ValueError),
                     (dict(k_weight=w.bfloat16()), TypeError), (dict(q_out=q.half()), ValueError), (dict(eps=-1.0), ValueError), (dict(q=q[None]), ValueError)):
        a = dict(q=q, k=k, positions=pos, inv_freq=inv, q_weight=w, k_weight=w)
        a.update(kw)
        with pytest.raises(want):
            pkg.ffpa_qk_norm_rope(**a)
    with pytest.raises(ValueError):
        pkg.ffpa_qk_norm_rope_bwd(q[:1], k, q, k, pos, inv)
    with pytest.raises(TypeError):
        pkg.ffpa_qk_norm_rope_bwd(q.half(), k, q, k, pos, inv)
    slots = torch.zeros(2, dtype=torch.int64)
    for kw, want in ((dict(v=k[:1]), ValueError), (dict(v=k.half()), TypeError), (dict(slots=slots.int()), TypeError), (dict(slots=slots[:1]), ValueError),
                     (dict(k_cache=kc[:, :, :1], v_cache=kc[:, :, :1]), ValueError), (dict(q=None, q_weight=w), ValueError)):
        a = dict(q=q, k=k, v=k, k_cache=kc, v_cache=kc, slots=slots)
        a.update(kw)
        with pytest.raises(want):
            pkg.ffpa_kv_append(**a)
    free, count = torch.zeros(4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for kw, want in ((dict(seq_lens=lens.long()), TypeError), (dict(new_lens=lens[:1]), ValueError), (dict(free_count=free), ValueError),
                     (dict(num_tokens=-1), ValueError), (dict(page_size=0), ValueError), (dict(block_table=table.long()), TypeError)):
        a = dict(block_table=table, seq_lens=lens, new_lens=lens, free_pages=free, free_count=count, page_size=16, num_tokens=4)
        a.update(kw)
        with pytest.raises(want):
            pkg.ffpa_page_plan(**a)


def test_frequencies():
    inv, scale = pkg.rope_inv_freq(64)
    assert inv.dtype == torch.float64 and scale == 1.0
    assert torch.equal(inv, 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64))
    assert torch.equal(pkg.rope_inv_freq(64, scaling="linear", factor=4.0)[0], inv / 4)
    grown = pkg.rope_inv_freq(64, scaling="base", factor=8.0)[0]
    assert grown[0] == 1 and abs(grown[-1] * 8 / inv[-1] - 1) < 1e-12
    parts, scale = pkg.rope_inv_freq(64, scaling="by_parts", factor=8.0, original_length=4096)
    assert abs(scale - (0.1 * math.log(8) + 1)) < 1e-12
    turns = 4096 * inv / (2 * math.pi)
    # whole pairs on either side of the ramp; between them the factor only grows
    assert torch.equal(parts[turns > 32 * 1.4], inv[turns > 32 * 1.4])
    assert torch.allclose(parts[turns < 1 / 1.4], inv[turns < 1 / 1.4] / 8, rtol=1e-15)
    ratio = inv / parts
    assert (ratio[1:] >= ratio[:-1] - 1e-12).all() and ratio.max() <= 8 + 1e-12
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, factor=0.5), dict(rot_dim=8, scaling="cubic"),
                dict(rot_dim=8, scaling="by_parts"), dict(rot_dim=8, base=-1.0), dict(rot_dim=2, scaling="base")):
        with pytest.raises(ValueError):
            pkg.rope_inv_freq(**bad)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_reference_gradients_match_differences(norm, interleaved):
    """The formula the kernel evaluates, and the 64-bit derivative its tests compare it with, against
    central differences (64 bits, step 1e-6: truncation and rounding stay below 1e-8)."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(3, 2, 16, generator=g, dtype=torch.float64)
    w = 1 + 0.3 * torch.randn(16, generator=g, dtype=torch.float64) if norm else None
    up = torch.randn(3, 2, 16, generator=g, dtype=torch.float64)
    pos, inv = torch.tensor([0, 5, 100003]), pkg.rope_inv_freq(8)[0]
    how = dict(interleaved=interleaved, rope_scale=1.25)

    def f(x, w):
        return (po.rope(x, pos, inv, w, **how) * up).sum()

    def slope(at, call):
        d = torch.zeros_like(at).flatten()
        for i in range(at.numel()):
            e = torch.zeros_like(at).flatten()
            e[i] = 1e-6
            e = e.view_as(at)
            d[i] = (call(at + e) - call(at - e)) / 2e-6
        return d.view_as(at)

    xd = x.clone().requires_grad_()
    wd = None if w is None else w.clone().requires_grad_()
    grads = torch.autograd.grad(f(xd, wd), [xd] + ([wd] if norm else []))
    assert (grads[0] - slope(x, lambda t: f(t, w))).abs().max() < 1e-7
    # the kernel's closed form
    back = po.rope(up, -pos, inv, None, **how)
    if norm:
        assert (grads[1] - slope(w, lambda t: f(x, t))).abs().max() < 1e-7
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        xn = x * r
        assert (grads[1] - (back * xn).sum((0, 1))).abs().max() < 1e-12
        back = r * (w * back - xn * (w * back * xn).mean(-1, keepdim=True))
    assert (grads[0] - back).abs().max() < 1e-12
