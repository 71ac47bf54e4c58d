"""Host side of the 8-bit paged cache and of decode attention behind shared pages: refusals of the C ABI
and of the binding, operators' registration and fakes, and the references that the GPU tests use."""
import contextlib
import ctypes
import functools
import math

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import exact_headdim_attention_gb300 as pkg
from exact_headdim_attention_gb300 import build as bld
from exact_headdim_attention_gb300._binding import Options
from tests import paged_fp8_oracle as p8
from tests.test_paged_host import FAKE, arr, rope_arg

DTYPE, INVALID, UNSUPPORTED, OK = pkg.FFPA_ERR_DTYPE, pkg.FFPA_ERR_INVALID, pkg.FFPA_ERR_UNSUPPORTED, pkg.FFPA_OK
BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    bld.build()
    return pkg.load_library()


def decode8_call(lib, dt=0, B=2, Hq=4, Hkv=2, D=128, pages=8, page=16, width=4, q=FAKE, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, o=FAKE,
                 lse=None, table=FAKE, table_str=4, lens=FAKE, q_str=None, k_str=None, s_str=None, scale=None, gqa=1, ws=FAKE,
                 ws_bytes=1 << 30):
    q_str = q_str or arr(Hq * D, D, 1)
    k_str = k_str or arr(page * Hkv * D, Hkv * D, D, 1)
    s_str = s_str or arr(Hkv * page, page, 1)
    sc = None if scale is None else ctypes.byref(ctypes.c_float(scale))
    return lib.ffpa_decode_paged_fp8(q, k, v, ks, vs, o, lse, dt, B, Hq, Hkv, D, pages, page, width, q_str, k_str, k_str, s_str,
                                     s_str, q_str, table, table_str, lens, sc, gqa, ws, ws_bytes, None, None)


def append8_call(lib, dt=0, T=16, Hq=4, Hkv=2, D=128, pages=8, page=16, q=FAKE, qo=FAKE, k=FAKE, kc=FAKE, ks=FAKE, vs=FAKE, slots=FAKE,
                 k_str=None, c_str=None, s_str=None, rope=None):
    a, b = arr(Hq * D, D, 1), arr(Hkv * D, D, 1)
    c_str = c_str or arr(page * Hkv * D, Hkv * D, D, 1)
    s_str = s_str or arr(Hkv * page, page, 1)
    return lib.ffpa_kv_append_fp8(q, k, FAKE, qo, kc, FAKE, ks, vs, dt, T, Hq, Hkv, D, pages, page, a, k_str or b, b, a, c_str, c_str,
                                  s_str, s_str, slots, rope or rope_arg(), None, None)


def read_call(lib, dt=0, T=20, B=2, Hkv=2, D=128, pages=8, page=16, width=4, kc=FAKE, ks=FAKE, vs=FAKE, k=FAKE, v=FAKE, table=FAKE,
              table_str=4, cu=FAKE, c_str=None, s_str=None, k_str=None):
    c_str = c_str or arr(page * Hkv * D, Hkv * D, D, 1)
    s_str = s_str or arr(Hkv * page, page, 1)
    k_str = k_str or arr(Hkv * D, D, 1)
    return lib.ffpa_kv_read(kc, FAKE, ks, vs, k, v, dt, T, B, Hkv, D, pages, page, width, c_str, c_str, s_str, s_str, k_str, k_str, table,
                            table_str, cu, None, None)


def shared_call(lib, dt=0, B=2, Hq=4, Hkv=2, D=128, pages=8, page=16, width=4, n=3, q=FAKE, k=FAKE, o=FAKE, sp=FAKE, sl=FAKE, table=FAKE,
                table_str=4, lens=FAKE, q_str=None, scale=None, gqa=1, ws=FAKE, ws_bytes=1 << 30,
                kernel=0):
    q_str = q_str or arr(Hq * D, D, 1)
    k_str = arr(page * Hkv * D, Hkv * D, D, 1)
    sc = None if scale is None else ctypes.byref(ctypes.c_float(scale))
    return lib.ffpa_decode_shared(q, k, FAKE, o, None, dt, B, Hq, Hkv, D, pages, page, width, n, q_str, k_str, k_str, q_str, sp, sl, table,
                                  table_str, lens, sc, gqa, ws, ws_bytes, None, ctypes.byref(Options(None, 0, kernel, 0)))


def test_decode_fp8_refusals(lib):
    for kw, want in ((dict(dt=2), DTYPE), (dict(D=56), UNSUPPORTED), (dict(D=72), UNSUPPORTED), (dict(D=1040), UNSUPPORTED), (dict(B=-1), INVALID),
                     (dict(Hkv=0), INVALID), (dict(Hq=5), INVALID), (dict(gqa=0), INVALID), (dict(page=0), INVALID), (dict(width=-1), INVALID),
                     (dict(width=1 << 20, page=1 << 12), INVALID), (dict(scale=math.inf), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
                     (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(ks=FAKE + 2), INVALID), (dict(vs=FAKE + 1), INVALID),
                     (dict(s_str=arr(32, 16, 2)), INVALID), (dict(s_str=arr(0, 16, 1)), INVALID), (dict(s_str=arr(32, -1, 1)), INVALID),
                     (dict(k_str=arr(4096, 256, 120, 1)), INVALID), (dict(k_str=arr(4096, 264, 128, 1)), INVALID), (dict(k=FAKE + 8), INVALID),
                     (dict(ws_bytes=1000), INVALID), (dict(ws=FAKE + 16), INVALID), (dict(table_str=3), INVALID), (dict(lens=None), INVALID)):
        assert decode8_call(lib, **kw) == want, kw
    assert decode8_call(lib, B=0) == OK and decode8_call(lib, dt=7, D=3, q=None) == DTYPE
    need = lib.ffpa_decode_paged_fp8_workspace_bytes(32, 8, 512)
    assert need == pkg.decode_paged_workspace_bytes(32, 8, 512) > 0 and lib.ffpa_decode_paged_fp8_workspace_bytes(32, 8, 72) == 0


def test_append_fp8_refusals(lib):
    for kw, want in ((dict(dt=3), DTYPE), (dict(D=40), UNSUPPORTED), (dict(D=72, rope=rope_arg(rot_dim=8)), UNSUPPORTED), (dict(T=-1), INVALID),
                     (dict(pages=0), INVALID), (dict(page=0), INVALID), (dict(qo=None), INVALID), (dict(k=None), INVALID), (dict(slots=None), INVALID),
                     (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(ks=FAKE + 2), INVALID), (dict(s_str=arr(32, 16, 3)), INVALID),
                     (dict(c_str=arr(4096, 264, 128, 1)), INVALID), (dict(kc=FAKE + 8), INVALID), (dict(rope=rope_arg(rot_dim=20)), INVALID)):
        assert append8_call(lib, **kw) == want, kw
    assert append8_call(lib, T=0) == OK


def test_read_refusals(lib):
    for kw, want in ((dict(dt=3), DTYPE), (dict(D=40), UNSUPPORTED), (dict(D=72), UNSUPPORTED), (dict(D=68, ks=None, vs=None), UNSUPPORTED),
                     (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(Hkv=0), INVALID), (dict(page=0), INVALID), (dict(width=-1), INVALID),
                     (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(kc=None), INVALID),
                     (dict(cu=None), INVALID), (dict(table=None), INVALID), (dict(cu=FAKE + 2), INVALID), (dict(k=FAKE + 8), INVALID),
                     (dict(k_str=arr(256, 132, 1)), INVALID), (dict(s_str=arr(32, 16, 2)), INVALID), (dict(c_str=arr(4096, 264, 128, 1)), INVALID),
                     (dict(table_str=3), INVALID), (dict(width=1 << 20, page=1 << 12, table_str=1 << 20), INVALID)):
        assert read_call(lib, **kw) == want, kw
    assert read_call(lib, T=0) == OK and read_call(lib, B=0) == OK


def test_shared_refusals(lib):
    for kw, want in ((dict(dt=2), DTYPE), (dict(D=56), UNSUPPORTED), (dict(D=72), UNSUPPORTED), (dict(D=1088), UNSUPPORTED), (dict(page=12), UNSUPPORTED),
                     (dict(Hq=258, Hkv=2), UNSUPPORTED), (dict(n=-1), INVALID), (dict(B=-1), INVALID), (dict(Hq=5), INVALID), (dict(gqa=0), INVALID),
                     (dict(sp=None), INVALID), (dict(sl=None), INVALID), (dict(sp=FAKE + 2), INVALID), (dict(sl=FAKE + 1), INVALID),
                     (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(o=None), INVALID), (dict(lens=None), INVALID), (dict(table=None), INVALID),
                     (dict(ws=None), INVALID), (dict(ws=FAKE + 16), INVALID), (dict(q_str=arr(512, 132, 1)), INVALID), (dict(scale=math.nan), INVALID),
                     (dict(kernel=-1), INVALID), (dict(kernel=2), INVALID), (dict(kernel=4), INVALID), (dict(kernel=5), INVALID)):
        assert shared_call(lib, **kw) == want, kw
    assert shared_call(lib, B=0) == OK
    need = pkg.decode_shared_workspace_bytes(2, 4, 2, 128)
    assert shared_call(lib, ws_bytes=need - 1) == INVALID and shared_call(lib, ws_bytes=need) in (pkg.FFPA_ERR_CUDA, INVALID)
    assert pkg.decode_shared_workspace_bytes(2, 4, 2, 72) == 0 and pkg.decode_shared_workspace_bytes(-1, 4, 2, 64) == 0
    assert pkg.decode_shared_workspace_bytes(0, 4, 2, 64) > 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_valid_calls_without_gpu_report_a_cuda_error(lib):
    for call in (decode8_call, append8_call, read_call, shared_call):
        assert call(lib) == pkg.FFPA_ERR_CUDA, call.__name__


def test_binding_refusals(lib):
    q, kc = torch.zeros(2, 4, 128, dtype=BF), torch.zeros(3, 16, 2, 128).to(E4M3)
    ks = torch.ones(3, 2, 16)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    for kw, want in ((dict(q=q[0]), ValueError), (dict(k_cache=kc.to(BF)), TypeError), (dict(k_cache=kc.view(torch.uint8)), TypeError),
                     (dict(k_scale=ks.double()), TypeError), (dict(k_scale=ks[:2]), ValueError), (dict(v_scale=ks.transpose(1, 2)), ValueError),
                     (dict(v_cache=kc[:2]), ValueError), (dict(block_table=table[:1]), ValueError), (dict(seq_lens=lens.long()), TypeError),
                     (dict(out=q[:1]), ValueError), (dict(enable_gqa=False), ValueError)):
        a = dict(q=q, k_cache=kc, v_cache=kc, k_scale=ks, v_scale=ks, block_table=table, seq_lens=lens, enable_gqa=True)
        a.update(kw)
        with pytest.raises(want):
            pkg.ffpa_decode_paged_fp8(**a)
    k, slots = torch.zeros(2, 2, 128, dtype=BF), torch.zeros(2, dtype=torch.int64)
    for kw, want in ((dict(v=k[:1]), ValueError), (dict(slots=slots.int()), TypeError), (dict(k_cache=kc.to(BF)), TypeError),
                     (dict(k_scale=ks.half()), TypeError), (dict(v_scale=ks[:, :1]), ValueError), (dict(q=None, q_weight=torch.ones(128)), ValueError)):
        a = dict(q=q, k=k, v=k, k_cache=kc, v_cache=kc, k_scale=ks, v_scale=ks, slots=slots)
        a.update(kw)
        with pytest.raises(want):
            pkg.ffpa_kv_append_fp8(**a)
    cu = torch.zeros(3, dtype=torch.int32)
    for kw, want in ((dict(cu_seqlens=cu[:2]), ValueError), (dict(cu_seqlens=cu.long()), TypeError), (dict(num_tokens=-1), ValueError),
                     (dict(k_scale=None), ValueError), (dict(k_scale=None, v_scale=None), ValueError), (dict(dtype=torch.float32), TypeError),
                     (dict(dtype="bf16"), TypeError), (dict(k_out=torch.zeros(4, 2, 128)), ValueError), (dict(k_cache=kc.to(BF), v_cache=kc.to(BF)), ValueError),
                     (dict(k_cache=kc.to(BF), v_cache=kc.to(BF), k_scale=None, v_scale=None, dtype=torch.float16), TypeError),
                     (dict(k_cache=kc[0], v_cache=kc[0]), ValueError)):
        a = dict(k_cache=kc, v_cache=kc, block_table=table, cu_seqlens=cu, num_tokens=4, k_scale=ks, v_scale=ks)
        a.update(kw)
        with pytest.raises(want):
            pkg.ffpa_kv_read(**a)
    k16, sp, sl = kc.to(BF), torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for kw, want in ((dict(q=q.half()), TypeError), (dict(k_cache=kc, v_cache=kc), TypeError), (dict(shared_pages=sp.long()), TypeError),
                     (dict(shared_pages=sp[None]), ValueError), (dict(shared_len=torch.zeros(2, dtype=torch.int32)), ValueError),
                     (dict(shared_len=sl.long()), TypeError), (dict(kernel="both"), ValueError), (dict(kernel="dual"), ValueError), (dict(block_table=table[:1]), ValueError)):
        a = dict(q=q, k_cache=k16, v_cache=k16, shared_pages=sp, shared_len=sl, block_table=table, seq_lens=lens, enable_gqa=True)
        a.update(kw)
        with pytest.raises(want):
            pkg.ffpa_decode_shared(**a)


def test_operators_are_registered_and_declare_their_writes():
    writes = {n: [a.name for a in getattr(torch.ops.ffpa, n).default._schema.arguments if a.alias_info and a.alias_info.is_write]
              for n in ("kv_append_fp8", "decode_paged_fp8", "kv_read", "decode_shared")}
    assert writes == {"kv_append_fp8": ["k_cache", "v_cache", "k_scale", "v_scale"], "decode_paged_fp8": [], "kv_read": [], "decode_shared": []}


def test_fakes():
    with FakeTensorMode():
        q, k = torch.empty(4, 8, 128, dtype=BF), torch.empty(4, 2, 128, dtype=BF)
        k16 = torch.empty(5, 16, 2, 128, dtype=BF)
        kc, ks = torch.empty(5, 16, 2, 128, dtype=E4M3), torch.empty(5, 2, 16)
        slots, table, n = torch.empty(4, dtype=torch.int64), torch.empty(4, 3, dtype=torch.int32), torch.empty(4, dtype=torch.int32)
        assert pkg.ffpa_kv_append_fp8_func(q, k, k, kc, kc.clone(), ks, ks.clone(), slots).shape == q.shape
        assert pkg.ffpa_kv_append_fp8_func(None, k, k, kc, kc.clone(), ks, ks.clone(), slots) is None
        for o, lse in (pkg.ffpa_attn_decode_fp8_func(q, kc, kc, ks, ks, table, n, enable_gqa=True, return_lse=True),
                       pkg.ffpa_attn_decode_shared_func(q, k16, k16, n, n[:1], table, n, enable_gqa=True, return_lse=True)):
            assert o.shape == q.shape and o.dtype == BF and lse.shape == (4, 8) and lse.dtype == torch.float32
        a, b = pkg.ffpa_kv_read_func(kc, kc, table, torch.empty(5, dtype=torch.int32), 7, k_scale=ks, v_scale=ks)
        assert a.shape == b.shape == (7, 2, 128) and a.dtype == BF
        a, b = pkg.ffpa_kv_read_func(k16.half(), k16.half(), table, torch.empty(5, dtype=torch.int32), 7)
        assert a.dtype == torch.float16


def test_the_reference_rounds_as_the_type_does():
    """Every finite fp16 value up to 448 (all e4m3 values, midpoints and subnormals among them) against torch's conversion."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.float16).float()
    x = x[torch.isfinite(x) & (x.abs() <= 448)]
    assert torch.equal(p8.nearest_e4m3(x.double()), x.to(E4M3).float().double())


def test_the_reference_decode_is_attention_over_the_values():
    g = torch.Generator().manual_seed(1)
    cache = p8.make_cache(g, [37], 2, 64, 16, spread=2.0)
    q = torch.randn(1, 4, 64, generator=g).to(BF)
    o, lse, _, _ = p8.decode(q, *cache)
    kc, vc, ks, vs, table, n = cache
    k, _ = p8.read(kc, ks, table, n, BF)
    v, _ = p8.read(vc, vs, table, n, BF)
    want = torch.nn.functional.scaled_dot_product_attention(q.double().transpose(0, 1)[None], k.transpose(0, 1)[None],
                                                            v.transpose(0, 1)[None], enable_gqa=True)[0].transpose(0, 1)
    assert (o - want).abs().max() < 1e-12


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_binding_refuses_tensors_without_memory(device):
    """The calls under the operators take tensors with memory only: traced ones (and such on no device) are refused."""
    with FakeTensorMode() if device == "cpu" else contextlib.nullcontext():
        e = functools.partial(torch.empty, device=device)
        q, k, kc = e(2, 4, 128, dtype=BF), e(2, 2, 128, dtype=BF), e(3, 16, 2, 128, dtype=BF)
        kq, ks = e(3, 16, 2, 128, dtype=E4M3), e(3, 2, 16)
        table, lens, slots = e(2, 2, dtype=torch.int32), e(2, dtype=torch.int32), e(2, dtype=torch.int64)
        for call in (lambda: pkg.ffpa_kv_append_fp8(q, k, k, kq, kq, ks, ks, slots),
                     lambda: pkg.ffpa_decode_paged_fp8(q, kq, kq, ks, ks, table, lens, enable_gqa=True),
                     lambda: pkg.ffpa_kv_read(kc, kc, table, e(3, dtype=torch.int32), 8),
                     lambda: pkg.ffpa_decode_shared(q, kc, kc, lens, lens[:1], table, lens, enable_gqa=True)):
            with pytest.raises(TypeError, match="memory of its own"):
                call()
