"""Caches whose offsets pass 32 bits: rows in far pages are those of near ones."""
import pytest
import torch

import exact_headdim_attention_gb300 as pkg
from tests.gpu_util import device_ok

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
PAGE, HKV, D, T = 16, 8, 512, 200


def rows(pages):
    """Scattered pages of T tokens, the last of the cache among them; their slots; keys, values and queries."""
    g = torch.Generator().manual_seed(1)
    ids = torch.tensor([pages - 1, pages // 2, 1, pages - 2, 30000, 10001, 32768, 33000, 32767, 32769, 39000, 37535, 25000], device=DEV)
    assert ids.unique().numel() == ids.numel()
    t = torch.arange(T, device=DEV)
    k, v, q = (torch.randn(n, h, D, generator=g).to(torch.bfloat16).to(DEV) for n, h in ((T, HKV), (T, HKV), (1, 32)))
    return ids, ids[t // PAGE] * PAGE + t % PAGE, k, v, q


def near(n):
    return torch.arange(n, dtype=torch.int32, device=DEV)[None]


def test_codes():
    pages = 70000                                              # 4.6 GB of codes each
    ids, slots, k, v, q = rows(pages)
    kc, vc = (torch.zeros(pages, PAGE, HKV, D, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = torch.zeros(2, pages, HKV, PAGE, device=DEV)
    pkg.ffpa_kv_append_fp8(None, k, v, kc, vc, ks, vs, slots)
    few = [c.view(torch.uint8)[ids].view(torch.float8_e4m3fn) for c in (kc, vc)] + [ks[ids], vs[ids]]
    again = [torch.zeros_like(x.view(torch.uint8)).view(x.dtype) if x.dtype != torch.float32 else torch.zeros_like(x) for x in few]
    pkg.ffpa_kv_append_fp8(None, k, v, *again, torch.arange(T, device=DEV))
    for a, b in zip(few, again):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    lens, table = torch.tensor([T], dtype=torch.int32, device=DEV), ids[None].int()
    o = pkg.ffpa_decode_paged_fp8(q, kc, vc, ks, vs, table, lens, enable_gqa=True)
    assert torch.equal(o, pkg.ffpa_decode_paged_fp8(q, *few, near(ids.numel()), lens, enable_gqa=True))
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    a = pkg.ffpa_kv_read(kc, vc, table, cu, T, k_scale=ks, v_scale=vs)
    b = pkg.ffpa_kv_read(few[0], few[1], near(ids.numel()), cu, T, k_scale=few[2], v_scale=few[3])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    device_ok()


def test_shared_pages():
    pages = 40000                                              # 5.2 GB each
    ids, slots, k, v, q = rows(pages)
    kc, vc = torch.zeros(2, pages, PAGE, HKV, D, dtype=torch.bfloat16, device=DEV)
    pkg.ffpa_kv_append(None, k, v, kc, vc, slots)
    table, lens = ids[None].int(), torch.tensor([T], dtype=torch.int32, device=DEV)
    shared = torch.tensor([128], dtype=torch.int32, device=DEV)
    few = near(ids.numel())
    for kernel in ("split", "single"):
        o = pkg.ffpa_decode_shared(q, kc, vc, table[0, :8].contiguous(), shared, table, lens, enable_gqa=True, kernel=kernel)
        want = pkg.ffpa_decode_shared(q, kc[ids], vc[ids], few[0, :8].contiguous(), shared, few, lens, enable_gqa=True, kernel=kernel)
        assert torch.equal(o, want)
    device_ok()
