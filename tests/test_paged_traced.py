"""The paged-cache calls and the head norm with rotation on tensors that have no memory (traced,
transformed, of shapes alone)."""

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import exact_headdim_attention_gb300 as pkg
from exact_headdim_attention_gb300 import build as bld

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    bld.build()


def calls(empty):
    """Every call of the binding, on tensors that `empty` makes."""
    q, k = empty(2, 4, 128, dtype=BF), empty(2, 2, 128, dtype=BF)
    kc, table = empty(3, 16, 2, 128, dtype=BF), empty(2, 2, dtype=torch.int32)
    lens, slots = empty(2, dtype=torch.int32), empty(2, dtype=torch.int64)
    return {"qk_norm_rope": lambda: pkg.ffpa_qk_norm_rope(q, k),
            "qk_norm_rope_bwd": lambda: pkg.ffpa_qk_norm_rope_bwd(q, k, q, k),
            "kv_append": lambda: pkg.ffpa_kv_append(q, k, k, kc, kc, slots),
            "decode_paged": lambda: pkg.ffpa_decode_paged(q, kc, kc, table, lens, enable_gqa=True),
            "page_plan": lambda: pkg.ffpa_page_plan(table, lens, lens, lens, lens[:1], 16, 4)}


@pytest.mark.parametrize("name", ["qk_norm_rope", "qk_norm_rope_bwd", "kv_append", "decode_paged", "page_plan"])
def test_binding_refuses_tensors_without_memory(name):
    with FakeTensorMode():
        with pytest.raises(TypeError, match="memory of its own"):
            calls(torch.empty)[name]()
    with pytest.raises(TypeError, match="memory of its own"):
        calls(lambda *s, dtype: torch.empty(*s, dtype=dtype, device="meta"))[name]()


def test_binding_refuses_transformed_tensors():
    q, k = torch.zeros(3, 2, 4, 128, dtype=BF), torch.zeros(2, 2, 128, dtype=BF)
    with pytest.raises(TypeError, match="memory of its own"):
        torch.vmap(lambda x: pkg.ffpa_qk_norm_rope(x, k)[0])(q)
    with pytest.raises(TypeError, match="memory of its own"):
        pkg.ffpa_qk_norm_rope(q[0].to_sparse(), k)
