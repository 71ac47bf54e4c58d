"""The operator of decode attention behind shared pages without a GPU: its way is an argument, and may be left out."""
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import exact_headdim_attention_gb300 as pkg

BF = torch.bfloat16


def test_the_way_is_an_argument():
    names = [a.name for a in torch.ops.ffpa.decode_shared.default._schema.arguments]
    assert names[-1] == "kernel"
    with FakeTensorMode():
        q, k = torch.empty(4, 8, 128, dtype=BF), torch.empty(5, 16, 2, 128, dtype=BF)
        table, n = torch.empty(4, 3, dtype=torch.int32), torch.empty(4, dtype=torch.int32)
        for kernel in (None, "single", "split"):
            o, lse = pkg.ffpa_attn_decode_shared_func(q, k, k, n, n[:1], table, n, enable_gqa=True, return_lse=True, kernel=kernel)
            assert o.shape == q.shape and lse.shape == (4, 8)
        o, _ = torch.ops.ffpa.decode_shared(q, k, k, n, n[:1], table, n, None, True)
        assert o.shape == q.shape
