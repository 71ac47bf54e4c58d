"""Which way ffpa_decode_shared takes by itself: one pass over all keys of each request, or the shared keys apart."""
import pytest
import torch

import exact_headdim_attention_gb300 as pkg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def call(B, Hq, Hkv, D, shared, own=40, page=32):
    """Arguments of a batch whose requests have `own` keys each behind `shared` shared ones, on random pages."""
    n, w = shared // page, -(-own // page)
    pages = n + B * w
    g = torch.Generator(device=DEV).manual_seed(B + Hq + D)
    k, v = (torch.randn(pages, page, Hkv, D, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, n + w), -1, dtype=torch.int32, device=DEV)
    table[:, n:] = order[n:].view(B, w)
    q = torch.randn(B, Hq, D, generator=g, device=DEV, dtype=torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)   # noqa: E731
    return q, k, v, order[:n].contiguous(), i32(shared), table, i32(*[shared + own] * B)


# (measured: where one way takes less than two thirds of the other's time)
@pytest.mark.parametrize("way,B,Hq,Hkv,D,shared", [
    ("split", 1, 128, 1, 512, 32768), ("split", 2, 64, 1, 256, 32768), ("split", 4, 128, 1, 128, 32768),
    ("split", 16, 40, 1, 64, 65536), ("split", 8, 12, 1, 512, 32768), ("split", 8, 32, 8, 256, 8192),
    ("single", 1, 16, 1, 512, 8192), ("single", 1, 8, 8, 128, 4096), ("single", 2, 17, 1, 64, 8192),
    ("single", 8, 4, 1, 64, 49152), ("single", 4, 4, 4, 128, 1024)])
def test_the_faster_way_is_taken(way, B, Hq, Hkv, D, shared):
    """By itself the call returns what the faster way returns, bit for bit (the two ways round differently)."""
    args = call(B, Hq, Hkv, D, shared)
    o = {w: pkg.ffpa_decode_shared(*args, enable_gqa=Hq != Hkv, kernel=w) for w in ("single", "split", None)}
    assert not torch.equal(o["single"], o["split"])
    assert torch.equal(o[None], o[way])


@pytest.mark.parametrize("way", ["single", "split"])
def test_a_traced_model_chooses_the_way(way):
    """The operator takes the way that its caller names, traced too, whatever the sizes would take."""
    args = call(4, 8, 2, 128, 512)
    want = pkg.ffpa_decode_shared(*args, enable_gqa=True, kernel=way)
    assert torch.equal(pkg.ffpa_attn_decode_shared_func(*args, enable_gqa=True, kernel=way), want)
    step = torch.compile(lambda q: pkg.ffpa_attn_decode_shared_func(q * 1, *args[1:], enable_gqa=True, kernel=way),
                         backend="eager", fullgraph=True)
    assert torch.equal(step(args[0]), want)
    with pytest.raises(ValueError):
        pkg.ffpa_attn_decode_shared_func(*args, enable_gqa=True, kernel="both")
