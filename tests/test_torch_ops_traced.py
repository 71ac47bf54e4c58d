"""The attention operators' backwards under tracing: operators of their own, of which a second
derivative is refused.  CPU: with shapes alone.  GPU: traced training steps against eager ones."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import exact_headdim_attention_gb300 as pkg

BF = torch.bfloat16


def dense(device="cpu"):
    g = torch.Generator().manual_seed(3)
    return [torch.randn(2, h, 40, 128, generator=g).to(device=device, dtype=BF).requires_grad_() for h in (4, 2, 2)]


def packed(device="cpu"):
    g = torch.Generator().manual_seed(4)
    return [torch.randn(80, h, 128, generator=g).to(device=device, dtype=BF).requires_grad_() for h in (4, 2, 2)]


def attend(q, k, v, cu=None, mask=None):
    if cu is None:
        return pkg.ffpa_attn_func(q, k, v, attn_mask=mask, is_causal=True, enable_gqa=True)
    return pkg.ffpa_attn_varlen_func(q, k, v, cu, None, 50, 50, causal=True, enable_gqa=True)


@pytest.mark.parametrize("varlen", [False, True])
def test_backward_of_shapes_alone(varlen):
    with FakeTensorMode():
        leaves = packed() if varlen else dense()
        cu = torch.empty(3, dtype=torch.int32) if varlen else None
        grads = torch.autograd.grad(attend(*leaves, cu).float().sum(), leaves)
        assert [(g.shape, g.dtype) for g in grads] == [(x.shape, x.dtype) for x in leaves]


@pytest.mark.parametrize("varlen", [False, True])
def test_second_derivative_is_refused(varlen):
    with FakeTensorMode():
        leaves = packed() if varlen else dense()
        cu = torch.empty(3, dtype=torch.int32) if varlen else None
        grad = torch.autograd.grad(attend(*leaves, cu).float().square().sum(), leaves, create_graph=True)[0]
        assert grad.requires_grad
        with pytest.raises(NotImplementedError, match="second derivative"):
            grad.float().sum().backward()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["causal", "mask", "varlen"])
def test_traced_training_step_equals_the_eager_one(kind):
    dev = torch.device("cuda:0")
    make = packed if kind == "varlen" else dense
    cu = torch.tensor([0, 30, 80], dtype=torch.int32, device=dev) if kind == "varlen" else None
    mask = torch.rand(40, 40, generator=torch.Generator().manual_seed(5)).to(dev) < 0.8 if kind == "mask" else None

    def step(q, k, v):
        return attend(q * 1.0, k, v, cu, mask).float().square().sum()

    def grads(f):
        ls = make(dev)
        f(*ls).backward()
        return [t.grad for t in ls]

    want, got = grads(step), grads(torch.compile(step, fullgraph=True, backend="aot_eager"))
    assert all(torch.isfinite(a).all() and a.abs().max() > 0 for a in want)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.gpu
@pytest.mark.parametrize("varlen", [False, True])
def test_second_derivative_is_refused_on_the_gpu(varlen):
    dev = torch.device("cuda:0")
    leaves = packed(dev) if varlen else dense(dev)
    cu = torch.tensor([0, 30, 80], dtype=torch.int32, device=dev) if varlen else None
    loss = attend(*leaves, cu).float().square().sum()
    plain = torch.autograd.grad(loss, leaves, retain_graph=True)
    grads = torch.autograd.grad(loss, leaves, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(plain, grads))
    with pytest.raises(NotImplementedError, match="second derivative"):
        grads[1].float().square().sum().backward()
