"""The torch operators around a paged cache.  CPU: registration, shape-only fakes, declared writes.
GPU: eager calls, gradients through autograd into the attention operators, tracing."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import exact_headdim_attention_gb300 as pkg
from exact_headdim_attention_gb300 import torch_ops
from tests import paged_oracle as po

BF = torch.bfloat16


def test_registered():
    for name in ("qk_norm_rope", "kv_append", "decode_paged", "page_plan"):
        assert hasattr(torch.ops.ffpa, name)
    assert torch._C._dispatch_has_kernel_for_dispatch_key("ffpa::qk_norm_rope", "Autograd")
    op = torch_ops.qk_norm_rope
    assert getattr(op, "_backward_fn", torch_ops._qk_norm_rope_backward) is torch_ops._qk_norm_rope_backward
    writes = {n: [a.name for a in getattr(torch.ops.ffpa, n).default._schema.arguments if a.alias_info and a.alias_info.is_write]
              for n in ("qk_norm_rope", "kv_append", "decode_paged", "page_plan")}
    assert writes == {"qk_norm_rope": [], "kv_append": ["k_cache", "v_cache"], "decode_paged": [], "page_plan": ["block_table"]}


def test_fakes():
    with FakeTensorMode():
        q, k = torch.empty(2, 8, 10, 128, dtype=BF), torch.empty(2, 2, 10, 128, dtype=BF)
        a, b = pkg.ffpa_qk_norm_rope_func(q, k)
        assert a.shape == q.shape and b.shape == k.shape and a.dtype == BF
        kc = torch.empty(5, 16, 2, 128, dtype=BF)
        q3, k3 = torch.empty(4, 8, 128, dtype=BF), torch.empty(4, 2, 128, dtype=BF)
        slots = torch.empty(4, dtype=torch.int64)
        assert pkg.ffpa_kv_append_func(q3, k3, k3, kc, kc.clone(), slots).shape == q3.shape
        assert pkg.ffpa_kv_append_func(None, k3, k3, kc, kc.clone(), slots) is None
        table, n = torch.empty(4, 3, dtype=torch.int32), torch.empty(4, dtype=torch.int32)
        o, lse = pkg.ffpa_attn_decode_func(q3, kc, kc, table, n, enable_gqa=True, return_lse=True)
        assert o.shape == q3.shape and lse.shape == (4, 8) and lse.dtype == torch.float32
        s, p, cu, ln, c = pkg.ffpa_page_plan_func(table, n, n, n, n[:1], 16, 9)
        assert s.shape == (9,) and s.dtype == torch.int64 and p.dtype == torch.int32
        assert cu.shape == (5,) and ln.shape == (4,) and c.shape == (1,)


@pytest.mark.gpu
def test_gradients_reach_leaves_and_skip_what_is_not_asked():
    dev = torch.device("cuda:0")
    g = torch.Generator().manual_seed(1)
    q, k = torch.randn(30, 4, 128, generator=g).to(BF), torch.randn(30, 2, 128, generator=g).to(BF)
    w = (1 + 0.2 * torch.randn(128, generator=g))
    pos, inv = torch.arange(30), pkg.rope_inv_freq(64)[0]
    up = torch.randn(30, 4, 128, generator=g).to(BF)
    ql, kl, wl = (t.to(dev).requires_grad_() for t in (q, k, w))
    qo, ko = pkg.ffpa_qk_norm_rope_func(ql, kl, pos.to(dev), inv.to(dev), wl, wl)
    (qo * up.to(dev)).sum().backward()                      # the keys' output is not used
    dx, dw, bx, bw = po.rope_grads(up, q, pos, inv, w)
    assert ((ql.grad.double().cpu() - dx).abs() <= bx).all()
    assert ((wl.grad.double().cpu() - dw).abs() <= bw).all()      # + the keys' share, which is zero
    assert (kl.grad == 0).all()
    # a gradient that is one broadcast value
    ql.grad = None
    qo, ko = pkg.ffpa_qk_norm_rope_func(ql, kl, pos.to(dev), inv.to(dev), wl, wl)
    (qo.sum() + ko.sum()).backward()
    dx, _, bx, _ = po.rope_grads(torch.ones_like(up), q, pos, inv, w)
    assert ((ql.grad.double().cpu() - dx).abs() <= bx).all()
    with pytest.raises(NotImplementedError):
        f = inv.to(dev).requires_grad_()
        pkg.ffpa_qk_norm_rope_func(ql, kl, pos.to(dev), f)[0].sum().backward()


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
def test_training_step_through_norm_rope_and_attention(packed):
    """Norm and rotation, then causal attention: the gradients of q, k, v and the weights against a
    64-bit chain.  Each stage rounds to bf16: the rounded rotated q and k perturb the scores, the
    attention's own bound is 2e-2 / 1e-2 of the largest / mean gradient (test_gpu_backward.py), and
    the rounded dq, dk pass through the norm's backward, which does not amplify (its gain is w r,
    near 1 for these inputs): twice that bound."""
    dev = torch.device("cuda:0")
    g = torch.Generator().manual_seed(4)
    B, Hq, Hkv, N, D = 2, 4, 2, 150, 256
    def rows(H):
        return torch.randn(B * N, H, D, generator=g).to(BF) if packed else torch.randn(B, H, N, D, generator=g).to(BF)
    q, k, v, up = rows(Hq), rows(Hkv), rows(Hkv), rows(Hq)
    w = 1 + 0.2 * torch.randn(2, D, generator=g)
    pos, inv = torch.arange(N), pkg.rope_inv_freq(D // 2)[0]
    if packed:
        pos = pos.repeat(B)
    leaves = [t.to(dev).requires_grad_() for t in (q, k, v, w[0], w[1])]
    qr, kr = pkg.ffpa_qk_norm_rope_func(leaves[0], leaves[1], pos.to(dev), inv.to(dev), leaves[3], leaves[4])
    if packed:
        cu = torch.arange(0, B * N + 1, N, dtype=torch.int32, device=dev)
        o = pkg.ffpa_attn_varlen_func(qr, kr, leaves[2], cu, None, N, N, causal=True, enable_gqa=True)
    else:
        o = pkg.ffpa_attn_func(qr, kr, leaves[2], is_causal=True, enable_gqa=True)
    o.backward(up.to(dev))
    ref = [t.double().requires_grad_() for t in (q, k, v, w[0], w[1])]

    def dense(t):     # [B, N, H, D] -> [B, H, N, D] of packed rows
        return t.view(B, N, -1, D).transpose(1, 2) if packed else t

    at = pos.view(B, N) if packed else pos.expand(B, N)
    qd = po.rope(dense(ref[0]).transpose(1, 2), at, inv, ref[3]).transpose(1, 2)
    kd = po.rope(dense(ref[1]).transpose(1, 2), at, inv, ref[4]).transpose(1, 2).repeat_interleave(Hq // Hkv, 1)
    vd = dense(ref[2]).repeat_interleave(Hq // Hkv, 1)
    s = (qd @ kd.transpose(2, 3)) * D ** -0.5
    s = s.masked_fill(torch.ones(N, N, dtype=torch.bool).triu(1), float("-inf"))
    (torch.softmax(s, -1) @ vd).backward(dense(up).double())
    for name, a, b in zip(("q", "k", "v", "q_weight", "k_weight"), leaves, ref):
        err = (a.grad.double().cpu() - b.grad).abs()
        assert err.max() <= 4e-2 * b.grad.abs().max() and err.mean() <= 2e-2 * b.grad.abs().mean(), name


@pytest.mark.gpu
def test_generation_step_through_the_operators_and_traced():
    dev = torch.device("cuda:0")
    g = torch.Generator().manual_seed(6)
    B, Hq, Hkv, D, page = 3, 4, 2, 128, 8
    qkv = torch.randn(7, Hq + 2 * Hkv, D, generator=g).to(BF).to(dev)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    inv = pkg.rope_inv_freq(D)[0].to(dev)
    free = torch.arange(20, dtype=torch.int32, device=dev)
    count, lens = torch.tensor([20], dtype=torch.int32, device=dev), torch.zeros(B, dtype=torch.int32, device=dev)
    new = torch.tensor([2, 4, 1], dtype=torch.int32, device=dev)
    last = torch.tensor([1, 5, 6], device=dev)

    def step(kc, vc, table):
        slots, pos, cu, n, c = pkg.ffpa_page_plan_func(table, lens, new, free, count, page, 7)
        qr = pkg.ffpa_kv_append_func(q, k, v, kc, vc, slots, pos, inv)
        return pkg.ffpa_attn_decode_func(qr[last], kc, vc, table, n, enable_gqa=True), n

    def fresh():
        return (torch.zeros(20, page, Hkv, D, dtype=BF, device=dev), torch.zeros(20, page, Hkv, D, dtype=BF, device=dev),
                torch.full((B, 4), -1, dtype=torch.int32, device=dev))

    o, n = step(*fresh())
    # the same through the binding
    kc, vc, table = fresh()
    slots, pos, cu, n2, c = pkg.ffpa_page_plan(table, lens, new, free, count, page, 7)
    qr = pkg.ffpa_kv_append(q, k, v, kc, vc, slots, pos, inv)
    want = pkg.ffpa_decode_paged(qr[last], kc, vc, table, n2, enable_gqa=True)
    assert torch.equal(o, want) and n.tolist() == [2, 4, 1]
    traced = torch.compile(step, fullgraph=True, backend="aot_eager")
    a = fresh()
    ot, nt = traced(*a)
    assert torch.equal(ot, want) and torch.equal(a[0], kc) and torch.equal(a[1], vc) and torch.equal(a[2], table)
