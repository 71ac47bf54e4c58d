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


# ---------------------------------------------------------------- the backward as an operator
def leaves(device="cpu", dtype=BF, wdtype=torch.float32, seed=1):
    g = torch.Generator().manual_seed(seed)
    q, k = torch.randn(6, 4, 128, generator=g), torch.randn(6, 2, 128, generator=g)
    w = 1 + 0.2 * torch.randn(128, generator=g)
    return [t.to(device=device, dtype=d).requires_grad_() for t, d in ((q, dtype), (k, dtype), (w, wdtype))]


def test_backward_of_shapes_alone():
    """The gradients have the leaves' shapes and types, with and without weights, norm and rotation."""
    with FakeTensorMode():
        q, k, w = leaves()
        inv = torch.empty(32, dtype=torch.float64)
        for how in (dict(positions=torch.empty(6, dtype=torch.int32), inv_freq=inv, q_weight=w, k_weight=w), dict(k_weight=w),
                    dict(positions=torch.empty(6, dtype=torch.int64), inv_freq=inv)):
            asked = [q, k] + ([w] if "k_weight" in how else [])
            grads = torch.autograd.grad(sum(t.sum() for t in pkg.ffpa_qk_norm_rope_func(q, k, **how)), asked)
            assert [(g.shape, g.dtype) for g in grads] == [(x.shape, x.dtype) for x in asked]


def test_second_derivative_is_refused():
    with FakeTensorMode():
        q, k, w = leaves()
        out = pkg.ffpa_qk_norm_rope_func(q, k, q_weight=w, k_weight=w)[0].float().square().sum()
        grad, = torch.autograd.grad(out, [w], create_graph=True)
        assert grad.requires_grad                       # a loss that uses it does not lose the term in silence
        with pytest.raises(NotImplementedError, match="second derivative"):
            grad.sum().backward()


def test_backward_operator_traces():
    """The joint graph of a compiled step names the backward operator (a trace that formed it from the
    binding's own calls would end in their refusal)."""
    from torch._functorch.aot_autograd import aot_function
    from torch._functorch.partitioners import default_partition
    seen = []

    def keep(joint, *a, **kw):
        seen.extend(str(n.target) for n in joint.graph.nodes if n.op == "call_function")
        return default_partition(joint, *a, **kw)

    q, k, w = leaves()
    pos, inv = torch.arange(6), pkg.rope_inv_freq(64)[0]
    step = aot_function(lambda q, k, w, pos, inv: pkg.ffpa_qk_norm_rope_func(q, k, pos, inv, w, w)[0].float().sum(),
                        fw_compiler=lambda gm, _: gm, partition_fn=keep)
    with pytest.raises((ValueError, RuntimeError)):     # traced; then the operator refuses memory of the host
        step(q, k, w, pos, inv)
    assert "ffpa.qk_norm_rope.default" in seen and "ffpa.qk_norm_rope_bwd.default" in seen


@pytest.mark.gpu
def test_traced_training_step_equals_the_eager_one():
    dev = torch.device("cuda:0")
    pos, inv = torch.arange(6, device=dev), pkg.rope_inv_freq(64)[0].to(dev)
    up = torch.randn(6, 4, 128, generator=torch.Generator().manual_seed(2)).to(BF).to(dev)

    def step(q, k, w):
        qo, ko = pkg.ffpa_qk_norm_rope_func(q, k, pos, inv, w, w)
        return ((qo * up).float().sum() + ko.float().square().sum())

    def grads(f):
        ls = leaves(dev)
        f(*ls).backward()
        return [t.grad for t in ls]

    want = grads(step)
    got = grads(torch.compile(step, fullgraph=True, backend="aot_eager"))
    assert all(torch.isfinite(a).all() and a.abs().max() > 0 for a in want)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # without weights, and with the queries' alone
    for kw in (dict(), dict(q_weight=leaves(dev)[2])):
        f = torch.compile(lambda q, k: sum(t.float().square().sum() for t in pkg.ffpa_qk_norm_rope_func(q, k, pos, inv, **kw)),
                          fullgraph=True, backend="aot_eager")
        q, k, _ = leaves(dev)
        f(q, k).backward()
        a, b, _ = leaves(dev)
        sum(t.float().square().sum() for t in pkg.ffpa_qk_norm_rope_func(a, b, pos, inv, **kw)).backward()
        assert torch.equal(a.grad, q.grad) and torch.equal(b.grad, k.grad)
