"""PyTorch custom operators over the C ABI.

``torch.ops.ffpa.attn_fwd`` and ``torch.ops.ffpa.attn_varlen_fwd`` wrap
``ffpa_fwd`` / ``ffpa_fwd_varlen`` as opaque operators: torch.compile and
other tracers see one node with a shape-only fake implementation and never
look inside, and eager calls go straight to the CUDA kernels through the
binding.  ``ffpa_attn_func`` takes the argument list of
``torch.nn.functional.scaled_dot_product_attention`` (the FFPA API
reference, ``ffpa_attn.ffpa_attn_func``, uses the same list), so it can
replace that call for the supported cases: bf16/fp16 CUDA tensors,
64 <= D <= 1024 with D % 8 == 0 (D % 64 == 0 for varlen and for the
backward), no dropout.  The dense operator is
differentiable through ``ffpa_bwd`` (the backward kernels; a mask enters
the recomputed scores, but no gradient is formed for the mask itself), and
the varlen operator through ``ffpa_bwd_varlen``.  Both backwards are operators
themselves (``attn_bwd``, ``attn_varlen_bwd``), so that a training step can be
traced; second derivatives are refused.

``torch.ops.ffpa.qk_norm_rope`` (differentiable through
``qk_norm_rope_bwd``, once), ``kv_append``, ``decode_paged`` and
``page_plan`` do the same for the calls around a paged key/value cache
(paged.py); the last three serve and have no gradient, and ``kv_append`` and
``page_plan`` declare the cache and the block table that they write.  As with
any operator of torch, a backward that is captured into a CUDA graph must
not meet leaves that an eager graph made on another stream still holds: free
that graph first, or capture ``ffpa_qk_norm_rope_bwd`` itself.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _binding, paged


def _eager(*tensors) -> bool:
    """Whether a backward may call the binding itself: no graph of the gradients is asked for, no
    tracer or mode looks on, and every tensor is a plain one.  (A backward's operator is for the
    rest: its dispatch takes 57 us of host time, of a step of 262 us.)"""
    return (not torch.is_grad_enabled() and torch._C._len_torch_dispatch_stack() == 0 and
            all(t is None or type(t) in (torch.Tensor, torch.nn.Parameter) for t in tensors))


@torch.library.custom_op("ffpa::attn_fwd", mutates_args=())
def attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, attn_mask: Optional[torch.Tensor],
             is_causal: bool, scale: Optional[float],
             enable_gqa: bool) -> tuple[torch.Tensor, torch.Tensor]:
    """O [B,Hq,Nq,D] and LSE [B,Hq,Nq] (fp32) of exact attention."""
    return _binding.ffpa_fwd(q, k, v, attn_mask=attn_mask, is_causal=is_causal, scale=scale,
                             enable_gqa=enable_gqa, return_lse=True)


@attn_fwd.register_fake
def _attn_fwd_fake(q, k, v, attn_mask, is_causal, scale, enable_gqa):
    B, Hq, Nq, _ = q.shape
    return (torch.empty_like(q, memory_format=torch.contiguous_format),
            q.new_empty((B, Hq, Nq), dtype=torch.float32))


def _attn_fwd_setup_context(ctx, inputs, output):
    q, k, v, attn_mask, is_causal, scale, enable_gqa = inputs
    o, lse = output
    ctx.save_for_backward(q, k, v, o, lse, attn_mask)
    ctx.is_causal, ctx.scale, ctx.enable_gqa = is_causal, scale, enable_gqa
    # An output the loss does not use arrives in backward as None (not as a
    # tensor of zeros), so the LSE check below needs no device read.
    ctx.set_materialize_grads(False)


def _check_grads(grad_o, grad_lse):
    if grad_lse is not None:
        raise NotImplementedError("gradients through the returned LSE are not supported")
    if grad_o is None:
        raise NotImplementedError("backward without a gradient for O")


def _no_second_derivative(ctx, *grads):
    raise NotImplementedError("no second derivative is formed")


def _like_inputs(q, k, v):
    return tuple(torch.empty_like(t, memory_format=torch.contiguous_format) for t in (q, k, v))


@torch.library.custom_op("ffpa::attn_bwd", mutates_args=())
def attn_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
             lse: torch.Tensor, attn_mask: Optional[torch.Tensor], is_causal: bool, scale: Optional[float],
             enable_gqa: bool) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of q, k and v."""
    return _binding.ffpa_bwd(dout, q, k, v, out, lse, is_causal=is_causal, scale=scale, enable_gqa=enable_gqa,
                             attn_mask=attn_mask)


@attn_bwd.register_fake
def _attn_bwd_fake(dout, q, k, v, out, lse, attn_mask, is_causal, scale, enable_gqa):
    return _like_inputs(q, k, v)


attn_bwd.register_autograd(_no_second_derivative)


def _attn_fwd_backward(ctx, grad_o, grad_lse):
    if ctx.needs_input_grad[3]:
        raise NotImplementedError("no gradient is formed for attn_mask")
    _check_grads(grad_o, grad_lse)
    q, k, v, o, lse, attn_mask = ctx.saved_tensors
    grad_o = grad_o.contiguous()
    if _eager(grad_o, q, k, v, o, lse, attn_mask):
        dq, dk, dv = _binding.ffpa_bwd(grad_o, q, k, v, o, lse, is_causal=ctx.is_causal, scale=ctx.scale,
                                       enable_gqa=ctx.enable_gqa, attn_mask=attn_mask)
    else:
        dq, dk, dv = torch.ops.ffpa.attn_bwd(grad_o, q, k, v, o, lse, attn_mask, ctx.is_causal, ctx.scale,
                                             ctx.enable_gqa)
    return dq, dk, dv, None, None, None, None


attn_fwd.register_autograd(_attn_fwd_backward, setup_context=_attn_fwd_setup_context)


@torch.library.custom_op("ffpa::attn_varlen_fwd", mutates_args=())
def attn_varlen_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                    cu_seqlens_k: Optional[torch.Tensor], max_seqlen_q: int, max_seqlen_k: int,
                    causal: bool, softmax_scale: Optional[float],
                    enable_gqa: bool) -> tuple[torch.Tensor, torch.Tensor]:
    """O [Tq,Hq,D] and LSE [Hq,Tq] (fp32) of packed variable-length attention."""
    return _binding.ffpa_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                                    max_seqlen_k, causal=causal, softmax_scale=softmax_scale,
                                    enable_gqa=enable_gqa, return_lse=True)


@attn_varlen_fwd.register_fake
def _attn_varlen_fwd_fake(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal,
                          softmax_scale, enable_gqa):
    Tq, Hq, _ = q.shape
    return (torch.empty_like(q, memory_format=torch.contiguous_format),
            q.new_empty((Hq, Tq), dtype=torch.float32))


def _attn_varlen_setup_context(ctx, inputs, output):
    (q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal, softmax_scale,
     enable_gqa) = inputs
    o, lse = output
    ctx.save_for_backward(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k)
    ctx.max_q, ctx.max_k = max_seqlen_q, max_seqlen_k
    ctx.causal, ctx.scale, ctx.enable_gqa = causal, softmax_scale, enable_gqa
    ctx.set_materialize_grads(False)


@torch.library.custom_op("ffpa::attn_varlen_bwd", mutates_args=())
def attn_varlen_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                    lse: torch.Tensor, cu_seqlens_q: torch.Tensor, cu_seqlens_k: Optional[torch.Tensor],
                    max_seqlen_q: int, max_seqlen_k: int, causal: bool, softmax_scale: Optional[float],
                    enable_gqa: bool) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of packed q, k and v."""
    return _binding.ffpa_bwd_varlen(dout, q, k, v, out, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                                    softmax_scale=softmax_scale, causal=causal, enable_gqa=enable_gqa)


@attn_varlen_bwd.register_fake
def _attn_varlen_bwd_fake(dout, q, k, v, out, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal,
                          softmax_scale, enable_gqa):
    return _like_inputs(q, k, v)


attn_varlen_bwd.register_autograd(_no_second_derivative)


def _attn_varlen_backward(ctx, grad_o, grad_lse):
    _check_grads(grad_o, grad_lse)
    q, k, v, o, lse, cu_q, cu_k = ctx.saved_tensors
    grad_o = grad_o.contiguous()
    if _eager(grad_o, q, k, v, o, lse, cu_q, cu_k):
        dq, dk, dv = _binding.ffpa_bwd_varlen(grad_o, q, k, v, o, lse, cu_q, cu_k, ctx.max_q, ctx.max_k,
                                              softmax_scale=ctx.scale, causal=ctx.causal, enable_gqa=ctx.enable_gqa)
    else:
        dq, dk, dv = torch.ops.ffpa.attn_varlen_bwd(grad_o, q, k, v, o, lse, cu_q, cu_k, ctx.max_q, ctx.max_k,
                                                    ctx.causal, ctx.scale, ctx.enable_gqa)
    return dq, dk, dv, None, None, None, None, None, None, None


attn_varlen_fwd.register_autograd(_attn_varlen_backward, setup_context=_attn_varlen_setup_context)


def ffpa_attn_func(query: torch.Tensor, key: torch.Tensor, value: torch.Tensor,
                   attn_mask: Optional[torch.Tensor] = None, dropout_p: float = 0.0,
                   is_causal: bool = False, scale: Optional[float] = None,
                   enable_gqa: bool = False, *, return_lse: bool = False):
    """Drop-in for ``F.scaled_dot_product_attention`` on [B,H,N,D] tensors.

    Causal masking is tail-aligned (query row r sees keys k <= r + Nkv - Nq),
    which equals SDPA's top-left alignment when Nq == Nkv.  Returns O, or
    (O, LSE) with return_lse."""
    if dropout_p != 0.0:
        raise NotImplementedError("dropout is not supported by this forward kernel")
    o, lse = torch.ops.ffpa.attn_fwd(query, key, value, attn_mask, bool(is_causal), scale,
                                     bool(enable_gqa))
    return (o, lse) if return_lse else o


def ffpa_attn_varlen_func(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                          cu_seqlens_q: torch.Tensor, cu_seqlens_k: Optional[torch.Tensor],
                          max_seqlen_q: int, max_seqlen_k: int, dropout_p: float = 0.0,
                          softmax_scale: Optional[float] = None, causal: bool = False,
                          enable_gqa: bool = False, *, return_lse: bool = False):
    """Packed THD variable-length forward (q [Tq,Hq,D], k/v [Tk,Hkv,D])."""
    if dropout_p != 0.0:
        raise NotImplementedError("dropout is not supported by this forward kernel")
    o, lse = torch.ops.ffpa.attn_varlen_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, int(max_seqlen_q),
                                            int(max_seqlen_k), bool(causal), softmax_scale,
                                            bool(enable_gqa))
    return (o, lse) if return_lse else o


@torch.library.custom_op("ffpa::qk_norm_rope", mutates_args=())
def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: Optional[torch.Tensor],
                 inv_freq: Optional[torch.Tensor], q_weight: Optional[torch.Tensor],
                 k_weight: Optional[torch.Tensor], eps: float, interleaved: bool,
                 rope_scale: float) -> tuple[torch.Tensor, torch.Tensor]:
    """Queries and keys normed per head and rotated by position."""
    return paged.ffpa_qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps=eps,
                                   interleaved=interleaved, rope_scale=rope_scale)


@qk_norm_rope.register_fake
def _qk_norm_rope_fake(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, rope_scale):
    return (torch.empty_like(q, memory_format=torch.contiguous_format),
            torch.empty_like(k, memory_format=torch.contiguous_format))


@torch.library.custom_op("ffpa::qk_norm_rope_bwd", mutates_args=())
def qk_norm_rope_bwd(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                     positions: Optional[torch.Tensor], inv_freq: Optional[torch.Tensor],
                     q_weight: Optional[torch.Tensor], k_weight: Optional[torch.Tensor], eps: float, interleaved: bool,
                     rope_scale: float) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of q, k, q_weight and k_weight (no entries for a weight that is None)."""
    dq, dk, dqw, dkw = paged.ffpa_qk_norm_rope_bwd(dq_out, dk_out, q, k, positions, inv_freq, q_weight, k_weight,
                                                   eps=eps, interleaved=interleaved, rope_scale=rope_scale)
    return dq, dk, q.new_empty(0) if dqw is None else dqw, k.new_empty(0) if dkw is None else dkw


@qk_norm_rope_bwd.register_fake
def _qk_norm_rope_bwd_fake(dq_out, dk_out, q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, rope_scale):
    return (torch.empty_like(q, memory_format=torch.contiguous_format),
            torch.empty_like(k, memory_format=torch.contiguous_format),
            q.new_empty(0) if q_weight is None else torch.empty_like(q_weight),
            k.new_empty(0) if k_weight is None else torch.empty_like(k_weight))


qk_norm_rope_bwd.register_autograd(_no_second_derivative)


def _qk_norm_rope_setup_context(ctx, inputs, output):
    q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, rope_scale = inputs
    ctx.save_for_backward(q, k, positions, inv_freq, q_weight, k_weight)
    ctx.eps, ctx.interleaved, ctx.rope_scale = eps, interleaved, rope_scale
    ctx.set_materialize_grads(False)


def _qk_norm_rope_backward(ctx, grad_q, grad_k):
    if ctx.needs_input_grad[3]:
        raise NotImplementedError("no gradient is formed for inv_freq")
    q, k, positions, inv_freq, q_weight, k_weight = ctx.saved_tensors
    # An output that the loss does not use has no gradient: zeros for its rows.
    grad_q = torch.zeros_like(q, memory_format=torch.contiguous_format) if grad_q is None else grad_q.contiguous()
    grad_k = torch.zeros_like(k, memory_format=torch.contiguous_format) if grad_k is None else grad_k.contiguous()
    how = (grad_q, grad_k, q, k, positions, inv_freq, q_weight, k_weight)
    if _eager(*how):
        dq, dk, dqw, dkw = paged.ffpa_qk_norm_rope_bwd(*how, eps=ctx.eps, interleaved=ctx.interleaved,
                                                       rope_scale=ctx.rope_scale)
    else:
        dq, dk, dqw, dkw = torch.ops.ffpa.qk_norm_rope_bwd(*how, ctx.eps, ctx.interleaved, ctx.rope_scale)
    return (dq, dk, None, None, None if q_weight is None else dqw, None if k_weight is None else dkw, None, None, None)


qk_norm_rope.register_autograd(_qk_norm_rope_backward, setup_context=_qk_norm_rope_setup_context)


@torch.library.custom_op("ffpa::kv_append", mutates_args=("k_cache", "v_cache"))
def kv_append(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
              v_cache: torch.Tensor, slots: torch.Tensor, positions: Optional[torch.Tensor],
              inv_freq: Optional[torch.Tensor], q_weight: Optional[torch.Tensor], k_weight: Optional[torch.Tensor],
              eps: float, interleaved: bool, rope_scale: float) -> torch.Tensor:
    """Keys and values into cache slots; the normed and rotated queries (no rows without q)."""
    out = paged.ffpa_kv_append(q, k, v, k_cache, v_cache, slots, positions, inv_freq, q_weight, k_weight, eps=eps,
                               interleaved=interleaved, rope_scale=rope_scale)
    return k.new_empty((0,) + tuple(k.shape[1:])) if out is None else out


@kv_append.register_fake
def _kv_append_fake(q, k, v, k_cache, v_cache, slots, positions, inv_freq, q_weight, k_weight, eps, interleaved,
                    rope_scale):
    if q is None:
        return k.new_empty((0,) + tuple(k.shape[1:]))
    return torch.empty_like(q, memory_format=torch.contiguous_format)


@torch.library.custom_op("ffpa::decode_paged", mutates_args=())
def decode_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                 seq_lens: torch.Tensor, scale: Optional[float],
                 enable_gqa: bool) -> tuple[torch.Tensor, torch.Tensor]:
    """O [B,Hq,D] and LSE [B,Hq] (fp32) of one new token per request over a paged cache."""
    return paged.ffpa_decode_paged(q, k_cache, v_cache, block_table, seq_lens, scale=scale, enable_gqa=enable_gqa,
                                   return_lse=True)


@decode_paged.register_fake
def _decode_paged_fake(q, k_cache, v_cache, block_table, seq_lens, scale, enable_gqa):
    B, Hq, _ = q.shape
    return (torch.empty_like(q, memory_format=torch.contiguous_format),
            q.new_empty((B, Hq), dtype=torch.float32))


@torch.library.custom_op("ffpa::page_plan", mutates_args=("block_table",))
def page_plan(block_table: torch.Tensor, seq_lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor,
              free_count: torch.Tensor, page_size: int, num_tokens: int
              ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Slots, positions, cumulative lengths, new lengths and free count; the table in place."""
    return paged.ffpa_page_plan(block_table, seq_lens, new_lens, free_pages, free_count, page_size, num_tokens)


@page_plan.register_fake
def _page_plan_fake(block_table, seq_lens, new_lens, free_pages, free_count, page_size, num_tokens):
    return (seq_lens.new_empty(num_tokens, dtype=torch.int64), seq_lens.new_empty(num_tokens),
            seq_lens.new_empty(seq_lens.shape[0] + 1), torch.empty_like(seq_lens), torch.empty_like(free_count))


def ffpa_qk_norm_rope_func(q: torch.Tensor, k: torch.Tensor, positions: Optional[torch.Tensor] = None,
                           inv_freq: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                           k_weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6, interleaved: bool = False,
                           rope_scale: float = 1.0):
    """RMS norm of every query and key head and rotation by position (see paged.ffpa_qk_norm_rope),
    differentiable in q, k and the weights.  Returns (q, k) for ffpa_attn_func ([B,H,N,D]) or
    ffpa_attn_varlen_func ([T,H,D])."""
    return torch.ops.ffpa.qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, float(eps), bool(interleaved),
                                       float(rope_scale))


def ffpa_kv_append_func(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                        v_cache: torch.Tensor, slots: torch.Tensor, positions: Optional[torch.Tensor] = None,
                        inv_freq: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                        k_weight: Optional[torch.Tensor] = None, *, eps: float = 1e-6, interleaved: bool = False,
                        rope_scale: float = 1.0):
    """Keys (normed and rotated) and values into cache slots (see paged.ffpa_kv_append).  Returns the
    queries, or None without q."""
    out = torch.ops.ffpa.kv_append(q, k, v, k_cache, v_cache, slots, positions, inv_freq, q_weight, k_weight,
                                   float(eps), bool(interleaved), float(rope_scale))
    return None if q is None else out


def ffpa_attn_decode_func(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                          seq_lens: torch.Tensor, scale: Optional[float] = None, enable_gqa: bool = False, *,
                          return_lse: bool = False):
    """Attention of one new token per request over a paged cache (see paged.ffpa_decode_paged)."""
    o, lse = torch.ops.ffpa.decode_paged(q, k_cache, v_cache, block_table, seq_lens, scale, bool(enable_gqa))
    return (o, lse) if return_lse else o


def ffpa_page_plan_func(block_table: torch.Tensor, seq_lens: torch.Tensor, new_lens: torch.Tensor,
                        free_pages: torch.Tensor, free_count: torch.Tensor, page_size: int, num_tokens: int):
    """Pages, slots and positions of one step's new tokens (see paged.ffpa_page_plan)."""
    return torch.ops.ffpa.page_plan(block_table, seq_lens, new_lens, free_pages, free_count, int(page_size),
                                    int(num_tokens))
