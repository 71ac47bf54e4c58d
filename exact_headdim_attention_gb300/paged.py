"""Generation over a paged key/value cache, and the head norm with rotation: argument marshalling.

One generation step of an attention layer:

    slots, positions, cu, lens, free_count = ffpa_page_plan(table, lens, new, free, free_count, page, tokens)
    q = ffpa_kv_append(q, k, v, k_cache, v_cache, slots, positions, inv_freq, q_weight, k_weight, rope_scale=scale)
    last = (cu[1:] - 1).clamp(min=0)
    o = ffpa_decode_paged(q[last], k_cache, v_cache, table, lens, enable_gqa=True)

with q, k, v the packed rows of the new tokens, (inv_freq, scale) those of training, and one row of
o for each request: of its last new token (for a request without one it is of no use).  And of a training step: ``ffpa_qk_norm_rope_func`` (torch_ops.py; differentiable through
``ffpa_qk_norm_rope_bwd``), then ``ffpa_attn_func`` or ``ffpa_attn_varlen_func``.  The step's plan
is shared by all layers.  As in _binding.py every computation runs in the CUDA kernels behind the C
ABI (include/ffpa.h); tensors are checked, outputs allocated and the ABI called in
csrc/paged_binding.cpp, because calls that serve single tokens are as short as a few microseconds.

A call on a stream of the caller's (stream=) makes its outputs in the current stream's memory, as the
attention calls do: the caller orders the two streams and keeps the outputs until the call is done.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import math

import torch

from . import build as _build
from ._binding import _options, _raise, load_library

_BOUND = ("ffpa_decode_paged", "ffpa_decode_paged_workspace_bytes", "ffpa_qk_norm_rope", "ffpa_qk_norm_rope_bwd",
          "ffpa_qk_norm_rope_bwd_workspace_bytes", "ffpa_kv_append", "ffpa_page_plan")
_module = _bound_to = None


def _native():
    """The marshalling module, bound to the library in use."""
    global _module, _bound_to
    lib = load_library()
    if lib is not _bound_to:
        if _module is None:
            path = _build.binding_path()
            if not path.exists():
                raise RuntimeError(f"{path.name} not found at {path}: build it with "
                                   "`python -m exact_headdim_attention_gb300.build` (no fallback path exists)")
            spec = importlib.util.spec_from_file_location("ffpa_paged_binding", path)
            _module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(_module)
        _module.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _BOUND))
        _bound_to = lib
    return _module


def _handle(stream):
    """cudaStream_t of a caller's stream; None leaves torch's current stream to the module."""
    return None if stream is None else stream.cuda_stream


def _on_stream(workspace, need, t, stream):
    """A workspace for a stream of the caller's (torch's, or any object with its handle as cuda_stream) is
    allocated in that stream's order (the module does so for the current one): it is free again for
    what the stream runs after the call, and for nothing else."""
    if workspace is not None or not t.is_cuda:
        return workspace
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=t.device)
    with torch.cuda.stream(stream):
        return torch.empty(max(need, 256), dtype=torch.uint8, device=t.device)


def _call_options(t, status, wait_timeout_ns=None, test_drop_first_copy=False):
    """(the call's ffpa_options, kept alive by the caller; their address), or (None, None)."""
    if status is None and not wait_timeout_ns and not test_drop_first_copy:
        return None, None
    ref = _options(t, None, status, wait_timeout_ns, test_drop_first_copy)
    return ref, ctypes.addressof(ref._obj)


def rope_inv_freq(rot_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                  original_length: int | None = None, beta_fast: float = 32.0, beta_slow: float = 1.0,
                  device=None) -> tuple[torch.Tensor, float]:
    """(inv_freq float64 [rot_dim / 2], rope_scale) of rotary positions: base ** (-2 i / rot_dim).

    scaling stretches them to contexts `factor` times as long:
      "linear"    every frequency is divided by factor;
      "base"      the base grows so that the slowest frequency is divided by factor and the
                  fastest stays: base * factor ** (rot_dim / (rot_dim - 2));
      "by_parts"  pairs that turn more than beta_fast times within original_length positions stay,
                  pairs that turn less than beta_slow times are divided by factor, a linear ramp
                  over the pair's number lies between (from whole pairs on either side: number 0
                  at the earliest, rot_dim - 1 at the latest); rope_scale = 0.1 ln(factor) + 1.
                  The published method is YaRN (arXiv 2309.00071)."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and at least 2")
    if not (base > 0 and math.isfinite(base)) or not (factor >= 1 and math.isfinite(factor)):
        raise ValueError("base must be positive and factor at least 1")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "base":
        if rot_dim < 4:
            raise ValueError('scaling "base" needs rot_dim of at least 4')
        base = base * factor ** (rot_dim / (rot_dim - 2))
    inv = base ** (-2.0 * i / rot_dim)
    if scaling == "linear":
        inv = inv / factor
    elif scaling == "by_parts":
        if not original_length or original_length < 1 or base <= 1:
            raise ValueError('scaling "by_parts" needs original_length and a base above 1')

        def pair_turning(times):     # (real) number of the pair that turns `times` times
            return rot_dim * math.log(original_length / (times * 2 * math.pi)) / (2 * math.log(base))

        # The ramp may end behind the last pair, which it then does not divide by the whole factor.
        lo = max(math.floor(pair_turning(beta_fast)), 0)
        hi = min(math.ceil(pair_turning(beta_slow)), rot_dim - 1)
        slow = ((i - lo) / (hi - lo)).clamp(0, 1) if hi > lo else (i >= hi).double()
        inv = inv * (1 - slow) + inv / factor * slow
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f'scaling must be None, "linear", "base" or "by_parts", got {scaling!r}')
    return inv.to(device) if device is not None else inv, scale


def ffpa_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions=None, inv_freq=None, q_weight=None,
                      k_weight=None, *, eps: float = 1e-6, interleaved: bool = False,
                      rope_scale: float = 1.0, q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head and rotation by position, through ``ffpa_qk_norm_rope``.

    q [B,Hq,N,D] and k [B,Hkv,N,D], or packed [T,H,D] (bf16 or fp16, D stride 1; slices of one
    projection's rows will do).  inv_freq [rot_dim/2] float64: radians per position (see
    rope_inv_freq); None does not rotate.  positions int32 or int64, [N] or [B,N].  q_weight,
    k_weight [D], float32 or the rows' type: None does not norm.  q_out, k_out may be q and k
    themselves.  Returns (q_out, k_out)."""
    r = _native().qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, rope_scale, q_out,
                               k_out, _handle(stream))
    if type(r) is int:
        _raise(r, "ffpa_qk_norm_rope")
    return r


def ffpa_qk_norm_rope_bwd(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                          positions=None, inv_freq=None, q_weight=None, k_weight=None, *, eps: float = 1e-6,
                          interleaved: bool = False, rope_scale: float = 1.0, dq=None, dk=None,
                          workspace=None, stream=None):
    """Gradients of ffpa_qk_norm_rope, through ``ffpa_qk_norm_rope_bwd``.

    dq_out, dk_out: gradients of the outputs, shaped as q and k; the other arguments are the
    forward's.  Returns (dq, dk, dq_weight, dk_weight), None for a weight that was None.
    workspace: a uint8 device tensor of qk_norm_rope_bwd_workspace_bytes(D) bytes (allocated here
    when None)."""
    if stream is not None and (q_weight is not None or k_weight is not None):
        workspace = _on_stream(workspace, qk_norm_rope_bwd_workspace_bytes(q.shape[-1]), q, stream)
    r = _native().qk_norm_rope_bwd(dq_out, dk_out, q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved,
                                   rope_scale, dq, dk, workspace, _handle(stream))
    if type(r) is int:
        _raise(r, "ffpa_qk_norm_rope_bwd")
    return r


@functools.lru_cache(maxsize=None)
def qk_norm_rope_bwd_workspace_bytes(D: int) -> int:
    """Bytes of the workspace of ffpa_qk_norm_rope_bwd (0 for an unsupported head dim)."""
    return int(load_library().ffpa_qk_norm_rope_bwd_workspace_bytes(D))


def ffpa_kv_append(q, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   slots: torch.Tensor, positions=None, inv_freq=None, q_weight=None, k_weight=None, *,
                   eps: float = 1e-6, interleaved: bool = False, rope_scale: float = 1.0, q_out=None,
                   stream=None, status=None):
    """ffpa_qk_norm_rope of packed rows whose keys and values go to a paged cache, through ``ffpa_kv_append``.

    q [T,Hq,D] (None: no queries), k, v [T,Hkv,D]; k_cache, v_cache [num_pages,page_size,Hkv,D] (any
    strides with D stride 1), written at slots (int64 [T], page * page_size + index in page; negative:
    padding, not stored).  Other arguments as for ffpa_qk_norm_rope; without inv_freq and k_weight
    keys are stored as they are.  Returns q_out (None without q).  A slot beyond the cache is not
    stored; the status word (see ffpa_fwd) receives FFPA_ERR_INVALID."""
    keep, options = _call_options(k, status)
    r = _native().kv_append(q, k, v, k_cache, v_cache, slots, positions, inv_freq, q_weight, k_weight, eps, interleaved,
                            rope_scale, q_out, _handle(stream), options)
    if type(r) is int:
        _raise(r, "ffpa_kv_append")
    return r


@functools.lru_cache(maxsize=None)
def decode_paged_workspace_bytes(Hq: int, Hkv: int, D: int) -> int:
    """Bytes of the workspace of ffpa_decode_paged, for any batch and lengths (0 for unsupported heads)."""
    return int(load_library().ffpa_decode_paged_workspace_bytes(Hq, Hkv, D))


def ffpa_decode_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                      seq_lens: torch.Tensor, *, scale: float | None = None, enable_gqa: bool = False,
                      return_lse: bool = False, out=None, lse=None, workspace=None, stream=None, status=None,
                      wait_timeout_ns=None, test_drop_first_copy=False):
    """Attention of one new token per request over a paged cache, through ``ffpa_decode_paged``.

    q [B,Hq,D]; k_cache, v_cache [num_pages,page_size,Hkv,D] (any strides with D stride 1);
    block_table int32 [B,max_pages]; seq_lens int32 [B], the keys each request sees (0: its row is
    0 and its LSE -inf).  Returns O [B,Hq,D], or (O, LSE [B,Hq] fp32) with return_lse.

    The lengths stay on the device, so a captured call serves any lengths.  A page or length out of
    range is not followed; the status word (see ffpa_fwd) receives FFPA_ERR_INVALID.  workspace: a
    uint8 device tensor of decode_paged_workspace_bytes(...) bytes, 256-byte aligned (allocated here
    when None); calls that may overlap on the GPU need one each.  wait_timeout_ns and
    test_drop_first_copy: as for ffpa_fwd."""
    if stream is not None:
        workspace = _on_stream(workspace, decode_paged_workspace_bytes(q.shape[1], k_cache.shape[2], q.shape[2]), q,
                               stream)
    keep, options = _call_options(q, status, wait_timeout_ns, test_drop_first_copy)
    r = _native().decode_paged(q, k_cache, v_cache, block_table, seq_lens, scale, enable_gqa, return_lse, out, lse,
                               workspace, _handle(stream), options)
    if type(r) is int:
        _raise(r, "ffpa_decode_paged")
    return r


def ffpa_page_plan(block_table: torch.Tensor, seq_lens: torch.Tensor, new_lens: torch.Tensor,
                   free_pages: torch.Tensor, free_count: torch.Tensor, page_size: int, num_tokens: int, *,
                   stream=None, status=None):
    """Pages, slots and positions of one step's new tokens, through ``ffpa_page_plan``.

    Request b holds seq_lens[b] tokens and gets new_lens[b] more (int32 [B]); pages for them come off
    the end of free_pages[:free_count] (int32; free_count int32 [1]) into block_table (int32
    [B,max_pages], written in place).  num_tokens: rows of the step, at least the new tokens.
    Returns (slots int64 [num_tokens], positions int32 [num_tokens], cu_seqlens int32 [B+1],
    seq_lens int32 [B] with the new tokens, free_count int32 [1] without the pages taken); rows
    behind the last token have slot -1 and position 0.  Everything stays on the device.  Tokens for
    which there is no page, or a negative one, get slot -1; the status word (see ffpa_fwd) receives
    FFPA_ERR_INVALID.

    Pages of a finished request go back by the caller: written at free_pages[free_count:]."""
    keep, options = _call_options(block_table, status)
    r = _native().page_plan(block_table, seq_lens, new_lens, free_pages, free_count, page_size, num_tokens,
                            _handle(stream), options)
    if type(r) is int:
        _raise(r, "ffpa_page_plan")
    return r
