"""Generation over a paged key/value cache, and the head norm with rotation: argument marshalling.

One generation step of an attention layer:

    slots, positions, cu, lens, free_count = ffpa_page_plan(table, lens, new, free, free_count, page, tokens)
    q = ffpa_kv_append(q, k, v, k_cache, v_cache, slots, positions, inv_freq, q_weight, k_weight)
    o = ffpa_decode_paged(q, k_cache, v_cache, table, lens)

and of a training step: ``ffpa_qk_norm_rope_func`` (torch_ops.py; differentiable through
``ffpa_qk_norm_rope_bwd``), then ``ffpa_attn_func`` or ``ffpa_attn_varlen_func``.  The step's plan
is shared by all layers.  As in _binding.py every computation runs in the CUDA kernels behind the C
ABI (include/ffpa.h), which also checks what this module does not.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from ._binding import (FFPA_OK, Rope, _check_buffer, _dtype_code, _options, _raise, _stream_handle,
                       load_library)


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
                  over the pair's number lies between; rope_scale = 0.1 ln(factor) + 1."""
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

        lo = max(math.floor(pair_turning(beta_fast)), 0)
        hi = min(math.ceil(pair_turning(beta_slow)), rot_dim // 2 - 1)
        slow = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        inv = inv * (1 - slow) + inv / factor * slow
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError(f'scaling must be None, "linear", "base" or "by_parts", got {scaling!r}')
    return inv.to(device) if device is not None else inv, scale


def _rope_args(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, rope_scale, B, N):
    """ctypes ffpa_rope of one call.  B, N: positions broadcast to [B, N]."""
    D = k.shape[-1]
    r = Rope()
    if inv_freq is not None:
        if inv_freq.dtype != torch.float64:
            raise TypeError(f"inv_freq must be float64, got {inv_freq.dtype}")
        if inv_freq.dim() != 1 or not inv_freq.is_contiguous() or not 0 < 2 * inv_freq.shape[0] <= D:
            raise ValueError(f"inv_freq must be contiguous [rot_dim / 2] with rot_dim in 8..{D}")
        if positions is None:
            raise ValueError("a rotation needs positions")
        if positions.dtype not in (torch.int32, torch.int64):
            raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
        shape = positions.shape
        if shape == (N,):
            r.position_str_n = positions.stride(0)
        elif shape == (B, N) or shape == (1, N):
            r.position_str_b = positions.stride(0) if shape[0] == B else 0
            r.position_str_n = positions.stride(1)
        else:
            shape = tuple(shape)
            raise ValueError(f"positions must have shape {(N,)} or {(B, N)}, got {shape}")
        r.positions, r.position_bits = positions.data_ptr(), 64 if positions.dtype == torch.int64 else 32
        r.inv_freq, r.rot_dim = inv_freq.data_ptr(), 2 * inv_freq.shape[0]
    if q_weight is not None:
        r.q_weight, r.weight_f32 = _weight_pointer(q_weight, "q_weight", k, D)
    if k_weight is not None:
        if q_weight is not None and q_weight.dtype != k_weight.dtype:
            raise TypeError("q_weight and k_weight must share one dtype")
        r.k_weight, r.weight_f32 = _weight_pointer(k_weight, "k_weight", k, D)
    r.interleaved, r.rope_scale, r.eps = bool(interleaved), rope_scale, eps
    return r


def _weight_pointer(w, name, k, D):
    f32 = w.dtype == torch.float32
    if not f32 and w.dtype != k.dtype:
        raise TypeError(f"{name} must be float32 or {k.dtype}, got {w.dtype}")
    if w.shape != (D,) or not w.is_contiguous():
        raise ValueError(f"{name} must be contiguous [{D}], got {tuple(w.shape)}")
    return w.data_ptr(), f32


def _strides(*tensors):
    """Strides of the tensors, one after the other, in one int64 array that the caller keeps alive
    over the call, and the address of each tensor's.  None has no strides."""
    flat, at = [], []
    for t in tensors:
        if t is None:
            at.append(None)
            continue
        at.append(8 * len(flat))
        flat += t.stride()
    keep = (ctypes.c_int64 * len(flat))(*flat)
    base = ctypes.addressof(keep)
    return keep, [None if x is None else base + x for x in at]


def _strides4(*tensors):
    """As _strides, for [B, H, N, D] or packed [T, H, D] rows as (b, h, n, d)."""
    flat = []
    for t in tensors:
        s = t.stride()
        flat += s if len(s) == 4 else (0, s[1], s[0], s[2])
    keep = (ctypes.c_int64 * len(flat))(*flat)
    base = ctypes.addressof(keep)
    return keep, range(base, base + 32 * len(tensors), 32)


def _stream_of(stream, t):
    """As _stream_handle, with a short way to torch's current stream of t's device."""
    if stream is None and t.is_cuda:
        return torch._C._cuda_getCurrentRawStream(t.device.index) or None
    return _stream_handle(stream, t)


def _qk_shape(q, k):
    """(B, Hq, Hkv, N, D) of [B, H, N, D] or packed [T, H, D] queries and keys.  (That every tensor of
    a call is memory of one device is the C ABI's check, here and below.)"""
    rank = q.dim()
    if rank != k.dim() or rank not in (3, 4):
        raise ValueError("q and k must both be 4-D [B, H, N, D] or 3-D [T, H, D]")
    if q.dtype != k.dtype:
        raise TypeError("q and k must share one dtype")
    if rank == 4:
        (B, Hq, N, D), (Bk, Hkv, Nk, Dk) = q.shape, k.shape
    else:
        (N, Hq, D), (Nk, Hkv, Dk) = q.shape, k.shape
        B = Bk = 1
    if (B, N, D) != (Bk, Nk, Dk):
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}")
    return B, Hq, Hkv, N, D


def _like(t, out, name):
    if out is None:
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    _check_buffer(out, name, t.shape, t.dtype, t.device)
    return out


def ffpa_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions=None, inv_freq=None, q_weight=None,
                      k_weight=None, *, eps: float = 1e-6, interleaved: bool = False,
                      rope_scale: float = 1.0, q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head and rotation by position, through ``ffpa_qk_norm_rope``.

    q [B,Hq,N,D] and k [B,Hkv,N,D], or packed [T,H,D] (bf16 or fp16, D stride 1; slices of one
    projection's rows will do).  inv_freq [rot_dim/2] float64: radians per position (see
    rope_inv_freq); None does not rotate.  positions int32 or int64, [N] or [B,N].  q_weight,
    k_weight [D], float32 or the rows' type: None does not norm.  q_out, k_out may be q and k
    themselves.  Returns (q_out, k_out)."""
    B, Hq, Hkv, N, D = _qk_shape(q, k)
    r = _rope_args(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, rope_scale, B, N)
    q_out, k_out = _like(q, q_out, "q_out"), _like(k, k_out, "k_out")
    keep, (qs, ks, qos, kos) = _strides4(q, k, q_out, k_out)
    st = load_library().ffpa_qk_norm_rope(q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(),
                                          _dtype_code(q), B, Hq, Hkv, N, D, qs, ks, qos, kos, r,
                                          _stream_of(stream, q))
    if st != FFPA_OK:
        _raise(st, "ffpa_qk_norm_rope")
    return q_out, k_out


def ffpa_qk_norm_rope_bwd(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                          positions=None, inv_freq=None, q_weight=None, k_weight=None, *, eps: float = 1e-6,
                          interleaved: bool = False, rope_scale: float = 1.0, dq=None, dk=None,
                          workspace=None, stream=None):
    """Gradients of ffpa_qk_norm_rope, through ``ffpa_qk_norm_rope_bwd``.

    dq_out, dk_out: gradients of the outputs, shaped as q and k; the other arguments are the
    forward's.  Returns (dq, dk, dq_weight, dk_weight), None for a weight that was None.
    workspace: a uint8 device tensor of qk_norm_rope_bwd_workspace_bytes(D) bytes (allocated here
    when None)."""
    B, Hq, Hkv, N, D = _qk_shape(q, k)
    for name, t, like in (("dq_out", dq_out, q), ("dk_out", dk_out, k)):
        if t.dtype != like.dtype:
            raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
        if t.shape != like.shape:
            raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(t.shape)}")
    r = _rope_args(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, rope_scale, B, N)
    dq, dk = _like(q, dq, "dq"), _like(k, dk, "dk")
    dqw = None if q_weight is None else torch.empty_like(q_weight)
    dkw = None if k_weight is None else torch.empty_like(k_weight)
    lib = load_library()
    ws = None
    if q_weight is not None or k_weight is not None:
        ws = _workspace(workspace, qk_norm_rope_bwd_workspace_bytes(D), q.device, stream)
    keep, (gqs, gks, qs, ks, dqs, dks) = _strides4(dq_out, dk_out, q, k, dq, dk)
    st = lib.ffpa_qk_norm_rope_bwd(dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(), dq.data_ptr(),
                                   dk.data_ptr(), None if dqw is None else dqw.data_ptr(),
                                   None if dkw is None else dkw.data_ptr(), _dtype_code(q), B, Hq, Hkv, N, D,
                                   gqs, gks, qs, ks, dqs, dks, r, None if ws is None else ws.data_ptr(),
                                   0 if ws is None else ws.numel(), _stream_of(stream, q))
    if st != FFPA_OK:
        _raise(st, "ffpa_qk_norm_rope_bwd")
    return dq, dk, dqw, dkw


@functools.lru_cache(maxsize=None)
def qk_norm_rope_bwd_workspace_bytes(D: int) -> int:
    """Bytes of the workspace of ffpa_qk_norm_rope_bwd (0 for an unsupported head dim)."""
    return int(load_library().ffpa_qk_norm_rope_bwd_workspace_bytes(D))


def _workspace(workspace, need: int, device, stream):
    """The caller's workspace, checked, or one of `need` bytes, which the caching allocator hands out
    and takes back in the order of the launch stream."""
    if workspace is None:
        if isinstance(stream, torch.cuda.Stream):
            with torch.cuda.stream(stream):
                return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    if (not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 or workspace.dim() != 1
            or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous 1-D uint8 tensor")
    return workspace


def _check_cache(k_cache, v_cache, dtype, D):
    """(num_pages, page_size, Hkv) of the cache."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be 4-D [num_pages, page_size, Hkv, D] of one shape")
    if k_cache.dtype != dtype or v_cache.dtype != dtype:
        raise TypeError(f"the cache must be {dtype}, got {k_cache.dtype} and {v_cache.dtype}")
    num_pages, page_size, Hkv, Dk = shape
    if Dk != D:
        raise ValueError(f"the cache has head dim {Dk}, the call {D}")
    return num_pages, page_size, Hkv


def _check_ints(t, name, n, dtype):
    """A contiguous 1-D integer tensor of the call with n entries (any number where n is None)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 1 or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must have shape {('any',) if n is None else (n,)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_table(t):
    """block_table [B, max_pages]: int32, entries of a row adjacent.  Returns its row stride."""
    if t.dtype != torch.int32:
        raise TypeError(f"block_table must be int32, got {t.dtype}")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("block_table must be 2-D [B, max_pages] with adjacent entries")
    return t.stride(0)


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
    if k.dim() != 3 or v.shape != k.shape:
        raise ValueError("k and v must be 3-D [T, Hkv, D] of one shape")
    if v.dtype != k.dtype:
        raise TypeError("k and v must share one dtype")
    T, Hkv, D = k.shape
    if q is not None:
        _, Hq, _, _, _ = _qk_shape(q, k)
        q_out = _like(q, q_out, "q_out")
    elif q_out is not None or q_weight is not None:
        raise ValueError("q_out and q_weight need q")
    else:
        Hq = Hkv
    num_pages, page_size, heads = _check_cache(k_cache, v_cache, k.dtype, D)
    if heads != Hkv:
        raise ValueError(f"the cache has {heads} key heads, the keys have {Hkv}")
    _check_ints(slots, "slots", T, torch.int64)
    r = _rope_args(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, rope_scale, 1, T)
    opts = None if status is None else _options(k, None, status, None, False)
    keep, (qs, ks, vs, qos, kcs, vcs) = _strides(q, k, v, q_out, k_cache, v_cache)
    st = load_library().ffpa_kv_append(
        None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(), None if q is None else q_out.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), _dtype_code(k), T, Hq, Hkv, D, num_pages, page_size, qs, ks, vs, qos,
        kcs, vcs, slots.data_ptr(), r, _stream_of(stream, k), opts)
    if st != FFPA_OK:
        _raise(st, "ffpa_kv_append")
    return q_out


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
    if q.dim() != 3:
        raise ValueError("q must be 3-D [B, Hq, D]")
    B, Hq, D = q.shape
    num_pages, page_size, Hkv = _check_cache(k_cache, v_cache, q.dtype, D)
    table_str = _check_table(block_table)
    rows, max_pages = block_table.shape
    if rows != B:
        raise ValueError(f"block_table has {rows} rows for {B} requests")
    _check_ints(seq_lens, "seq_lens", B, torch.int32)
    out = _like(q, out, "out")
    if lse is not None:
        _check_buffer(lse, "lse", (B, Hq), torch.float32, q.device, contiguous=True)
    elif return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    ws = _workspace(workspace, decode_paged_workspace_bytes(Hq, Hkv, D), q.device, stream)
    sc = None if scale is None else ctypes.byref(ctypes.c_float(float(scale)))
    opts = None
    if status is not None or wait_timeout_ns or test_drop_first_copy:
        opts = _options(q, None, status, wait_timeout_ns, test_drop_first_copy)
    keep, (qs, ks, vs, os) = _strides(q, k_cache, v_cache, out)
    st = load_library().ffpa_decode_paged(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
        _dtype_code(q), B, Hq, Hkv, D, num_pages, page_size, max_pages, qs, ks, vs, os, block_table.data_ptr(),
        table_str, seq_lens.data_ptr(), sc, bool(enable_gqa), ws.data_ptr(), ws.numel(), _stream_of(stream, q), opts)
    if st != FFPA_OK:
        _raise(st, "ffpa_decode_paged")
    return (out, lse) if return_lse else out


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
    which there is no page get slot -1; the status word (see ffpa_fwd) receives FFPA_ERR_INVALID.

    Pages of a finished request go back by the caller: written at free_pages[free_count:]."""
    device = block_table.device
    table_str = _check_table(block_table)
    B, max_pages = block_table.shape
    _check_ints(seq_lens, "seq_lens", B, torch.int32)
    _check_ints(new_lens, "new_lens", B, torch.int32)
    _check_ints(free_pages, "free_pages", None, torch.int32)
    _check_ints(free_count, "free_count", 1, torch.int32)
    if num_tokens < 0 or page_size < 1:
        raise ValueError("num_tokens must not be negative and page_size must be positive")
    slots = torch.empty(num_tokens, dtype=torch.int64, device=device)
    positions = torch.empty(num_tokens, dtype=torch.int32, device=device)
    cu = torch.empty(B + 1, dtype=torch.int32, device=device)
    lens, count = torch.empty_like(seq_lens), torch.empty_like(free_count)
    opts = None if status is None else _options(block_table, None, status, None, False)
    st = load_library().ffpa_page_plan(block_table.data_ptr(), table_str, B, max_pages, seq_lens.data_ptr(),
                                       new_lens.data_ptr(), free_pages.data_ptr(), free_pages.numel(),
                                       free_count.data_ptr(), int(page_size), int(num_tokens), slots.data_ptr(),
                                       positions.data_ptr(), cu.data_ptr(), lens.data_ptr(), count.data_ptr(),
                                       _stream_of(stream, block_table), opts)
    if st != FFPA_OK:
        _raise(st, "ffpa_page_plan")
    return slots, positions, cu, lens, count
