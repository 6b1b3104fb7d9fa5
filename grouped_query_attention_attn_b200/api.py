"""Tensor-level calls on top of the C ABI.

PyTorch supplies device memory, shapes and the current stream; every step of
the computation runs in libgqa.so.  Non-OK statuses become exceptions:
``ValueError`` for invalid arguments and workspace problems,
``NotImplementedError`` for unsupported shapes, ``RuntimeError`` otherwise.
"""

import math
from typing import NamedTuple

import torch

from . import _binding as _b

_EXC = {
    _b.GQA_ERR_INVALID_ARG: ValueError,
    _b.GQA_ERR_WORKSPACE: ValueError,
    _b.GQA_ERR_UNSUPPORTED: NotImplementedError,
}


def _check(rc, what):
    if rc != _b.GQA_OK:
        raise _EXC.get(rc, RuntimeError)(f"{what}: {_b.gqa_last_error()} (status {rc})")


def _stream(t):
    return torch.cuda.current_stream(t.device).cuda_stream


def _need(t, name, dtype, ndim):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _shapes(q, k, v):
    B, Tq, Hq, d = q.shape
    Bk, Tkv, Hkv, dk = k.shape
    if Bk != B or dk != d or tuple(v.shape) != tuple(k.shape):
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    return B, Tq, Tkv, Hq, Hkv, d


def attn(q, k, v, causal=True, scale=None, out=None, return_lse=False, window=None, sinks=0,
         rope_theta=None, q_pos0=None):
    """Grouped-query attention forward, bf16.

    q [B, Tq, Hq, d], k/v [B, Tkv, Hkv, d] (bf16, contiguous, on one GPU);
    query head h reads K/V head h // (Hq // Hkv).  Returns o [B, Tq, Hq, d]
    (and lse [B, Hq, Tq] fp32 when ``return_lse``).  ``window`` (an int >= 1)
    selects causal sliding-window attention with ``sinks`` always-visible
    leading keys.  ``rope_theta`` rotates q as it is loaded (query row t at
    position ``q_pos0`` + t, default Tkv - Tq); k must already be rotated.
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.bfloat16, 4)
    B, Tq, Tkv, Hq, Hkv, d = _shapes(q, k, v)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if out is None else out
    _need(o, "out", torch.bfloat16, 4)
    lse = torch.empty((B, Hq, Tq), dtype=torch.float32, device=q.device) if return_lse else None
    lp = lse.data_ptr() if lse is not None else None
    if rope_theta is not None:
        if window is not None:
            raise NotImplementedError("rope_theta with a sliding window")
        pos0 = Tkv - Tq if q_pos0 is None else int(q_pos0)
        rc = _b.gqa_attn_fwd_rope(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lp,
                                  B, Tq, Tkv, Hq, Hkv, d, int(bool(causal)), scale, pos0,
                                  float(rope_theta), _stream(q))
    elif window is None:
        rc = _b.gqa_attn_fwd_lse(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lp,
                                 B, Tq, Tkv, Hq, Hkv, d, int(bool(causal)), scale, _stream(q))
    else:
        if not causal:
            raise ValueError("a sliding window needs causal=True")
        rc = _b.gqa_attn_fwd_window(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lp,
                                    B, Tq, Tkv, Hq, Hkv, d, int(window), int(sinks), scale,
                                    _stream(q))
    _check(rc, "gqa_attn_fwd")
    return (o, lse) if return_lse else o


def _need_host(t, name, ndim):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-d tensor, got {tuple(t.shape)}")


def host_staging(q, k, device=None):
    """Device staging buffers (q, k, v, o) for ``attn_host`` on host tensors shaped like q, k."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    return (torch.empty(q.shape, dtype=torch.bfloat16, device=dev),
            torch.empty(k.shape, dtype=torch.bfloat16, device=dev),
            torch.empty(k.shape, dtype=torch.bfloat16, device=dev),
            torch.empty(q.shape, dtype=torch.bfloat16, device=dev))


def attn_host(q, k, v, out=None, causal=True, scale=None, staging=None, done=None):
    """``attn`` on host (CPU, preferably pinned) bf16 tensors: the copies up and down
    run in the library, overlapped with the attention chunk by chunk.  ``staging``
    is a (q, k, v, o) tuple of device buffers (``host_staging``).  The call is
    asynchronous on the staging device's current stream and returns ``out``: valid
    once that stream has reached this point, or, with ``done`` (a torch.cuda.Event),
    once ``done`` has completed (the stream is then not held for the copies down, so
    consecutive calls overlap).  The host tensors must stay alive and unchanged until
    then: the copies run after this function returns."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need_host(t, n, 4)
    B, Tq, Tkv, Hq, Hkv, d = _shapes(q, k, v)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty(q.shape, dtype=torch.bfloat16, pin_memory=q.is_pinned()) if out is None else out
    _need_host(o, "out", 4)
    if tuple(o.shape) != tuple(q.shape):
        raise ValueError(f"out shape {tuple(o.shape)} != q shape {tuple(q.shape)}")
    st = host_staging(q, k) if staging is None else staging
    for t, ref, n in zip(st, (q, k, k, q), ("q_dev", "k_dev", "v_dev", "o_dev")):
        _need(t, n, torch.bfloat16, 4)
        if tuple(t.shape) != tuple(ref.shape):
            raise ValueError(f"{n} shape {tuple(t.shape)} != {tuple(ref.shape)}")
    ev = None
    if done is not None:
        done.record(torch.cuda.current_stream(st[0].device))   # makes sure the event exists
        ev = done.cuda_event
    rc = _b.gqa_attn_fwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                              *(t.data_ptr() for t in st), B, Tq, Tkv, Hq, Hkv, d,
                              int(bool(causal)), scale, _stream(st[0]), ev)
    _check(rc, "gqa_attn_fwd_host")
    return o


def attn_f32(q, k, v, causal=True, scale=None, return_lse=False):
    """The same operation in fp32 (FP32 pipe); q/k/v fp32 in the same layouts."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, torch.float32, 4)
    B, Tq, Tkv, Hq, Hkv, d = _shapes(q, k, v)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, Tq), dtype=torch.float32, device=q.device) if return_lse else None
    rc = _b.gqa_attn_fwd_f32(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                             lse.data_ptr() if lse is not None else None,
                             B, Tq, Tkv, Hq, Hkv, d, int(bool(causal)), scale, _stream(q))
    _check(rc, "gqa_attn_fwd_f32")
    return (o, lse) if return_lse else o


def decode_workspace_size(B, Hq, Hkv, d, Lmax):
    return int(_b.gqa_decode_workspace_size(B, Hq, Hkv, d, Lmax))


def decode(q, k_cache, v_cache, seqlens, scale=None, workspace=None, out=None, window=None,
           sinks=0, rope_theta=None):
    """One query token per sequence against a bf16 KV cache.

    q [B, Hq, d], caches [B, Lmax, Hkv, d], seqlens int32 [B] on the device.
    ``workspace``: a uint8 CUDA tensor of at least decode_workspace_size(...)
    bytes (allocated here when None).  ``rope_theta`` rotates q as it is loaded
    (position max(seqlens[b] - 1, 0)); the cached keys must already be rotated.
    """
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(seqlens, "seqlens", torch.int32, 1)
    B, Hq, d = q.shape
    Bc, Lmax, Hkv, dc = k_cache.shape
    if Bc != B or dc != d or tuple(v_cache.shape) != tuple(k_cache.shape) or seqlens.shape[0] != B:
        raise ValueError("decode shape mismatch")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    need = decode_workspace_size(B, Hq, Hkv, d, Lmax)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q) if out is None else out
    if rope_theta is not None:
        if window is not None:
            raise NotImplementedError("rope_theta with a sliding window")
        rc = _b.gqa_decode_rope(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                seqlens.data_ptr(), o.data_ptr(), B, Hq, Hkv, d, Lmax, scale,
                                float(rope_theta), workspace.data_ptr(), workspace.numel(),
                                _stream(q))
    elif window is None:
        rc = _b.gqa_decode(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                           seqlens.data_ptr(), o.data_ptr(), B, Hq, Hkv, d, Lmax, scale,
                           workspace.data_ptr(), workspace.numel(), _stream(q))
    else:
        rc = _b.gqa_decode_window(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                  seqlens.data_ptr(), o.data_ptr(), B, Hq, Hkv, d, Lmax,
                                  int(window), int(sinks), scale, workspace.data_ptr(),
                                  workspace.numel(), _stream(q))
    _check(rc, "gqa_decode")
    return o


def fold_kv(kv, g):
    """Mean-pool the heads of a bf16 [B, T, H, d] K or V tensor into g contiguous groups."""
    _need(kv, "kv", torch.bfloat16, 4)
    B, T, H, d = kv.shape
    out = torch.empty((B, T, g, d), dtype=kv.dtype, device=kv.device)
    rc = _b.gqa_fold_kv(kv.data_ptr(), out.data_ptr(), B, T, H, g, d, _stream(kv))
    _check(rc, "gqa_fold_kv")
    return out


def attn_bwd_workspace_size(B, Tq, Hq):
    return int(_b.gqa_attn_bwd_workspace_size(B, Tq, Hq))


def attn_bwd(q, k, v, o, lse, dout, causal=True, scale=None, window=None, sinks=0,
             workspace=None):
    """Gradients (dq, dk, dv) of attn(q, k, v) for the upstream gradient dout.

    o and lse are the forward's outputs (attn(..., return_lse=True)).  dk / dv
    of a K/V head are summed over the G query heads that share it.
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _need(t, n, torch.bfloat16, 4)
    _need(lse, "lse", torch.float32, 3)
    B, Tq, Tkv, Hq, Hkv, d = _shapes(q, k, v)
    if tuple(o.shape) != tuple(q.shape) or tuple(dout.shape) != tuple(q.shape):
        raise ValueError("o and dout must have q's shape")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    need = int(_b.gqa_attn_bwd_workspace_size(B, Tq, Hq))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    rc = _b.gqa_attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(),
                         lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                         B, Tq, Tkv, Hq, Hkv, d, int(bool(causal)),
                         0 if window is None else int(window), int(sinks), scale,
                         workspace.data_ptr(), workspace.numel(), _stream(q))
    _check(rc, "gqa_attn_bwd")
    return dq, dk, dv


def rope_(x, pos0=0, theta=10000.0):
    """Rotary position embedding of a bf16 [B, T, H, d] q or k tensor, in place
    (row t at position pos0 + t).  Returns x."""
    _need(x, "x", torch.bfloat16, 4)
    B, T, H, d = x.shape
    _check(_b.gqa_rope(x.data_ptr(), B, T, H, d, int(pos0), float(theta), _stream(x)), "gqa_rope")
    return x


def rope_qk_(q, k, pos0=0, theta=10000.0):
    """RoPE of bf16 q [B, T, Hq, d] and k [B, T, Hkv, d] in place, in one launch
    (row t of both at position pos0 + t).  Returns (q, k)."""
    _need(q, "q", torch.bfloat16, 4)
    _need(k, "k", torch.bfloat16, 4)
    B, T, Hq, d = q.shape
    if k.shape[0] != B or k.shape[1] != T or k.shape[3] != d:
        raise ValueError(f"k shape {tuple(k.shape)} does not match q {tuple(q.shape)}")
    _check(_b.gqa_rope_qk(q.data_ptr(), k.data_ptr(), B, T, Hq, k.shape[2], d, int(pos0),
                          float(theta), _stream(q)), "gqa_rope_qk")
    return q, k


def rope_decode_q_(q, seqlens, theta=10000.0):
    """RoPE of bf16 decode queries [B, H, d] in place, sequence b at position seqlens[b] - 1."""
    _need(q, "q", torch.bfloat16, 3)
    _need(seqlens, "seqlens", torch.int32, 1)
    B, H, d = q.shape
    _check(_b.gqa_rope_decode_q(q.data_ptr(), seqlens.data_ptr(), B, H, d, float(theta),
                                _stream(q)), "gqa_rope_decode_q")
    return q


# ------------------------------------------------- the paged 8-bit K/V cache --

class Cache8(NamedTuple):
    """K and V in pages of 8-bit values: k, v [n_pages, Hkv, page, d] (float8_e4m3fn or
    int8) and the fp32 scales k_scale, v_scale [n_pages, Hkv, page // block] of each
    block of tokens and head.  A table [B, M] int32 names each sequence's pages."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def cache8(n_pages, Hkv, d, page=64, block=64, dtype=torch.float8_e4m3fn, device=None):
    """An empty Cache8 of n_pages pages of ``page`` rows, scales per ``block`` rows."""
    if page < 1 or block < 1 or page % block:
        raise ValueError(f"block={block} must divide page={page}")
    if dtype not in (torch.float8_e4m3fn, torch.int8):
        raise ValueError(f"dtype={dtype} must be torch.float8_e4m3fn or torch.int8")
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    pool, scale = (n_pages, Hkv, page, d), (n_pages, Hkv, page // block)
    return Cache8(torch.zeros(pool, dtype=torch.uint8, device=dev).view(dtype),
                  torch.zeros(pool, dtype=torch.uint8, device=dev).view(dtype),
                  torch.zeros(scale, dtype=torch.float32, device=dev),
                  torch.zeros(scale, dtype=torch.float32, device=dev))


def cache8_append_(cache, table, seqlens, k, v, counts=None):
    """Quantise new rows into a Cache8, in place: the first counts[b] (default T) rows
    of bf16 k, v [B, T, Hkv, d] become rows seqlens[b], seqlens[b] + 1, ... of sequence
    b (table [B, M], seqlens, counts [B] int32; seqlens is not changed).  The scale of a
    block is the smallest power of two that covers its rows (int8 loses up to one of its
    seven bits against max / 127); rows already in a block are requantised, and so
    rounded again, when its scale grows.  The page of row seqlens[b] must belong to
    sequence b alone.  Returns cache."""
    return _b.torch_binding().cache8_append_(cache, table, seqlens, k, v, counts)


def cache8_read(cache, table, seqlens, T, out=None):
    """Rows 0 .. T - 1 of every sequence as bf16 (k, v), each [B, T, Hkv, d] (``out``: that
    pair of tensors); rows at and past seqlens[b] are zeros."""
    return _b.torch_binding().cache8_read(cache, table, seqlens, T, out)


def cache8_copy_(cache, moves):
    """Apply page moves (int32 [1 + cap, 3], from pages_fork_ or pages_compact_) to a Cache8,
    in place: moves[0, 0] moves (src, dst, rows), each replacing the first ``rows`` rows of
    page dst by those of page src.  A page may be the destination of one move only and
    then occur in no other.  Returns cache."""
    return _b.torch_binding().cache8_copy_(cache, moves)


def decode8_workspace_size(B, Hq, Hkv, d, Lmax):
    """Bytes of workspace for decode8 on tables of Lmax = M * page rows."""
    return int(_b.gqa_decode8_workspace_size(B, Hq, Hkv, d, Lmax))


def decode8(q, cache, table, seqlens, scale=None, workspace=None, out=None, window=None, sinks=0,
            rope_theta=None):
    """One query token per sequence against a Cache8: ``decode`` for a paged 8-bit cache.

    q [B, Hq, d] bf16, table [B, M] and seqlens [B] int32 on the device; returns
    [B, Hq, d].  ``window`` (an int >= 1) leaves the newest ``window`` rows and the first
    ``sinks`` visible.  ``rope_theta`` rotates q as it is loaded (position
    max(seqlens[b] - 1, 0)); the cached keys must already be rotated.  Weights enter the
    product with V in fp16 (11 bits) and elements of q below 2^-14 of their row's largest
    count to 2^-25 of it; scores, statistics and sums are fp32.  ``workspace``:
    a uint8 CUDA tensor of at least decode8_workspace_size(...) bytes (allocated here
    when None)."""
    return _b.torch_binding().decode8(q, cache, table, seqlens, scale, workspace, out, window, sinks,
                                      rope_theta)


def pages_workspace_size(B, M, n_pages):
    """Bytes of workspace for the pages_* calls on a table [B, M] and refs [n_pages]."""
    return int(_b.gqa_pages_workspace_size(B, M, n_pages))


def pages_resize_(table, refs, lengths, page, workspace=None):
    """Give row b of a page table [B, M] exactly the pages that lengths[b] rows need, in
    place: pages past them are released (refs [n_pages] counts the entries that name a
    page), missing ones taken from the free pages, lowest first.  lengths[b] = 0 frees
    the row.  device_status raises if the pool ran out.  Returns table."""
    return _b.torch_binding().pages_resize_(table, refs, lengths, page, workspace)


def pages_fork_(table, refs, seqlens, parents, page, workspace=None):
    """Row b becomes a copy of the old row parents[b] (int32 [B]; negative: empty), all rows
    at once and in place, seqlens too: full pages are shared, and every child but one
    gets a page of its own for the last, partly filled one.  Returns the moves
    [1 + B, 3] to apply with cache8_copy_ to each cache that uses the table."""
    return _b.torch_binding().pages_fork_(table, refs, seqlens, parents, page, workspace)


def pages_compact_(table, refs, page, workspace=None):
    """Move the pages in use to the lowest numbers, in place.  Returns the moves
    [1 + n_pages // 2, 3] to apply with cache8_copy_ to each cache that uses the table."""
    return _b.torch_binding().pages_compact_(table, refs, page, workspace)


def device_status(reset=True):
    """Synchronise, then raise if a kernel recorded an error (e.g. a wait timeout)."""
    _check(_b.gqa_device_status(int(bool(reset))), "gqa_device_status")
