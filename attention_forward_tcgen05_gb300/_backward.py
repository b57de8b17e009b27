"""Gradients of the prefill attention (the last part of include/attn.h).

As in ``_binding``: the raw entry points keep the C names and argument order, and the
torch helpers only check, allocate outputs and workspaces and pass pointers and the
stream.
"""
from __future__ import annotations

import functools
import math

from ._binding import ATTN_OK, AttnError, _keys, _launching, load
from ._serving import _device, _elsewhere, _need, _out_code, _sized, _torch, _workspace


# ------------------------------------------------------------------ raw C ABI
def attn_prefill_backward(*args) -> int:
    return load().attn_prefill_backward(*args)


def attn_prefill_varlen_backward(*args) -> int:
    return load().attn_prefill_varlen_backward(*args)


def attn_prefill_backward_workspace(B, Hq, Hkv, total_q, max_sq, max_kv, d) -> int:
    return int(load().attn_prefill_backward_workspace(B, Hq, Hkv, total_q, max_sq, max_kv, d))


# ------------------------------------------------------------------ torch helpers
_KEPT = 64 << 20  # bytes; a larger call takes far longer than an allocation


@functools.lru_cache(maxsize=1024)
def _work_bytes(*sizes):
    return attn_prefill_backward_workspace(*sizes)


def _work(n, dev, handle):
    """A workspace of n bytes and its pointer: the stream's kept one, or a large call's own, which
    goes back to the stream's allocations."""
    if n <= _KEPT:
        t = _workspace((n + 3) // 4, dev, handle)
    else:
        t = _torch().empty(n, dtype=_torch().uint8, device="cuda")
    return t, t.data_ptr()


def _gradients(out, q, k, v, dev):
    """(tensors, pointers) of dq, dk, dv."""
    torch = _torch()
    if out is None:
        out = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        return out, (out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr())
    if len(out) != 3:
        raise ValueError("out must be (dq, dk, dv)")
    return tuple(out), [_sized(t, f"out[{i}]", torch.bfloat16, dev, *like.shape)
                        for i, (t, like) in enumerate(zip(out, (q, k, v)))]


def _saved(do, o, lse, dlse, q, lse_shape, dev):
    """(dout, o, lse, dlse pointers, o's type code)."""
    torch = _torch()
    gp = _sized(do, "do", torch.bfloat16, dev, *q.shape)
    if not isinstance(o, torch.Tensor):
        raise TypeError("o must be a CUDA tensor")
    code = _out_code(o.dtype)
    op = _sized(o, "o", o.dtype, dev, *q.shape)
    lp = _sized(lse, "lse", torch.float32, dev, *lse_shape)
    dp = None if dlse is None else _sized(dlse, "dlse", torch.float32, dev, *lse_shape)
    return gp, op, lp, dp, code


def prefill_backward(do, q, k, v, o, lse, causal: bool = True, window: int = 0, n_sink: int = 0,
                     scale: float | None = None, dlse=None, out=None, stream=None):
    """Gradients of ``prefill`` and (window > 0) ``prefill_window`` (attn_prefill_backward):
    (dq, dk, dv) bf16, shaped like q, k, v, into ``out`` if given.

    do [B,Sq,Hq,d] bf16 is the gradient of o; q, k, v are the forward call's inputs, o (bf16
    or fp32) and lse its results; causal, window, n_sink and scale as there.  dlse fp32
    [B,Hq,Sq]: the gradient of lse, for a loss that uses it."""
    torch = _torch()
    dev = _device(q, "q")
    if stream is not None or dev != torch._C._cuda_getDevice():
        return _elsewhere(lambda: prefill_backward(do, q, k, v, o, lse, causal, window, n_sink, scale, dlse, out), q,
                          stream, (do, q, k, v, o, lse, dlse, out))
    handle = torch._C._cuda_getCurrentRawStream(dev)
    qp = _need(q, "q", torch.bfloat16, 4, dev)
    kp = _need(k, "k", torch.bfloat16, 4, dev)
    B, Sq, Hq, d = q.shape
    _, Skv, Hkv, _ = k.shape
    if k.shape[0] != B or k.shape[3] != d:
        raise ValueError(f"q and k differ in batch or head dim: {list(q.shape)} and {list(k.shape)}")
    vp = _sized(v, "v", torch.bfloat16, dev, *k.shape)
    gp, op, lp, dp, code = _saved(do, o, lse, dlse, q, (B, Hq, Sq), dev)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, (dq, dk, dv) = _gradients(out, q, k, v, dev)
    n = _work_bytes(B, Hq, Hkv, B * Sq, Sq, Skv, d)
    work, wp = _work(n, dev, handle)
    with _launching:
        rc = load().attn_prefill_backward(gp, qp, kp, vp, op, lp, dp, dq, dk, dv, B, Hq, Hkv, Sq, Skv, d, int(causal),
                                          _keys(window), _keys(n_sink), scale, code, wp, n, handle)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_prefill_backward")
    return out


def prefill_varlen_backward(do, q, kcache, vcache, o, lse, cu_seqlens_q, kv_lens, max_sq: int, causal: bool = True,
                            window: int = 0, n_sink: int = 0, scale: float | None = None, dlse=None, out=None,
                            stream=None):
    """Gradients of ``prefill_varlen`` (attn_prefill_varlen_backward): (dq, dkcache, dvcache)
    bf16, shaped like q, kcache, vcache.

    do and o [total_q,Hq,d], lse and dlse [Hq,total_q], the rest as in the forward call.
    Rows of no sequence and cache slots at or past kv_lens[b] are not used: their gradients
    are 0, or stay as they are in ``out``."""
    torch = _torch()
    dev = _device(q, "q")
    if stream is not None or dev != torch._C._cuda_getDevice():
        return _elsewhere(lambda: prefill_varlen_backward(do, q, kcache, vcache, o, lse, cu_seqlens_q, kv_lens, max_sq,
                                                          causal, window, n_sink, scale, dlse, out), q, stream,
                          (do, q, kcache, vcache, o, lse, cu_seqlens_q, kv_lens, dlse, out))
    handle = torch._C._cuda_getCurrentRawStream(dev)
    qp = _need(q, "q", torch.bfloat16, 3, dev)
    kp = _need(kcache, "kcache", torch.bfloat16, 4, dev)
    total, Hq, d = q.shape
    B, max_kv, Hkv, dk_ = kcache.shape
    if dk_ != d:
        raise ValueError(f"q and the cache differ in head dim: {d} and {dk_}")
    vp = _sized(vcache, "vcache", torch.bfloat16, dev, *kcache.shape)
    cu = _sized(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev, B + 1)
    np_ = _sized(kv_lens, "kv_lens", torch.int32, dev, B)
    gp, op, lp, dp, code = _saved(do, o, lse, dlse, q, (Hq, total), dev)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    max_sq = int(max_sq)
    fill = int(out is None)
    out, (dq, dk, dv) = _gradients(out, q, kcache, vcache, dev)
    if fill and B == 0:
        out[0].zero_()  # (a call of no sequences writes nothing)
    n = _work_bytes(B, Hq, Hkv, total, max_sq, max_kv, d)
    work, wp = _work(n, dev, handle)
    with _launching:
        rc = load().attn_prefill_varlen_backward(gp, qp, kp, vp, op, lp, dp, dq, dk, dv, cu, np_, B, Hq, Hkv, total,
                                                 max_sq, max_kv, d, int(causal), _keys(window), _keys(n_sink), scale,
                                                 code, fill, wp, n, handle)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_prefill_varlen_backward")
    return out
