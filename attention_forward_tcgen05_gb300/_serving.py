"""The paged-cache serving calls: rotary positions with the cache append, attention of
new tokens over pages (chunks and single tokens), accumulated attention weights and
eviction by them (the second half of include/attn.h).

As in ``_binding``: the raw entry points keep the C names and argument order, and the
torch helpers only check, allocate outputs and pass pointers and the stream.

A paged cache is a pair of pools ``kcache``/``vcache`` [num_pages, page_size, Hkv, d] and
a ``page_table`` int32 [B, max_pages]; key j of sequence b lies in slot j % page_size of
page ``page_table[b, j // page_size]``.  Table entries past a sequence's keys are never
read.  Where ``page_table`` is optional, None means the dense cache [B, max_kv, Hkv, d]
of the other calls.
"""
from __future__ import annotations

import ctypes
import functools
import math

from ._binding import ATTN_BF16, ATTN_F32, ATTN_OK, AttnError, _counters, _launching, _lock, load


_module = None


def _torch():
    global _module
    if _module is None:
        import torch
        _module = torch
    return _module


# ------------------------------------------------------------------ raw C ABI
def attn_rope_append(*args) -> int:
    return load().attn_rope_append(*args)


def attn_prefill_paged(*args) -> int:
    return load().attn_prefill_paged(*args)


def attn_prefill_paged_splits(B, Hq, Hkv, total_q, max_sq, max_kv, d, min_rows) -> int:
    return load().attn_prefill_paged_splits(B, Hq, Hkv, total_q, max_sq, max_kv, d, min_rows)


def attn_decode_paged(*args) -> int:
    return load().attn_decode_paged(*args)


def attn_decode_paged_splits(B, Hq, Hkv, max_kv, d, o_dtype, min_rows) -> int:
    return load().attn_decode_paged_splits(B, Hq, Hkv, max_kv, d, o_dtype, min_rows)


def attn_key_weights(*args) -> int:
    return load().attn_key_weights(*args)


def attn_evict(*args) -> int:
    return load().attn_evict(*args)


# ------------------------------------------------------------------ argument checks
# A decode step makes these calls many times over on a few microseconds of GPU work, so the
# checks are kept short: one pass over a tensor's attributes, device and stream as integers.
def _device(lead, name):
    try:
        dev = lead.get_device()
    except AttributeError:
        dev = -1
    if dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    return dev


def _record(x, stream):
    """Mark the tensors of nested arguments as used by a stream: their memory is not given
    out again before what it has queued is done."""
    if isinstance(x, (tuple, list)):
        for y in x:
            _record(y, stream)
    elif isinstance(x, _torch().Tensor):
        x.record_stream(stream)


def _elsewhere(call, lead, stream, inputs):
    """``call()`` with the tensors' device and the given stream current: outputs and
    workspaces then belong to that stream, and the outputs are marked as used by the
    caller's, the inputs as used by the given one."""
    torch = _torch()
    if stream is not None and stream.device != lead.device:
        raise ValueError("the stream belongs to another device than the tensors")
    with torch.cuda.device(lead.device):
        own = torch.cuda.current_stream()
        if stream is None or stream == own:
            return call()
        with torch.cuda.stream(stream):
            result = call()
        _record(inputs, stream)
        _record(result, own)
        return result


def _refuse(t, name, dtype, ndim, dev, contiguous=True):
    """Why a tensor is not what the call reads or writes."""
    if not isinstance(t, _torch().Tensor) or not t.is_cuda or t.get_device() != dev:
        raise TypeError(f"{name} must be a CUDA tensor on device {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be a {'contiguous ' if contiguous else ''}{ndim}-D tensor")


def _need(t, name, dtype, ndim, dev):
    """A contiguous tensor's pointer."""
    try:
        if t.get_device() == dev and t.dtype is dtype and t.is_contiguous() and t.dim() == ndim:
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, ndim, dev)


def _sized(t, name, dtype, dev, *want):
    """A contiguous tensor of exactly that shape: its pointer."""
    try:
        if t.get_device() == dev and t.dtype is dtype and t.is_contiguous() and t.shape == want:
            return t.data_ptr()
    except AttributeError:
        pass
    if _need(t, name, dtype, len(want), dev) is not None:
        raise ValueError(f"{name} must have shape {list(want)}, got {list(t.shape)}")


def _cache(kcache, vcache, page_table, B, dev, need_table=False):
    """(k, v, table pointers, Hkv, d, max_pages, page_size, num_pages) of a cache."""
    torch = _torch()
    kp = _need(kcache, "kcache", torch.bfloat16, 4, dev)
    n, page, Hkv, d = shape = kcache.shape
    vp = None
    if vcache is not None:
        vp = _need(vcache, "vcache", torch.bfloat16, 4, dev)
        if vcache.shape != shape:
            raise ValueError("kcache and vcache must have the same shape")
    if page_table is None and not need_table:
        if n != B:
            raise ValueError(f"a dense cache must have one row per sequence: {n} for {B}")
        return kp, vp, None, Hkv, d, 1, page, n
    tp = _need(page_table, "page_table", torch.int32, 2, dev)
    rows, width = page_table.shape
    if rows != B:
        raise ValueError(f"page_table must have one row per sequence: {rows} for {B}")
    return kp, vp, tp, Hkv, d, width, page, n


def _out_code(dtype):
    torch = _torch()
    if dtype is torch.bfloat16:
        return ATTN_BF16
    if dtype is torch.float32:
        return ATTN_F32
    raise TypeError(f"unsupported output dtype {dtype}")


# The split rules, kept by their sizes: the loops of a decode come with the same ones, and a
# foreign call takes 3 us of a helper's 20.
@functools.lru_cache(maxsize=1024)
def _prefill_splits(B, Hq, Hkv, total, max_sq, max_kv, d):
    rows = ctypes.c_int(1)
    n = attn_prefill_paged_splits(B, Hq, Hkv, total, max_sq, max_kv, d, ctypes.addressof(rows))
    return max(n, 1), rows.value


@functools.lru_cache(maxsize=1024)
def _decode_splits(B, Hq, Hkv, max_kv, d, code):
    rows = ctypes.c_int(1)
    n = attn_decode_paged_splits(B, Hq, Hkv, max_kv, d, code, ctypes.addressof(rows))
    return max(n, 1), rows.value


# Workspaces of prefill_paged and decode_paged: kept for each stream, whose launches are
# ordered; a call holds _launching while it makes its launches, so that another thread's on the
# same stream do not come between two of them.  A call being captured gets its own (two graphs
# may replay at the same time).  They grow to the largest call seen and stay for the process.
_partials = {}  # (device, stream handle) -> fp32


def _workspace(floats, dev, handle):
    """fp32 workspace for split partials."""
    torch = _torch()
    if torch._C._cuda_isCurrentStreamCapturing():
        return torch.empty(floats, dtype=torch.float32, device="cuda")
    work = _partials.get((dev, handle))
    if work is None or work.numel() < floats:
        work = _partials[dev, handle] = torch.empty(floats, dtype=torch.float32, device="cuda")
    return work


def _stream_counters(n, dev, handle):
    """Zeroed completion counters of n rows."""
    torch = _torch()
    if torch._C._cuda_isCurrentStreamCapturing():
        return torch.zeros(n, dtype=torch.int32, device="cuda")
    counters = _counters.get((dev, handle))
    if counters is None or counters.numel() < n:
        with _lock:
            counters = torch.zeros(max(n, 4096), dtype=torch.int32, device="cuda")
            torch.cuda.synchronize(dev)  # zeroed before the stream uses it, and no longer in use
            _counters[dev, handle] = counters
    return counters


# ------------------------------------------------------------------ rotary positions
def rope_frequencies(rot_dim: int, base: float = 10000.0, device="cuda", factor: float = 1.0,
                     method: str = "none", original_length: int = 4096, low_turns: float = 1.0,
                     high_turns: float = 32.0):
    """Frequencies for ``rope_append``: (inv_freq float64 [rot_dim / 2] in radians per
    position, amp).

    f_i = base^(-2i / rot_dim), stretched for contexts ``factor`` times the original ones:
    ``"linear"`` divides every f_i by factor; ``"ntk"`` raises the base by
    factor^(rot_dim / (rot_dim - 2)); ``"yarn"`` keeps the pairs that turn at least
    ``high_turns`` times over ``original_length`` positions, divides those that turn at
    most ``low_turns`` times, blends between (linearly in the number of turns), and sets
    amp = 0.1 ln(factor) + 1.  (A checkpoint whose frequencies were blended otherwise, over
    the pair's index between rounded bounds, say, brings its own: pass them as inv_freq.)"""
    torch = _torch()
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    if not (base > 0 and factor > 0 and math.isfinite(base) and math.isfinite(factor)):
        raise ValueError("base and factor must be positive and finite")
    if method == "ntk" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    f = torch.pow(torch.tensor(base, dtype=torch.float64), -i / rot_dim)
    amp = 1.0
    if method == "linear":
        f = f / factor
    elif method == "yarn":
        if not (original_length > 0 and high_turns > low_turns >= 0):
            raise ValueError("yarn needs original_length > 0 and high_turns > low_turns >= 0")
        turns = original_length * f / (2 * math.pi)
        keep = ((turns - low_turns) / (high_turns - low_turns)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
        amp = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif method not in ("none", "ntk"):
        raise ValueError(f"unknown method {method!r}")
    return f.to(device), amp


def _token_rows(t, name, bf16, dev, total, H, d):
    """Rows of tokens [total, H, d] with any stride between tokens (a view of a fused
    projection's output, say): (pointer, stride in elements)."""
    try:
        good = t.get_device() == dev and t.dtype is bf16 and t.dim() == 3
    except AttributeError:
        good = False
    if not good:
        _refuse(t, name, bf16, 3, dev, contiguous=False)
    if t.shape != (total, H, d):
        raise ValueError(f"{name} must have shape {[total, H, d]}, got {list(t.shape)}")
    row, head, one = t.stride()
    if one != 1 or (H > 1 and head != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), (row if total > 1 else H * d)


def rope_append(q, k, v, kcache, vcache, kv_lens, inv_freq, page_table=None, cu_seqlens_q=None, positions=None,
                interleaved: bool = False, amp: float = 1.0, out=None, stream=None):
    """Rotate the new tokens' queries and keys and append keys and values to the cache
    (attn_rope_append).

    q [total,Hq,d] (or None: keys and values only), k/v [total,Hkv,d] bf16, rows of tokens
    at any stride; kv_lens int32 [B] counts each sequence's keys after the append: its new
    tokens are its last ones.  cu_seqlens_q int32 [B+1] gives each sequence's tokens; None
    means one token per sequence.  inv_freq float64 [rot_dim / 2] (None: no rotation), amp
    as from ``rope_frequencies``; positions int32 [total] (None: a token's key index).
    Writes kcache / vcache; returns the rotated q [total,Hq,d] (``out`` if given; it may be
    q itself when q is contiguous), or None without q."""
    torch = _torch()
    dev = _device(k, "k")
    if stream is not None or dev != torch._C._cuda_getDevice():
        return _elsewhere(lambda: rope_append(q, k, v, kcache, vcache, kv_lens, inv_freq, page_table, cu_seqlens_q,
                                              positions, interleaved, amp, out), k, stream,
                          (q, k, v, kcache, vcache, kv_lens, inv_freq, page_table, cu_seqlens_q, positions, out))
    handle = torch._C._cuda_getCurrentRawStream(dev)
    np_ = _need(kv_lens, "kv_lens", torch.int32, 1, dev)
    total, B = k.shape[0], kv_lens.shape[0]
    kp, vp, tp, Hkv, d, max_pages, page, n_pages = _cache(kcache, vcache, page_table, B, dev)
    kr, ks = _token_rows(k, "k", torch.bfloat16, dev, total, Hkv, d)
    vr, vs = _token_rows(v, "v", torch.bfloat16, dev, total, Hkv, d)
    Hq, qr, qs, op = Hkv, None, 0, None
    if q is not None:
        Hq = q.shape[1]
        qr, qs = _token_rows(q, "q", torch.bfloat16, dev, total, Hq, d)
        if out is None:
            out = torch.empty((total, Hq, d), dtype=torch.bfloat16, device="cuda")  # (q may be strided)
            op = out.data_ptr()
        else:
            op = _sized(out, "out", torch.bfloat16, dev, total, Hq, d)
    elif out is not None:
        raise ValueError("out without q")
    cu = pos = fr = None
    if cu_seqlens_q is not None:
        cu = _sized(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev, B + 1)
    elif total != B:
        raise ValueError("without cu_seqlens_q there must be one token per sequence")
    if positions is not None:
        pos = _sized(positions, "positions", torch.int32, dev, total)
    rot = 0
    if inv_freq is not None:
        fr = _need(inv_freq, "inv_freq", torch.float64, 1, dev)
        rot = 2 * inv_freq.shape[0]
    rc = load().attn_rope_append(qr, kr, vr, qs, ks, vs, pos, fr, op, kp, vp, tp, cu, np_, B, Hq, Hkv, total, d, rot,
                                 int(interleaved), amp, max_pages, page, n_pages, handle)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_rope_append")
    return out


# ------------------------------------------------------------------ attention over pages
def prefill_paged(q, kcache, vcache, page_table, cu_seqlens_q, kv_lens, max_sq: int, causal: bool = True,
                  scale: float | None = None, out_dtype=None, stream=None, out=None, window: int = 0,
                  n_sink: int = 0, n_splits: int = 0, min_rows_per_split: int = 1, max_kv: int | None = None,
                  parts=None):
    """``prefill_varlen`` over a paged cache (attn_prefill_paged): the same arguments and
    results, with page_table.  n_splits key splits of each sequence (0: chosen from the
    sizes and max_kv, the longest sequence's keys, by default the table's width) are
    joined through ``parts``, optional fp32 (part_o [total_q,Hq,n_splits,d], part_lse
    [total_q,Hq,n_splits]; by default a workspace kept for the stream).  window > 0 takes
    no splits.  Give max_kv where the table is wider than its sequences are long: sized
    for the table, most splits would hold no keys."""
    torch = _torch()
    dev = _device(q, "q")
    if stream is not None or dev != torch._C._cuda_getDevice():
        return _elsewhere(lambda: prefill_paged(q, kcache, vcache, page_table, cu_seqlens_q, kv_lens, max_sq, causal,
                                                scale, out_dtype, None, out, window, n_sink, n_splits,
                                                min_rows_per_split, max_kv, parts), q, stream,
                          (q, kcache, vcache, page_table, cu_seqlens_q, kv_lens, out, parts))
    handle = torch._C._cuda_getCurrentRawStream(dev)
    qp = _need(q, "q", torch.bfloat16, 3, dev)
    np_ = _need(kv_lens, "kv_lens", torch.int32, 1, dev)
    B = kv_lens.shape[0]
    kp, vp, tp, Hkv, d, max_pages, page, n_pages = _cache(kcache, vcache, page_table, B, dev, need_table=True)
    total, Hq, dq = q.shape
    max_sq = int(max_sq)
    if dq != d:
        raise ValueError(f"q and the cache differ in head dim: {dq} and {d}")
    cu = _sized(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev, B + 1)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        o = torch.empty_like(q) if out_dtype in (None, torch.bfloat16) else torch.empty_like(q, dtype=out_dtype)
        lse = torch.empty((Hq, total), dtype=torch.float32, device="cuda")
        op, lp = o.data_ptr(), lse.data_ptr()
    else:
        o, lse = out
        op = _sized(o, "out[0]", o.dtype, dev, total, Hq, d)
        lp = _sized(lse, "out[1]", torch.float32, dev, Hq, total)
    code = _out_code(o.dtype)
    lib = load()
    if n_splits == 0:
        n_splits = 1
        if parts is not None:
            n_splits = parts[0].shape[2]
        elif not window:
            n_splits, min_rows_per_split = _prefill_splits(B, Hq, Hkv, total, max_sq,
                                                           max_pages * page if max_kv is None else max_kv, d)
    pp = ps = None
    if n_splits > 1:
        if parts is None:
            rows = total * Hq * n_splits
            work = _workspace(rows * (d + 1), dev, handle)
            pp = work.data_ptr()
            ps = pp + rows * d * 4
        else:
            pp = _sized(parts[0], "parts[0]", torch.float32, dev, total, Hq, n_splits, d)
            ps = _sized(parts[1], "parts[1]", torch.float32, dev, total, Hq, n_splits)
    with _launching:
        rc = lib.attn_prefill_paged(qp, kp, vp, op, lp, tp, cu, np_, B, Hq, Hkv, total, max_sq, max_pages, page,
                                    n_pages, d, int(causal), int(window), int(n_sink), scale, n_splits, min_rows_per_split, pp,
                                    ps, code, handle)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_prefill_paged")
    return o, lse


def decode_paged(q, kcache, vcache, page_table, kv_lens, n_splits: int = 0, min_rows_per_split: int = 1,
                 scale: float | None = None, out_dtype=None, stream=None, out=None, parts=None, counters=None,
                 max_kv: int | None = None):
    """``decode`` over a paged cache (attn_decode_paged): the same arguments and results,
    with page_table.  n_splits = 0 chooses the splits and their least rows from the sizes
    and max_kv (the longest sequence's keys, by default the table's width; give it where
    the table is wider).  The split partials and counters are kept for the stream."""
    torch = _torch()
    dev = _device(q, "q")
    if stream is not None or dev != torch._C._cuda_getDevice():
        return _elsewhere(lambda: decode_paged(q, kcache, vcache, page_table, kv_lens, n_splits, min_rows_per_split,
                                               scale, out_dtype, None, out, parts, counters, max_kv), q, stream,
                          (q, kcache, vcache, page_table, kv_lens, out, parts, counters))
    handle = torch._C._cuda_getCurrentRawStream(dev)
    qp = _need(q, "q", torch.bfloat16, 3, dev)
    B, Hq, dq = q.shape
    np_ = _sized(kv_lens, "kv_lens", torch.int32, dev, B)
    kp, vp, tp, Hkv, d, max_pages, page, n_pages = _cache(kcache, vcache, page_table, B, dev, need_table=True)
    if dq != d:
        raise ValueError(f"q and the cache differ in head dim: {dq} and {d}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        o = torch.empty_like(q) if out_dtype in (None, torch.bfloat16) else torch.empty_like(q, dtype=out_dtype)
        lse = torch.empty((B, Hq), dtype=torch.float32, device="cuda")
        op, lp = o.data_ptr(), lse.data_ptr()
    else:
        o, lse = out
        op = _sized(o, "out[0]", o.dtype, dev, B, Hq, d)
        lp = _sized(lse, "out[1]", torch.float32, dev, B, Hq)
    code = _out_code(o.dtype)
    lib = load()
    if n_splits == 0:
        if parts is not None:
            n_splits = parts[0].shape[2]
        else:
            n_splits, min_rows_per_split = _decode_splits(B, Hq, Hkv, max_pages * page if max_kv is None else max_kv,
                                                          d, code)
    pp = ps = cp = None
    if n_splits > 1:
        rows = B * Hq * n_splits
        if parts is None:
            work = _workspace(rows * (d + 1), dev, handle)
            pp = work.data_ptr()
            ps = pp + rows * d * 4
        else:
            pp = _sized(parts[0], "parts[0]", torch.float32, dev, B, Hq, n_splits, d)
            ps = _sized(parts[1], "parts[1]", torch.float32, dev, B, Hq, n_splits)
        if counters is None:
            counters = _stream_counters(B * Hq, dev, handle)
        elif counters.dtype != torch.int32 or counters.get_device() != dev or counters.numel() < B * Hq:
            raise TypeError("counters must be a CUDA int32 tensor of at least B*Hq entries")
        cp = counters.data_ptr()
    with _launching:
        rc = lib.attn_decode_paged(qp, kp, vp, tp, np_, B, Hq, Hkv, d, max_pages, page, n_pages, scale, n_splits,
                                   min_rows_per_split, pp, ps, op, lp, code, cp, handle)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_decode_paged")
    return o, lse


# ------------------------------------------------------------------ weights and eviction
def _weight_rows(weights, dev, B, Hkv, capacity):
    p = _need(weights, "weights", _torch().float32, 3, dev)
    b, h, n = weights.shape
    if b != B or h != Hkv or n < capacity:
        raise ValueError(f"weights must be [{B}, {Hkv}, at least {capacity}], got {[b, h, n]}")
    return p, n


def key_weights(q, lse, kcache, kv_lens, weights, page_table=None, cu_seqlens_q=None, max_sq: int | None = None,
                causal: bool = True, window: int = 0, n_sink: int = 0, scale: float | None = None,
                accumulate: bool = True, stream=None):
    """Add the attention weight that each cached key received from the new rows to
    ``weights`` fp32 [B,Hkv,>= capacity] (attn_key_weights), or set it (accumulate=False).

    q and lse are an attention call's: q [total_q,Hq,d], lse [Hq,total_q] with cu_seqlens_q
    int32 [B+1] and max_sq, the longest sequence's rows (a longer one is reported by
    sync_check); or, without cu_seqlens_q, a decode's q [B,Hq,d], lse [B,Hq].  causal,
    window, n_sink and scale as in that call.  Entries at or past kv_lens[b] stay as they
    are.  Returns weights."""
    torch = _torch()
    if cu_seqlens_q is None:
        max_sq = 1
    elif max_sq is None:
        raise ValueError("cu_seqlens_q needs max_sq, the longest sequence's rows")
    dev = _device(q, "q")
    if stream is not None or dev != torch._C._cuda_getDevice():
        return _elsewhere(lambda: key_weights(q, lse, kcache, kv_lens, weights, page_table, cu_seqlens_q, max_sq,
                                              causal, window, n_sink, scale, accumulate), q, stream,
                          (q, lse, kcache, kv_lens, weights, page_table, cu_seqlens_q))
    handle = torch._C._cuda_getCurrentRawStream(dev)
    qp = _need(q, "q", torch.bfloat16, 3, dev)
    np_ = _need(kv_lens, "kv_lens", torch.int32, 1, dev)
    B = kv_lens.shape[0]
    kp, _, tp, Hkv, d, max_pages, page, n_pages = _cache(kcache, None, page_table, B, dev)
    total, Hq, dq = q.shape
    if dq != d:
        raise ValueError(f"q and the cache differ in head dim: {dq} and {d}")
    cu = None
    if cu_seqlens_q is not None:
        cu = _sized(cu_seqlens_q, "cu_seqlens_q", torch.int32, dev, B + 1)
        lp = _sized(lse, "lse", torch.float32, dev, Hq, total)
    else:
        if total != B:
            raise ValueError("without cu_seqlens_q there must be one row per sequence")
        lp = _sized(lse, "lse", torch.float32, dev, B, Hq)
    wp, w_stride = _weight_rows(weights, dev, B, Hkv, max_pages * page)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    rc = load().attn_key_weights(qp, lp, kp, tp, cu, np_, wp, w_stride, B, Hq, Hkv, total, int(max_sq), d, max_pages, page,
                                 n_pages, int(causal), int(window), int(n_sink), scale, int(accumulate), handle)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_key_weights")
    return weights


def evict(weights, kcache, vcache, kv_lens, budget: int, n_recent: int = 0, n_sink: int = 0, page_table=None,
          dst=None, out=None, stream=None):
    """Shrink every sequence to at most ``budget`` keys per KV head (attn_evict): the first
    n_sink, the last n_recent and the largest ``weights`` fp32 [B,Hkv,>= capacity] between
    them (equal ones: the lowest index) stay, moved to the front in order.

    In place by default: kcache, vcache and weights (the freed entries become 0) change;
    pages that other sequences share must not be among them.  ``dst`` = (kcache, vcache,
    page_table or None, weights or None) writes to other pages instead and leaves the source
    as it is; the two must not overlap.  Returns (kept int32 [B,Hkv,budget]: the old index
    of each key, -1 past the end; new kv_lens int32 [B]), into ``out`` if given (the new
    lengths may be kv_lens itself)."""
    torch = _torch()
    dev = _device(kcache, "kcache")
    if stream is not None or dev != torch._C._cuda_getDevice():
        return _elsewhere(lambda: evict(weights, kcache, vcache, kv_lens, budget, n_recent, n_sink, page_table, dst,
                                        out), kcache, stream, (weights, kcache, vcache, kv_lens, page_table, dst, out))
    handle = torch._C._cuda_getCurrentRawStream(dev)
    budget, n_recent, n_sink = int(budget), int(n_recent), int(n_sink)
    np_ = _need(kv_lens, "kv_lens", torch.int32, 1, dev)
    B = kv_lens.shape[0]
    if vcache is None:
        raise TypeError("vcache must be a CUDA tensor")
    kp, vp, tp, Hkv, d, max_pages, page, n_pages = _cache(kcache, vcache, page_table, B, dev)
    wp, w_stride = _weight_rows(weights, dev, B, Hkv, max_pages * page)
    k2 = v2 = t2 = None
    m2 = p2 = n2 = 0
    w2 = wp
    if dst is not None:
        dk, dv, dt, dw = dst
        if dv is None:
            raise TypeError("dst needs both caches")
        k2, v2, t2, H2, d2, m2, p2, n2 = _cache(dk, dv, dt, B, dev)
        if H2 != Hkv or d2 != d:
            raise ValueError("dst must have the cache's heads and head dim")
        w2 = None if dw is None else _sized(dw, "dst weights", torch.float32, dev, B, Hkv, w_stride)
    if out is None:
        kept = torch.empty((B, Hkv, max(budget, 0)), dtype=torch.int32, device="cuda")
        lens = torch.empty_like(kv_lens)
        ep, lp = kept.data_ptr(), lens.data_ptr()
    else:
        kept, lens = out
        ep = _sized(kept, "out[0]", torch.int32, dev, B, Hkv, budget)
        lp = _sized(lens, "out[1]", torch.int32, dev, B)
    rc = load().attn_evict(wp, w2, w_stride, kp, vp, tp, np_, B, Hkv, d, max_pages, page, n_pages, budget, n_recent,
                           n_sink, k2, v2, t2, m2, p2, n2, ep, lp, handle)
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_evict")
    return kept, lens
