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
import math

from ._binding import ATTN_BF16, ATTN_F32, ATTN_OK, AttnError, _counters, _lock, _torch, load


# ------------------------------------------------------------------ raw C ABI
def attn_rope_append(*args) -> int:
    return load().attn_rope_append(*args)


def attn_prefill_paged(*args) -> int:
    return load().attn_prefill_paged(*args)


def attn_prefill_paged_splits(B, Hq, Hkv, total_q, max_sq, max_kv, d) -> int:
    return load().attn_prefill_paged_splits(B, Hq, Hkv, total_q, max_sq, max_kv, d)


def attn_decode_paged(*args) -> int:
    return load().attn_decode_paged(*args)


def attn_decode_paged_splits(B, Hkv, max_kv, min_rows) -> int:
    return load().attn_decode_paged_splits(B, Hkv, max_kv, min_rows)


def attn_key_weights(*args) -> int:
    return load().attn_key_weights(*args)


def attn_evict(*args) -> int:
    return load().attn_evict(*args)


# ------------------------------------------------------------------ argument checks
class _Call:
    """The device of a call (every tensor lies on it) and the stream it goes to."""

    def __init__(self, lead, name, stream):
        torch = _torch()
        if not isinstance(lead, torch.Tensor) or not lead.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        self.device = lead.device
        self.stream = stream
        current = torch.cuda.current_device()
        self._guard = None if self.device.index == current else torch.cuda.device(self.device)
        if self._guard is not None:
            self._guard.__enter__()
        try:
            own = torch.cuda.current_stream()
            if stream is not None and stream.device != self.device:
                raise ValueError("the stream belongs to another device than the tensors")
            self.handle = (stream or own).cuda_stream
            self._foreign = stream is not None and stream.cuda_stream != own.cuda_stream
        except BaseException:
            self.close()
            raise

    def close(self):
        if self._guard is not None:
            self._guard.__exit__(None, None, None)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def check(self, t, name, dtype, ndim, contiguous=True):
        if not isinstance(t, _torch().Tensor) or t.device != self.device:
            raise TypeError(f"{name} must be a CUDA tensor on {self.device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.dim() != ndim or (contiguous and not t.is_contiguous()):
            raise ValueError(f"{name} must be a {'contiguous ' if contiguous else ''}{ndim}-D tensor")
        return t.data_ptr()

    def shape(self, t, name, *want):
        if tuple(t.shape) != want:
            raise ValueError(f"{name} must have shape {list(want)}, got {list(t.shape)}")

    def output(self, t, name, dtype, *want):
        """An output given by the caller, checked."""
        p = self.check(t, name, dtype, len(want))
        self.shape(t, name, *want)
        return p

    def scratch(self, *shape):
        """fp32 workspace that lives until the call's work on its stream is done."""
        t = _torch().empty(shape, dtype=_torch().float32, device=self.device)
        if self._foreign:
            t.record_stream(self.stream)
        return t

    def result(self, shape, dtype):
        t = _torch().empty(shape, dtype=dtype, device=self.device)
        if self._foreign:
            t.record_stream(self.stream)
        return t

    def cache(self, kcache, vcache, page_table, B, need_table=False):
        """(k, v, table pointers, Hkv, d, max_pages, page_size, num_pages) of a cache."""
        bf16 = _torch().bfloat16
        kp = self.check(kcache, "kcache", bf16, 4)
        vp = self.check(vcache, "vcache", bf16, 4) if vcache is not None else None
        n, page, Hkv, d = kcache.shape
        if vcache is not None and vcache.shape != kcache.shape:
            raise ValueError("kcache and vcache must have the same shape")
        if page_table is None:
            if need_table:
                raise TypeError("page_table must be a CUDA tensor")
            if n != B:
                raise ValueError(f"a dense cache must have one row per sequence: {n} for {B}")
            return kp, vp, None, Hkv, d, 1, page, n
        tp = self.check(page_table, "page_table", _torch().int32, 2)
        if page_table.shape[0] != B:
            raise ValueError(f"page_table must have one row per sequence: {page_table.shape[0]} for {B}")
        return kp, vp, tp, Hkv, d, page_table.shape[1], page, n


def _out_code(dtype):
    torch = _torch()
    if dtype == torch.bfloat16:
        return ATTN_BF16
    if dtype == torch.float32:
        return ATTN_F32
    raise TypeError(f"unsupported output dtype {dtype}")


def _stream_counters(n, c):
    """Zeroed completion counters for a decode_paged call on c's stream: a buffer for each
    stream (its calls are ordered), and one of its own for a call being captured (two graphs
    may replay at the same time)."""
    torch = _torch()
    if torch.cuda.is_current_stream_capturing():
        return torch.zeros(n, dtype=torch.int32, device=c.device)
    key = (c.device.type, c.device.index, c.handle)
    buf = _counters.get(key)
    if buf is None or buf.numel() < n:
        with _lock:
            buf = torch.zeros(max(n, 4096), dtype=torch.int32, device=c.device)
            torch.cuda.synchronize(c.device)  # zeroed before the stream uses it, and no longer in use
            _counters[key] = buf
    return buf


def _raise(rc, what):
    if rc != ATTN_OK:
        raise AttnError(rc, what)


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
    most ``low_turns`` times, blends linearly between, and sets amp = 0.1 ln(factor) + 1."""
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


def _token_rows(c, t, name, total, H, d):
    """Rows of tokens [total, H, d] with any stride between tokens (a view of a fused
    projection's output, say): (pointer, stride in elements)."""
    p = c.check(t, name, _torch().bfloat16, 3, contiguous=False)
    c.shape(t, name, total, H, d)
    if t.stride(2) != 1 or (H > 1 and t.stride(1) != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return p, (t.stride(0) if total > 1 else H * d)


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
    with _Call(k, "k", stream) as c:
        if k.dim() != 3:
            raise ValueError("k must be a 3-D tensor")
        total = k.shape[0]
        np_ = c.check(kv_lens, "kv_lens", torch.int32, 1)
        B = kv_lens.shape[0]
        kp, vp, tp, Hkv, d, max_pages, page, n_pages = c.cache(kcache, vcache, page_table, B)
        kr, ks = _token_rows(c, k, "k", total, Hkv, d)
        vr, vs = _token_rows(c, v, "v", total, Hkv, d)
        Hq, qr, qs, op = Hkv, None, 0, None
        if q is not None:
            Hq = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else 0
            qr, qs = _token_rows(c, q, "q", total, Hq, d)
            if out is None:
                out = c.result((total, Hq, d), torch.bfloat16)
            op = c.output(out, "out", torch.bfloat16, total, Hq, d)
        elif out is not None:
            raise ValueError("out without q")
        cu = pos = fr = None
        if cu_seqlens_q is not None:
            cu = c.output(cu_seqlens_q, "cu_seqlens_q", torch.int32, B + 1)
        elif total != B:
            raise ValueError("without cu_seqlens_q there must be one token per sequence")
        if positions is not None:
            pos = c.output(positions, "positions", torch.int32, total)
        rot = 0
        if inv_freq is not None:
            fr = c.check(inv_freq, "inv_freq", torch.float64, 1)
            rot = 2 * inv_freq.shape[0]
        _raise(load().attn_rope_append(qr, kr, vr, qs, ks, vs, pos, fr, op, kp, vp, tp, cu, np_, B, Hq, Hkv, total, d,
                                       rot, int(interleaved), amp, max_pages, page, n_pages, c.handle),
               "attn_rope_append")
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
    [total_q,Hq,n_splits]).  window > 0 takes no splits."""
    torch = _torch()
    with _Call(q, "q", stream) as c:
        qp = c.check(q, "q", torch.bfloat16, 3)
        np_ = c.check(kv_lens, "kv_lens", torch.int32, 1)
        B = kv_lens.shape[0]
        kp, vp, tp, Hkv, d, max_pages, page, n_pages = c.cache(kcache, vcache, page_table, B, need_table=True)
        total, Hq = q.shape[0], q.shape[1]
        c.shape(q, "q", total, Hq, d)
        cu = c.output(cu_seqlens_q, "cu_seqlens_q", torch.int32, B + 1)
        if scale is None:
            scale = 1.0 / math.sqrt(d)
        if out is None:
            o, lse = c.result((total, Hq, d), out_dtype or torch.bfloat16), c.result((Hq, total), torch.float32)
        else:
            o, lse = out
        code = _out_code(o.dtype)
        op = c.output(o, "out[0]", o.dtype, total, Hq, d)
        lp = c.output(lse, "out[1]", torch.float32, Hq, total)
        if n_splits == 0:
            if window or parts is not None or Hq % Hkv:
                n_splits = 1 if parts is None else parts[0].shape[2]
            else:
                n_splits = max(1, load().attn_prefill_paged_splits(B, Hq, Hkv, total, int(max_sq),
                                                                   max_pages * page if max_kv is None else max_kv, d))
        pp = ps = None
        if n_splits > 1:
            if parts is None:
                parts = c.scratch(total, Hq, n_splits, d), c.scratch(total, Hq, n_splits)
            pp = c.output(parts[0], "parts[0]", torch.float32, total, Hq, n_splits, d)
            ps = c.output(parts[1], "parts[1]", torch.float32, total, Hq, n_splits)
        _raise(load().attn_prefill_paged(qp, kp, vp, op, lp, tp, cu, np_, B, Hq, Hkv, total, int(max_sq), max_pages,
                                         page, n_pages, d, int(causal), window, n_sink, scale, n_splits,
                                         min_rows_per_split, pp, ps, code, c.handle), "attn_prefill_paged")
    return o, lse


def decode_paged(q, kcache, vcache, page_table, kv_lens, n_splits: int = 0, min_rows_per_split: int = 1,
                 scale: float | None = None, out_dtype=None, stream=None, out=None, parts=None, counters=None,
                 max_kv: int | None = None):
    """``decode`` over a paged cache (attn_decode_paged): the same arguments and results,
    with page_table.  n_splits = 0 chooses the splits and their least rows from the sizes
    and max_kv (the longest sequence's keys, by default the table's width)."""
    torch = _torch()
    with _Call(q, "q", stream) as c:
        qp = c.check(q, "q", torch.bfloat16, 3)
        np_ = c.check(kv_lens, "kv_lens", torch.int32, 1)
        B, Hq = q.shape[0], q.shape[1]
        c.shape(kv_lens, "kv_lens", B)
        kp, vp, tp, Hkv, d, max_pages, page, n_pages = c.cache(kcache, vcache, page_table, B, need_table=True)
        c.shape(q, "q", B, Hq, d)
        if scale is None:
            scale = 1.0 / math.sqrt(d)
        if n_splits == 0:
            if parts is not None:
                n_splits = parts[0].shape[2]
            else:
                rows = ctypes.c_int(1)
                n_splits = load().attn_decode_paged_splits(B, Hkv, max_pages * page if max_kv is None else max_kv,
                                                           ctypes.addressof(rows))
                min_rows_per_split = rows.value
        if parts is None:
            parts = c.scratch(B, Hq, n_splits, d), c.scratch(B, Hq, n_splits)
        pp = c.output(parts[0], "parts[0]", torch.float32, B, Hq, n_splits, d)
        ps = c.output(parts[1], "parts[1]", torch.float32, B, Hq, n_splits)
        if out is None:
            o, lse = c.result((B, Hq, d), out_dtype or torch.bfloat16), c.result((B, Hq), torch.float32)
        else:
            o, lse = out
        code = _out_code(o.dtype)
        op = c.output(o, "out[0]", o.dtype, B, Hq, d)
        lp = c.output(lse, "out[1]", torch.float32, B, Hq)
        if counters is None:
            counters = _stream_counters(B * Hq, c)
        elif counters.dtype != torch.int32 or counters.device != c.device or counters.numel() < B * Hq:
            raise TypeError("counters must be a CUDA int32 tensor of at least B*Hq entries")
        _raise(load().attn_decode_paged(qp, kp, vp, tp, np_, B, Hq, Hkv, d, max_pages, page, n_pages, scale, n_splits,
                                        min_rows_per_split, pp, ps, op, lp, code, counters.data_ptr(), c.handle),
               "attn_decode_paged")
    return o, lse


# ------------------------------------------------------------------ weights and eviction
def key_weights(q, lse, kcache, kv_lens, weights, page_table=None, cu_seqlens_q=None, max_sq: int = 1,
                causal: bool = True, window: int = 0, n_sink: int = 0, scale: float | None = None,
                accumulate: bool = True, stream=None):
    """Add the attention weight that each cached key received from the new rows to
    ``weights`` fp32 [B,Hkv,>= capacity] (attn_key_weights), or set it (accumulate=False).

    q and lse are an attention call's: q [total_q,Hq,d], lse [Hq,total_q] with cu_seqlens_q
    int32 [B+1] and max_sq; or, without cu_seqlens_q, a decode's q [B,Hq,d], lse [B,Hq].
    causal, window, n_sink and scale as in that call.  Entries at or past kv_lens[b] stay
    as they are.  Returns weights."""
    torch = _torch()
    with _Call(q, "q", stream) as c:
        qp = c.check(q, "q", torch.bfloat16, 3)
        np_ = c.check(kv_lens, "kv_lens", torch.int32, 1)
        B = kv_lens.shape[0]
        kp, _, tp, Hkv, d, max_pages, page, n_pages = c.cache(kcache, None, page_table, B)
        total, Hq = q.shape[0], q.shape[1]
        c.shape(q, "q", total, Hq, d)
        cu = None
        if cu_seqlens_q is not None:
            cu = c.output(cu_seqlens_q, "cu_seqlens_q", torch.int32, B + 1)
            lp = c.output(lse, "lse", torch.float32, Hq, total)
        else:
            if total != B:
                raise ValueError("without cu_seqlens_q there must be one row per sequence")
            lp = c.output(lse, "lse", torch.float32, B, Hq)
            max_sq = 1
        wp = c.check(weights, "weights", torch.float32, 3)
        if weights.shape[0] != B or weights.shape[1] != Hkv or weights.shape[2] < max_pages * page:
            raise ValueError(f"weights must be [B, Hkv, at least {max_pages * page}], got {list(weights.shape)}")
        if scale is None:
            scale = 1.0 / math.sqrt(d)
        _raise(load().attn_key_weights(qp, lp, kp, tp, cu, np_, wp, weights.shape[2], B, Hq, Hkv, total, int(max_sq),
                                       d, max_pages, page, n_pages, int(causal), window, n_sink, scale,
                                       int(accumulate), c.handle), "attn_key_weights")
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
    with _Call(kcache, "kcache", stream) as c:
        np_ = c.check(kv_lens, "kv_lens", torch.int32, 1)
        B = kv_lens.shape[0]
        kp, vp, tp, Hkv, d, max_pages, page, n_pages = c.cache(kcache, vcache, page_table, B)
        wp = c.check(weights, "weights", torch.float32, 3)
        if weights.shape[0] != B or weights.shape[1] != Hkv or weights.shape[2] < max_pages * page:
            raise ValueError(f"weights must be [B, Hkv, at least {max_pages * page}], got {list(weights.shape)}")
        k2 = v2 = t2 = None
        m2 = p2 = n2 = 0
        w2 = wp
        if dst is not None:
            dk, dv, dt, dw = dst
            if dv is None:
                raise TypeError("dst needs both caches")
            k2, v2, t2, H2, d2, m2, p2, n2 = c.cache(dk, dv, dt, B)
            if (H2, d2) != (Hkv, d):
                raise ValueError("dst must have the cache's heads and head dim")
            w2 = None
            if dw is not None:
                w2 = c.output(dw, "dst weights", torch.float32, *weights.shape)
        budget = int(budget)
        if out is None:
            kept, lens = c.result((B, Hkv, max(budget, 0)), torch.int32), c.result((B,), torch.int32)
        else:
            kept, lens = out
        ep = c.output(kept, "out[0]", torch.int32, B, Hkv, budget)
        lp = c.output(lens, "out[1]", torch.int32, B)
        _raise(load().attn_evict(wp, w2, weights.shape[2], kp, vp, tp, np_, B, Hkv, d, max_pages, page, n_pages,
                                 budget, n_recent, n_sink, k2, v2, t2, m2, p2, n2, ep, lp, c.handle), "attn_evict")
    return kept, lens
