"""The paged serving calls reject bad arguments on the host: the C entry points before any
CUDA call (no GPU needed), the torch helpers before they call them."""
import ctypes

import pytest
import torch

import attention_forward_tcgen05_gb300 as attn
from attention_forward_tcgen05_gb300 import build as attn_build

N = None
P = 16   # an aligned non-null dummy (never dereferenced: validation fails first)
M = 18   # misaligned
INVALID, UNSUPPORTED, OK = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED, attn.ATTN_OK


@pytest.fixture(scope="module", autouse=True)
def lib():
    attn_build.build()
    return attn.load()


class Call:
    """An entry point with valid arguments by name; a test changes some of them."""

    def __init__(self, fn, **args):
        self.fn, self.args = fn, args

    def __call__(self, **changes):
        assert set(changes) <= set(self.args), set(changes) - set(self.args)
        return self.fn(*{**self.args, **changes}.values())


ROPE = Call(attn.attn_rope_append, q=P, k=P, v=P, qs=256, ks=128, vs=128, positions=P, inv_freq=P, q_out=P, kc=P,
            vc=P, table=P, cu=P, lens=P, B=2, Hq=4, Hkv=2, total=7, d=64, rot=64, inter=0, amp=1.0, max_pages=4,
            page=16, pages=9, stream=N)
PREFILL = Call(attn.attn_prefill_paged, q=P, kc=P, vc=P, o=P, lse=P, table=P, cu=P, lens=P, B=2, Hq=4, Hkv=2, total=7,
               max_sq=5, max_pages=4, page=16, pages=9, d=64, causal=1, window=0, sink=0, scale=0.5, n_splits=1,
               min_rows=1, po=N, pl=N, o_dtype=0, stream=N)
DECODE = Call(attn.attn_decode_paged, q=P, kc=P, vc=P, table=P, lens=P, B=2, Hq=4, Hkv=2, d=64, max_pages=4, page=16,
              pages=9, scale=0.5, n_splits=2, min_rows=1, po=P, pl=P, o=P, lse=P, o_dtype=0, counters=P, stream=N)
WEIGHTS = Call(attn.attn_key_weights, q=P, lse=P, kc=P, table=P, cu=P, lens=P, w=P, stride=64, B=2, Hq=4, Hkv=2,
               total=7, max_sq=5, d=64, max_pages=4, page=16, pages=9, causal=1, window=0, sink=0, scale=0.5, acc=1,
               stream=N)
EVICT = Call(attn.attn_evict, w=P, wo=P, stride=64, kc=P, vc=P, table=P, lens=P, B=2, Hkv=2, d=64, max_pages=4,
             page=16, pages=9, budget=8, recent=2, sink=1, k2=N, v2=N, table2=N, max_pages2=0, page2=0, pages2=0,
             kept=P, new_lens=P, stream=N)


@pytest.mark.parametrize("call", [ROPE, PREFILL, DECODE, WEIGHTS, EVICT], ids=["rope", "prefill", "decode", "weights", "evict"])
def test_common_refusals(call):
    a = call.args
    if "Hq" in a:
        assert call(Hq=3) == INVALID
        assert call(Hq=0) == INVALID
    assert call(Hkv=0) == INVALID
    assert call(B=-1) == INVALID
    for d in (0, 32, 96, 512):
        assert call(d=d) == UNSUPPORTED
    # the cache's sizes
    assert call(max_pages=0) == INVALID
    assert call(page=0) == INVALID
    assert call(pages=-1) == INVALID
    assert call(max_pages=1 << 20, page=1 << 11) == INVALID  # 2^31 keys
    assert call(pages=1 << 20, page=1 << 11) == INVALID      # 2^31 slots
    for name in ("kc", "vc", "lens"):
        if name in a:
            assert call(**{name: N}) == INVALID
    for name in ("kc", "vc"):
        if name in a:
            assert call(**{name: M}) == INVALID
    assert call(lens=M + 1) == INVALID
    assert call(table=M) == INVALID
    # without a table: one page per sequence (dense), or refused
    if call in (PREFILL, DECODE):
        assert call(table=N) == INVALID
    else:
        assert call(table=N) == INVALID                                  # several pages a sequence
        assert call(table=N, max_pages=1, page=64, pages=1) == INVALID   # fewer rows than sequences
    if "scale" in a:
        for s in (0.0, -1.0, float("nan"), float("inf")):
            assert call(scale=s) == INVALID
    if "o_dtype" in a:
        assert call(o_dtype=2) == UNSUPPORTED


def test_empty_work_is_a_no_op():
    assert ROPE(B=0, total=0, q=N, k=N, v=N, q_out=N, lens=N, cu=P) == OK
    assert ROPE(total=0, k=N, v=N) == OK
    assert PREFILL(B=0, q=N, o=N) == OK
    assert PREFILL(total=0, q=N, o=N) == OK
    assert PREFILL(max_sq=0, q=N) == OK
    assert DECODE(B=0) == OK
    assert WEIGHTS(B=0, q=N, w=N) == OK
    assert EVICT(B=0, w=N, kept=N) == OK


def test_rope():
    for rot in (-16, 8, 20, 80):
        assert ROPE(rot=rot) == UNSUPPORTED
    assert ROPE(inv_freq=N) == INVALID
    assert ROPE(inv_freq=20) == INVALID  # fp64 on 4 bytes
    assert ROPE(amp=float("nan")) == INVALID
    assert ROPE(q=N) == INVALID and ROPE(q_out=N) == INVALID  # both or neither
    assert ROPE(cu=N) == INVALID         # one token each, but 7 for 2
    assert ROPE(qs=248) == INVALID and ROPE(qs=257) == INVALID
    assert ROPE(ks=120) == INVALID and ROPE(vs=132) == INVALID
    assert ROPE(q_out=P, qs=512) == INVALID  # in place over a strided q
    assert ROPE(q=M) == INVALID and ROPE(k=M) == INVALID and ROPE(positions=M) == INVALID
    assert ROPE(total=-1) == INVALID


def test_prefill():
    assert PREFILL(total=-1) == INVALID and PREFILL(max_sq=-1) == INVALID
    assert PREFILL(window=-1) == INVALID and PREFILL(sink=-1) == INVALID
    assert PREFILL(window=4, causal=0) == INVALID
    assert PREFILL(window=4, n_splits=2, po=P, pl=P) == UNSUPPORTED
    for n in (0, -1, 1025):
        assert PREFILL(n_splits=n) == INVALID
    assert PREFILL(n_splits=2) == INVALID  # no partials
    assert PREFILL(n_splits=2, po=M, pl=P) == INVALID
    assert PREFILL(min_rows=-1) == INVALID
    for name in ("q", "o", "lse"):
        assert PREFILL(**{name: N}) == INVALID and PREFILL(**{name: M}) == INVALID
    assert PREFILL(cu=N) == INVALID and PREFILL(cu=M) == INVALID
    assert PREFILL(total=1 << 30) == INVALID  # 2^32 rows of heads
    assert PREFILL(max_sq=1 << 30) == INVALID


def test_decode():
    for n in (0, 1025):
        assert DECODE(n_splits=n) == INVALID
    assert DECODE(min_rows=-1) == INVALID
    for name in ("q", "o", "lse", "po", "pl", "counters"):
        assert DECODE(**{name: N}) == INVALID
    assert DECODE(Hq=258, Hkv=2) == INVALID  # groups above 128
    assert DECODE(counters=M) == INVALID


def test_weights():
    assert WEIGHTS(stride=63) == INVALID
    assert WEIGHTS(cu=N) == INVALID  # one row each, but 7 for 2
    assert WEIGHTS(cu=N, total=2) == INVALID  # and max_sq 1
    assert WEIGHTS(window=4, causal=0) == INVALID and WEIGHTS(window=-1) == INVALID and WEIGHTS(sink=-1) == INVALID
    for name in ("q", "lse", "w"):
        assert WEIGHTS(**{name: N}) == INVALID
    assert WEIGHTS(q=M) == INVALID
    assert WEIGHTS(scale=1e-31) == UNSUPPORTED and WEIGHTS(scale=2e30) == UNSUPPORTED
    assert WEIGHTS(total=1 << 30) == INVALID and WEIGHTS(max_sq=1 << 30) == INVALID


def test_evict():
    assert EVICT(budget=0) == INVALID and EVICT(budget=2) == INVALID  # below n_recent + n_sink
    assert EVICT(recent=-1) == INVALID and EVICT(sink=-1) == INVALID
    assert EVICT(recent=2 ** 31 - 1, sink=2 ** 31 - 1) == INVALID
    assert EVICT(stride=63) == INVALID
    for name in ("w", "kept", "new_lens"):
        assert EVICT(**{name: N}) == INVALID
    dst = dict(k2=32, v2=32, table2=P, max_pages2=1, page2=16, pages2=4)
    assert EVICT(**{**dst, "v2": N}) == INVALID and EVICT(**{**dst, "k2": N}) == INVALID
    assert EVICT(**{**dst, "page2": 7}) == INVALID  # no room for the budget
    assert EVICT(**{**dst, "table2": N, "pages2": 1}) == INVALID
    # the source as its own destination
    assert EVICT(k2=P, v2=P, table2=P, max_pages2=4, page2=16, pages2=9) == INVALID


def test_split_rules():
    rows = ctypes.c_int(0)
    r = ctypes.addressof(rows)
    assert attn.attn_prefill_paged_splits(1, 3, 2, 1, 1, 1, 64, r) == INVALID
    assert attn.attn_prefill_paged_splits(1, 4, 2, 1, 1, 1, 96, r) == INVALID
    assert attn.attn_prefill_paged_splits(1, 4, 2, 1, 1, 1, 64, N) == INVALID
    assert attn.attn_decode_paged_splits(1, 3, 2, 1, 64, 0, r) == INVALID
    assert attn.attn_decode_paged_splits(1, 4, 2, -1, 64, 0, r) == INVALID
    assert attn.attn_decode_paged_splits(1, 4, 2, 1, 64, 0, N) == INVALID
    assert attn.attn_decode_paged_splits(1, 4, 2, 1, 64, 2, r) == INVALID
    for B in (0, 1, 7, 64, 4096):
        for Hq, Hkv in ((1, 1), (28, 4), (32, 2), (128, 1), (300, 2)):
            for kv in (0, 1, 300, 5000, 1 << 20, 1 << 30):
                for d in (64, 128, 256):
                    for dtype in (0, 1):
                        n = attn.attn_decode_paged_splits(B, Hq, Hkv, kv, d, dtype, r)
                        assert 1 <= n <= 1024 and rows.value >= 0 and (n == 1 or n * 192 < kv + 192)
                    for sq in (0, 1, 9, 600, 70000):
                        n = attn.attn_prefill_paged_splits(B, Hq, Hkv, B * sq, sq, kv, d, r)
                        # enough splits of rows.value rows for every key, and none of them idle
                        assert 1 <= n <= 32 and rows.value % 128 == 0 and n * rows.value >= kv, (B, Hq, kv, d, sq)
    # the largest length an int holds
    for B in (1, 4096):
        assert 1 <= attn.attn_prefill_paged_splits(B, 28, 4, B, 1, (1 << 31) - 1, 128, r) <= 32
        assert 0 < rows.value and rows.value % 128 == 0
        assert 1 <= attn.attn_decode_paged_splits(B, 64, 2, (1 << 31) - 1, 128, 1, r) <= 48 and rows.value > 0
    # few rows against many keys are split, a full batch is not
    assert attn.attn_prefill_paged_splits(1, 28, 4, 8, 8, 30000, 128, r) >= 8
    assert attn.attn_prefill_paged_splits(64, 28, 4, 64 * 512, 512, 4096, 128, r) == 1
    assert attn.attn_decode_paged_splits(1, 28, 4, 30000, 128, 0, r) >= 16
    assert attn.attn_decode_paged_splits(512, 32, 8, 4096, 128, 0, r) == 1


def test_helpers_refuse_host_tensors():
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    lens = torch.ones(2, dtype=torch.int32)
    t = torch.zeros(2, 1, dtype=torch.int32)
    w = torch.zeros(2, 2, 16)
    for lead in (x, None):
        with pytest.raises(TypeError):
            attn.rope_append(x, lead, x, c, c, lens, None)
        with pytest.raises(TypeError):
            attn.prefill_paged(lead, c, c, t, lens, lens, 1)
        with pytest.raises(TypeError):
            attn.decode_paged(lead, c, c, t, lens)
        with pytest.raises(TypeError):
            attn.key_weights(lead, w, c, lens, w)
    with pytest.raises(TypeError):
        attn.evict(w, c, c, lens, 4)


@pytest.mark.gpu
def test_helpers_check_shapes_and_types():
    bf = dict(dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    q, k = torch.zeros(2, 4, 64, **bf), torch.zeros(2, 2, 64, **bf)
    c, lens, t = torch.zeros(3, 16, 2, 64, **bf), torch.ones(2, **i32), torch.zeros(2, 1, **i32)
    cu, f = torch.tensor([0, 1, 2], **i32), torch.zeros(32, dtype=torch.float64, device="cuda")
    w, lse = torch.zeros(2, 2, 16, device="cuda"), torch.zeros(2, 4, device="cuda")

    def no(error, fn, *args, **kw):
        with pytest.raises(error):
            fn(*args, **kw)

    r = attn.rope_append
    no(TypeError, r, q, k, k, c, c, lens, f.float(), page_table=t)
    no(TypeError, r, q.float(), k, k, c, c, lens, f, page_table=t)
    no(TypeError, r, q, k, k, c, c, lens.long(), f, page_table=t)
    no(TypeError, r, q, k, k, c, c, lens, f, page_table=t.cpu())
    no(ValueError, r, q, k, k[:, :1], c, c, lens, f, page_table=t)
    no(ValueError, r, q, k, k, c, c[:2], lens, f, page_table=t)
    no(ValueError, r, q, k, k, c, c, lens, f)                       # dense: 3 rows for 2 sequences
    no(ValueError, r, q, k, k, c, c, lens, f, page_table=t[:1])
    no(ValueError, r, q.transpose(0, 1).contiguous().transpose(0, 1), k, k, c, c, lens, f, page_table=t)
    no(ValueError, r, q, k, k, c, c, lens, f, page_table=t, out=torch.zeros(2, 4, 32, **bf))
    no(ValueError, r, None, k, k, c, c, lens, f, page_table=t, out=q)
    no(ValueError, r, q, k, k, c, c, lens, f, page_table=t, positions=lens[:1])
    no(ValueError, r, q, k, k, c, c, lens[:1], f, page_table=t[:1])  # two tokens, one sequence
    p = attn.prefill_paged
    no(TypeError, p, q, c, c, None, cu, lens, 1)
    no(ValueError, p, q, c, c, t, cu[:2], lens, 1)
    no(ValueError, p, q[..., :32].contiguous(), c, c, t, cu, lens, 1)
    no(TypeError, p, q, c, c, t, cu, lens, 1, out_dtype=torch.float16)
    no(ValueError, p, q, c, c, t, cu, lens, 1, out=(q, lse[:1]))
    no(ValueError, p, q, c, c, t, cu, lens, 1, n_splits=2, parts=(q.float(), lse))
    no(attn.AttnError, p, q, c, c, t, cu, lens, 1, window=4, causal=False)
    d = attn.decode_paged
    no(ValueError, d, q, c, c, t, lens[:1])
    no(TypeError, d, q, c, c, t, lens, 2, counters=lens.long())
    no(TypeError, d, q, c, c, t, lens, 2, counters=lens)  # too few
    no(attn.AttnError, d, q, c, c, t, lens, scale=0.0)
    kw = attn.key_weights
    no(ValueError, kw, q, lse, c, lens, w[:, :, :15].contiguous(), page_table=t)
    no(ValueError, kw, q, lse.T.contiguous(), c, lens, w, page_table=t)
    no(ValueError, kw, q, lse, c, lens, w, page_table=t, cu_seqlens_q=cu)  # lse [Hq, total]
    no(TypeError, kw, q, lse, c, lens, w.bfloat16(), page_table=t)
    e = attn.evict
    no(attn.AttnError, e, w, c, c, lens, 0, page_table=t)
    no(attn.AttnError, e, w, c, c, lens, 4, n_recent=4, n_sink=1, page_table=t)
    no(TypeError, e, w, c, None, lens, 4, page_table=t)
    no(ValueError, e, w, c, c, lens, 4, page_table=t, dst=(c[..., :1, :].contiguous(), c[..., :1, :].contiguous(), t, None))
    no(ValueError, e, w, c, c, lens, 4, page_table=t, out=(lens, lens))
    no(ValueError, e, w.transpose(0, 1), c, c, lens, 4, page_table=t)
    if torch.cuda.device_count() == 1:
        torch.cuda.synchronize()
    attn.sync_check()
