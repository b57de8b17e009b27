"""The windowed decode, the rotations with several axes and the prefill's gradients reject bad
arguments on the host: the C entry points before any CUDA call (no GPU needed), the torch
helpers before they call them."""
import ctypes
import math

import pytest
import torch

import attention_forward_tcgen05_gb300 as attn
from attention_forward_tcgen05_gb300 import build as attn_build
from tests.test_paged_boundary import Call

N = None
P = 256  # an aligned non-null dummy (never dereferenced: validation fails first)
M = 258  # misaligned
INVALID, UNSUPPORTED, OK = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED, attn.ATTN_OK
BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def lib():
    attn_build.build()
    return attn.load()


DECODE = Call(attn.attn_decode_window, q=P, kc=P, vc=P, table=P, lens=P, B=2, Hq=4, Hkv=2, d=64, max_pages=4, page=16,
              pages=9, window=8, sink=2, scale=0.5, n_splits=2, min_rows=1, po=P, pl=P, o=P, lse=P, o_dtype=0,
              counters=P, stream=N)
APPEND = Call(attn.attn_rope_append_axes, q=P, k=P, v=P, qs=256, ks=128, vs=128, positions=P, axes=P, n_axes=3,
              inv_freq=P, q_out=P, kc=P, vc=P, table=P, cu=P, lens=P, B=2, Hq=4, Hkv=2, total=7, d=64, rot=64, inter=0,
              amp=1.0, max_pages=4, page=16, pages=9, stream=N)
ROTATE = Call(attn.attn_rope_rotate, q=P, k=5 * P, qs=256, ks=128, positions=P, axes=P, n_axes=3, inv_freq=P, qo=2 * P,
              ko=3 * P, qos=256, kos=128, Hq=4, Hk=2, total=7, d=64, rot=64, inter=0, inverse=0, amp=1.0, stream=N)
GRAD = Call(attn.attn_prefill_backward, do=P, q=2 * P, k=3 * P, v=4 * P, o=5 * P, lse=6 * P, dlse=N, dq=7 * P,
            dk=8 * P, dv=9 * P, B=2, Hq=4, Hkv=2,
            Sq=70, Skv=90, d=64, causal=1, window=0, sink=0, scale=0.5, o_dtype=1, work=P, work_bytes=BIG, stream=N)
VARLEN = Call(attn.attn_prefill_varlen_backward, do=P, q=2 * P, k=3 * P, v=4 * P, o=5 * P, lse=6 * P, dlse=N, dq=7 * P,
              dk=8 * P, dv=9 * P, cu=P,
              lens=P, B=2, Hq=4, Hkv=2, total=70, max_sq=50, max_kv=90, d=64, causal=1, window=0, sink=0, scale=0.5,
              o_dtype=1, fill=1, work=P, work_bytes=BIG, stream=N)


def refused(call, status, **changes):
    for name, values in changes.items():
        for v in values:
            assert call(**{name: v}) == status, (name, v)


def test_decode_window():
    refused(DECODE, INVALID, window=(0, -1), sink=(-1,), Hq=(3, 0, -4), Hkv=(0,), B=(-1,), max_pages=(0,), page=(0,),
            scale=(0.0, -1.0, math.inf, math.nan), n_splits=(0, 1025), min_rows=(-1,), q=(N, M), kc=(N, M), vc=(N, M),
            lens=(N, M), o=(N, M), lse=(N, M), po=(N, M), pl=(N, M), counters=(N, M), table=(M,))
    refused(DECODE, UNSUPPORTED, d=(32, 96, 512), o_dtype=(2, -1))
    assert DECODE(Hq=258, Hkv=2) == INVALID            # groups of more than 128 heads
    assert DECODE(page=1 << 29) == INVALID             # 2^30 keys a table, 2^31 slots a pool
    assert DECODE(table=N) == INVALID                  # a dense cache has one page a sequence
    assert DECODE(B=0) == OK


def test_decode_window_splits():
    rows = ctypes.c_int(0)
    f = lambda *a: attn.attn_decode_window_splits(*a, ctypes.addressof(rows))
    for bad in ((-1, 4, 2, 99, 8, 0, 64), (2, 3, 2, 99, 8, 0, 64), (2, 4, 2, -1, 8, 0, 64), (2, 4, 2, 99, 0, 0, 64),
                (2, 4, 2, 99, 8, -1, 64), (2, 4, 2, 99, 8, 0, 32)):
        assert f(*bad) == INVALID
    assert attn.attn_decode_window_splits(2, 4, 2, 99, 8, 0, 64, N) == INVALID
    # by the keys that are read, not by the cache's: the same as a cache of the window's size
    top = 2 ** 31 - 1
    for args in ((1, 28, 4, 128), (64, 32, 8, 128), (3, 40, 2, 64), (1, 128, 1, 256)):
        B, Hq, Hkv, d = args
        n = f(B, Hq, Hkv, 1 << 20, 1024, 4, d)
        assert n >= 1 and rows.value >= 1 and n == f(B, Hq, Hkv, 1028, 1024, 4, d)
        assert f(B, Hq, Hkv, top, top, top, d) >= 1 and f(B, Hq, Hkv, 0, 1, 0, d) == 1


def test_rope_append_axes():
    refused(APPEND, INVALID, n_axes=(0, -1, 9), axes=(N, M), positions=(N, M), Hq=(3, 0), Hkv=(0,), B=(-1,), total=(-1,),
            amp=(math.inf, math.nan), inv_freq=(N, 260), k=(N, M), v=(N, M), kc=(N, M), vc=(N, M), lens=(N, M), q=(N, M),
            q_out=(N, M), qs=(248, 257), ks=(120, 129), vs=(0,), cu=(M,), page=(0,), max_pages=(0,))
    refused(APPEND, UNSUPPORTED, rot=(0, 8, 80, -16), d=(32, 96, 512))
    assert APPEND(cu=N) == INVALID  # seven tokens of two sequences
    assert APPEND(total=0, axes=N, positions=N) == OK


def test_rope_rotate():
    refused(ROTATE, INVALID, n_axes=(0, 9), axes=(N, M), positions=(N, M), Hq=(-1,), Hk=(-1,), total=(-1,),
            amp=(math.inf, math.nan), inv_freq=(N, 260), q=(N, M), k=(N, M), qo=(N, M), ko=(N, M), qs=(248, 257),
            ks=(120,), qos=(255, 0), kos=(127,))
    refused(ROTATE, UNSUPPORTED, d=(0, 8, 40, 272), rot=(0, 8, 24, 80, -16))
    assert ROTATE(Hq=0, Hk=0) == INVALID
    assert ROTATE(qo=P, qs=264) == INVALID  # in place at another stride
    assert ROTATE(Hq=1 << 30, qs=1 << 36, qos=1 << 36) == INVALID
    assert ROTATE(Hq=(1 << 25) - 1, qs=1 << 32, qos=1 << 32) == INVALID  # two heads of k beside them
    # one output for both, or over the other's input
    assert ROTATE(qo=2 * P, ko=2 * P) == INVALID
    assert ROTATE(k=4 * P, qo=4 * P, ko=6 * P) == INVALID
    assert ROTATE(q=4 * P, qo=6 * P, ko=4 * P) == INVALID
    assert ROTATE(total=0, q=N, k=N, positions=N, axes=N, n_axes=1) == OK


@pytest.mark.parametrize("call", [GRAD, VARLEN], ids=["fixed", "varlen"])
def test_gradients(call):
    refused(call, INVALID, B=(-1,), Hq=(3, 0), Hkv=(0, -2), window=(-1,), sink=(-1,), scale=(0.0, -1.0, math.inf, math.nan),
            do=(N, M), q=(N, M), k=(N, M), v=(N, M), o=(N, M), lse=(N, M), dlse=(M,), dq=(N, M), dk=(N, M), dv=(N, M),
            work=(N, M), work_bytes=(0, 1000))
    refused(call, UNSUPPORTED, d=(32, 256, 512), o_dtype=(2, -1), scale=(1e-31, 1e31))
    assert call(window=4, causal=0) == INVALID
    assert call(B=0) == OK


@pytest.mark.parametrize("call", [GRAD, VARLEN], ids=["fixed", "varlen"])
def test_gradients_over_inputs(call):
    for out in ("dq", "dk", "dv"):
        for i, x in enumerate(("do", "q", "k", "v", "o", "lse", "dq", "dk", "dv")):
            if x not in (out, "lse"):
                assert call(**{out: (i + 1) * P}) == INVALID, (out, x)


def test_gradients_sizes():
    refused(GRAD, INVALID, Sq=(-1,), Skv=(-1,))
    refused(VARLEN, INVALID, total=(-1,), max_sq=(-1,), max_kv=(-1,), cu=(N, M), lens=(N, M))
    # rows of all heads, cache rows and tiles of all heads below 2^31
    assert GRAD(B=1, Hq=1 << 10, Hkv=1 << 10, Sq=1 << 21) == INVALID
    assert GRAD(B=1, Hq=1 << 10, Hkv=1 << 10, Skv=1 << 21) == INVALID
    assert GRAD(B=1, Hq=64, Hkv=8, Sq=1 << 24, Skv=1 << 24) == INVALID
    assert GRAD(Sq=0, Skv=0) == OK
    assert VARLEN(total=0, max_sq=0, max_kv=0) == OK


def test_workspace():
    w = attn.attn_prefill_backward_workspace
    for bad in ((-1, 4, 2, 70, 70, 90, 64), (1, 3, 2, 70, 70, 90, 64), (1, 4, 2, -1, 70, 90, 64), (1, 4, 2, 70, 70, 90, 256),
                (1, 1 << 10, 1 << 10, 1 << 21, 1 << 21, 5, 64)):
        assert w(*bad) == 0
    # eight sequences of 128k rows, one of a million; items of all heads past 2 * 10^9
    assert w(8, 64, 8, 8 << 17, 1 << 17, 1 << 17, 128) > 0
    assert w(1, 8, 1, 1 << 20, 1 << 20, 1 << 20, 128) > 0
    assert w(1, 32, 8, 1 << 20, 1 << 20, 1 << 20, 128) == 0
    n = w(1, 4, 2, 70, 70, 90, 64)
    assert n > 0 and n % 256 == 0
    assert GRAD(B=1, Sq=70, Skv=90, work_bytes=n - 1) == INVALID
    # grows with the rows, not with their square
    assert w(1, 28, 4, 16384, 16384, 16384, 128) < 8 * w(1, 28, 4, 4096, 4096, 4096, 128)


def test_helpers_refuse_host_tensors():
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    f = torch.zeros(32, dtype=torch.float64)
    for call in (lambda: attn.decode_window(b(2, 4, 64), b(2, 9, 2, 64), b(2, 9, 2, 64), i(2), 4),
                 lambda: attn.rope_rotate(b(3, 4, 64), b(3, 2, 64), f, i(3)),
                 lambda: attn.rope_rotate(None, None, f, i(3)),
                 lambda: attn.rope_append(b(2, 4, 64), b(2, 2, 64), b(2, 2, 64), b(2, 9, 2, 64), b(2, 9, 2, 64), i(2), f,
                                          positions=i(3, 2), axes=i(32)),
                 lambda: attn.prefill_backward(*(b(1, 5, 4, 64) for _ in range(5)), torch.zeros(1, 4, 5)),
                 lambda: attn.prefill_varlen_backward(b(5, 4, 64), b(5, 4, 64), b(1, 9, 4, 64), b(1, 9, 4, 64),
                                                      b(5, 4, 64), torch.zeros(4, 5), i(2), i(1), 5)):
        with pytest.raises(TypeError):
            call()


@pytest.mark.gpu
def test_helpers_check_shapes_and_types():
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    fl = lambda *s: torch.zeros(*s, device="cuda")
    f = torch.zeros(32, dtype=torch.float64, device="cuda")
    dec = dict(q=b(2, 4, 64), kcache=b(2, 9, 2, 64), vcache=b(2, 9, 2, 64), kv_lens=i(2), window=4)
    for change in (dict(q=b(2, 4, 128)), dict(kv_lens=i(3)), dict(vcache=b(2, 8, 2, 64)), dict(vcache=None),
                   dict(kcache=b(3, 9, 2, 64), vcache=b(3, 9, 2, 64)), dict(page_table=i(3, 4)), dict(q=fl(2, 4, 64)),
                   dict(out=(b(2, 4, 64), fl(2, 5))), dict(n_splits=2, counters=i(7)), dict(out_dtype=torch.float16),
                   dict(q=b(2, 64, 4).transpose(1, 2))):
        with pytest.raises((TypeError, ValueError)):
            attn.decode_window(**{**dec, **change})
    for change in (dict(window=0), dict(n_sink=-1), dict(scale=0.0), dict(q=b(2, 3, 64))):
        with pytest.raises(attn.AttnError):
            attn.decode_window(**{**dec, **change})
    rot = dict(q=b(3, 4, 64), k=b(3, 2, 64), inv_freq=f, positions=i(2, 3), axes=i(32))
    for change in (dict(q=b(3, 4, 128)), dict(k=b(4, 2, 64)), dict(positions=i(3)), dict(positions=i(2, 4)),
                   dict(axes=i(31)), dict(axes=i(32).long()), dict(inv_freq=f.float()), dict(q=b(3, 64, 4).transpose(1, 2)),
                   dict(out=(b(3, 4, 64), b(3, 3, 64))), dict(q=None, out=(b(3, 4, 64), None)), dict(q=b(3, 4))):
        with pytest.raises((TypeError, ValueError)):
            attn.rope_rotate(**{**rot, **change})
    with pytest.raises(attn.AttnError):
        attn.rope_rotate(**{**rot, "positions": i(9, 3)})
    app = dict(q=b(2, 4, 64), k=b(2, 2, 64), v=b(2, 2, 64), kcache=b(2, 9, 2, 64), vcache=b(2, 9, 2, 64), kv_lens=i(2),
               inv_freq=f, positions=i(3, 2), axes=i(32))
    for change in (dict(positions=None), dict(inv_freq=None), dict(positions=i(2)), dict(positions=i(3, 3)), dict(axes=i(16))):
        with pytest.raises((TypeError, ValueError)):
            attn.rope_append(**{**app, **change})
    grad = dict(do=b(1, 5, 4, 64), q=b(1, 5, 4, 64), k=b(1, 6, 2, 64), v=b(1, 6, 2, 64), o=b(1, 5, 4, 64), lse=fl(1, 4, 5))
    for change in (dict(do=b(1, 5, 4, 32)), dict(k=b(2, 6, 2, 64)), dict(v=b(1, 5, 2, 64)), dict(lse=fl(1, 5, 4)),
                   dict(dlse=fl(1, 4, 6)), dict(o=b(1, 5, 4, 64).half()), dict(o=None), dict(out=(b(1, 5, 4, 64),)),
                   dict(out=(b(1, 5, 4, 64), b(1, 6, 2, 64), fl(1, 6, 2, 64))), dict(do=b(1, 1, 4, 64).expand(1, 5, 4, 64))):
        with pytest.raises((TypeError, ValueError)):
            attn.prefill_backward(**{**grad, **change})
    for change in (dict(window=-1), dict(window=3, causal=False), dict(scale=math.nan)):
        with pytest.raises(attn.AttnError):
            attn.prefill_backward(**{**grad, **change})
    var = dict(do=b(5, 4, 64), q=b(5, 4, 64), kcache=b(2, 6, 2, 64), vcache=b(2, 6, 2, 64), o=b(5, 4, 64), lse=fl(4, 5),
               cu_seqlens_q=i(3), kv_lens=i(2), max_sq=5)
    for change in (dict(cu_seqlens_q=i(2)), dict(kv_lens=i(3)), dict(lse=fl(5, 4)), dict(kcache=b(2, 6, 2, 128))):
        with pytest.raises((TypeError, ValueError)):
            attn.prefill_varlen_backward(**{**var, **change})
    attn.sync_check()


@pytest.mark.gpu
def test_a_sequence_above_max_sq_is_reported():
    b = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 3, 9], dtype=torch.int32, device="cuda")
    lens = torch.tensor([3, 6], dtype=torch.int32, device="cuda")
    args = (b(9, 2, 64), b(9, 2, 64), b(2, 6, 1, 64), b(2, 6, 1, 64), b(9, 2, 64), torch.zeros(2, 9, device="cuda"), cu, lens)
    attn.prefill_varlen_backward(*args, 5)
    with pytest.raises(attn.AttnError) as e:
        attn.sync_check()
    assert e.value.status == attn.ATTN_ERR_DEVICE_INPUT
    attn.prefill_varlen_backward(*args, 6)
    attn.sync_check()
