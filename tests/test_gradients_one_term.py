"""The gradients' ordinary form, one bf16 term of P and dS (sequences of more pairs than
test_gradient_forms.LIMIT), at the sizes and masks where tiles, windows and tails can go wrong.

Every sequence is checked against its form's bound, and one of one term also for not keeping the
bound of two (Batch.check), so that a case cannot move to the other form unseen."""
import math

import pytest
import torch

import attention_forward_tcgen05_gb300 as attn
from tests.test_gradient_forms import LIMIT, Batch, pairs
from tests.test_prefill_backward import F

EVEN = [  # as a fixed-length batch and as a packed one: rows, keys, sequences, heads, mask
    (1, 24700, 2, (2, 1), {}), (1, 24700, 1, (4, 2), dict(causal=False)),
    (127, 400, 1, (2, 2), {}), (128, 400, 2, (4, 2), {}), (129, 400, 1, (4, 2), {}), (129, 257, 1, (3, 3), dict(causal=False)),
    (257, 400, 1, (3, 3), dict(causal=False)), (400, 257, 2, (4, 4), dict(causal=False)),
    (300, 300, 2, (7, 1), {}), (300, 300, 1, (32, 1), {}),
    (500, 230, 1, (4, 2), {}),                             # rows that admit nothing, whole tiles of them
    (500, 230, 1, (4, 2), dict(window=70, sink=3)),
    (601, 601, 1, (4, 2), dict(window=1, sink=40)),        # the own key and the sinks
    (700, 700, 1, (2, 1), dict(window=100, sink=130)),     # sinks past a tile
    (700, 700, 2, (2, 1), dict(window=128)), (513, 513, 2, (6, 2), dict(window=129, sink=4)),
    (300, 300, 1, (4, 1), dict(window=5000, sink=7)),      # wider than the sequence
    (260, 640, 3, (8, 2), dict(window=200, sink=200)), (130, 1300, 1, (4, 2), dict(window=250, sink=2)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("i", range(len(EVEN)))
def test_even(i, d):
    n, L, B, (Hq, Hkv), mask = EVEN[i]
    assert pairs(n, L, **mask) > LIMIT
    x = Batch([n] * B, [L] * B, Hq, Hkv, d, **mask, dlse=i % 2 == 1, o_dtype=torch.float32 if i % 3 == 1 else torch.bfloat16)
    x.check(x.fixed())
    x.check(x.packed(L + 13, first=i % 4, spare=5))


UNEVEN = [  # packed, all of one term but sequences of no rows or no keys
    dict(lens_q=[100, 90, 200], lens_k=[300, 437, 1000], Hq=7, Hkv=1, d=128),
    dict(lens_q=[0, 229, 0, 300], lens_k=[40, 229, 0, 400], Hq=4, Hkv=4, d=64),
    dict(lens_q=[400, 1, 310], lens_k=[700, 25000, 310], Hq=4, Hkv=2, d=128, dlse=True),
    dict(lens_q=[457, 455], lens_k=[457, 290], Hq=4, Hkv=2, d=64, window=60, sink=3),
    dict(lens_q=[1, 400, 255], lens_k=[90, 700, 400], Hq=8, Hkv=2, d=64, window=128, sink=1, dlse=True),
    dict(lens_q=[400, 255], lens_k=[700, 400], Hq=8, Hkv=2, d=128, window=128, sink=1, dlse=True),
    dict(lens_q=[177, 240], lens_k=[300, 120], Hq=2, Hkv=1, d=128, causal=False),
    dict(lens_q=[177, 240], lens_k=[300, 120], Hq=2, Hkv=1, d=64, causal=False, dlse=True),
    dict(lens_q=[31] * 40, lens_k=[820] * 40, Hq=2, Hkv=2, d=64),   # many short sequences
    dict(lens_q=[31] * 40, lens_k=[820] * 40, Hq=2, Hkv=1, d=128),
    dict(lens_q=[31] * 40, lens_k=[820] * 40, Hq=2, Hkv=2, d=64, causal=False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("i", range(len(UNEVEN)))
def test_uneven(i, o_dtype):
    x = Batch(**UNEVEN[i], o_dtype=o_dtype)
    assert any(not s["few"] for s in x.seqs)
    x.check(x.packed(max(x.lens_k) + 50, first=(0, 3, 130)[i % 3], spare=(9, 0, 200)[i % 3], give_out=i % 2 == 0))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_own_key_only(d):
    """window = 1: P = 1, o = v of the own key, dP = D, so dS, dq and dk are 0 and dv is a sum of g over the
    group.  Off by: 2^-8 of dv and F of its terms; dP - D by 2 F of what they are sums of, in every
    term of dq and dk."""
    S, Hq, Hkv = LIMIT + 130, 4, 2
    G, scale = Hq // Hkv, 1 / math.sqrt(d)
    assert pairs(S, S, window=1) > LIMIT
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda H: torch.randn(1, S, H, d, generator=g, device="cuda").bfloat16()
    q, do, k, v = rnd(Hq), rnd(Hq), rnd(Hkv), rnd(Hkv)
    kr, vr = k.repeat_interleave(G, 2), v.repeat_interleave(G, 2)
    lse = ((q.double() * kr.double()).sum(-1) * scale).float().transpose(1, 2).contiguous()
    dq, dk, dv = attn.prefill_backward(do, q, k, v, vr.contiguous(), lse, window=1)
    attn.sync_check()
    fold = lambda t: t.unflatten(2, (Hkv, G)).sum(3)
    gd = do.double()
    want = fold(gd)
    assert ((dv.double() - want).abs() <= 2.0 ** -8 * want.abs() + F * fold(gd.abs()) + 1e-30).all()
    off = 4 * F * (gd.abs() * vr.double().abs()).sum(-1, keepdim=True) * scale
    assert (dq.double().abs() <= off * kr.double().abs() + 1e-30).all()
    assert (dk.double().abs() <= fold(off * q.double().abs()) + 1e-30).all()
