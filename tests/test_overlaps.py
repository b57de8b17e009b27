"""Outputs that overlap inputs or one another in part are refused, and only those: the gradients and
the rotation write while other work of the call still reads."""
import random

import pytest
import torch

import attention_forward_tcgen05_gb300 as attn
from attention_forward_tcgen05_gb300 import build as attn_build
from tests.test_paged_boundary import Call

INVALID, UNSUPPORTED = attn.ATTN_ERR_INVALID_ARG, attn.ATTN_ERR_UNSUPPORTED
A = 1 << 24  # between dummies (never dereferenced: refused first)


@pytest.fixture(scope="module", autouse=True)
def lib():
    attn_build.build()
    return attn.load()


# 2 x 70 rows of 4 heads of 64, 2 x 90 keys of 2 heads
Q, K, STAT = 2 * 70 * 4 * 64 * 2, 2 * 90 * 2 * 64 * 2, 2 * 4 * 70 * 4
GRAD = Call(attn.attn_prefill_backward, do=A, q=2 * A, k=3 * A, v=4 * A, o=5 * A, lse=6 * A, dlse=10 * A, dq=7 * A, dk=8 * A,
            dv=9 * A, B=2, Hq=4, Hkv=2, Sq=70, Skv=90, d=64, causal=1, window=0, sink=0, scale=0.5, o_dtype=1, work=1 << 30,
            work_bytes=1 << 40, stream=None)
VARLEN = Call(attn.attn_prefill_varlen_backward, do=A, q=2 * A, k=3 * A, v=4 * A, o=5 * A, lse=6 * A, dlse=10 * A, dq=7 * A,
              dk=8 * A, dv=9 * A, cu=11 * A, lens=12 * A, B=2, Hq=4, Hkv=2, total=140, max_sq=70, max_kv=90, d=64, causal=1,
              window=0, sink=0, scale=0.5, o_dtype=1, fill=1, work=1 << 30, work_bytes=1 << 40, stream=None)
AT = dict(do=A, q=2 * A, k=3 * A, v=4 * A, o=5 * A, lse=6 * A, dlse=10 * A, dq=7 * A, dk=8 * A, dv=9 * A)
SIZE = dict(do=Q, q=Q, k=K, v=K, o=Q, lse=STAT, dlse=STAT, dq=Q, dk=K, dv=K)


@pytest.mark.parametrize("call", [GRAD, VARLEN], ids=["fixed", "varlen"])
def test_gradients_over_parts_of_inputs(call):
    for out in ("dq", "dk", "dv"):
        for x, size in SIZE.items():
            if x == out:
                continue
            at = AT[x]
            for p in (at, at + 512, at + size - 16, at - 16, at - SIZE[out] + 16):
                assert call(**{out: p}) == INVALID, (out, x, p - at)
    n = attn.attn_prefill_backward_workspace(2, 4, 2, 140, 70, 90, 64)
    for x, size in SIZE.items():
        for p in ((1 << 30) + 256, (1 << 30) + n - 16, (1 << 30) - size + 16):
            assert call(**{x: p}) == INVALID, (x, p)
    # fp32 o is twice as long
    assert call(o_dtype=0, dq=5 * A + Q + 16) == INVALID


ROTATE = Call(attn.attn_rope_rotate, q=A, k=2 * A, qs=256, ks=128, positions=5 * A, axes=6 * A, n_axes=3, inv_freq=7 * A,
              qo=3 * A, ko=4 * A, qos=256, kos=128, Hq=4, Hk=2, total=7, d=64, rot=64, inter=0, inverse=0, amp=1.0, stream=None)


def test_rotation_over_parts_of_inputs():
    row = 256 * 2
    for p in (A + row, A - row, A + 16, A + 6 * row):          # q_out over q, a row later, ...
        assert ROTATE(qo=p) == INVALID, p - A
    for p in (2 * A + 16, 2 * A + 6 * 256, 2 * A - 6 * row):   # over k
        assert ROTATE(qo=p) == INVALID, p - 2 * A
    for p in (3 * A + 16, 3 * A + 6 * row + 256):              # k_out over q_out
        assert ROTATE(ko=p) == INVALID, p - 3 * A
    # one fused buffer of 6 heads a row: a head too far
    assert ROTATE(qo=8 * A, qos=384, ko=8 * A + 3 * 128, kos=384) == INVALID
    assert ROTATE(qo=8 * A, qos=384, ko=8 * A + 5 * 128, kos=384) == INVALID  # k's second head in the next row's first
    assert ROTATE(qo=A, qs=256, qos=264) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="dummies: where there is a GPU the call would be made")
def test_the_calls_are_good_otherwise():
    for call in (GRAD, VARLEN, ROTATE):
        assert call() == attn.ATTN_ERR_CUDA  # (past the checks, and no GPU)
    assert ROTATE(qo=A) == ROTATE(ko=2 * A) == ROTATE(qo=A, ko=2 * A) == attn.ATTN_ERR_CUDA  # in place
    # a row of 6 heads each, in and out
    fused = dict(q=A, qs=384, k=A + 4 * 128, ks=384, qos=384, kos=384)
    assert ROTATE(**fused, qo=8 * A, ko=8 * A + 4 * 128) == ROTATE(**fused, qo=A, ko=A + 4 * 128) == attn.ATTN_ERR_CUDA
    assert GRAD(dq=2 * A + Q, dk=2 * A + 2 * Q, dv=2 * A + 2 * Q + K) == attn.ATTN_ERR_CUDA  # side by side


@pytest.mark.gpu
def test_views_of_one_buffer():
    """Random strided views of a buffer against the elements that they are."""
    rng = random.Random(5)
    buf = torch.zeros(1 << 16, dtype=torch.bfloat16, device="cuda")
    freq = torch.zeros(8, dtype=torch.float64, device="cuda")
    seen = {True: 0, False: 0}
    for _ in range(3000):
        total, d = rng.randint(1, 9), 16
        pos = torch.zeros(total, dtype=torch.int32, device="cuda")

        def view(H):
            s = H * d + 8 * rng.choice([0, 0, 2, 4, 4, 6, 11])
            at = 8 * rng.randint(0, rng.choice([20, 120, 3000]))
            return buf.as_strided((total, H, d), (s, d, 1), at), {at + t * s + e for t in range(total) for e in range(H * d)}, (at, s)

        Hq, Hk = rng.randint(1, 3), rng.randint(0, 2)
        q, qe, qa = view(Hq)
        qo, qoe, qoa = (q, qe, qa) if rng.random() < 0.3 else view(Hq)
        k = ko = None
        bad = bool(qoe & qe) and qoa != qa and not (total == 1 and qoa[0] == qa[0])
        if Hk:
            k, ke, ka = view(Hk)
            ko, koe, koa = (k, ke, ka) if rng.random() < 0.3 else view(Hk)
            bad |= bool(koe & ke) and koa != ka and not (total == 1 and koa[0] == ka[0])
            bad |= bool(qoe & ke) or bool(koe & qe) or bool(koe & qoe)
        seen[bad] += 1
        if bad:
            with pytest.raises(attn.AttnError) as e:
                attn.rope_rotate(q, k, freq, pos, out=(qo, ko))
            assert e.value.status == INVALID
        else:
            attn.rope_rotate(q, k, freq, pos, out=(qo, ko))
    assert min(seen.values()) > 300
    x = torch.zeros(2, 60, 4, 64, dtype=torch.bfloat16, device="cuda").flatten()
    one = lambda at: x[at:at + 40 * 4 * 64].view(1, 40, 4, 64)
    q, k, v, do, o = (torch.zeros(1, 40, 4, 64, dtype=torch.bfloat16, device="cuda") for _ in range(5))
    lse = torch.zeros(1, 4, 40, device="cuda")
    free = lambda: torch.zeros_like(q)
    with pytest.raises(attn.AttnError):
        attn.prefill_backward(do, q, k, v, o, lse, out=(one(0), one(256), free()))
    with pytest.raises(attn.AttnError):
        attn.prefill_backward(do, one(0), k, v, o, lse, out=(free(), free(), one(39 * 256)))
    attn.prefill_backward(do, one(0), k, v, o, lse, out=(free(), free(), one(40 * 256)))
    attn.sync_check()
