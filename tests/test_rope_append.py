"""Rotary positions and the cache append against fp64.

Tolerance: the kernel rounds an fp32 result once to bf16, so an output is off by half a bf16
step of its value plus the fp32 error: the angle's (2^-31 turn from the fixed point and
2^-25 of a half turn from its rounding to fp32, together below 2^-23 rad), two products and
a sum, each 2^-24, sincospi's 2 units in the last place and the amplitude's rounding, all
relative to amp * (|x1| + |x2|): below 2^-20 of that."""
import math

import numpy as np
import pytest
import torch

import attention_forward_tcgen05_gb300 as attn
from tests.paged_cases import make_pages
from tests.tolerances import half_ulp_bf16


def rotate(x, pos, freq, amp, inter):
    """fp64 rotation of x [T,H,d], and |x1| + |x2| of each output."""
    x = np.asarray(x, np.float64).copy()
    mag = np.zeros_like(x)
    rot = 2 * len(freq)
    a = pos[:, None] * np.asarray(freq, np.float64)[None]
    c, s = np.cos(a)[:, None] * amp, np.sin(a)[:, None] * amp
    i1 = np.arange(0, rot, 2) if inter else np.arange(rot // 2)
    i2 = i1 + (1 if inter else rot // 2)
    x1, x2 = x[..., i1].copy(), x[..., i2].copy()
    x[..., i1], x[..., i2] = x1 * c - x2 * s, x1 * s + x2 * c
    m = (abs(x1) + abs(x2)) * abs(amp)
    mag[..., i1] = mag[..., i2] = m
    return x, mag


def check(got, ref, mag):
    got = got.float().cpu().numpy().astype(np.float64)
    delta = mag * 2.0 ** -20
    assert (abs(got - ref) <= half_ulp_bf16(abs(ref) + delta) + delta).all()


def test_frequencies():
    f, amp = attn.rope_frequencies(64, device="cpu")
    assert f.dtype == torch.float64 and amp == 1.0
    np.testing.assert_allclose(f.numpy(), [10000.0 ** (-2 * i / 64) for i in range(32)], rtol=1e-14)
    g, _ = attn.rope_frequencies(64, factor=4, method="linear", device="cpu")
    np.testing.assert_allclose(g.numpy(), f.numpy() / 4, rtol=1e-14)
    g, _ = attn.rope_frequencies(64, factor=4, method="ntk", device="cpu")
    assert g[0] == 1.0
    np.testing.assert_allclose(g[-1].item(), f[-1].item() / 4, rtol=1e-12)  # the slowest pair: stretched in full
    g, amp = attn.rope_frequencies(64, factor=4, method="yarn", original_length=2048, device="cpu")
    assert amp == pytest.approx(0.1 * math.log(4) + 1)
    turns = 2048 * f / (2 * math.pi)
    assert torch.equal(g[turns >= 32], f[turns >= 32])
    np.testing.assert_allclose(g[turns <= 1].numpy(), f[turns <= 1].numpy() / 4, rtol=1e-14)
    assert ((g <= f) & (g >= f / 4 * (1 - 1e-12))).all()
    for kw in (dict(rot_dim=63), dict(rot_dim=0), dict(rot_dim=64, method="other"), dict(rot_dim=64, factor=0.0),
               dict(rot_dim=64, method="yarn", low_turns=8, high_turns=8)):
        with pytest.raises(ValueError):
            attn.rope_frequencies(device="cpu", **kw)


SEQS = [(1, 1), (7, 40), (0, 5), (16, 16), (33, 100), (1, 65)]  # (new tokens, keys with them)


def _case(Hq, Hkv, d, page, seed, seqs=SEQS):
    g = torch.Generator().manual_seed(seed)
    T = sum(n for n, _ in seqs)
    x = torch.randn(T, Hq + 2 * Hkv, d, generator=g).bfloat16()
    lens = torch.tensor([L for _, L in seqs], dtype=torch.int32)
    cu = torch.zeros(len(seqs) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor([n for n, _ in seqs]), 0)
    kc = torch.randn(len(seqs), int(lens.max()), Hkv, d, generator=g).bfloat16()
    kp, vp, table = make_pages(kc, -kc, lens, page, seed)
    idx = [(b, L - n + i) for b, (n, L) in enumerate(seqs) for i in range(n)]
    return x, lens, cu, kp, vp, table, idx


def _check_cache(kp, vp, kp0, vp0, table, page, idx, ref_k, mag, v):
    """The appended rows, and every other row as it was."""
    kp, vp = kp.cpu(), vp.cpu()
    rows = [(int(table[b, j // page]), j % page) for b, j in idx]
    for t, (g, s) in enumerate(rows):
        check(kp[g, s], ref_k[t], mag[t])
        assert torch.equal(vp[g, s], v[t])
        kp[g, s], vp[g, s] = kp0[g, s], vp0[g, s]
    assert torch.equal(kp.view(torch.int16), kp0.view(torch.int16))
    assert torch.equal(vp.view(torch.int16), vp0.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (256, 256), (256, 96)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("Hq,Hkv,page", [(4, 2, 16), (7, 1, 5), (3, 3, 1)])
def test_rotate_and_append(d, rot, inter, Hq, Hkv, page):
    x, lens, cu, kp, vp, table, idx = _case(Hq, Hkv, d, page, 500 + d + rot)
    freq, amp = attn.rope_frequencies(rot, factor=2.0, method="yarn", device="cpu")
    # strided views of one projection's rows, and contiguous tensors; far and negative positions
    T = x.shape[0]
    rng = np.random.default_rng(1)
    for strided in (True, False):
        for pos in (None, rng.integers(-5, 2 ** 31 - 1, T).astype(np.int32)):
            xg = x.cuda()
            q, k, v = xg[:, :Hq], xg[:, Hq:Hq + Hkv], xg[:, Hq + Hkv:]
            if not strided:
                q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
            kg, vg = kp.cuda(), vp.cuda()
            pt = None if pos is None else torch.from_numpy(pos).cuda()
            out = attn.rope_append(q, k, v, kg, vg, lens.cuda(), freq.cuda(), page_table=table.cuda(),
                                   cu_seqlens_q=cu.cuda(), positions=pt, interleaved=inter, amp=amp)
            attn.sync_check()
            p = np.array([j for _, j in idx]) if pos is None else pos.astype(np.int64)
            ref, mag = rotate(x.float().numpy(), p.astype(np.float64), freq.numpy(), amp, inter)
            check(out, ref[:, :Hq], mag[:, :Hq])
            _check_cache(kg, vg, kp, vp, table, page, idx, ref[:, Hq:Hq + Hkv], mag[:, Hq:Hq + Hkv], x[:, Hq + Hkv:])


@pytest.mark.gpu
def test_one_token_each_dense_cache_and_in_place():
    """Without cu_seqlens_q, on the dense cache, q rotated in place."""
    B, Hq, Hkv, d, cap = 9, 8, 2, 128, 50
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(B, h, d, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
    lens = torch.tensor([1, 50, 7, 8, 9, 20, 33, 2, 49], dtype=torch.int32)
    freq, _ = attn.rope_frequencies(d, device="cpu")
    kc = torch.zeros(B, cap, Hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    qg = q.cuda()
    out = attn.rope_append(qg, k.cuda(), v.cuda(), kc, vc, lens.cuda(), freq.cuda(), out=qg)
    attn.sync_check()
    assert out is qg
    pos = (lens - 1).numpy().astype(np.float64)
    rq, mq = rotate(q.float().numpy(), pos, freq.numpy(), 1.0, False)
    rk, mk = rotate(k.float().numpy(), pos, freq.numpy(), 1.0, False)
    check(qg, rq, mq)
    b = torch.arange(B)
    check(kc[b, (lens - 1).long()], rk, mk)
    assert torch.equal(vc.cpu()[b, (lens - 1).long()], v)
    kc[b, (lens - 1).long()] = 0
    assert not kc.any()


@pytest.mark.gpu
def test_append_only_padding_and_bad_slots():
    """No rotation, no queries; tokens behind the last sequence are not stored; a token
    without a place (before the first key, past the table) is reported, the others stand."""
    x, lens, cu, kp, vp, table, idx = _case(2, 2, 64, 16, 9)
    T = x.shape[0]
    pad = torch.cat([x, x[:5] * 0 + 3])
    kg, vg = kp.cuda(), vp.cuda()
    k, v = pad[:, 2:4].contiguous(), pad[:, 4:].contiguous()
    assert attn.rope_append(None, k.cuda(), v.cuda(), kg, vg, lens.cuda(), None, page_table=table.cuda(),
                            cu_seqlens_q=cu.cuda()) is None
    attn.sync_check()
    ref = k.float().numpy().astype(np.float64)
    _check_cache(kg, vg, kp, vp, table, 16, idx, ref[:T], 0 * ref[:T], v[:T])
    # queries behind the last sequence keep the bytes of `out`
    freq, _ = attn.rope_frequencies(64, device="cuda")
    q = pad[:, :2].contiguous().cuda()
    out = torch.full_like(q, 5.0)
    attn.rope_append(q, k.cuda(), v.cuda(), kg, vg, lens.cuda(), freq, page_table=table.cuda(),
                     cu_seqlens_q=cu.cuda(), out=out)
    attn.sync_check()
    assert (out[T:] == 5).all()
    for bad in (0, 16 * table.shape[1] + 1):  # sequence 5's single token: key -1, key past the table
        l2 = lens.clone()
        l2[5] = bad
        kg, vg = kp.cuda(), vp.cuda()
        attn.rope_append(None, k.cuda(), v.cuda(), kg, vg, l2.cuda(), None, page_table=table.cuda(),
                         cu_seqlens_q=cu.cuda())
        with pytest.raises(attn.AttnError) as e:
            attn.sync_check()
        assert e.value.status == attn.ATTN_ERR_DEVICE_INPUT
        _check_cache(kg, vg, kp, vp, table, 16, idx[:-1], ref[:T - 1], 0 * ref[:T - 1], v[:T - 1])
