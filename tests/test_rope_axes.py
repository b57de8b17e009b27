"""Rotary positions with several axes: the append, the rotation without a cache and its inverse,
against fp64.  Tolerance as in test_rope_append.py: half a bf16 step of the value plus
2^-20 amp (|x1| + |x2|)."""
import math

import numpy as np
import pytest
import torch

import attention_forward_tcgen05_gb300 as attn
from tests.paged_cases import gather, make_pages
from tests.test_rope_append import check


def rotate(x, pos, freq, axes, amp, inter, sign=1.0):
    """fp64 rotation of x [T,H,d] by pos [A,T], and |x1| + |x2| of each output."""
    x = np.asarray(x, np.float64).copy()
    mag = np.zeros_like(x)
    rot = 2 * len(freq)
    a = sign * np.asarray(pos, np.float64)[np.asarray(axes)].T * np.asarray(freq, np.float64)[None]
    c, s = np.cos(a)[:, None] * amp, np.sin(a)[:, None] * amp
    i1 = np.arange(0, rot, 2) if inter else np.arange(rot // 2)
    i2 = i1 + (1 if inter else rot // 2)
    x1, x2 = x[..., i1].copy(), x[..., i2].copy()
    x[..., i1], x[..., i2] = x1 * c - x2 * s, x1 * s + x2 * c
    mag[..., i1] = mag[..., i2] = (abs(x1) + abs(x2)) * abs(amp)
    return x, mag


def test_axes_layouts():
    f, a = attn.rope_axes([2, 3, 1], base=100.0, device="cpu")
    assert f.dtype == torch.float64 and a.dtype == torch.int32
    assert a.tolist() == [0, 0, 1, 1, 1, 2]
    np.testing.assert_allclose(f.numpy(), [100.0 ** (-i / 6) for i in range(6)], rtol=1e-14)
    g, a = attn.rope_axes([2, 3, 1], base=100.0, layout="dealt", device="cpu")
    assert a.tolist() == [0, 1, 2, 0, 1, 1] and torch.equal(f, g)
    g, a = attn.rope_axes([2, 3], base=100.0, layout="separate", device="cpu")
    assert a.tolist() == [0, 0, 1, 1, 1]
    np.testing.assert_allclose(g.numpy(), [1, 0.1, 1, 100 ** (-1 / 3), 100 ** (-2 / 3)], rtol=1e-14)
    # one axis is the plain series
    assert torch.equal(attn.rope_axes([32], device="cpu")[0], attn.rope_frequencies(64, device="cpu")[0])
    assert attn.rope_axes([4, 0, 4], device="cpu")[1].tolist() == [0] * 4 + [2] * 4
    for bad in (dict(sections=[]), dict(sections=[0, 0]), dict(sections=[4, -1]), dict(sections=[1] * 9),
                dict(sections=[4], base=0.0), dict(sections=[4], layout="other")):
        with pytest.raises(ValueError):
            attn.rope_axes(device="cpu", **bad)


def _inputs(T, Hq, Hk, d, n_axes, seed, fused=False, far=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, Hq + 2 * Hk, d, generator=g).bfloat16()
    pos = torch.randint(-3, 5000, (n_axes, T), generator=g, dtype=torch.int32) + far
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    if fused:
        y = x.cuda()
        return (q, k, v), (y[:, :Hq], y[:, Hq:Hq + Hk], y[:, Hq + Hk:]), pos
    return (q, k, v), tuple(t.contiguous().cuda() for t in (q, k, v)), pos


CASES = [
    # T, Hq, Hk, d, sections, layout, interleaved, fused, far
    (1, 4, 2, 64, (8, 12, 12), "blocks", False, False, 0),
    (7, 3, 1, 128, (24, 40), "separate", True, True, 0),
    (65, 28, 4, 128, (16, 24, 24), "dealt", False, True, 1000000),
    (300, 2, 2, 256, (60, 4, 32, 32), "blocks", True, False, 0),
    (33, 5, 5, 64, (1, 2, 1, 1, 1, 1, 1, 8), "dealt", False, False, -2000000000),
    (3001, 4, 1, 64, (16,), "blocks", False, True, 0),
    (2433, 2, 1, 128, (20, 12), "blocks", True, False, 50000),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("inverse", [False, True])
def test_rotate(case, inverse):
    T, Hq, Hk, d, sections, layout, inter, fused, far = case
    f, ax = attn.rope_axes(sections, layout=layout)
    host, dev, pos = _inputs(T, Hq, Hk, d, len(sections), 3 + T, fused, far)
    q, k = attn.rope_rotate(dev[0], dev[1], f, pos.cuda(), axes=ax, interleaved=inter, amp=1.25, inverse=inverse)
    attn.sync_check()
    for got, x in ((q, host[0]), (k, host[1])):
        assert got.shape == x.shape and got.is_contiguous()
        check(got, *rotate(x.float(), pos, f.cpu(), ax.cpu(), 1.25, inter, -1.0 if inverse else 1.0))
    # into rows at another stride, beside what stays
    y = torch.full((T, Hq + Hk + 1, d), 9.0, dtype=torch.bfloat16, device="cuda")
    out = attn.rope_rotate(dev[0], dev[1], f, pos.cuda(), axes=ax, interleaved=inter, amp=1.25, inverse=inverse,
                           out=(y[:, :Hq], y[:, Hq + 1:]))
    attn.sync_check()
    assert torch.equal(out[0], q) and torch.equal(out[1], k) and (y[:, Hq] == 9).all()
    # in place, and each side alone
    a, b = attn.rope_rotate(dev[0], None, f, pos.cuda(), axes=ax, interleaved=inter, amp=1.25, inverse=inverse,
                            out=(dev[0], None))
    c, e = attn.rope_rotate(None, dev[1], f, pos.cuda(), axes=ax, interleaved=inter, amp=1.25, inverse=inverse,
                            out=(None, dev[1]))
    attn.sync_check()
    assert b is None and c is None and torch.equal(dev[0], q) and torch.equal(dev[1], k)


@pytest.mark.gpu
@pytest.mark.parametrize("d,rot", [(16, 16), (48, 32), (80, 80), (112, 48), (240, 224)])
def test_rotate_head_dims_and_one_axis(d, rot):
    """Any multiple of 16; without axes the positions are one row, as in rope_append."""
    f, amp = attn.rope_frequencies(rot)
    host, dev, pos = _inputs(50, 3, 2, d, 1, d)
    q, k = attn.rope_rotate(dev[0], dev[1], f, pos[0].cuda())
    z = torch.zeros(rot // 2, dtype=torch.int32, device="cuda")
    q2, k2 = attn.rope_rotate(dev[0], dev[1], f, pos.cuda(), axes=z)
    attn.sync_check()
    assert torch.equal(q, q2) and torch.equal(k, k2)
    check(q, *rotate(host[0].float(), pos, f.cpu(), [0] * (rot // 2), amp, False))
    check(k, *rotate(host[1].float(), pos, f.cpu(), [0] * (rot // 2), amp, False))


@pytest.mark.gpu
def test_inverse_is_the_gradient():
    """L = <rotate(x), y>: dL/dx is inverse(y) (a linear map and its transpose), against the
    difference quotients of the fp64 rotation along random directions."""
    f, ax = attn.rope_axes((16, 24, 24))
    host, dev, pos = _inputs(40, 4, 2, 128, 3, 8)
    amp = 1.1
    y = torch.randn(40, 4, 128, generator=torch.Generator().manual_seed(1)).bfloat16()
    grad, _ = attn.rope_rotate(y.cuda(), None, f, pos.cuda(), axes=ax, amp=amp, inverse=True)
    attn.sync_check()
    x, grad = host[0].double().numpy(), grad.double().cpu().numpy()
    _, mag = rotate(y.float(), pos, f.cpu(), ax.cpu(), amp, False, -1.0)
    rng = np.random.default_rng(2)
    for _ in range(3):
        u, h = rng.standard_normal(x.shape), 1e-3
        up = (rotate(x + h * u, pos, f.cpu(), ax.cpu(), amp, False)[0] * y.double().numpy()).sum()
        dn = (rotate(x - h * u, pos, f.cpu(), ax.cpu(), amp, False)[0] * y.double().numpy()).sum()
        # each element of grad is off by half a bf16 step and 2^-20 of its terms; the quotient of a linear
        # map by 1e-16 * |terms| / h
        tol = ((2.0 ** -8 * abs(grad) + 2.0 ** -20 * mag) * abs(u)).sum() + 1e-9 * abs(x).sum()
        assert abs((up - dn) / (2 * h) - (grad * u).sum()) <= tol


@pytest.mark.gpu
@pytest.mark.parametrize("case", [c for c in CASES if c[3] in (64, 128, 256)], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("dense", [False, True])
def test_append(case, dense):
    T, Hq, Hk, d, sections, layout, inter, fused, far = case
    f, ax = attn.rope_axes(sections, layout=layout)
    host, dev, pos = _inputs(T, Hq, Hk, d, len(sections), 5 + T, fused, far)
    hist = 9
    cuts = [0, T // 3, T // 3, T]  # one sequence without new tokens
    new = [b - a for a, b in zip(cuts, cuts[1:])]
    lens = torch.tensor([n + hist for n in new], dtype=torch.int32)
    kc = torch.randn(3, int(lens.max()), Hk, d).bfloat16()
    vc = torch.randn(3, int(lens.max()), Hk, d).bfloat16()
    if dense:
        kp, vp, table = kc.cuda(), vc.cuda(), None
    else:
        kp, vp, table = make_pages(kc, vc, lens, 16, 4)
        kp, vp, table = kp.cuda(), vp.cuda(), table.cuda()
    q = attn.rope_append(*dev, kp, vp, lens.cuda(), f, page_table=table,
                         cu_seqlens_q=torch.tensor(cuts, dtype=torch.int32).cuda(), positions=pos.cuda(),
                         interleaved=inter, amp=0.75, axes=ax)
    attn.sync_check()
    check(q, *rotate(host[0].float(), pos, f.cpu(), ax.cpu(), 0.75, inter))
    rk, mk = rotate(host[1].float(), pos, f.cpu(), ax.cpu(), 0.75, inter)
    kp, vp = kp.cpu(), vp.cpu()
    for b, n in enumerate(new):
        L, t = int(lens[b]), slice(cuts[b], cuts[b + 1])
        k = kp[b, :L] if dense else gather(kp, table.cpu(), b, L, 16)
        v = vp[b, :L] if dense else gather(vp, table.cpu(), b, L, 16)
        assert torch.equal(k[:hist], kc[b, :hist]) and torch.equal(v[:hist], vc[b, :hist])
        check(k[hist:], rk[t], mk[t])
        assert torch.equal(v[hist:], host[2][t])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 2500])
def test_equal_axes_give_the_bits_of_one_axis(T):
    """A text token has the same position on every axis: the rotation of rope_append."""
    f, ax = attn.rope_axes((16, 24, 24))
    _, dev, pos = _inputs(T, 4, 2, 128, 1, 6)
    lens = torch.tensor([T], dtype=torch.int32).cuda()
    cu = torch.tensor([0, T], dtype=torch.int32).cuda()
    res = []
    for p, axes in ((pos[0].cuda(), None), (pos.expand(3, T).contiguous().cuda(), ax)):
        kc = torch.zeros(1, T, 2, 128, dtype=torch.bfloat16, device="cuda")
        vc = torch.zeros_like(kc)
        res.append((attn.rope_append(*dev, kc, vc, lens, f, cu_seqlens_q=cu, positions=p, axes=axes), kc, vc))
    q, k = attn.rope_rotate(dev[0], dev[1], f, pos.expand(3, T).contiguous().cuda(), axes=ax)
    attn.sync_check()
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert torch.equal(q, res[0][0]) and torch.equal(k, res[0][1][0])


@pytest.mark.gpu
def test_an_axis_out_of_range_is_reported():
    f, ax = attn.rope_axes((16, 16))
    _, dev, pos = _inputs(4, 2, 1, 64, 2, 6)
    for bad in (2, -1):
        wrong = ax.clone()
        wrong[3] = bad
        attn.rope_rotate(dev[0], dev[1], f, pos.cuda(), axes=wrong)
        with pytest.raises(attn.AttnError) as e:
            attn.sync_check()
        assert e.value.status == attn.ATTN_ERR_DEVICE_INPUT
    attn.rope_rotate(dev[0], dev[1], f, pos.cuda(), axes=ax)
    attn.sync_check()


@pytest.mark.gpu
def test_no_tokens_a_stream_and_a_graph():
    f, ax = attn.rope_axes((16, 24, 24))
    e = lambda H: torch.empty(0, H, 128, dtype=torch.bfloat16, device="cuda")
    q, k = attn.rope_rotate(e(4), e(2), f, torch.empty(3, 0, dtype=torch.int32, device="cuda"), axes=ax)
    assert q.shape == (0, 4, 128) and k.shape == (0, 2, 128)
    host, dev, pos = _inputs(20, 4, 2, 128, 3, 2)
    p, side = pos.cuda(), torch.cuda.Stream()
    want = attn.rope_rotate(dev[0], dev[1], f, p, axes=ax)
    side.wait_stream(torch.cuda.current_stream())
    got = attn.rope_rotate(dev[0], dev[1], f, p, axes=ax, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gq, gk = attn.rope_rotate(dev[0], dev[1], f, p, axes=ax, inverse=True)
    for shift in (0, 11):
        p.copy_((pos + shift).cuda())
        graph.replay()
        torch.cuda.synchronize()
        check(gq, *rotate(host[0].float(), pos + shift, f.cpu(), ax.cpu(), 1.0, False, -1.0))
    attn.sync_check()
