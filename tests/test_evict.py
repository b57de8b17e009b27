"""Accumulated attention weights and eviction by them.

Weights tolerance, from the arithmetic: the exponent's argument carries the fp32 dot product
((d + 1) 2^-24 of scale * sum |q k|), one fma and the rounding of -lse log2 e (2^-23 of
|scale s| + |lse|), and ex2.approx 2^-22 of the term; the sum of n terms adds n 2^-24 at
most.  All terms are positive, so the bounds add."""
import numpy as np
import pytest
import torch

import attention_forward_tcgen05_gb300 as attn
from attention_forward_tcgen05_gb300 import workloads as W
from tests.paged_cases import admitted, gather, make_pages

pytestmark = pytest.mark.gpu


def weights_ref(q, lse, kc, cu, kv, Hkv, scale, causal, window=0, n_sink=0):
    """fp64 (W [B][Hkv][L], bound) lists; lse [Hq][T]."""
    q, kc, lse = q.double().numpy(), kc.double().numpy(), lse.double().numpy()
    G, d = q.shape[1] // Hkv, q.shape[2]
    out = []
    for b in range(len(kv)):
        a, e, L = int(cu[b]), int(cu[b + 1]), int(kv[b])
        ok = admitted(e - a, L, causal, window, n_sink)
        w, bound = np.zeros((Hkv, L)), np.zeros((Hkv, L))
        for h in range(q.shape[1]):
            hk = h // G
            s = scale * (q[a:e, h] @ kc[b, :L, hk].T)
            m = scale * (abs(q[a:e, h]) @ abs(kc[b, :L, hk]).T)
            l = lse[h, a:e, None]
            live = ok & np.isfinite(l)
            with np.errstate(invalid="ignore", over="ignore"):
                p = np.where(live, np.exp(s - l), 0.0)
                arg = np.where(live, (d + 1) * 2.0 ** -24 * m + 2.0 ** -23 * (abs(s) + abs(l)), 0.0)
            w[hk] += p.sum(0)
            bound[hk] += (p * (1.1 * arg + 2.0 ** -22)).sum(0)
        out.append((w, bound + w * G * max(1, e - a) * 2.0 ** -24 + 1e-30))
    return out


def lse_of(q, kc, cu, kv, Hkv, scale, causal, window=0, n_sink=0):
    """fp32 LSE [Hq][T] of an attention call, as its kernel would leave it."""
    G = q.shape[1] // Hkv
    lse = np.full((q.shape[1], q.shape[0]), -np.inf)
    qd, kd = q.double().numpy(), kc.double().numpy()
    for b in range(len(kv)):
        a, e, L = int(cu[b]), int(cu[b + 1]), int(kv[b])
        ok = admitted(e - a, L, causal, window, n_sink)
        for h in range(q.shape[1]):
            s = np.where(ok, scale * (qd[a:e, h] @ kd[b, :L, h // G].T), -np.inf)
            if L:
                m = s.max(1, keepdims=True)
                m = np.where(np.isfinite(m), m, 0)
                with np.errstate(divide="ignore"):
                    lse[h, a:e] = (m + np.log(np.exp(s - m).sum(1, keepdims=True)))[:, 0]
    return torch.from_numpy(lse).float()


FEW = [(1, 1), (0, 40), (2, 300), (1, 0), (2, 129), (2, 1)]
MANY = [(1, 1), (77, 300), (128, 128), (0, 50), (200, 150), (129, 900), (40, 40), (3, 0)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv,page", [(4, 2, 16), (7, 1, 48), (5, 5, None), (24, 1, 64)])
@pytest.mark.parametrize("seqs", [FEW, MANY], ids=["few", "many"])
@pytest.mark.parametrize("mask", [(True, 0, 0), (False, 0, 0), (True, 60, 3)], ids=["causal", "full", "window"])
def test_weights(d, Hq, Hkv, page, seqs, mask):
    causal, window, n_sink = mask
    scale = 1.0 / np.sqrt(d)
    sq = torch.tensor([a for a, _ in seqs], dtype=torch.int32)
    kv = torch.tensor([b for _, b in seqs], dtype=torch.int32)
    q, kc, vc, cu = W.varlen_inputs(len(seqs), Hq, Hkv, d, sq, kv, 600 + d + Hq)
    lse = lse_of(q, kc, cu, kv, Hkv, scale, causal, window, n_sink)
    if page is None:
        pool, table, cap = kc.clone(), None, kc.shape[1]
        for b in range(len(seqs)):
            pool[b, int(kv[b]):] = float("nan")
    else:
        pool, _, table = make_pages(kc, vc, kv, page, 600)
        cap = table.shape[1] * page
    w0 = torch.rand(len(seqs), Hkv, cap + 3)
    ref = weights_ref(q, lse, kc, cu, kv, Hkv, scale, causal, window, n_sink)
    for acc in (False, True):
        w = w0.cuda()
        r = attn.key_weights(q.cuda(), lse.cuda(), pool.cuda(), kv.cuda(), w,
                             page_table=None if table is None else table.cuda(), cu_seqlens_q=cu.cuda(),
                             max_sq=int(sq.max()), causal=causal, window=window, n_sink=n_sink, scale=scale,
                             accumulate=acc)
        attn.sync_check()
        assert r is w
        got = w.cpu().double().numpy()
        for b, (wr, bound) in enumerate(ref):
            L = int(kv[b])
            want = wr + (w0[b, :, :L].double().numpy() if acc else 0)
            assert (abs(got[b, :, :L] - want) <= bound + (abs(want) * 2.0 ** -24 if acc else 0)).all(), (b, acc)
            assert np.array_equal(got[b, :, L:], w0[b, :, L:].double().numpy())


@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (28, 4), (40, 2)])
def test_weights_of_a_decode(Hq, Hkv):
    """One row per sequence, lse [B][Hq] as the decode leaves it; each head's weights sum to 1."""
    lens = torch.tensor([1, 700, 64, 0, 129], dtype=torch.int32)
    q, kc, vc = W.decode_inputs(5, Hq, Hkv, 128, lens, 610)
    kp, vp, table = make_pages(kc, vc, lens, 32, 610)
    cap = table.shape[1] * 32
    args = q.cuda(), kp.cuda()
    o, lse = attn.decode_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda())
    w = torch.full((5, Hkv, cap), 9.0, device="cuda")
    attn.key_weights(*args[:1], lse, args[1], lens.cuda(), w, page_table=table.cuda(), accumulate=False)
    attn.sync_check()
    ref = weights_ref(q, lse.cpu().T, kc, list(range(6)), lens, Hkv, 1 / np.sqrt(128), True)
    for b, (wr, bound) in enumerate(ref):
        L = int(lens[b])
        assert (abs(w[b, :, :L].cpu().double().numpy() - wr) <= bound).all()
        if L:
            np.testing.assert_allclose(w[b, :, :L].sum(-1).cpu().numpy(), Hq // Hkv, rtol=2e-3)


def test_weights_same_bits_each_time():
    sq, kv = torch.tensor([700], dtype=torch.int32), torch.tensor([900], dtype=torch.int32)
    q, kc, vc, cu = W.varlen_inputs(1, 8, 2, 128, sq, kv, 611)
    lse = lse_of(q, kc, cu, kv, 2, 0.09, True).cuda()
    got = []
    for _ in range(4):
        w = torch.zeros(1, 2, 900, device="cuda")
        attn.key_weights(q.cuda(), lse, kc.cuda(), kv.cuda(), w, cu_seqlens_q=cu.cuda(), max_sq=700, scale=0.09)
        got.append(w)
    attn.sync_check()
    assert all(torch.equal(got[0], g) for g in got[1:])


# ------------------------------------------------------------------ eviction
def kept_ref(w, L, budget, n_recent, n_sink):
    """Kept indices of one row of weights: numpy's order by (-weight, index)."""
    if L <= budget:
        return np.arange(L)
    mid = np.arange(n_sink, L - n_recent)
    x = w[mid].astype(np.float64)
    nan = np.isnan(x)  # above everything
    top = mid[np.lexsort((mid, np.where(nan, 0, -x), ~nan))][:budget - n_sink - n_recent]
    return np.sort(np.concatenate([np.arange(n_sink), top, np.arange(L - n_recent, L)])).astype(int)


def weird_weights(B, Hkv, cap, kind, seed):
    rng = np.random.default_rng(seed)
    if kind == "random":
        w = rng.random((B, Hkv, cap)) ** 6
    elif kind == "ties":
        w = rng.integers(0, 3, (B, Hkv, cap)) * 0.25
    elif kind == "equal":
        w = np.zeros((B, Hkv, cap))
        w[..., ::2] = -0.0
    else:  # infinities, NaN, negatives, denormals
        w = rng.choice([np.inf, -np.inf, -1.5, 1e-42, 0.0, -0.0, 3e38, 1.0, 1.0000001], (B, Hkv, cap))
        w[:, :, 5::11] = np.nan
    return torch.from_numpy(w).float()


LENS = [0, 1, 30, 31, 64, 100, 500, 1025]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["random", "ties", "equal", "special"])
@pytest.mark.parametrize("budget,n_recent,n_sink", [(31, 8, 2), (1, 0, 0), (64, 64, 0), (64, 60, 4), (300, 0, 4)])
@pytest.mark.parametrize("where", ["in_place", "pages", "dense"])
def test_evict(d, kind, budget, n_recent, n_sink, where):
    Hkv, page = 3, 48
    B = len(LENS)
    lens = torch.tensor(LENS, dtype=torch.int32)
    g = torch.Generator().manual_seed(budget + d)
    kc = torch.randn(B, max(LENS), Hkv, d, generator=g).bfloat16()
    vc = torch.randn(B, max(LENS), Hkv, d, generator=g).bfloat16()
    if where == "dense":
        kp, vp, table, page = kc.clone(), vc.clone(), None, max(LENS)
        cap = page
    else:
        kp, vp, table = make_pages(kc, vc, lens, page, 620)
        cap = table.shape[1] * page
    w = weird_weights(B, Hkv, cap + 1, kind, 621)
    kg, vg, wg, lg = kp.cuda(), vp.cuda(), w.cuda(), lens.cuda()
    tg = None if table is None else table.cuda()
    dst, t2 = None, table
    out_lens = torch.empty(B, dtype=torch.int32, device="cuda")
    if where == "pages":
        per = -(-min(budget, cap) // 16)
        t2 = torch.randperm(B * per, generator=g).to(torch.int32).view(B, per)
        dst = (torch.full((B * per, 16, Hkv, d), 3.0, dtype=torch.bfloat16, device="cuda"),
               torch.full((B * per, 16, Hkv, d), 4.0, dtype=torch.bfloat16, device="cuda"), t2.cuda(),
               torch.full_like(wg, 5.0))
    else:
        out_lens = lg  # the new lengths over the old ones
    kept = torch.empty(B, Hkv, budget, dtype=torch.int32, device="cuda")
    r = attn.evict(wg, kg, vg, lg, budget, n_recent, n_sink, page_table=tg, dst=dst, out=(kept, out_lens))
    attn.sync_check()
    assert r[0] is kept and r[1] is out_lens
    kept = kept.cpu().numpy()
    assert out_lens.cpu().tolist() == [min(L, budget) for L in LENS]
    pg = 16 if where == "pages" else page
    k2, v2, w2 = (x.cpu() for x in ((dst[0], dst[1], dst[3]) if dst else (kg, vg, wg)))
    t2 = torch.arange(B, dtype=torch.int32)[:, None] if t2 is None else t2
    for b, L in enumerate(LENS):
        n = min(L, budget)
        for h in range(Hkv):
            idx = kept_ref(w[b, h].numpy(), L, budget, n_recent, n_sink)
            assert np.array_equal(kept[b, h, :n], idx), (b, h)
            assert (kept[b, h, n:] == -1).all()
            assert torch.equal(gather(k2, t2, b, n, pg)[:, h], kc[b, idx, h])
            assert torch.equal(gather(v2, t2, b, n, pg)[:, h], vc[b, idx, h])
            assert torch.equal(w2[b, h, :n].view(torch.int32), w[b, h, idx].view(torch.int32))
            assert (w2[b, h, n:L] == 0).all()
            rest = w[b, h, L:] if dst is None else torch.full_like(w[b, h, L:], 5.0)
            assert torch.equal(w2[b, h, L:].view(torch.int32), rest.view(torch.int32))
    if dst:  # the source stays
        assert torch.equal(kg.cpu().view(torch.int16), kp.view(torch.int16))
        assert torch.equal(wg.cpu().view(torch.int32), w.view(torch.int32))


@pytest.mark.parametrize("kind", ["random", "ties", "special"])
@pytest.mark.parametrize("in_place", [True, False], ids=["in_place", "pages"])
@pytest.mark.parametrize("B,Hkv,cap", [(9, 1, 9000), (60, 1, 8200), (5, 8, 3000)])
def test_evict_rows_in_slices(kind, in_place, B, Hkv, cap):
    """Rows that 4, 2 and 1 CTAs share, some shorter than a slice; the weights alone."""
    rng = np.random.default_rng(6)
    L = rng.integers(0, cap + 1, B)
    L[:5] = [cap, 33, 0, 1, cap // 8]
    w = weird_weights(B, Hkv, cap, kind, 7)
    kc = torch.zeros(B, cap, Hkv, 64, dtype=torch.bfloat16, device="cuda")
    wg, w2 = w.cuda(), torch.full((B, Hkv, cap), 9.0, device="cuda")
    dst = None if in_place else (torch.zeros_like(kc), torch.zeros_like(kc), None, w2)
    lens = torch.from_numpy(L.astype(np.int32)).cuda()
    for budget, n_recent, n_sink in ((700, 100, 4), (33, 0, 0)):
        if in_place:
            wg.copy_(w)
        kept, new = attn.evict(wg, kc, kc.clone(), lens, budget, n_recent, n_sink, dst=dst)
        attn.sync_check()
        kept, got = kept.cpu().numpy(), (wg if in_place else w2).cpu()
        for b in range(B):
            n = min(int(L[b]), budget)
            assert new[b].item() == n
            for h in range(Hkv):
                idx = kept_ref(w[b, h].numpy(), int(L[b]), budget, n_recent, n_sink)
                assert np.array_equal(kept[b, h, :n], idx) and (kept[b, h, n:] == -1).all(), (b, h)
                assert torch.equal(got[b, h, :n].view(torch.int32), w[b, h, idx].view(torch.int32)), (b, h)
                assert (got[b, h, n:int(L[b])] == 0).all()


@pytest.mark.parametrize("L", [60000, 64000, 130000])
def test_evict_rows_of_several_blocks(L):
    """60,000 and 64,000 keys: four and eight slices of a block each.  130,000: blocks that each
    pass reads again."""
    d = 64
    g = torch.Generator().manual_seed(5)
    kc = torch.randn(1, L, 1, d, generator=g).bfloat16()
    w = torch.rand(1, 1, L, generator=g).mul(50).round()  # many ties
    kg, vg, wg = kc.cuda(), (-kc).cuda(), w.cuda()
    kept, lens = attn.evict(wg, kg, vg, torch.tensor([L], dtype=torch.int32, device="cuda"), 5000, 100, 4)
    attn.sync_check()
    idx = kept_ref(w[0, 0].numpy(), L, 5000, 100, 4)
    assert np.array_equal(kept[0, 0].cpu().numpy(), idx) and lens.item() == 5000
    assert torch.equal(kg[0, :5000, 0].cpu(), kc[0, idx, 0]) and torch.equal(vg[0, :5000, 0].cpu(), -kc[0, idx, 0])
    assert torch.equal(wg[0, 0, :5000].cpu(), w[0, 0, idx]) and (wg[0, 0, 5000:] == 0).all()
