"""Gradients of the prefill attention against their formula in fp64 and against differences.

Bounds, element by element.  bf16 rounds by at most 2^-8 of a value, fp32 by 2^-24.  P goes
into its product rounded to bf16 (R = 2^-8 of it) and is itself off by F = 2^-13 of it: its
exponent is a score in fp32 (|scale q.k - lse| below 200 here, 128 products summed and three
bf16 terms of lse / scale: 2^-16 in all) and ex2.approx adds 2^-22.  So
  |d dv| <= (R + F) sum P |g| + R |dv|.
dS = P (dP - D) likewise is off by R |dS| + 2 F P (sum |g||v| + |D|) (dP and D are fp32 sums of
up to 128 products; their own errors, 2^-17 of the absolute sums, are inside the second F), so
  |d dq| <= scale sum (R |dS| + 2 F P (|g||v| + |D|)) |k| + R |dq|,
dk alike.  The products' fp32 accumulation (2^-24 a term over up to 4096 terms) is inside F.
"""
import math

import pytest
import torch

import attention_forward_tcgen05_gb300 as attn

R, F = 2.0 ** -8, 2.0 ** -13


def _inputs(B, Hq, Hkv, Sq, Skv, d, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    q = (rnd(B, Sq, Hq, d) * spread).bfloat16()
    k, v, do = rnd(B, Skv, Hkv, d).bfloat16(), rnd(B, Skv, Hkv, d).bfloat16(), rnd(B, Sq, Hq, d).bfloat16()
    return q, k, v, do


def _mask(Sq, L, causal, window, sink, dev):
    p = torch.arange(Sq, device=dev)[:, None] + L - Sq
    j = torch.arange(L, device=dev)[None]
    ok = (j <= p) if causal else torch.ones(Sq, L, dtype=torch.bool, device=dev)
    if window:
        ok = ok & ((j > p - window) | (j < sink))
    return ok


def _forward(q, k, v, ok, scale):
    """fp64 o, lse of one sequence: q [n,Hq,d], k, v [L,Hkv,d]."""
    G = q.shape[1] // k.shape[1]
    kk, vv = k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    s = torch.einsum("ihd,jhd->hij", q.double(), kk) * scale
    s = s.masked_fill(~ok, -math.inf)
    lse = s.logsumexp(-1)
    p = torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[..., None])
    p = p.masked_fill(~ok, 0.0)
    return torch.einsum("hij,jhd->ihd", p, vv), lse


def _reference(do, q, k, v, o, lse, dlse, ok, scale):
    """fp64 gradients of one sequence and the bounds of the module's docstring."""
    Hkv = k.shape[1]
    G = q.shape[1] // Hkv
    rep = lambda x: x.double().repeat_interleave(G, 1)
    qd, g, kk, vv = q.double(), do.double(), rep(k), rep(v)
    s = torch.einsum("ihd,jhd->hij", qd, kk) * scale
    live = torch.isfinite(lse.double())
    p = torch.exp(s - torch.where(live, lse.double(), torch.zeros_like(lse.double()))[..., None])
    p = torch.where(ok & live[..., None], p, 0.0)
    D = torch.einsum("ihd,ihd->hi", g, o.double())
    if dlse is not None:
        D = D - dlse.double()
    ds = p * (torch.einsum("ihd,jhd->hij", g, vv) - D[..., None])
    e = R * ds.abs() + 2 * F * p * (torch.einsum("ihd,jhd->hij", g.abs(), vv.abs()) + D.abs()[..., None])
    head = lambda x: x.unflatten(1, (Hkv, G)).sum(2)
    dq = torch.einsum("hij,jhd->ihd", ds, kk) * scale
    dk = head(torch.einsum("hij,ihd->jhd", ds, qd)) * scale
    dv = head(torch.einsum("hij,ihd->jhd", p, g))
    bq = torch.einsum("hij,jhd->ihd", e, kk.abs()) * scale + R * dq.abs()
    bk = head(torch.einsum("hij,ihd->jhd", e, qd.abs())) * scale + R * dk.abs()
    bv = head(torch.einsum("hij,ihd->jhd", p, g.abs())) * (R + F) + R * dv.abs()
    return (dq, dk, dv), (bq, bk, bv)


def _within(got, want, bound, what):
    assert torch.isfinite(got).all(), f"{what}: not finite"
    # (1e-30: bf16 subnormals)
    over = (got.double() - want).abs() - bound - 1e-30
    assert not over.numel() or over.max().item() <= 0, \
        f"{what}: off by {(got.double() - want).abs().max().item():.3e}, {int((over > 0).sum())} beyond the bound"


def _check_fixed(B, Hq, Hkv, Sq, Skv, d, causal=True, window=0, sink=0, o_dtype=torch.bfloat16, dlse=False, seed=1,
                 scale=None, spread=1.5):
    q, k, v, do = (t.cuda() for t in _inputs(B, Hq, Hkv, Sq, Skv, d, seed, spread))
    sc = 1 / math.sqrt(d) if scale is None else scale
    ok = _mask(Sq, Skv, causal, window, sink, "cuda")
    fw = [_forward(q[b], k[b], v[b], ok, sc) for b in range(B)]
    o = torch.stack([x[0] for x in fw]).to(o_dtype)
    lse = torch.stack([x[1] for x in fw]).float()
    dl = torch.randn(B, Hq, Sq, generator=torch.Generator().manual_seed(seed + 5)).cuda() if dlse else None
    got = attn.prefill_backward(do, q, k, v, o, lse, causal=causal, window=window, n_sink=sink, scale=scale, dlse=dl)
    attn.sync_check()
    for b in range(B):
        want, bound = _reference(do[b], q[b], k[b], v[b], o[b], lse[b], None if dl is None else dl[b], ok, sc)
        for x, w, e, name in zip(got, want, bound, ("dq", "dk", "dv")):
            _within(x[b], w, e, f"{name}[{b}]")
    return got


FIXED = [
    # B, Hq, Hkv, Sq, Skv, d, causal, window, sink
    (1, 1, 1, 1, 1, 64, True, 0, 0),
    (1, 1, 1, 1, 1, 128, False, 0, 0),
    (2, 2, 1, 1, 300, 128, True, 0, 0),        # one row, as a decode step
    (1, 2, 2, 127, 127, 64, True, 0, 0),
    (1, 2, 2, 128, 128, 128, True, 0, 0),
    (1, 4, 2, 129, 129, 128, True, 0, 0),
    (2, 7, 1, 300, 300, 128, True, 0, 0),
    (1, 3, 3, 257, 400, 64, False, 0, 0),
    (1, 4, 4, 400, 257, 128, False, 0, 0),
    (1, 4, 2, 200, 500, 128, True, 0, 0),      # cached keys before the rows
    (1, 4, 2, 500, 200, 128, True, 0, 0),      # rows that admit nothing, whole tiles of them
    (1, 4, 2, 500, 200, 64, True, 70, 3),
    (1, 4, 2, 600, 600, 128, True, 1, 0),      # the own key only
    (1, 4, 2, 600, 600, 64, True, 1, 1),
    (1, 2, 1, 700, 700, 128, True, 100, 130),  # sinks past a tile
    (1, 2, 1, 700, 700, 64, True, 128, 0),
    (2, 6, 2, 513, 513, 128, True, 129, 4),
    (1, 4, 1, 300, 300, 64, True, 5000, 7),    # wider than the sequence
    (1, 2, 2, 1, 1000, 64, True, 10, 2),       # keys that nobody sees
    (3, 8, 2, 260, 640, 64, True, 200, 200),
    (1, 32, 1, 200, 200, 128, True, 0, 0),     # one group of 32 heads
    (1, 16, 16, 1100, 1100, 64, False, 0, 0),
    (1, 5, 5, 2100, 2100, 128, True, 300, 4),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", FIXED, ids=lambda c: "-".join(map(str, c)))
def test_fixed(case):
    _check_fixed(*case, seed=sum(map(int, case)))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_fp32_o_and_lse_gradient(d):
    _check_fixed(2, 4, 2, 300, 333, d, True, 100, 2, o_dtype=torch.float32, dlse=True)
    _check_fixed(1, 4, 2, 300, 200, d, True, 0, 0, o_dtype=torch.float32, dlse=True)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.01, 1.0])
def test_scale(scale):
    _check_fixed(1, 4, 2, 300, 300, 64, True, 0, 0, scale=scale, spread=0.5)


def _check_varlen(lens_q, lens_k, Hq, Hkv, d, causal=True, window=0, sink=0, dlse=False, spare_q=0, spare_k=0, seed=3,
                  give_out=False, first=0):
    """Packed rows; rows of no sequence and slots behind a sequence's keys hold NaN."""
    B, max_kv = len(lens_q), max(lens_k) + spare_k
    total = first + sum(lens_q) + spare_q
    g = torch.Generator().manual_seed(seed)
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16)
    q, do, o, lse = nan(total, Hq, d), nan(total, Hq, d), nan(total, Hq, d), torch.full((Hq, total), float("nan"))
    dl = torch.full((Hq, total), float("nan")) if dlse else None
    kc, vc = nan(B, max_kv, Hkv, d), nan(B, max_kv, Hkv, d)
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(lens_q), 0)
    cu += first
    sc, refs = 1 / math.sqrt(d), []
    for b in range(B):
        r, n, L = slice(int(cu[b]), int(cu[b + 1])), lens_q[b], lens_k[b]
        q[r] = (torch.randn(n, Hq, d, generator=g) * 1.5).bfloat16()
        do[r] = torch.randn(n, Hq, d, generator=g).bfloat16()
        kc[b, :L] = torch.randn(L, Hkv, d, generator=g).bfloat16()
        vc[b, :L] = torch.randn(L, Hkv, d, generator=g).bfloat16()
        ok = _mask(n, L, causal, window, sink, "cpu")
        x, y = _forward(q[r], kc[b, :L], vc[b, :L], ok, sc)
        o[r], lse[:, r] = x.bfloat16(), y.float()
        if dlse:
            dl[:, r] = torch.randn(Hq, n, generator=g)
        refs.append(_reference(do[r], q[r], kc[b, :L], vc[b, :L], o[r], lse[:, r], dl[:, r] if dlse else None, ok, sc))
    dev = lambda t: None if t is None else t.cuda()
    out = None
    if give_out:
        out = tuple(torch.full(t.shape, 7.0, dtype=torch.bfloat16, device="cuda") for t in (q, kc, vc))
    got = attn.prefill_varlen_backward(dev(do), dev(q), dev(kc), dev(vc), dev(o), dev(lse), dev(cu),
                                       torch.tensor(lens_k, dtype=torch.int32).cuda(), max(max(lens_q), 1),
                                       causal=causal, window=window, n_sink=sink, dlse=dev(dl), out=out)
    attn.sync_check()
    rest = 7.0 if give_out else 0.0
    dq, dk, dv = (t.cpu() for t in got)
    for b, (want, bound) in enumerate(refs):
        r, L = slice(int(cu[b]), int(cu[b + 1])), lens_k[b]
        _within(dq[r], want[0], bound[0], f"dq of sequence {b}")
        _within(dk[b, :L], want[1], bound[1], f"dk[{b}]")
        _within(dv[b, :L], want[2], bound[2], f"dv[{b}]")
        assert (dk[b, L:] == rest).all() and (dv[b, L:] == rest).all()
    assert (dq[:first] == rest).all() and (dq[int(cu[B]):] == rest).all()


VARLEN = [
    dict(lens_q=[5, 130, 1, 64], lens_k=[5, 130, 1, 64], Hq=4, Hkv=2, d=128),
    dict(lens_q=[100, 37, 200], lens_k=[300, 37, 1000], Hq=7, Hkv=1, d=128, spare_q=9, spare_k=50),
    dict(lens_q=[0, 129, 0, 3], lens_k=[40, 129, 0, 0], Hq=4, Hkv=4, d=64, spare_q=200, spare_k=300),
    dict(lens_q=[257, 255], lens_k=[257, 90], Hq=4, Hkv=2, d=64, window=60, sink=3, spare_q=1, first=3),
    dict(lens_q=[400, 1, 310], lens_k=[700, 500, 310], Hq=8, Hkv=2, d=128, window=128, sink=1, dlse=True, first=130),
    dict(lens_q=[77, 140], lens_k=[300, 20], Hq=2, Hkv=1, d=128, causal=False, spare_k=1),
    dict(lens_q=[31] * 40, lens_k=[31] * 40, Hq=2, Hkv=2, d=64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("give_out", [False, True])
@pytest.mark.parametrize("i", range(len(VARLEN)))
def test_varlen(i, give_out):
    _check_varlen(**VARLEN[i], give_out=give_out)


@pytest.mark.gpu
def test_no_rows_no_keys():
    for d in (64, 128):
        e = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
        full = lambda *s: torch.full(s, 3.0, dtype=torch.bfloat16, device="cuda")
        out = full(2, 5, 4, d), full(2, 0, 2, d), full(2, 0, 2, d)
        dq, _, _ = attn.prefill_backward(full(2, 5, 4, d), full(2, 5, 4, d), e(2, 0, 2, d), e(2, 0, 2, d),
                                         e(2, 5, 4, d), torch.full((2, 4, 5), -math.inf, device="cuda"), out=out)
        assert (dq == 0).all()
        out = e(2, 0, 4, d), full(2, 5, 2, d), full(2, 5, 2, d)
        _, dk, dv = attn.prefill_backward(e(2, 0, 4, d), e(2, 0, 4, d), full(2, 5, 2, d), full(2, 5, 2, d),
                                          e(2, 0, 4, d), torch.zeros(2, 4, 0, device="cuda"), out=out)
        assert (dk == 0).all() and (dv == 0).all()
        out = attn.prefill_backward(*(e(0, 5, 4, d) for _ in range(2)), *(e(0, 5, 2, d) for _ in range(2)),
                                    e(0, 5, 4, d), torch.zeros(0, 4, 5, device="cuda"))
        assert out[0].shape == (0, 5, 4, d)
        # packed rows, none of them of a sequence
        cu, kl = torch.zeros(3, dtype=torch.int32).cuda(), torch.tensor([3, 0], dtype=torch.int32).cuda()
        out = attn.prefill_varlen_backward(full(4, 4, d), full(4, 4, d), full(2, 6, 2, d), full(2, 6, 2, d),
                                           full(4, 4, d), torch.zeros(4, 4, device="cuda"), cu, kl, 0)
        assert all((t == 0).all() for t in out)
    attn.sync_check()


@pytest.mark.gpu
def test_packed_rows_of_no_sequences_at_all():
    torch.full((1 << 20,), 3.0, device="cuda")  # (what the outputs' memory may hold)
    full = lambda *s: torch.full(s, 3.0, dtype=torch.bfloat16, device="cuda")
    cu, kl = torch.zeros(1, dtype=torch.int32).cuda(), torch.zeros(0, dtype=torch.int32).cuda()
    args = (full(5, 4, 64), full(5, 4, 64), full(0, 6, 2, 64), full(0, 6, 2, 64), full(5, 4, 64),
            torch.zeros(4, 5, device="cuda"), cu, kl, 0)
    out = attn.prefill_varlen_backward(*args)
    assert (out[0] == 0).all() and out[1].shape == out[2].shape == (0, 6, 2, 64)
    given = full(5, 4, 64), full(0, 6, 2, 64), full(0, 6, 2, 64)
    attn.prefill_varlen_backward(*args, out=given)
    assert (given[0] == 3).all()
    attn.sync_check()


@pytest.mark.gpu
@pytest.mark.parametrize("d,window,sink", [(64, 0, 0), (128, 40, 2)])
def test_against_differences(d, window, sink):
    """dL/dx . u against (L(x + h u) - L(x - h u)) / 2h of the fp64 forward, L = <o, do> + <lse, dlse>,
    through the package's own forward call.  The directional derivative is a sum of n bounded
    terms, so its bound is the elementwise one summed with |u|, plus what o in bf16 (2^-8 of it,
    in D) and lse in fp32 leave: 2^-8 sum P sum |g||o| and its products; the differences' own
    error at h = 1e-4 is below 1e-6 of the terms."""
    B, Hq, Hkv, S = 1, 4, 2, 150
    q, k, v, do = (t.cuda() for t in _inputs(B, Hq, Hkv, S, S, d, 11, spread=1.0))
    dl = torch.randn(B, Hq, S, generator=torch.Generator().manual_seed(2)).cuda()
    sc = 1 / math.sqrt(d)
    if window:
        o, lse = attn.prefill_window(q, k, v, window, sink, out_dtype=torch.float32)
    else:
        o, lse = attn.prefill(q, k, v, out_dtype=torch.float32)
    got = attn.prefill_backward(do, q, k, v, o, lse, window=window, n_sink=sink, dlse=dl)
    attn.sync_check()
    ok = _mask(S, S, True, window, sink, "cuda")
    want, bound = _reference(do[0], q[0], k[0], v[0], o[0], lse[0], dl[0], ok, sc)

    def loss(q, k, v):
        o, lse = _forward(q, k, v, ok, sc)
        return (o * do[0].double()).sum() + (lse * dl[0].double()).sum()

    x = [t[0].double() for t in (q, k, v)]
    # the forward's o is within 5e-3 of the exact one (P in bf16): its share of D
    dO = 5e-3 * do[0].double().abs().sum(-1).T
    G = Hq // Hkv
    p = torch.exp(torch.einsum("ihd,jhd->hij", x[0], x[1].repeat_interleave(G, 1)) * sc - lse[0].double()[..., None])
    p = torch.where(ok, p, 0.0) * dO[..., None] * sc
    more = (torch.einsum("hij,jhd->ihd", p, x[1].abs().repeat_interleave(G, 1)),
            torch.einsum("hij,ihd->jhd", p, x[0].abs()).unflatten(1, (Hkv, G)).sum(2), torch.zeros_like(x[2]))
    for i in range(3):
        u = torch.randn(x[i].shape, generator=torch.Generator().manual_seed(20 + i), dtype=torch.float64).cuda()
        h = 1e-4
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + h * u, x[i] - h * u
        diff = (loss(*up) - loss(*down)) / (2 * h)
        mine = (got[i][0].double() * u).sum()
        tol = ((bound[i] + more[i]) * u.abs()).sum() + 1e-6 * (want[i].abs() * u.abs()).sum()
        assert (mine - diff).abs() <= tol
        # and far nearer than that bound, which adds every error with the same sign
        assert (mine - diff).abs() <= 0.02 * ((want[i] * u).square().sum().sqrt() + want[i].norm())


@pytest.mark.gpu
def test_same_bits_each_time():
    q, k, v, do = (t.cuda() for t in _inputs(1, 8, 2, 900, 900, 128, 5))
    o, lse = attn.prefill_window(q, k, v, 200, 4)
    a = attn.prefill_backward(do, q, k, v, o, lse, window=200, n_sink=4)
    junk = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")  # the next workspace may be any memory
    del junk
    b = attn.prefill_backward(do, q, k, v, o, lse, window=200, n_sink=4)
    attn.sync_check()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


FEW = [  # B, Hq, Hkv, Sq, Skv, causal, window, sink: at most 131072 rows x heads x admitted keys
    (3, 8, 1, 3, 3, True, 0, 0), (1, 4, 4, 2, 2, True, 0, 0), (1, 8, 2, 17, 200, True, 20, 1), (1, 4, 2, 64, 256, False, 0, 0),
    (1, 6, 2, 64, 64, True, 9, 3), (1, 2, 1, 1, 256, True, 0, 0), (1, 4, 2, 63, 129, True, 0, 0), (5, 4, 1, 40, 33, True, 0, 0),
    (1, 2, 1, 1500, 1500, True, 12, 2), (2, 4, 1, 1, 8000, True, 0, 0), (1, 1, 1, 300, 200, True, 0, 0), (4, 32, 8, 16, 64, True, 0, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", FEW, ids=lambda c: "-".join(map(str, c)))
def test_few_pairs_show_no_rounding_of_terms(case, d):
    """P and dS enter their products as two terms (2^-17 of each left out), so that a gradient is off by
    its own rounding, 2^-8 of it, and by far less of the sum of its terms' magnitudes: 2^-16 for the terms,
    2^-20 for exponentials and fp32 sums.  In D and dP the same happens before the difference dP - D:
    2^-20 of what they are sums of, in every term."""
    B, Hq, Hkv, Sq, Skv, causal, window, sink = case
    q, k, v, do = (t.cuda() for t in _inputs(B, Hq, Hkv, Sq, Skv, d, 31))
    sc, G = 1 / math.sqrt(d), Hq // Hkv
    ok = _mask(Sq, Skv, causal, window, sink, "cuda")
    o, lse = torch.empty(q.shape, device="cuda"), torch.empty(B, Hq, Sq, device="cuda")
    for b in range(B):
        x, y = _forward(q[b], k[b], v[b], ok, sc)
        o[b], lse[b] = x.float(), y.float()
    for fixed in (True, False):
        if fixed:
            got = attn.prefill_backward(do, q, k, v, o, lse, causal=causal, window=window, n_sink=sink)
        else:
            cu = torch.arange(B + 1, dtype=torch.int32).cuda() * Sq
            flat = lambda t: t.reshape(B * Sq, Hq, d)
            got = attn.prefill_varlen_backward(flat(do), flat(q), k, v, flat(o),
                                               lse.transpose(0, 1).reshape(Hq, B * Sq).contiguous(), cu,
                                               torch.full((B,), Skv, dtype=torch.int32).cuda(), Sq, causal=causal,
                                               window=window, n_sink=sink)
            got = got[0].view(q.shape), got[1], got[2]
        attn.sync_check()
        for b in range(B):
            x, kk, vv, g = (t[b].double() for t in (q, k, v, do))
            kr, vr = kk.repeat_interleave(G, 1), vv.repeat_interleave(G, 1)
            l = lse[b].double()[..., None]
            p = torch.exp(torch.einsum("ihd,jhd->hij", x, kr) * sc - torch.where(l.isinf(), 0.0, l))
            p = torch.where(ok & ~l.isinf(), p, 0.0)
            dd = (g * o[b].double()).sum(-1).T[..., None]
            dp = torch.einsum("ihd,jhd->hij", g, vr)
            ds = p * (dp - dd)
            # off by: two terms of it, and 2^-20 of what P's exponent, dP and D are made of
            size = torch.einsum("ihd,jhd->hij", g.abs(), vr.abs()) + (g * o[b].double()).abs().sum(-1).T[..., None]
            expo = torch.einsum("ihd,jhd->hij", x.abs(), kr.abs()) * sc + torch.where(l.isinf(), 0.0, l).abs() + 1
            dp_off = p * 2.0 ** -16 + p * expo * 2.0 ** -20
            ds_off = ds.abs() * 2.0 ** -16 + ds.abs() * expo * 2.0 ** -20 + p * size * 2.0 ** -20
            fold = lambda t: t.unflatten(1, (Hkv, G)).sum(2)
            want = (torch.einsum("hij,jhd->ihd", ds, kr) * sc, fold(torch.einsum("hij,ihd->jhd", ds, x)) * sc,
                    fold(torch.einsum("hij,ihd->jhd", p, g)))
            off = (torch.einsum("hij,jhd->ihd", ds_off, kr.abs()) * sc,
                   fold(torch.einsum("hij,ihd->jhd", ds_off, x.abs())) * sc,
                   fold(torch.einsum("hij,ihd->jhd", dp_off, g.abs())))
            for i, name in enumerate(("dq", "dk", "dv")):
                bad = (got[i][b].double() - want[i]).abs() > want[i].abs() * 2.0 ** -8 + off[i] * 1.01 + 1e-30
                assert not bad.any(), (name, int(bad.sum()))
