"""The two forms of the prefill's gradients: P and dS as two bf16 terms each in sequences of few pairs
of a row and a key, as one in others (include/attn.h).  Which one it is goes by the sequence's own
pairs, not by the batch, the heads or the cache around it.

Bounds: of one term, those of test_prefill_backward.  Of two, a gradient is off by its own
rounding, 2^-8 of it, and by far less of the sum of its terms' magnitudes: 2^-16 for the terms (2^-17 of P
and of dS left out), 2^-20 for exponentials and fp32 sums, and before the difference dP - D 2^-20 of what
the two are sums of, in every term.  One term cannot keep the second bound: its rounding of up to
2^-8 a term is 2^8 of it, and shows wherever a gradient is small beside its terms.
"""
import math

import pytest
import torch

import attention_forward_tcgen05_gb300 as attn
from tests.test_prefill_backward import _forward, _mask, _reference, _within

LIMIT = 24576


def pairs(rows, keys, causal=True, window=0, sink=0):
    """Pairs of a row and a key by which a sequence has one form or the other."""
    n = min(rows, keys) if causal else rows
    p = n * (keys - n) + n * (n + 1) // 2 if causal else n * keys
    return min(p, rows * (window + sink)) if window else p


def _tight(do, q, k, v, o, lse, dlse, ok, scale):
    """Bounds of two terms beside the gradients' own rounding."""
    Hkv = k.shape[1]
    G = q.shape[1] // Hkv
    x, g, kr, vr = q.double(), do.double(), *(t.double().repeat_interleave(G, 1) for t in (k, v))
    l = lse.double()[..., None]
    p = torch.exp(torch.einsum("ihd,jhd->hij", x, kr) * scale - torch.where(l.isinf(), 0.0, l))
    p = torch.where(ok & ~l.isinf(), p, 0.0)
    D = (g * o.double()).sum(-1).T[..., None]
    if dlse is not None:
        D = D - dlse.double()[..., None]
    ds = p * (torch.einsum("ihd,jhd->hij", g, vr) - D)
    size = torch.einsum("ihd,jhd->hij", g.abs(), vr.abs()) + (g * o.double()).abs().sum(-1).T[..., None]
    if dlse is not None:
        size = size + dlse.double().abs()[..., None]
    expo = torch.einsum("ihd,jhd->hij", x.abs(), kr.abs()) * scale + torch.where(l.isinf(), 0.0, l).abs() + 1
    p_off = p * 2.0 ** -16 + p * expo * 2.0 ** -20
    ds_off = ds.abs() * 2.0 ** -16 + ds.abs() * expo * 2.0 ** -20 + p * size * 2.0 ** -20
    fold = lambda t: t.unflatten(1, (Hkv, G)).sum(2)
    off = (torch.einsum("hij,jhd->ihd", ds_off, kr.abs()) * scale, fold(torch.einsum("hij,ihd->jhd", ds_off, x.abs())) * scale,
           fold(torch.einsum("hij,ihd->jhd", p_off, g.abs())))
    return off


class Batch:
    """Sequences of lens_q new rows over lens_k keys, and each one's gradients in fp64 with the bounds of
    either form."""

    def __init__(self, lens_q, lens_k, Hq, Hkv, d, causal=True, window=0, sink=0, o_dtype=torch.bfloat16, dlse=False,
                 seed=7):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.lens_q, self.lens_k, self.Hq, self.Hkv, self.d = list(lens_q), list(lens_k), Hq, Hkv, d
        self.mask = dict(causal=causal, window=window, n_sink=sink)
        self.seqs = []
        scale = 1 / math.sqrt(d)
        for n, L in zip(lens_q, lens_k):
            q, do = (rnd(n, Hq, d) * 1.5).bfloat16(), rnd(n, Hq, d).bfloat16()
            k, v = rnd(L, Hkv, d).bfloat16(), rnd(L, Hkv, d).bfloat16()
            ok = _mask(n, L, causal, window, sink, "cuda")
            o, lse = _forward(q, k, v, ok, scale)
            o, lse = o.to(o_dtype), lse.float()
            dl = rnd(Hq, n) if dlse else None
            want, one = _reference(do, q, k, v, o, lse, dl, ok, scale)
            two = [w.abs() * 2.0 ** -8 + 1.01 * t for w, t in zip(want, _tight(do, q, k, v, o, lse, dl, ok, scale))]
            few = pairs(n, L, causal, window, sink) <= LIMIT
            self.seqs.append(dict(q=q, do=do, k=k, v=v, o=o, lse=lse, dl=dl, want=want, one=one, two=two, few=few))

    def packed(self, max_kv=None, first=0, spare=0, give_out=False, **kw):
        """first, spare: rows of no sequence before and behind, which with the slots behind a sequence's keys
        hold NaN."""
        max_kv = max_kv or max(self.lens_k)
        nan = lambda *s, dtype=torch.bfloat16: torch.full(s, math.nan, dtype=dtype, device="cuda")

        def rows(name):
            x = [s[name] for s in self.seqs]
            return torch.cat([nan(first, self.Hq, self.d, dtype=x[0].dtype), *x, nan(spare, self.Hq, self.d, dtype=x[0].dtype)])

        def stats(name):
            if self.seqs[0][name] is None:
                return None
            f = lambda n: nan(self.Hq, n, dtype=torch.float32)
            return torch.cat([f(first), *(s[name] for s in self.seqs), f(spare)], 1).contiguous()

        cache = lambda name: torch.stack([torch.cat([s[name], nan(max_kv - s[name].shape[0], self.Hkv, self.d)])
                                          for s in self.seqs])
        cu = torch.zeros(len(self.seqs) + 1, dtype=torch.int32)
        cu[1:] = torch.cumsum(torch.tensor(self.lens_q), 0)
        cu += first
        q, k = rows("q"), cache("k")
        out = tuple(torch.full_like(t, 7.0) for t in (q, k, k)) if give_out else None
        dq, dk, dv = attn.prefill_varlen_backward(rows("do"), q, k, cache("v"), rows("o"), stats("lse"), cu.cuda(),
                                                  torch.tensor(self.lens_k, dtype=torch.int32).cuda(),
                                                  max(self.lens_q), dlse=stats("dl"), out=out, **self.mask, **kw)
        attn.sync_check()
        rest = 7.0 if give_out else 0.0
        assert (dq[:first] == rest).all() and (dq[int(cu[-1]):] == rest).all()
        for b, L in enumerate(self.lens_k):
            assert (dk[b, L:] == rest).all() and (dv[b, L:] == rest).all()
        return [(dq[cu[b]:cu[b + 1]], dk[b, :L], dv[b, :L]) for b, L in enumerate(self.lens_k)]

    def fixed(self, **kw):
        st = lambda name: None if self.seqs[0][name] is None else torch.stack([s[name] for s in self.seqs])
        got = attn.prefill_backward(st("do"), st("q"), st("k"), st("v"), st("o"), st("lse"), dlse=st("dl"), **self.mask, **kw)
        attn.sync_check()
        return list(zip(*got))

    def check(self, got):
        """Every sequence within its form's bound, and those of one term not within that of two."""
        for b, (s, out) in enumerate(zip(self.seqs, got)):
            beyond = 0
            for name, x, w, one, two in zip(("dq", "dk", "dv"), out, s["want"], s["one"], s["two"]):
                _within(x, w, two if s["few"] else one, f"{name} of sequence {b}")
                beyond += int(((x.double() - w).abs() > two + 1e-30).sum())
            assert s["few"] or beyond, f"sequence {b} is not of one term"


OWN = [  # sequences of few pairs each: alone, many of them, in a cache far longer than they are
    (dict(lens_q=[5] * 200, lens_k=[5] * 200, Hq=32, Hkv=8, d=64), None),
    (dict(lens_q=[5] * 200, lens_k=[5] * 200, Hq=32, Hkv=8, d=128), None),
    (dict(lens_q=[5], lens_k=[5], Hq=28, Hkv=4, d=128), 4096),
    (dict(lens_q=[64] * 6, lens_k=[64] * 6, Hq=28, Hkv=4, d=64, window=9, sink=3), None),
    (dict(lens_q=[64, 1, 30], lens_k=[200, 900, 30], Hq=16, Hkv=4, d=128, dlse=True), 1100),
    (dict(lens_q=[128] * 3, lens_k=[128] * 3, Hq=32, Hkv=8, d=64, causal=False), None),
]


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(OWN)))
def test_few_pairs_whatever_is_around_them(i):
    kw, max_kv = OWN[i]
    x = Batch(**kw, o_dtype=torch.float32)
    assert all(s["few"] for s in x.seqs)
    x.check(x.packed(max_kv))
    if len({*zip(x.lens_q, x.lens_k)}) == 1:
        x.check(x.fixed())


EDGE = [  # just below the limit and just above it
    (dict(causal=False), (64, 384), (64, 385)), (dict(), (221, 221), (222, 222)), (dict(), (96, 303), (96, 304)),
    (dict(), (300, 221), (300, 222)), (dict(window=40, sink=8), (512, 600), (513, 600)), (dict(), (1, 24576), (1, 24577)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("i", range(len(EDGE)))
def test_limit(i, d):
    kw, below, above = EDGE[i]
    for (n, L), few in ((below, True), (above, False)):
        x = Batch([n, n], [L, L], 4, 2, d, **kw)
        assert [s["few"] for s in x.seqs] == [few, few]
        x.check(x.fixed())
        x.check(x.packed())


MIXED = [
    dict(lens_q=[5, 700, 64, 300, 1], lens_k=[5, 700, 64, 420, 3000], Hq=8, Hkv=2, d=128),
    dict(lens_q=[300, 5, 64, 700], lens_k=[420, 40, 64, 700], Hq=4, Hkv=4, d=64),
    dict(lens_q=[31] * 20 + [900], lens_k=[40] * 20 + [1000], Hq=4, Hkv=2, d=64, window=100, sink=3, dlse=True),
    dict(lens_q=[900, 0, 130, 17], lens_k=[900, 50, 130, 0], Hq=7, Hkv=1, d=128, window=128, sink=1, dlse=True),
    dict(lens_q=[129, 20, 257], lens_k=[300, 100, 128], Hq=4, Hkv=2, d=64, causal=False),
    dict(lens_q=[129, 20, 257], lens_k=[300, 100, 128], Hq=4, Hkv=2, d=128, causal=False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("o_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("i", range(len(MIXED)))
def test_both_forms_in_one_batch(i, o_dtype):
    x = Batch(**MIXED[i], o_dtype=o_dtype)
    assert {s["few"] for s in x.seqs} == {True, False}
    x.check(x.packed(max(x.lens_k) + 77))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_a_graph_replayed_with_other_lengths(d):
    """The lengths are read when the call runs: a replay has each sequence in its form of then."""
    first = dict(lens_q=[700, 5, 300, 64], lens_k=[700, 90, 300, 64])
    then = dict(lens_q=[5, 700, 64, 300], lens_k=[90, 700, 64, 300])
    a, b = Batch(**first, Hq=4, Hkv=2, d=d), Batch(**then, Hq=4, Hkv=2, d=d, seed=8)

    def tensors(x):
        pad = lambda t: torch.cat([t, t.new_zeros(700 - t.shape[0], *t.shape[1:])])
        cat = lambda n, dim=0: torch.cat([s[n] for s in x.seqs], dim).contiguous()
        cu = torch.zeros(5, dtype=torch.int32)
        cu[1:] = torch.cumsum(torch.tensor(x.lens_q), 0)
        return [cat("do"), cat("q"), *(torch.stack([pad(s[n]) for s in x.seqs]) for n in "kv"), cat("o"), cat("lse", 1),
                cu.cuda(), torch.tensor(x.lens_k, dtype=torch.int32).cuda()]

    def outputs(x, got):
        cu = [sum(x.lens_q[:i]) for i in range(5)]
        return [(got[0][cu[i]:cu[i + 1]], got[1][i, :L], got[2][i, :L]) for i, L in enumerate(x.lens_k)]

    args = tensors(a)
    a.check(outputs(a, attn.prefill_varlen_backward(*args, 700)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = attn.prefill_varlen_backward(*args, 700)
    for x in (a, b, a):
        for t, new in zip(args, tensors(x)):
            t.copy_(new)
        graph.replay()
        attn.sync_check()
        x.check(outputs(x, got))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_many_short_and_empty_sequences_between_long_ones(d):
    x = Batch([300] + [0] * 200 + [8] * 100 + [0] * 100 + [300, 1], [300] + [9] * 200 + [8] * 100 + [0] * 100 + [340, 60], 4, 2, d)
    x.check(x.packed(400, first=3, spare=2))


@pytest.mark.gpu
def test_time_beside_many_short_and_empty_sequences():
    """Item lists are searched, not walked, where sequences have no items of a form: 1 and 2.2 ms here (one by
    one, 26 and 41 ms)."""
    for between in (0, 8):
        lens = [2000] + [between] * 4000 + [2000]
        B, T, mk = len(lens), sum(lens), 2000
        z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
        cu = torch.tensor([0] + lens).cumsum(0).int().cuda()
        q, k, lse = z(T, 4, 64), z(B, mk, 2, 64), torch.full((4, T), 7.0, device="cuda")
        out = z(T, 4, 64), z(B, mk, 2, 64), z(B, mk, 2, 64)
        call = lambda: attn.prefill_varlen_backward(q, q, k, k, q, lse, cu, torch.tensor(lens).int().cuda(), mk, out=out)
        call()
        times = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda.synchronize()
            a.record()
            call()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        attn.sync_check()
        assert sorted(times)[2] < 10.0, times
