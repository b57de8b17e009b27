"""The rotations, the windowed attention and their gradients together, as a training step makes
them, and a windowed serving loop over pages whose far pages are given back."""
import math
import threading

import pytest
import torch

import attention_forward_tcgen05_gb300 as attn
from tests.test_prefill_backward import F, R, _forward, _mask, _reference, _within

pytestmark = pytest.mark.gpu


def _turn(x, pos, f, axes, sign=1.0):
    """fp64 rotation of x [T,H,d] (pairs m, m + rot/2) by pos [A,T]."""
    rot = 2 * f.shape[0]
    a = pos.double()[axes.long()].T * f * sign
    c, s = a.cos()[:, None], a.sin()[:, None]
    x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
    return torch.cat((x1 * c - x2 * s, x1 * s + x2 * c, x[..., rot:]), -1)


class Step:
    """One attention layer's part of a training step on [B,S] tokens with three positions each."""

    def __init__(self, B, S, Hq, Hkv, d, window, sink, seed):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
        self.shape, self.window, self.sink = (B, S, Hq, Hkv, d), window, sink
        self.q, self.k, self.v = rnd(B, S, Hq, d), rnd(B, S, Hkv, d), rnd(B, S, Hkv, d)
        self.do = rnd(B, S, Hq, d)
        self.f, self.axes = attn.rope_axes((d // 8, d // 8, d // 4))
        self.pos = torch.randint(0, 3000, (3, B * S), generator=g, dtype=torch.int32).cuda()

    def run(self):
        B, S, Hq, Hkv, d = self.shape
        qr, kr = attn.rope_rotate(self.q.flatten(0, 1), self.k.flatten(0, 1), self.f, self.pos, axes=self.axes)
        qr, kr = qr.view_as(self.q), kr.view_as(self.k)
        o, lse = attn.prefill_window(qr, kr, self.v, self.window, self.sink)
        dqr, dkr, dv = attn.prefill_backward(self.do, qr, kr, self.v, o, lse, window=self.window, n_sink=self.sink)
        dq, dk = attn.rope_rotate(dqr.flatten(0, 1), dkr.flatten(0, 1), self.f, self.pos, axes=self.axes, inverse=True)
        return o, lse, dq.view_as(self.q), dk.view_as(self.k), dv

    def exact(self):
        """(o, dq, dk, dv) of the whole chain in fp64, by torch's own differentiation."""
        B, S, Hq, Hkv, d = self.shape
        ok = _mask(S, S, True, self.window, self.sink, "cuda")
        leaves = [t.double().requires_grad_() for t in (self.q, self.k, self.v)]
        q = _turn(leaves[0].flatten(0, 1), self.pos, self.f, self.axes).view(B, S, Hq, d)
        k = _turn(leaves[1].flatten(0, 1), self.pos, self.f, self.axes).view(B, S, Hkv, d)
        G = Hq // Hkv
        s = torch.einsum("bihd,bjhd->bhij", q, k.repeat_interleave(G, 2)) / math.sqrt(d)
        p = s.masked_fill(~ok, -math.inf).softmax(-1)
        o = torch.einsum("bhij,bjhd->bihd", p, leaves[2].repeat_interleave(G, 2))
        return (o.detach(), *torch.autograd.grad((o * self.do.double()).sum(), leaves))


def _near(got, want, what):
    """Relative distance in the 2-norm.  The chain rounds to bf16 at seven places (q and k
    rotated, P and o forward, P and dS backward, the gradients twice), each by at most 2^-8 of a
    value, independently: 2^-8 * sqrt(7 / 3) of the norm for sums without cancellation; scores'
    errors (2^-8 of 1 from the rotated q and k, times a spread of the scores of about 1) enter P and
    dS once more each.  2^-5 leaves a factor of three; a wrong sign, scale, axis or mask is off by
    more than 2^-2."""
    rel = ((got.double() - want).norm() / want.norm()).item()
    assert rel <= 2.0 ** -5, f"{what}: {rel:.2e}"


@pytest.mark.parametrize("case", [(2, 300, 4, 2, 64, 90, 4), (1, 700, 14, 2, 128, 256, 1), (3, 129, 2, 2, 128, 1000, 0)])
def test_training_step(case):
    step = Step(*case, seed=5)
    o, lse, dq, dk, dv = step.run()
    attn.sync_check()
    for got, want, what in zip((o, dq, dk, dv), step.exact(), ("o", "dq", "dk", "dv")):
        _near(got, want, what)


def test_training_step_in_a_graph_and_on_two_streams():
    """Replays on new inputs, with eager steps of other tensors on another stream at the same time."""
    a, b = Step(2, 260, 4, 2, 64, 90, 4, seed=6), Step(2, 260, 4, 2, 64, 90, 4, seed=7)
    want = [[t.clone() for t in s.run()] for s in (a, b)]
    attn.sync_check()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        got = a.run()
    inputs = [[t.clone() for t in (s.q, s.k, s.v, s.do, s.pos)] for s in (a, b)]
    for x, w in ((inputs[1], want[1]), (inputs[0], want[0]), (inputs[1], want[1])):
        for dst, src in zip((a.q, a.k, a.v, a.do, a.pos), x):
            dst.copy_(src)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            other = b.run()
        torch.cuda.synchronize()
        assert all(torch.equal(g, e) for g, e in zip(got, w))
        assert all(torch.equal(g, e) for g, e in zip(other, want[1]))
    attn.sync_check()


def test_threads_on_one_stream():
    """Calls of several threads on the same stream share its kept workspace and keep their results, small
    calls beside ones whose workspace is larger."""
    g = torch.Generator().manual_seed(8)
    sets = []
    for i, (S, H, d) in enumerate(((40, 4, 64), (700, 8, 128), (333, 2, 64), (1500, 4, 128))):
        q, do = ((torch.randn(1, S, H, d, generator=g)).bfloat16().cuda() for _ in range(2))
        k, v = ((torch.randn(1, S, 2, d, generator=g)).bfloat16().cuda() for _ in range(2))
        o, lse = attn.prefill(q, k, v)
        sets.append((do, q, k, v, o, lse))
    want = [attn.prefill_backward(*x) for x in sets]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        for _ in range(25):
            got = attn.prefill_backward(*sets[i])
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    attn.sync_check()
    assert not bad


def test_a_stream_given():
    s = Step(1, 300, 4, 1, 128, 64, 2, seed=8)
    o, lse, *_ = want = s.run()
    qr, kr = attn.rope_rotate(s.q.flatten(0, 1), s.k.flatten(0, 1), s.f, s.pos, axes=s.axes)
    qr, kr = qr.view_as(s.q), kr.view_as(s.k)
    side = torch.cuda.Stream()
    plain = attn.prefill_backward(s.do, qr, kr, s.v, o, lse, window=64, n_sink=2)
    side.wait_stream(torch.cuda.current_stream())
    got = attn.prefill_backward(s.do, qr, kr, s.v, o, lse, window=64, n_sink=2, stream=side)
    out = tuple(torch.empty_like(t) for t in (s.q, s.k, s.v))
    attn.prefill_backward(s.do, qr, kr, s.v, o, lse, window=64, n_sink=2, stream=side, out=out)
    side.synchronize()
    assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(plain, got, out))
    assert torch.equal(plain[2], want[4])
    attn.sync_check()


def test_rows_past_four_billion_bytes():
    """q, do, o and dq of 4.6 GB each (offsets above 2^32 bytes and 2^31 elements), one group of 128
    heads: the last rows and keys against the formula over the end alone, which a short window
    allows."""
    S, H, d, win, n = 140000, 128, 128, 64, 320
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)
    q, k, v, do = rnd(1, S, H, d), rnd(1, S, 1, d), rnd(1, S, 1, d), rnd(1, S, H, d)
    o, lse = attn.prefill_window(q, k, v, win)
    dq, dk, dv = attn.prefill_backward(do, q, k, v, o, lse, window=win)
    attn.sync_check()
    ok = _mask(n, n, True, win, 0, "cuda")
    ok[:win] = False  # rows whose window begins before the slice
    cut = lambda t: t[0, -n:]
    want, bound = _reference(cut(do), cut(q), cut(k), cut(v), cut(o), lse[0, :, -n:], None, ok, 1 / math.sqrt(d))
    keep = 2 * win  # rows and keys that only rows of the slice concern
    _within(cut(dq)[keep:], want[0][keep:], bound[0][keep:], "dq")
    _within(cut(dk)[keep:], want[1][keep:], bound[1][keep:], "dk")
    _within(cut(dv)[keep:], want[2][keep:], bound[2][keep:], "dv")


def test_windowed_serving_loop():
    """A prompt with three positions a token, then tokens one by one, over pages; pages behind the
    window leave the table after every step.  Each output against fp64 attention over the rotated,
    rounded keys: P in bf16 for the prompt (R of it, relative to |v|), in two terms for the tokens."""
    B, Hq, Hkv, d, page, window, sink, n_new = 2, 8, 2, 64, 16, 70, 3, 40
    g = torch.Generator().manual_seed(4)
    prompt = [133, 50]
    total = [p + n_new for p in prompt]
    f, axes = attn.rope_axes((8, 12, 12), layout="dealt")
    x = [torch.randn(t, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda() for t in total]
    pos = [torch.randint(0, 500, (3, t), generator=g, dtype=torch.int32).cuda() for t in total]
    width = -(-max(total) // page)
    table = torch.arange(B * width, dtype=torch.int32).view(B, width)[:, torch.randperm(width, generator=g)].contiguous().cuda()
    kp = torch.full((B * width, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    scale = 1 / math.sqrt(d)
    rot = [_turn(t.double(), p, f, axes) for t, p in zip(x, pos)]
    rq = [r[:, :Hq].bfloat16() for r in rot]
    rk = [r[:, Hq:Hq + Hkv].bfloat16() for r in rot]

    def check(o, b, rows, err):
        L = rows.stop
        ok = _mask(L, L, True, window, sink, "cuda")[rows]
        v = x[b][:L, Hq + Hkv:]
        want, _ = _forward(rq[b][rows], rk[b][:L], v, ok, scale)
        mag, _ = _forward(rq[b][rows], rk[b][:L], v.abs(), ok, scale)
        # rotated q and k may round to the next bf16 value here and there: a score moves by up to
        # scale * 2^-8 * sum |q||k|; below 0.05 for these, of which e^0.05 - 1 reaches P
        assert ((o.double() - want).abs() <= (err + 0.06) * mag + R * want.abs()).all()
        assert ((o.double() - want).norm() / want.norm()).item() <= 0.01

    lens = torch.tensor(prompt, dtype=torch.int32).cuda()
    cu = torch.tensor([0, prompt[0], sum(prompt)], dtype=torch.int32).cuda()
    rows = torch.cat([t[:p] for t, p in zip(x, prompt)])
    q = attn.rope_append(rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], kp, vp, lens, f, page_table=table,
                         cu_seqlens_q=cu, positions=torch.cat([p[:, :n] for p, n in zip(pos, prompt)], 1).contiguous(),
                         axes=axes)
    o, _ = attn.prefill_paged(q, kp, vp, table, cu, lens, max(prompt), window=window, n_sink=sink)
    attn.sync_check()
    for b in range(B):
        check(o[cu[b]:cu[b + 1]], b, slice(0, prompt[b]), R + F)
    for i in range(n_new):
        lens += 1
        rows = torch.stack([t[p + i] for t, p in zip(x, prompt)])
        q = attn.rope_append(rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], kp, vp, lens, f, page_table=table,
                             positions=torch.stack([p[:, n + i] for p, n in zip(pos, prompt)], 1).contiguous(), axes=axes)
        o, _ = attn.decode_window(q, kp, vp, lens, window, sink, page_table=table)
        attn.sync_check()
        for b in range(B):
            L = prompt[b] + i + 1
            check(o[b:b + 1], b, slice(L - 1, L), 2.0 ** -16)
            for e in range(width):  # given back: out of the next window, no sink in it
                if e * page >= sink and (e + 1) * page <= L + 1 - window and table[b, e] >= 0:
                    kp[table[b, e]], vp[table[b, e]] = float("nan"), float("nan")
                    table[b, e] = -1
    assert (table < 0).any()
