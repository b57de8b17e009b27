"""The paged calls together, as a serving loop makes them: prompts in chunks, single tokens,
key weights after each call, eviction in between; then captured into graphs, on other
streams and two at a time."""
import math

import numpy as np
import pytest
import torch

import attention_forward_tcgen05_gb300 as attn
from tests.paged_cases import admitted
from tests.test_evict import kept_ref
from tests.test_rope_append import rotate
from tests.tolerances import check_lse, check_o

pytestmark = pytest.mark.gpu

Hq, Hkv, d, G = 8, 2, 64, 4
ROT = 32


class Model:
    """The loop's state in fp64: each sequence's keys, values and weights per KV head."""

    def __init__(self, B, freq):
        self.k = [[np.zeros((0, d))] * Hkv for _ in range(B)]
        self.v = [[np.zeros((0, d))] * Hkv for _ in range(B)]
        self.w = [[np.zeros(0)] * Hkv for _ in range(B)]
        self.seen = [0] * B  # tokens so far: positions go on after an eviction
        self.freq = freq

    def step(self, b, q, k, v):
        """New rows of sequence b (as the cache holds them: k rounded to bf16): o, lse."""
        n = q.shape[0]
        o, lse = np.zeros((n, Hq, d)), np.zeros((Hq, n))
        for hk in range(Hkv):
            self.k[b][hk] = np.concatenate([self.k[b][hk], k[:, hk]])
            self.v[b][hk] = np.concatenate([self.v[b][hk], v[:, hk]])
            L = len(self.k[b][hk])
            w = np.concatenate([self.w[b][hk], np.zeros(n)])
            ok = admitted(n, L, True)
            for h in range(hk * G, (hk + 1) * G):
                s = np.where(ok, q[:, h] @ self.k[b][hk].T / math.sqrt(d), -np.inf)
                lse[h] = np.log(np.exp(s).sum(1))
                p = np.exp(s - lse[h][:, None])
                o[:, h] = p @ self.v[b][hk]
                w += p.sum(0)
            self.w[b][hk] = w
        self.seen[b] += n
        return o, lse

    def keep(self, b, hk, idx):
        self.k[b][hk], self.v[b][hk], self.w[b][hk] = (x[b][hk][idx] for x in (self.k, self.v, self.w))


def test_serving_loop():
    B, page, cap = 3, 16, 256
    rng = np.random.default_rng(7)
    freq, amp = attn.rope_frequencies(ROT, device="cuda")
    m = Model(B, freq.cpu().numpy())
    table = torch.from_numpy(rng.permutation(B * cap // page).astype(np.int32)).view(B, -1).cuda()
    kc = torch.full((B * cap // page, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    w = torch.zeros(B, Hkv, cap, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    steps = [("chunk", [40, 100, 7]), ("chunk", [64, 0, 130]), ("one",), ("evict", 60), ("one",), ("one",),
             ("chunk", [20, 33, 1]), ("evict", 48), ("one",)]
    for step in steps:
        if step[0] == "evict":
            N, recent, sink = step[1], 8, 2
            before = w.cpu().numpy()
            kept, _ = attn.evict(w, kc, vc, lens, N, recent, sink, page_table=table, out=(
                torch.empty(B, Hkv, N, dtype=torch.int32, device="cuda"), lens))
            attn.sync_check()
            for b in range(B):
                for hk in range(Hkv):
                    L = len(m.k[b][hk])
                    idx = kept_ref(before[b, hk], L, N, recent, sink)  # by the weights the kernel had
                    assert np.array_equal(kept[b, hk, :len(idx)].cpu().numpy(), idx)
                    m.keep(b, hk, idx)
                assert lens[b].item() == len(m.k[b][0])
            continue
        new = step[1] if step[0] == "chunk" else [1] * B
        T = sum(new)
        x = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hkv, d))).to(torch.bfloat16).cuda()
        pos = np.concatenate([np.arange(n) + m.seen[b] for b, n in enumerate(new)]).astype(np.int32)
        lens += torch.tensor(new, dtype=torch.int32, device="cuda")
        cu = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
        chunk = step[0] == "chunk"
        q = attn.rope_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kc, vc, lens, freq, page_table=table,
                             cu_seqlens_q=cu if chunk else None, positions=torch.from_numpy(pos).cuda())
        if chunk:
            o, lse = attn.prefill_paged(q, kc, vc, table, cu, lens, max(new), out_dtype=torch.float32)
        else:
            o, lse = attn.decode_paged(q, kc, vc, table, lens, out_dtype=torch.float32)
        attn.key_weights(q, lse, kc, lens, w, page_table=table, cu_seqlens_q=cu if chunk else None, max_sq=max(new))
        attn.sync_check()
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        lse = lse if chunk else lse.T
        # the reference takes q and k as the kernels have them: rotated, rounded to bf16 (the
        # rotation itself is checked to half a step)
        ref, mag = rotate(x.float().cpu().numpy()[:, :Hq + Hkv], pos.astype(np.float64), m.freq, amp, False)
        qn = q.double().cpu().numpy()
        assert (abs(qn - ref[:, :Hq]) <= 2.0 ** -8 * (abs(ref[:, :Hq]) + mag[:, :Hq] * 2.0 ** -20) + mag[:, :Hq] * 2.0 ** -20).all()
        kn = torch.from_numpy(ref[:, Hq:]).to(torch.bfloat16).double().numpy()
        vn = x[:, Hq + Hkv:].double().cpu().numpy()
        at = 0
        for b, n in enumerate(new):
            if n:
                ro, rl = m.step(b, qn[at:at + n], kn[at:at + n], vn[at:at + n])
                check_o(o[at:at + n], ro, False, f"{step} {b}")
                check_lse(lse[:, at:at + n], rl)
            for hk in range(Hkv):  # every weight of every step so far: off by a part in 1000 at most
                L = len(m.w[b][hk])
                np.testing.assert_allclose(w[b, hk, :L].cpu().numpy(), m.w[b][hk], rtol=1e-3, atol=1e-5)
            at += n
    total = sum(m.seen)
    assert total == sum(sum(s[1]) if s[0] == "chunk" else B for s in steps if s[0] != "evict")


# ------------------------------------------------------------------ graphs, streams
def _state(seed, B=5, page=16, cap=160, new=None):
    g = torch.Generator().manual_seed(seed)
    new = new or [1] * B
    lens = torch.randint(20, cap + 1, (B,), generator=g).to(torch.int32)
    T = sum(new)
    n = B * cap // page
    s = dict(x=torch.randn(T, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda(), lens=lens.cuda(),
             table=torch.randperm(n, generator=g).to(torch.int32).view(B, -1).cuda(),
             kc=torch.randn(n, page, Hkv, d, generator=g).bfloat16().cuda(),
             vc=torch.randn(n, page, Hkv, d, generator=g).bfloat16().cuda(),
             w=torch.zeros(B, Hkv, cap, device="cuda"), max_sq=max(new),
             cu=torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32).cuda())
    return s


FREQ = {}


def _step(s, n_splits=3, stream=None):
    """One whole step; every output and the state after it."""
    if "f" not in FREQ:
        FREQ["f"] = attn.rope_frequencies(ROT, device="cuda")[0]
    kw = dict(page_table=s["table"], stream=stream)
    one = s["max_sq"] == 1
    cu = None if one else s["cu"]
    x = s["x"]
    q = attn.rope_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], s["kc"], s["vc"], s["lens"], FREQ["f"],
                         cu_seqlens_q=cu, **kw)
    if one:
        o, lse = attn.decode_paged(q, s["kc"], s["vc"], s["table"], s["lens"], n_splits, stream=stream)
    else:
        o, lse = attn.prefill_paged(q, s["kc"], s["vc"], s["table"], s["cu"], s["lens"], s["max_sq"],
                                    n_splits=n_splits, stream=stream)
    attn.key_weights(q, lse, s["kc"], s["lens"], s["w"], cu_seqlens_q=cu, max_sq=s["max_sq"], **kw)
    kept, lens = attn.evict(s["w"], s["kc"], s["vc"], s["lens"], 30, 6, 2, **kw)
    return q, o, lse, kept, lens


def _all(s, out):
    return [t.clone() for t in out] + [s[n].clone() for n in ("kc", "vc", "w")]


def _same(a, b):
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("new", [[1] * 5, [30, 1, 0, 17, 3]], ids=["tokens", "chunks"])
def test_captured_step_replays_on_new_inputs(new):
    want = []
    for seed in (1, 2):
        s = _state(seed, new=new)
        want.append(_all(s, _step(s)))
    attn.sync_check()
    s = _state(1, new=new)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _step(s)
    for seed in (1, 2, 1):
        for name, t in _state(seed, new=new).items():
            if isinstance(t, torch.Tensor):
                s[name].copy_(t)
        g.replay()
        torch.cuda.synchronize()
        _same(_all(s, out), want[seed - 1])
    attn.sync_check()


def test_two_graphs_replay_at_the_same_time():
    """Two captured decode steps with workspaces and counters of their own, replayed on two
    streams without an order between them."""
    want, graphs = [], []
    for seed in (3, 4):
        s = _state(seed, B=40, cap=480)
        ref = attn.decode_paged(s["x"][:, :Hq].contiguous(), s["kc"], s["vc"], s["table"], s["lens"], 6)
        torch.cuda.synchronize()
        q = s["x"][:, :Hq].contiguous()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(20):
                out = attn.decode_paged(q, s["kc"], s["vc"], s["table"], s["lens"], 6)
        graphs.append((g, out, s, q))
        want.append(ref)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for (g, *_), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (g, out, *_), ref in zip(graphs, want):
        _same(list(out), list(ref))
    attn.sync_check()


def test_steps_on_two_streams_at_once():
    """Eager steps on two streams (their counters and workspaces do not meet), and the
    stream argument."""
    want = []
    for seed in (5, 6):
        s = _state(seed, B=33, cap=320)
        want.append(_all(s, _step(s)))
    torch.cuda.synchronize()
    states = [_state(seed, B=33, cap=320) for seed in (5, 6)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for s, st in zip(states, streams):
        outs.append(_step(s, stream=st))  # given as an argument
    torch.cuda.synchronize()
    for s, out, w in zip(states, outs, want):
        _same(_all(s, out), w)
    for t, (s, st) in enumerate(zip([_state(5, B=33, cap=320), _state(6, B=33, cap=320)], streams)):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):  # as the current stream
            out = _step(s)
        torch.cuda.synchronize()
        _same(_all(s, out), want[t])
    attn.sync_check()


def test_threads_on_one_stream():
    """Two host threads make split calls on the same stream: their launches and workspaces do
    not mix."""
    import threading
    states = [_state(11, new=[30, 1, 0, 17, 3]), _state(12, new=[9, 20, 5, 1, 30])]
    one = [_state(13, B=9), _state(14, B=9)]
    want, got, errors = [], [[], []], []

    def chunk(s):
        q = s["x"][:, :Hq].contiguous()
        return attn.prefill_paged(q, s["kc"], s["vc"], s["table"], s["cu"], s["lens"], s["max_sq"], n_splits=3)

    def token(s):
        return attn.decode_paged(s["x"][:, :Hq].contiguous(), s["kc"], s["vc"], s["table"], s["lens"], 4)

    want = [(chunk(s), token(o)) for s, o in zip(states, one)]
    torch.cuda.synchronize()

    def work(i):
        try:
            for _ in range(50):
                got[i].append((chunk(states[i]), token(one[i])))
        except Exception as e:  # pragma: no cover
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for i in (0, 1):
        for c, o in got[i]:
            _same(list(c) + list(o), list(want[i][0]) + list(want[i][1]))
    attn.sync_check()


def test_long_pools():
    """Rows behind 2^31 elements of a pool: append, weights and both forms of eviction."""
    page, H, D = 256, 8, 256
    n_pages = 2 ** 31 // (page * H * D) + 4
    kc = torch.zeros(n_pages, page, H, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(8)
    k, v, q = (torch.randn(300, H, D, generator=g).bfloat16() for _ in range(3))
    attn.rope_append(None, k.cuda(), v.cuda(), kc, vc, lens, None, page_table=table, cu_seqlens_q=cu)
    attn.sync_check()
    assert torch.equal(kc[n_pages - 1].cpu(), k[:256]) and torch.equal(kc[n_pages - 2, :44].cpu(), k[256:])
    assert torch.equal(vc[n_pages - 1].cpu(), v[:256]) and not kc[:n_pages - 2].any()
    o, lse = attn.prefill_paged(q.cuda(), kc, vc, table, cu, lens, 300)
    w = torch.zeros(1, H, 512, device="cuda")
    attn.key_weights(q.cuda(), lse, kc, lens, w, page_table=table, cu_seqlens_q=cu, max_sq=300)
    attn.sync_check()
    np.testing.assert_allclose(w.sum(-1).cpu().numpy(), 300.0, rtol=1e-4)  # each row's weights sum to 1
    small = torch.zeros(2, page, H, D, dtype=torch.bfloat16, device="cuda")
    t2 = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    kept, _ = attn.evict(w, kc, vc, lens, 100, 10, 4, page_table=table, dst=(small, torch.zeros_like(small), t2, None))
    kept2, n2 = attn.evict(w, kc, vc, lens, 100, 10, 4, page_table=table)
    attn.sync_check()
    assert torch.equal(kept, kept2) and n2.item() == 100
    for h in range(H):
        idx = kept[0, h].cpu().long()
        assert torch.equal(small[1, :100, h].cpu(), k[idx, h]) and torch.equal(kc[n_pages - 1, :100, h].cpu(), k[idx, h])


def test_append_of_a_long_batch():
    """Enough tokens for the eight-token CTAs: sequences that start inside one, an empty one,
    tokens behind the last."""
    new = [1003, 0, 5, 1500, 1]
    lens = torch.tensor([1003, 4, 40, 1501, 1], dtype=torch.int32)
    T, page = sum(new), 32
    g = torch.Generator().manual_seed(9)
    x = torch.randn(T + 11, 3 + 2, 128, generator=g).bfloat16()
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
    n_pages = [-(-int(L) // page) for L in lens]
    table = torch.full((5, max(n_pages)), -1, dtype=torch.int32)
    order = torch.randperm(sum(n_pages), generator=g).to(torch.int32)
    at = 0
    for b, n in enumerate(n_pages):
        table[b, :n] = order[at:at + n]
        at += n
    kc = torch.zeros(sum(n_pages), page, 1, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    freq, _ = attn.rope_frequencies(128, device="cuda")
    xg = x.cuda()
    out = torch.full((T + 11, 3, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    attn.rope_append(xg[:, :3], xg[:, 3:4], xg[:, 4:], kc, vc, lens.cuda(), freq, page_table=table.cuda(),
                     cu_seqlens_q=cu.cuda(), out=out)
    attn.sync_check()
    pos = np.concatenate([np.arange(n) + int(L) - n for n, L in zip(new, lens)])
    ref, mag = rotate(x[:T].float().numpy(), pos.astype(np.float64), freq.cpu().numpy(), 1.0, False)
    from tests.test_rope_append import check
    check(out[:T], ref[:, :3], mag[:, :3])
    assert (out[T:] == 9).all()
    used = torch.zeros(kc.shape[:2], dtype=torch.bool)
    i = 0
    for b, n in enumerate(new):
        for j in range(int(lens[b]) - n, int(lens[b])):
            used[int(table[b, j // page]), j % page] = True
    rows = [(int(table[b, j // page]), j % page) for b, n in enumerate(new) for j in range(int(lens[b]) - n, int(lens[b]))]
    r = torch.tensor(rows)
    check(kc.cpu()[r[:, 0], r[:, 1]], ref[:, 3:4], mag[:, 3:4])
    assert torch.equal(vc.cpu()[r[:, 0], r[:, 1]], x[:T, 4:])
    assert not kc.cpu()[~used].any() and not vc.cpu()[~used].any()
