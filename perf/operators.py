"""The paged-cache serving operators, as cases to time: rotary positions with the
cache append, attention of new tokens over a paged cache (chunks and single
tokens), accumulated attention weights, and eviction by them.

Every case is one call of a serving step.  ``prepare`` makes the inputs a serving
loop holds before the call; ``run`` makes the call, in its plain form (elementary
torch operations in fp32, angles in fp64) or, with ``own`` set, through the
package's entry points; ``exact`` computes the same in fp64.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
# Common keys: B sequences, Hq / Hkv heads, head dim d, page size of the cache.
# new_lo..new_hi: new tokens of a sequence, hist_lo..hist_hi: cached ones before
# them (uniform per sequence, from the seed).  d = 128 with 28/4 or 32/8 heads are
# the package's GQA workloads.
def listed():
    return [
        # the smallest call of a step: one new token for each of 64 sequences
        dict(name="rope_decode_b64", op="rope", B=64, Hq=32, Hkv=8, d=128, rot=128, interleaved=False,
             scaled=False, page=16, new_lo=1, new_hi=1, hist_lo=64, hist_hi=512, far=0, fused=True),
        # a long prompt, a quarter to a half of each head rotated, positions far out
        dict(name="rope_prompt_32k_far", op="rope", B=1, Hq=32, Hkv=8, d=128, rot=64, interleaved=True,
             scaled=True, page=128, new_lo=32768, new_hi=32768, hist_lo=0, hist_hi=0, far=1000000, fused=True),
        # one sequence, one token: latency only (the package's 1641-key decode)
        dict(name="decode_1641", op="decode", B=1, Hq=28, Hkv=4, d=128, page=16, new_lo=1, new_hi=1,
             hist_lo=1640, hist_hi=1640, f32=False),
        # the package's ragged decode batch, from pages
        dict(name="decode_ragged_b64", op="decode", B=64, Hq=32, Hkv=8, d=128, page=64, new_lo=1, new_hi=1,
             hist_lo=511, hist_hi=8191, f32=False),
        # few sequences, very long contexts, small heads: split over the keys
        dict(name="decode_long_b3_d64", op="decode", B=3, Hq=16, Hkv=2, d=64, page=32, new_lo=1, new_hi=1,
             hist_lo=100000, hist_hi=131071, f32=True),
        # checking a few drafted tokens of each sequence: few rows, many keys
        dict(name="chunk_draft_b16", op="chunk", B=16, Hq=28, Hkv=4, d=128, page=16, new_lo=5, new_hi=9,
             hist_lo=1000, hist_hi=8000, window=0, sink=0, f32=False),
        # the package's chunked prefill batch, from pages
        dict(name="chunk_b8", op="chunk", B=8, Hq=28, Hkv=4, d=128, page=64, new_lo=64, new_hi=1024,
             hist_lo=0, hist_hi=4096, window=0, sink=0, f32=False),
        # one chunk of a long prompt: the largest amount of work
        dict(name="chunk_long", op="chunk", B=1, Hq=28, Hkv=4, d=128, page=128, new_lo=2000, new_hi=2048,
             hist_lo=30000, hist_hi=30720, window=0, sink=0, f32=False),
        # weights after each decode step of the ragged batch
        dict(name="weights_decode_b64", op="weights", B=64, Hq=32, Hkv=8, d=128, page=64, new_lo=1, new_hi=1,
             hist_lo=511, hist_hi=8191),
        # weights of a whole prompt (the package's 3314-token GQA prefill)
        dict(name="weights_prompt_3314", op="weights", B=1, Hq=28, Hkv=4, d=128, page=64, new_lo=3314,
             new_hi=3314, hist_lo=0, hist_hi=0),
        # a batch whose caches outgrew their budget
        dict(name="evict_b64", op="evict", B=64, Hq=32, Hkv=8, d=128, page=64, hist_lo=4096, hist_hi=8192,
             budget=2048, recent=256, sink=4),
        # one long sequence
        dict(name="evict_one", op="evict", B=1, Hq=28, Hkv=4, d=128, page=16, hist_lo=16000, hist_hi=16384,
             budget=4096, recent=1024, sink=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "decode", "chunk", "weights", "evict"])
    d = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    G = rng.choice([1, 2, 4, 7, 8])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    c = dict(op=op, Hq=Hkv * G, Hkv=Hkv, d=d, page=page)
    if op == "rope":
        B = _log_int(rng, 1, 64)
        one = rng.random() < 0.4
        new = 1 if one else _log_int(rng, 2, max(2, 24000 // (B * Hkv)))
        hist = _log_int(rng, 1, 512)
        c.update(B=B, rot=rng.choice([r for r in (32, 64, 96, 128, 256) if r <= d]),
                 interleaved=rng.random() < 0.5, scaled=rng.random() < 0.5, new_lo=1 if one else (new + 1) // 2,
                 new_hi=new, hist_lo=hist // 2, hist_hi=hist, far=rng.choice([0, 0, 100000, 1000000]),
                 fused=rng.random() < 0.5)
    elif op == "decode":
        keys = max(1, 1500000 // (Hkv * d // 64))  # K rows of 128 bytes in all: below the ragged batch's
        B = _log_int(rng, 1, 128)
        hi = _log_int(rng, 2, max(2, min(131072, keys // B)))
        c.update(B=B, new_lo=1, new_hi=1, hist_lo=rng.choice([hi, hi // 2, hi // 8]), hist_hi=hi,
                 f32=rng.random() < 0.5)
    elif op in ("chunk", "weights"):
        B = _log_int(rng, 1, 16)
        one = op == "weights" and rng.random() < 0.5
        new = 1 if one else _log_int(rng, 2, 2048)
        hist = _log_int(rng, 1, 16384)
        while B * new * (hist + new) * Hkv * G * d > 2e11 or B * (hist + new) * Hkv * d > 1e8:
            B, new, hist = max(1, B // 2), max(1, new * 3 // 4), max(1, hist * 3 // 4)
        c.update(B=B, new_lo=max(1, new // 2), new_hi=new, hist_lo=hist // 4, hist_hi=hist)
        if op == "chunk":
            win = rng.choice([0, 0, 0, _log_int(rng, 16, 2048)])
            c.update(window=win, sink=rng.choice([0, 4]) if win else 0, f32=rng.random() < 0.3)
    else:
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 64, max(64, min(32768, 40000000 // (B * Hkv * d))))
        budget = max(8, int(hi * rng.uniform(0.1, 0.6)))
        c.update(B=B, hist_lo=rng.choice([budget, budget // 2]), hist_hi=hi, budget=budget, recent=rng.randint(0, budget // 2),
                 sink=rng.choice([0, 1, 4]))
    return c


# ------------------------------------------------------------------ inputs
def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g)


def _lengths(case):
    """New tokens and keys (new ones last) of each sequence: part of the case, the
    same for every seed."""
    B = case["B"]
    g = torch.Generator().manual_seed(B * 100003 + case["hist_hi"] * 31 + case["Hq"])
    new = _ints(g, case.get("new_lo", 0), case.get("new_hi", 0), B)
    hist = _ints(g, case["hist_lo"], case["hist_hi"], B)
    return new.tolist(), (new + hist).tolist()


def _pages(g, lens, page):
    """A table whose pages lie in the pool in no order, as an allocator leaves them."""
    per = [-(-n // page) for n in lens]
    pool = max(1, sum(per))
    order = torch.randperm(pool, generator=g, dtype=torch.int64).to(torch.int32)
    table = torch.full((len(lens), max(1, max(per))), -1, dtype=torch.int32)  # unused entries: -1
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pool


def _frequencies(rot, scaled):
    """Radians per position of each rotated pair, and the amplitude: plain, or
    stretched by 8 for long contexts with the fast pairs kept (a ramp between)."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = 10000.0 ** (-i / rot)
    if not scaled:
        return f, 1.0
    turns = 4096 * f / (2 * math.pi)
    keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
    return f * keep + f / 8 * (1 - keep), 0.1 * math.log(8) + 1.0


def _randn(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(torch.bfloat16)


def prepare(case, seed):
    op, B, Hq, Hkv, d, page = (case[k] for k in ("op", "B", "Hq", "Hkv", "d", "page"))
    new, lens = _lengths(case)
    g = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    table, pool = _pages(g, lens, page)
    s = dict(case=case, op=op, new=new, lens=lens, scale=1.0 / math.sqrt(d),
             table=table.to(DEV), kv_lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
             kcache=_randn(gen, pool, page, Hkv, d), vcache=_randn(gen, pool, page, Hkv, d))
    T = sum(new)
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(new), 0)
    s["one"] = all(n == 1 for n in new)
    s["cu"] = None if s["one"] and op != "chunk" else cu.to(DEV)
    s["max_sq"] = max(new)
    if op == "rope":
        if case["fused"]:  # rows of one projection's output: q, k and v side by side
            x = _randn(gen, T, (Hq + 2 * Hkv), d)
            s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            s["q"], s["k"], s["v"] = _randn(gen, T, Hq, d), _randn(gen, T, Hkv, d), _randn(gen, T, Hkv, d)
        f, s["amp"] = _frequencies(case["rot"], case["scaled"])
        s["freq"] = f.to(DEV)
        pos = torch.cat([torch.arange(L - n, L) for n, L in zip(new, lens)]) + case["far"]
        s["pos"] = pos.to(torch.int32).to(DEV)
        s["slot"] = _slots(table, new, lens, page).to(DEV)
        return s
    if op == "evict":
        s["weights"] = torch.rand(B, Hkv, table.shape[1] * page, generator=gen, device=DEV).pow(4)
        s["weights"][..., ::7] = 0.125  # equal weights: ties go to the lowest index
        out_lens = [min(n, case["budget"]) for n in lens]
        t2, pool2 = _pages(g, out_lens, page)
        s["table2"] = t2.to(DEV)
        s["kcache2"] = torch.zeros(pool2, page, Hkv, d, dtype=torch.bfloat16, device=DEV)
        s["vcache2"] = torch.zeros_like(s["kcache2"])
        s["weights2"] = torch.zeros_like(s["weights"])
        return s
    s["q"] = _randn(gen, T, Hq, d, scale=1.5)  # scores a little peaked
    if op == "weights":
        s["lse"] = _lse(s)
        s["weights"] = torch.zeros(B, Hkv, table.shape[1] * page, device=DEV)
    return s


def _slots(table, new, lens, page):
    """Row of the pool that each new token's key goes to."""
    out = []
    for b, (n, L) in enumerate(zip(new, lens)):
        j = torch.arange(L - n, L)
        out.append(table[b, j // page].to(torch.int64) * page + j % page)
    return torch.cat(out)


def _rows(table, b, L, page):
    """Rows of the pool that hold keys 0..L-1 of sequence b."""
    j = torch.arange(L, device=table.device)
    return table[b, j // page].to(torch.int64) * page + j % page


def _seqs(s):
    at = 0
    for b, (n, L) in enumerate(zip(s["new"], s["lens"])):
        yield b, at, n, L
        at += n


def _mask(n, L, window, sink, dev):
    """Keys that new row i (position L - n + i) admits."""
    p = torch.arange(L - n, L, device=dev)[:, None]
    j = torch.arange(L, device=dev)[None]
    ok = j <= p
    if window:
        ok = ok & ((j > p - window) | (j < sink))
    return ok


def _lse(s):
    """Log-sum-exp of each row's scores: what the attention call before returned."""
    c = s["case"]
    G = c["Hq"] // c["Hkv"]
    out = torch.empty(c["Hq"], s["q"].shape[0], device=DEV)
    for b, at, n, L in _seqs(s):
        k = s["kcache"].view(-1, c["Hkv"], c["d"])[_rows(s["table"], b, L, c["page"])].float()
        ok = _mask(n, L, 0, 0, DEV)
        for h in range(c["Hkv"]):
            q = s["q"][at:at + n, h * G:(h + 1) * G].transpose(0, 1).float()
            sc = (q @ k[:, h].T) * s["scale"]
            out[h * G:(h + 1) * G, at:at + n] = sc.masked_fill_(~ok, -math.inf).logsumexp(-1)
    return out.T.contiguous() if s["one"] else out


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    import attention_forward_tcgen05_gb300 as attn
    c, op = s["case"], s["op"]
    if op == "rope":
        q = attn.rope_append(s["q"], s["k"], s["v"], s["kcache"], s["vcache"], s["kv_lens"], s["freq"],
                             page_table=s["table"], cu_seqlens_q=s["cu"], positions=s["pos"],
                             interleaved=c["interleaved"], amp=s["amp"])
        return q, s["kcache"], s["vcache"]
    if op == "decode":
        return attn.decode_paged(s["q"], s["kcache"], s["vcache"], s["table"], s["kv_lens"],
                                 out_dtype=torch.float32 if c["f32"] else torch.bfloat16)
    if op == "chunk":
        return attn.prefill_paged(s["q"], s["kcache"], s["vcache"], s["table"], s["cu"], s["kv_lens"],
                                  s["max_sq"], window=c["window"], n_sink=c["sink"],
                                  out_dtype=torch.float32 if c["f32"] else torch.bfloat16)
    if op == "weights":
        return attn.key_weights(s["q"], s["lse"], s["kcache"], s["kv_lens"], s["weights"], page_table=s["table"],
                                cu_seqlens_q=s["cu"], max_sq=s["max_sq"], accumulate=False)
    kept, lens = attn.evict(s["weights"], s["kcache"], s["vcache"], s["kv_lens"], c["budget"],
                            n_recent=c["recent"], n_sink=c["sink"], page_table=s["table"],
                            dst=(s["kcache2"], s["vcache2"], s["table2"], s["weights2"]))
    return kept, lens, s["kcache2"], s["vcache2"], s["weights2"]


def _plain_rope(s):
    c, rot = s["case"], s["case"]["rot"]
    a = s["pos"].double()[:, None] * s["freq"][None]  # far positions: angles in 64 bits
    cos, sin = (a.cos() * s["amp"]).float()[:, None], (a.sin() * s["amp"]).float()[:, None]

    def turn(x):
        y = x.float()
        if c["interleaved"]:
            x1, x2 = y[..., 0:rot:2], y[..., 1:rot:2]
            r = torch.stack((x1 * cos - x2 * sin, x1 * sin + x2 * cos), -1).flatten(-2)
        else:
            x1, x2 = y[..., :rot // 2], y[..., rot // 2:rot]
            r = torch.cat((x1 * cos - x2 * sin, x1 * sin + x2 * cos), -1)
        return torch.cat((r, y[..., rot:]), -1).to(torch.bfloat16)

    s["kcache"].view(-1, c["Hkv"], c["d"])[s["slot"]] = turn(s["k"])
    s["vcache"].view(-1, c["Hkv"], c["d"])[s["slot"]] = s["v"]
    return turn(s["q"]), s["kcache"], s["vcache"]


def _plain_attend(s):
    c = s["case"]
    G, d, win = c["Hq"] // c["Hkv"], c["d"], c.get("window", 0)
    o = torch.empty(s["q"].shape, dtype=torch.float32 if c["f32"] else torch.bfloat16, device=DEV)
    lse = torch.empty(c["Hq"], s["q"].shape[0], device=DEV)
    for b, at, n, L in _seqs(s):
        rows = _rows(s["table"], b, L, c["page"])
        k = s["kcache"].view(-1, c["Hkv"], d)[rows].float()
        v = s["vcache"].view(-1, c["Hkv"], d)[rows].float()
        ok = _mask(n, L, win, c.get("sink", 0), DEV)
        for h in range(c["Hkv"]):
            q = s["q"][at:at + n, h * G:(h + 1) * G].transpose(0, 1).float()
            sc = (q @ k[:, h].T) * s["scale"]
            sc = sc.masked_fill_(~ok, -math.inf)
            m = sc.amax(-1, keepdim=True)
            p = (sc - m).exp_()
            l = p.sum(-1, keepdim=True)
            o[at:at + n, h * G:(h + 1) * G] = ((p @ v[:, h]) / l).transpose(0, 1).to(o.dtype)
            lse[h * G:(h + 1) * G, at:at + n] = (m + l.log())[..., 0]
    return o, (lse.T.contiguous() if s["op"] == "decode" else lse)


def _plain_weights(s):
    c = s["case"]
    G, d = c["Hq"] // c["Hkv"], c["d"]
    lse = s["lse"].T if s["one"] else s["lse"]
    for b, at, n, L in _seqs(s):
        k = s["kcache"].view(-1, c["Hkv"], d)[_rows(s["table"], b, L, c["page"])].float()
        ok = _mask(n, L, 0, 0, DEV)
        for h in range(c["Hkv"]):
            q = s["q"][at:at + n, h * G:(h + 1) * G].transpose(0, 1).float()
            sc = (q @ k[:, h].T) * s["scale"] - lse[h * G:(h + 1) * G, at:at + n, None]
            s["weights"][b, h, :L] = sc.masked_fill_(~ok, -math.inf).exp_().sum((0, 1))
    return s["weights"]


def _plain_evict(s):
    c = s["case"]
    budget, recent, sink = c["budget"], c["recent"], c["sink"]
    kept = torch.full((c["B"], c["Hkv"], budget), -1, dtype=torch.int32, device=DEV)
    for b, L in enumerate(s["lens"]):
        n = min(L, budget)
        if L <= budget:
            idx = torch.arange(L, device=DEV).expand(c["Hkv"], L)
        else:
            w = s["weights"][b, :, sink:L - recent]
            top = torch.sort(w, dim=-1, descending=True, stable=True).indices[:, :budget - sink - recent] + sink
            ends = torch.cat((torch.arange(sink, device=DEV), torch.arange(L - recent, L, device=DEV)))
            idx = torch.cat((top, ends.expand(c["Hkv"], -1)), -1).sort(-1).values
        kept[b, :, :n] = idx.to(torch.int32)
        src = _rows(s["table"], b, L, c["page"])[idx]           # [Hkv, n]
        dst = _rows(s["table2"], b, n, c["page"])
        heads = torch.arange(c["Hkv"], device=DEV)[:, None]
        for a, z in (("kcache", "kcache2"), ("vcache", "vcache2")):
            s[z].view(-1, c["Hkv"], c["d"])[dst] = s[a].view(-1, c["Hkv"], c["d"])[src, heads].transpose(0, 1)
        s["weights2"][b, :, :n] = s["weights"][b].gather(-1, idx)
        s["weights2"][b, :, n:L] = 0
    return kept, s["kv_lens"].clamp(max=budget), s["kcache2"], s["vcache2"], s["weights2"]


_PLAIN = dict(rope=_plain_rope, decode=_plain_attend, chunk=_plain_attend, weights=_plain_weights,
              evict=_plain_evict)


# ------------------------------------------------------------------ work
def work(case):
    """One pass's bytes and operations, from the lengths of its sequences."""
    op, B, Hq, Hkv, d = (case[k] for k in ("op", "B", "Hq", "Hkv", "d"))
    new, lens = _lengths(case)
    if op == "evict":
        n = sum(min(L, case["budget"]) for L in lens)
        moved = Hkv * n * (2 * d * 2 * 2 + 4 + 4)  # K and V rows in and out, weight and index out
        return {"bytes": moved + Hkv * sum(lens) * 4, "flops": Hkv * sum(lens)}
    T = sum(new)
    if op == "rope":
        return {"bytes": T * (Hq + 2 * Hkv) * d * 2 * 2, "flops": T * (Hq + Hkv) * case["rot"] * 3}
    pairs, keys, win, sink = 0, 0, case.get("window", 0), case.get("sink", 0)
    for n, L in zip(new, lens):
        if win:
            for p in range(L - n, L):
                lo = max(0, p - win + 1)
                pairs += p + 1 - lo + min(sink, lo)
            lo = max(0, L - n - win + 1)
            keys += L - lo + min(sink, lo)
        else:
            pairs += n * (L - n) + n * (n + 1) // 2
            keys += L
    if op == "weights":
        return {"bytes": keys * Hkv * (d * 2 + 4) + T * Hq * (d * 2 + 4), "flops": 2 * d * Hq * pairs}
    o = 4 if case["f32"] else 2
    return {"bytes": keys * Hkv * d * 2 * 2 + T * Hq * (d * (2 + o) + 4), "flops": 4 * d * Hq * pairs}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The definitions, head by head in fp64, from the same inputs."""
    s = prepare(case, seed)
    op, Hq, Hkv, d, page = case["op"], case["Hq"], case["Hkv"], case["d"], case["page"]
    table = s["table"].long()
    pool_k, pool_v = s["kcache"].flatten(0, 1), s["vcache"].flatten(0, 1)
    if op == "rope":
        turn = torch.polar(torch.full((), s["amp"], dtype=torch.float64, device=DEV),
                           s["pos"].double()[:, None, None] * s["freq"])

        def rotated(x):
            y, r = x.double(), case["rot"]
            even = y[..., :r].unflatten(-1, (r // 2, 2) if case["interleaved"] else (2, r // 2))
            if not case["interleaved"]:
                even = even.transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(even.contiguous()) * turn)
            y[..., :r] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
            return y

        kc, vc = pool_k.double(), pool_v.double()
        kc[s["slot"]] = rotated(s["k"])
        vc[s["slot"]] = s["v"].double()
        return rotated(s["q"]), kc.view(s["kcache"].shape), vc.view(s["vcache"].shape)
    where = lambda b, L: (table[b, :, None] * page + torch.arange(page, device=DEV)).flatten()[:L]
    if op == "evict":
        keep = torch.full((case["B"], Hkv, case["budget"]), -1, dtype=torch.int32)
        w_all = s["weights"].cpu()
        k2, v2 = s["kcache2"].flatten(0, 1).double(), s["vcache2"].flatten(0, 1).double()
        w2 = s["weights2"].double()
        t2 = s["table2"].long()
        for b, L in enumerate(s["lens"]):
            n = min(L, case["budget"])
            dst = (t2[b, :, None] * page + torch.arange(page, device=DEV)).flatten()[:n]
            src = where(b, L)
            for h in range(Hkv):
                rank = w_all[b, h, :L].double().clone()
                rank[:case["sink"]] = math.inf
                rank[L - case["recent"]:] = math.inf
                idx = torch.from_numpy(np.sort(np.argsort(-rank.numpy(), kind="stable")[:n]))
                keep[b, h, :n] = idx.to(torch.int32)
                at = idx.to(DEV)
                k2[dst, h] = pool_k[src[at], h].double()
                v2[dst, h] = pool_v[src[at], h].double()
                w2[b, h, :n] = s["weights"][b, h, at].double()
                w2[b, h, n:L] = 0
        lens = torch.tensor([min(n, case["budget"]) for n in s["lens"]], dtype=torch.int32)
        return keep, lens, k2.view(s["kcache2"].shape), v2.view(s["vcache2"].shape), w2
    G, T = Hq // Hkv, s["q"].shape[0]
    o = torch.zeros(T, Hq, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(T, Hq, dtype=torch.float64, device=DEV)
    w = s["weights"].double() if op == "weights" else None
    given = None if op != "weights" else (s["lse"] if s["one"] else s["lse"].T).double()
    at = 0
    for b, L in enumerate(s["lens"]):
        n = s["new"][b]
        rows = where(b, L)
        p = torch.arange(L - n, L, device=DEV)
        j = torch.arange(L, device=DEV)
        hidden = j[None] > p[:, None]
        if case.get("window"):
            hidden = hidden | ((j[None] <= p[:, None] - case["window"]) & (j[None] >= case["sink"]))
        for hk in range(Hkv):
            k = pool_k[rows, hk].double()
            v = pool_v[rows, hk].double()
            total = torch.zeros(L, dtype=torch.float64, device=DEV)
            for h in range(hk * G, (hk + 1) * G):
                sc = torch.einsum("id,jd->ij", s["q"][at:at + n, h].double(), k) * s["scale"]
                sc[hidden] = -math.inf
                if op == "weights":
                    total += torch.exp(sc - given[at:at + n, h, None]).sum(0)
                else:
                    ls = torch.logsumexp(sc, -1)
                    lse[at:at + n, h] = ls
                    o[at:at + n, h] = torch.exp(sc - ls[:, None]) @ v
            if op == "weights":
                w[b, hk, :L] = total
        at += n
    if op == "weights":
        return w
    return o, (lse if op == "decode" else lse.T)
