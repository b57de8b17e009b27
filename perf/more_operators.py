"""Windowed attention of single tokens, the gradients of attention, and rotary positions
with several axes, as cases to time.

Every case is one call of a serving or training step.  ``prepare`` makes the inputs such a
program holds before the call; ``run`` makes the call, in its plain form (elementary torch
operations in fp32, angles in fp64) or, with ``own`` set, through the package's entry
points; ``exact`` computes the same in fp64.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
# Common keys: B sequences, Hq / Hkv heads, head dim d.
#   decode: window and sink first keys; hist_lo..hist_hi keys of a sequence (uniform, fixed
#     by the case); page = 0: dense caches; freed: pages that no key of the window or the
#     sinks lies in have left the table.
#   grad: S tokens and keys a sequence, or (ragged) S_lo..S_hi new tokens of each after
#     hist_lo..hist_hi cached keys, packed; window = 0: none.
#   append, rotate: T tokens, sections of the rotated pairs that follow each axis.
# 28/4 and 32/8 heads of 128 are the package's GQA workloads, 16 heads of 64 its sweep's.
def listed():
    return [
        # the smallest call: one sequence of the package's 1641 keys, one token
        dict(name="decode_1641_w1024", op="decode", B=1, Hq=28, Hkv=4, d=128, page=16, window=1024, sink=4,
             hist_lo=1641, hist_hi=1641, freed=False, f32=False),
        # a serving batch far past its window, pages behind it given back
        dict(name="decode_ragged_b64_w4096", op="decode", B=64, Hq=32, Hkv=8, d=128, page=64, window=4096, sink=4,
             hist_lo=512, hist_hi=32768, freed=True, f32=False),
        # dense caches, small heads, a large group, fp32 outputs
        dict(name="decode_dense_b16_d64_f32", op="decode", B=16, Hq=40, Hkv=2, d=64, page=0, window=2000, sink=0,
             hist_lo=100, hist_hi=8001, freed=False, f32=True),
        # training on one sequence of the package's window workload
        dict(name="grad_window_3314", op="grad", ragged=False, B=1, Hq=28, Hkv=4, d=128, S=3314, causal=True,
             window=1024, sink=4, dlse=False),
        # the same without a window
        dict(name="grad_causal_3314", op="grad", ragged=False, B=1, Hq=28, Hkv=4, d=128, S=3314, causal=True,
             window=0, sink=0, dlse=False),
        # an encoder: every token sees every token, small heads, no groups
        dict(name="grad_full_4096_d64", op="grad", ragged=False, B=2, Hq=16, Hkv=16, d=64, S=4096, causal=False,
             window=0, sink=0, dlse=False),
        # short sequences of unequal length, packed, a short window, a loss on the log-sum-exps too
        dict(name="grad_packed_b8", op="grad", ragged=True, B=8, Hq=32, Hkv=8, d=128, S_lo=100, S_hi=1500,
             hist_lo=0, hist_hi=300, causal=True, window=512, sink=1, dlse=True),
        # a long sequence: the largest amount of work
        dict(name="grad_long_16k_w4096", op="grad", ragged=False, B=1, Hq=32, Hkv=8, d=128, S=16384, causal=True,
             window=4096, sink=4, dlse=False),
        # one new token for each of 64 sequences, three axes
        dict(name="append_decode_b64", op="append", B=64, T=64, Hq=32, Hkv=8, d=128, sections="16,24,24",
             layout="blocks", interleaved=False, page=16, hist_hi=512, fused=True),
        # a prompt of pictures and text, axes dealt in turn, half of each head rotated
        dict(name="append_prompt_24k", op="append", B=1, T=24576, Hq=32, Hkv=8, d=128, sections="12,10,10",
             layout="dealt", interleaved=True, page=64, hist_hi=0, fused=True),
        # a picture encoder's tokens: height and width, each with its own frequencies
        dict(name="rotate_pictures_2x4096", op="rotate", T=8192, Hq=16, Hkv=16, d=64, sections="16,16",
             layout="separate", interleaved=False, fused=False, inverse=False),
        # the gradient of a video prompt's rotation, inside one projection's gradient
        dict(name="rotate_inverse_32k", op="rotate", T=32768, Hq=28, Hkv=4, d=128, sections="16,24,24",
             layout="blocks", interleaved=False, fused=True, inverse=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "grad", "grad", "append", "rotate"])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    G = rng.choice([1, 2, 4, 7, 8])
    if op == "decode":
        G = rng.choice([1, 2, 4, 7, 8, 12, 16, 20, 32])
        d = rng.choice([64, 128, 128, 256])
        B = _log_int(rng, 1, 128)
        rows = max(2, 1500000 // (Hkv * d // 64) // B)  # of 128 bytes, in all: below the ragged batch's
        window = _log_int(rng, 1, min(8192, rows))
        page = rng.choice([0, 16, 32, 48, 64, 128, 256])
        freed = page > 0 and rng.random() < 0.5
        hi = _log_int(rng, 2, 131072 if freed else max(2, min(32768, rows)))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, page=page, window=window, sink=rng.choice([0, 1, 4, 64]),
                    hist_lo=rng.choice([hi, (hi + 1) // 2, (hi + 7) // 8]), hist_hi=hi, freed=freed,
                    f32=rng.random() < 0.4)
    if op == "grad":
        d = rng.choice([64, 128, 128])
        ragged = rng.random() < 0.4
        B = _log_int(rng, 1, 16 if ragged else 4)
        S = _log_int(rng, 2, 6000)  # (a row that sees one key has no gradient in its scores)
        hist = _log_int(rng, 1, 2000) if ragged and rng.random() < 0.5 else 0
        while B * S * (S + hist) * Hkv * G * d > 1.5e11:  # the whole square's, without a window
            B, S, hist = max(1, B // 2), max(2, S * 3 // 4), hist * 3 // 4
        causal = rng.random() < 0.8
        window = _log_int(rng, 8, 4096) if causal and rng.random() < 0.6 else 0
        c = dict(op=op, ragged=ragged, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, causal=causal, window=window,
                 sink=rng.choice([0, 1, 4, 130]) if window else 0, dlse=rng.random() < 0.3)
        if ragged:
            c.update(S_lo=max(2, S // 8), S_hi=S, hist_lo=0, hist_hi=hist)
        else:
            c.update(S=S)
        return c
    d = rng.choice([64, 128, 128, 256])
    rot = rng.choice([r for r in (32, 64, 96, 128, 256) if r <= d])
    first = rng.randint(1, rot // 2 - 2)
    second = rng.randint(1, rot // 2 - first)
    sections = [s for s in (first, second, rot // 2 - first - second) if s]
    c = dict(op=op, Hq=Hkv * G, Hkv=Hkv, d=d, sections=",".join(map(str, sections)),
             layout=rng.choice(["blocks", "dealt", "separate"]), interleaved=rng.random() < 0.5,
             fused=rng.random() < 0.5)
    T = _log_int(rng, 1, max(2, 33000000 // (Hkv * (G + 2) * d)))
    if op == "append":
        B = min(T, _log_int(rng, 1, 64))
        one = rng.random() < 0.3
        c.update(B=B, T=B if one else T, page=rng.choice([16, 32, 48, 64, 128]), hist_hi=rng.choice([0, 100, 500]))
    else:
        c.update(T=T, inverse=rng.random() < 0.5)
    return c


# ------------------------------------------------------------------ inputs
def _ints(g, lo, hi, n):
    return torch.randint(lo, hi + 1, (n,), generator=g)


def _lengths(case):
    """Keys (and new tokens) of each sequence: part of the case, the same for every seed."""
    op, B = case["op"], case.get("B", 1)
    g = torch.Generator().manual_seed(B * 100003 + case.get("hist_hi", 0) * 31 + case["Hq"])
    if op == "decode":
        return [1] * B, _ints(g, case["hist_lo"], case["hist_hi"], B).tolist()
    if op == "append":  # B sequences share the T tokens, one at least each
        cuts = sorted((torch.randperm(case["T"] - 1, generator=g)[:B - 1] + 1).tolist())
        new = [b - a for a, b in zip([0] + cuts, cuts + [case["T"]])]
        hist = _ints(g, 0, case["hist_hi"], B).tolist()
    elif case["ragged"]:
        new = _ints(g, case["S_lo"], case["S_hi"], B).tolist()
        hist = _ints(g, case["hist_lo"], case["hist_hi"], B).tolist()
    else:
        new, hist = [case["S"]] * B, [0] * B
    return new, [n + h for n, h in zip(new, hist)]


def _randn(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(torch.bfloat16)


def _table(g, lens, page, used):
    """A table whose pages lie in the pool in no order, as an allocator leaves them; used:
    for each sequence the entries that hold a page (the others are -1)."""
    table = torch.full((len(lens), max(1, max(-(-n // page) for n in lens))), -1, dtype=torch.int32)
    pool = max(1, sum(len(u) for u in used))
    order = torch.randperm(pool, generator=g, dtype=torch.int64).to(torch.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, u] = order[at:at + len(u)]
        at += len(u)
    return table, pool


def _rotation(case):
    """Radians per position of each rotated pair, and the axis whose position it follows."""
    sections = [int(s) for s in case["sections"].split(",")]
    pairs = sum(sections)
    if case["layout"] == "dealt":  # t h w t h w ... while an axis has pairs left
        left, axes = list(sections), []
        while len(axes) < pairs:
            for a in range(len(sections)):
                if left[a]:
                    axes.append(a)
                    left[a] -= 1
    else:
        axes = [a for a, s in enumerate(sections) for _ in range(s)]
    i = torch.arange(pairs, dtype=torch.float64)
    f = 10000.0 ** (-i / pairs)
    if case["layout"] == "separate":  # each axis its own series over its pairs
        f = torch.cat([10000.0 ** (-torch.arange(s, dtype=torch.float64) / s) for s in sections])
    return f.to(DEV), torch.tensor(axes, dtype=torch.int32, device=DEV), len(sections)


def _positions(g, T, n_axes):
    """Text (all axes alike) with pictures and clips in it: rows and columns inside a frame."""
    t = torch.arange(T)
    frame = t // 600
    side = int(torch.randint(10, 40, (1,), generator=g))
    text = (frame % 3 == 0)
    base = int(torch.randint(0, 5000, (1,), generator=g))
    rows, cols = base + frame + (t % 600) // side, base + frame + t % side
    where = [torch.where(text, base + t, base + frame), torch.where(text, base + t, rows),
             torch.where(text, base + t, cols)]
    return torch.stack(where[3 - n_axes:]).to(torch.int32).to(DEV)


def prepare(case, seed):
    op, Hq, Hkv, d = (case[k] for k in ("op", "Hq", "Hkv", "d"))
    g = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case=case, op=op, scale=1.0 / math.sqrt(d))
    if op in ("append", "rotate"):
        T = case["T"]
        s["freq"], s["axes"], n_axes = _rotation(case)
        s["pos"] = _positions(g, T, n_axes)
        if case["fused"]:  # rows of one projection's output: q, k and v side by side
            x = _randn(gen, T, Hq + 2 * Hkv, d)
            s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            s["q"], s["k"], s["v"] = _randn(gen, T, Hq, d), _randn(gen, T, Hkv, d), _randn(gen, T, Hkv, d)
        if op == "rotate":
            if case["fused"]:  # the same of the results
                y = torch.zeros(T, Hq + 2 * Hkv, d, dtype=torch.bfloat16, device=DEV)
                s["out"] = (y[:, :Hq], y[:, Hq:Hq + Hkv])
            return s
    new, lens = _lengths(case)
    B = len(lens)
    s.update(new=new, lens=lens, kv_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(new), 0)
    if op == "append":
        page = case["page"]
        table, pool = _table(g, lens, page, [list(range(-(-n // page))) for n in lens])
        s["table"], s["cu"] = table.to(DEV), None if case["T"] == B else cu.to(DEV)
        s["kcache"], s["vcache"] = _randn(gen, pool, page, Hkv, d), _randn(gen, pool, page, Hkv, d)
        b = torch.repeat_interleave(torch.arange(B), torch.tensor(new))
        j = torch.cat([torch.arange(L - n, L) for n, L in zip(new, lens)])
        s["slot"] = (table[b, j // page].long() * page + j % page).to(DEV)  # row of the pool of each token's key
        return s
    if op == "decode":
        page, W, sink = case["page"], case["window"], case["sink"]
        s["q"] = _randn(gen, B, Hq, d, scale=1.5)  # scores a little peaked
        if page == 0:
            s["table"] = None
            s["kcache"], s["vcache"] = (_randn(gen, B, max(lens), Hkv, d) for _ in range(2))
            return s
        used = [[e for e in range(-(-L // page)) if not case["freed"] or e * page < sink or (e + 1) * page > L - W]
                for L in lens]
        table, pool = _table(g, lens, page, used)
        s["table"] = table.to(DEV)
        s["kcache"], s["vcache"] = _randn(gen, pool, page, Hkv, d), _randn(gen, pool, page, Hkv, d)
        return s
    # grad: the forward call's inputs, its outputs, and the gradient that comes back
    T, max_kv = sum(new), max(lens)
    s.update(cu=cu.to(DEV), max_sq=max(new), q=_randn(gen, T, Hq, d, scale=1.5), do=_randn(gen, T, Hq, d),
             kcache=_randn(gen, B, max_kv, Hkv, d), vcache=_randn(gen, B, max_kv, Hkv, d),
             o=torch.zeros(T, Hq, d, dtype=torch.bfloat16, device=DEV), lse=torch.empty(Hq, T, device=DEV),
             dlse=torch.randn(Hq, T, generator=gen, device=DEV) if case["dlse"] else None)
    G = Hq // Hkv
    for b, at, n, L in _seqs(s):
        ok = _mask(case, n, L)
        for h in range(Hkv):
            sc = _scores(s, b, at, n, L, h).masked_fill_(~ok, -math.inf)
            lse = sc.logsumexp(-1)
            s["lse"][h * G:(h + 1) * G, at:at + n] = lse
            o = sc.sub_(lse[..., None]).exp_() @ s["vcache"][b, :L, h].float()
            s["o"][at:at + n, h * G:(h + 1) * G] = o.transpose(0, 1).to(torch.bfloat16)
    if not case["ragged"]:  # [B][S][H][d] and [B][H][S], as the fixed-length call has them
        S = case["S"]
        for k in ("q", "do", "o"):
            s[k] = s[k].view(B, S, Hq, d)
        for k in ("lse", "dlse"):
            s[k] = None if s[k] is None else s[k].view(Hq, B, S).transpose(0, 1).contiguous()
    return s


def _seqs(s):
    at = 0
    for b, (n, L) in enumerate(zip(s["new"], s["lens"])):
        yield b, at, n, L
        at += n


def _mask(case, n, L):
    """Keys that new row i (position L - n + i) admits."""
    p = torch.arange(L - n, L, device=DEV)[:, None]
    j = torch.arange(L, device=DEV)[None]
    if not case["causal"]:
        return torch.ones(n, L, dtype=torch.bool, device=DEV)
    ok = j <= p
    if case["window"]:
        ok = ok & ((j > p - case["window"]) | (j < case["sink"]))
    return ok


def _scores(s, b, at, n, L, h):
    """[G, n, L] of sequence b and KV head h, in fp32."""
    c = s["case"]
    G = c["Hq"] // c["Hkv"]
    q = s["q"].reshape(-1, c["Hq"], c["d"])[at:at + n, h * G:(h + 1) * G].transpose(0, 1).float()
    return (q @ s["kcache"][b, :L, h].float().T) * s["scale"]


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    import attention_forward_tcgen05_gb300 as attn
    c, op = s["case"], s["op"]
    if op == "decode":
        return attn.decode_window(s["q"], s["kcache"], s["vcache"], s["kv_lens"], c["window"], c["sink"],
                                  page_table=s["table"], out_dtype=torch.float32 if c["f32"] else torch.bfloat16)
    if op == "append":
        q = attn.rope_append(s["q"], s["k"], s["v"], s["kcache"], s["vcache"], s["kv_lens"], s["freq"],
                             page_table=s["table"], cu_seqlens_q=s["cu"], positions=s["pos"],
                             interleaved=c["interleaved"], axes=s["axes"])
        return q, s["kcache"], s["vcache"]
    if op == "rotate":
        return attn.rope_rotate(s["q"], s["k"], s["freq"], s["pos"], axes=s["axes"], interleaved=c["interleaved"],
                                inverse=c["inverse"], out=s.get("out"))
    if c["ragged"]:
        return attn.prefill_varlen_backward(s["do"], s["q"], s["kcache"], s["vcache"], s["o"], s["lse"], s["cu"],
                                            s["kv_lens"], s["max_sq"], causal=c["causal"], window=c["window"],
                                            n_sink=c["sink"], dlse=s["dlse"])
    return attn.prefill_backward(s["do"], s["q"], s["kcache"], s["vcache"], s["o"], s["lse"], causal=c["causal"],
                                 window=c["window"], n_sink=c["sink"], dlse=s["dlse"])


def _plain_decode(s):
    c = s["case"]
    B, Hkv, d, W, page = c["B"], c["Hkv"], c["d"], c["window"], c["page"]
    L = s["kv_lens"].long()[:, None]
    lo = (L - W).clamp(min=0)
    ns = lo.clamp(max=c["sink"])  # sinks before the window, then the window's keys
    u = torch.arange(min(max(s["lens"]), W + c["sink"]), device=DEV)[None]
    j = torch.where(u < ns, u, u - ns + lo)
    ok = j < L
    j = j.clamp(max=max(s["lens"]) - 1)
    if page:
        row = s["table"].long().gather(1, j // page) * page + j % page
    else:
        row = torch.arange(B, device=DEV)[:, None] * s["kcache"].shape[1] + j
    row = row.clamp(min=0)
    k = s["kcache"].view(-1, Hkv, d)[row].float()
    v = s["vcache"].view(-1, Hkv, d)[row].float()
    q = s["q"].float().view(B, Hkv, -1, d)
    sc = torch.einsum("bhgd,bjhd->bhgj", q, k) * s["scale"]
    sc = sc.masked_fill_(~ok[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = (sc - m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgj,bjhd->bhgd", p, v) / l
    return (o.reshape(B, -1, d).to(torch.float32 if c["f32"] else torch.bfloat16),
            (m + l.log())[..., 0].reshape(B, -1))


def _plain_grad(s):
    c = s["case"]
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    G = Hq // Hkv
    T = sum(s["new"])
    do, lse, dlse = s["do"].reshape(T, Hq, d), s["lse"], s["dlse"]
    delta = (do.float() * s["o"].reshape(T, Hq, d).float()).sum(-1).T
    if not c["ragged"]:
        lse = lse.transpose(0, 1).reshape(Hq, T)
        dlse = None if dlse is None else dlse.transpose(0, 1).reshape(Hq, T)
    if dlse is not None:
        delta = delta - dlse
    dq = torch.zeros(T, Hq, d, dtype=torch.bfloat16, device=DEV)
    dk, dv = torch.zeros_like(s["kcache"]), torch.zeros_like(s["vcache"])
    for b, at, n, L in _seqs(s):
        ok = _mask(c, n, L)
        for h in range(Hkv):
            rows, heads = slice(at, at + n), slice(h * G, (h + 1) * G)
            p = _scores(s, b, at, n, L, h).sub_(lse[heads, rows, None]).masked_fill_(~ok, -math.inf).exp_()
            g = do[rows, heads].transpose(0, 1).float()
            dv[b, :L, h] = (p.transpose(1, 2) @ g).sum(0).to(torch.bfloat16)
            ds = g @ s["vcache"][b, :L, h].float().T
            ds = p.mul_(ds.sub_(delta[heads, rows, None])).mul_(s["scale"])
            dq[rows, heads] = (ds @ s["kcache"][b, :L, h].float()).transpose(0, 1).to(torch.bfloat16)
            q = s["q"].reshape(T, Hq, d)[rows, heads].transpose(0, 1).float()
            dk[b, :L, h] = (ds.transpose(1, 2) @ q).sum(0).to(torch.bfloat16)
    return dq.view(s["q"].shape), dk, dv


def _turn(s, x, sign):
    """x [T, H, d] with its pairs turned, in fp32 (angles in 64 bits), rounded once."""
    rot = 2 * s["freq"].shape[0]
    a = s["pos"].double()[s["axes"].long()].T * (s["freq"] * sign)  # [T, pairs]
    cos, sin = a.cos().float()[:, None], a.sin().float()[:, None]
    y = x.float()
    if s["case"]["interleaved"]:
        x1, x2 = y[..., 0:rot:2], y[..., 1:rot:2]
        r = torch.stack((x1 * cos - x2 * sin, x1 * sin + x2 * cos), -1).flatten(-2)
    else:
        x1, x2 = y[..., :rot // 2], y[..., rot // 2:rot]
        r = torch.cat((x1 * cos - x2 * sin, x1 * sin + x2 * cos), -1)
    return torch.cat((r, y[..., rot:]), -1).to(torch.bfloat16)


def _plain_append(s):
    Hkv, d = s["case"]["Hkv"], s["case"]["d"]
    s["kcache"].view(-1, Hkv, d)[s["slot"]] = _turn(s, s["k"], 1)
    s["vcache"].view(-1, Hkv, d)[s["slot"]] = s["v"]
    return _turn(s, s["q"], 1), s["kcache"], s["vcache"]


def _plain_rotate(s):
    sign = -1 if s["case"]["inverse"] else 1
    q, k = _turn(s, s["q"], sign), _turn(s, s["k"], sign)
    if "out" in s:
        s["out"][0].copy_(q)
        s["out"][1].copy_(k)
        return s["out"]
    return q, k


_PLAIN = dict(decode=_plain_decode, grad=_plain_grad, append=_plain_append, rotate=_plain_rotate)


# ------------------------------------------------------------------ work
def work(case):
    """One pass's bytes and operations, from the lengths of its sequences."""
    op, Hq, Hkv, d = (case[k] for k in ("op", "Hq", "Hkv", "d"))
    if op in ("append", "rotate"):
        T = case["T"]
        heads = Hq + (2 if op == "append" else 1) * Hkv
        pairs = sum(int(x) for x in case["sections"].split(","))
        return {"bytes": T * heads * d * 2 * 2, "flops": T * (Hq + Hkv) * pairs * 6}
    new, lens = _lengths(case)
    if op == "decode":
        W, sink = case["window"], case["sink"]
        keys = sum(min(L, W) + min(sink, max(0, L - W)) for L in lens)
        o = 4 if case["f32"] else 2
        return {"bytes": keys * Hkv * d * 2 * 2 + len(lens) * Hq * (d * (2 + o) + 4), "flops": 4 * d * Hq * keys}
    pairs, T, win, sink = 0, sum(new), case["window"], case["sink"]
    for n, L in zip(new, lens):
        if not case["causal"]:
            pairs += n * L
        elif win:
            pairs += sum(min(p + 1, win) + min(sink, max(0, p + 1 - win)) for p in range(L - n, L))
        else:
            pairs += n * (L - n) + n * (n + 1) // 2
    dlse = T * Hq * 4 if case["dlse"] else 0
    return {"bytes": T * Hq * (4 * d * 2 + 4) + sum(lens) * Hkv * d * 2 * 4 + dlse, "flops": 10 * d * Hq * pairs}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The definitions in fp64, from the same inputs: attention a sequence and a block of
    rows at a time (gradients with the forward call's o and lse, which are inputs), rotations
    as complex products."""
    s = prepare(case, seed)
    op, Hq, Hkv, d = (case[k] for k in ("op", "Hq", "Hkv", "d"))
    if op in ("append", "rotate"):
        sign = -1.0 if case.get("inverse") else 1.0
        rot = 2 * s["freq"].shape[0]
        angle = torch.stack([s["pos"][a].double() * f for a, f in zip(s["axes"].tolist(), s["freq"].tolist())], -1)
        unit = torch.polar(torch.ones_like(angle), sign * angle)[:, None]

        def turned(x):
            y = x.double()
            e = y[..., :rot].unflatten(-1, (rot // 2, 2) if case["interleaved"] else (2, rot // 2))
            if not case["interleaved"]:
                e = e.transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(e.contiguous()) * unit)
            z = z if case["interleaved"] else z.transpose(-1, -2)
            return torch.cat((z.flatten(-2), y[..., rot:]), -1)

        if op == "rotate":
            return turned(s["q"]), turned(s["k"])
        kc, vc = s["kcache"].flatten(0, 1).double(), s["vcache"].flatten(0, 1).double()
        kc[s["slot"]] = turned(s["k"])
        vc[s["slot"]] = s["v"].double()
        return turned(s["q"]), kc.view(s["kcache"].shape), vc.view(s["vcache"].shape)
    G = Hq // Hkv
    if op == "decode":
        o = torch.zeros(case["B"], Hq, d, dtype=torch.float64, device=DEV)
        lse = torch.zeros(case["B"], Hq, dtype=torch.float64, device=DEV)
        for b, L in enumerate(s["lens"]):
            j = torch.arange(L, device=DEV)
            j = j[(j >= L - case["window"]) | (j < case["sink"])]
            if case["page"]:
                at = s["table"][b].long()[j // case["page"]], j % case["page"]
            else:
                at = torch.full_like(j, b), j
            k, v = s["kcache"][at].double(), s["vcache"][at].double()
            sc = torch.einsum("hgd,jhd->hgj", s["q"][b].double().view(Hkv, G, d), k) * s["scale"]
            lse[b] = sc.logsumexp(-1).flatten()
            o[b] = torch.einsum("hgj,jhd->hgd", sc.softmax(-1), v).flatten(0, 1)
        return o, lse
    T, step = sum(s["new"]), 1024
    q, do, o = (s[x].reshape(T, Hq, d) for x in ("q", "do", "o"))
    by_head = lambda x: x.double() if case["ragged"] else x.double().transpose(0, 1).reshape(Hq, T)
    lse, dlse = by_head(s["lse"]), None if s["dlse"] is None else by_head(s["dlse"])
    dq = torch.zeros(T, Hq, d, dtype=torch.float64, device=DEV)
    dk, dv = torch.zeros_like(s["kcache"], dtype=torch.float64), torch.zeros_like(s["vcache"], dtype=torch.float64)
    at = 0
    for b, (n, L) in enumerate(zip(s["new"], s["lens"])):
        for i0 in range(0, n, step):
            i1 = min(n, i0 + step)
            p = torch.arange(L - n + i0, L - n + i1, device=DEV)
            j = torch.arange(L, device=DEV)
            if case["causal"]:
                j = j[:L - n + i1]
            if case["window"]:  # the block's keys
                j = j[(j > L - n + i0 - case["window"]) | (j < case["sink"])]
            seen = torch.ones(i1 - i0, len(j), dtype=torch.bool, device=DEV)
            if case["causal"]:
                seen = j[None] <= p[:, None]
            if case["window"]:
                seen &= (p[:, None] - j[None] < case["window"]) | (j[None] < case["sink"])
            for h in range(Hq):
                r, hk = slice(at + i0, at + i1), h // G
                k, v = s["kcache"][b, j, hk].double(), s["vcache"][b, j, hk].double()
                x, g = q[r, h].double(), do[r, h].double()
                w = torch.exp(x @ k.T * s["scale"] - lse[h, r, None]).masked_fill(~seen, 0.0)
                back = g @ v.T - torch.einsum("id,id->i", g, o[r, h].double())[:, None]
                if dlse is not None:
                    back = back + dlse[h, r, None]
                back = w * back * s["scale"]
                dq[r, h] = back @ k
                dk[b, j, hk] += back.T @ x
                dv[b, j, hk] += w.T @ g
        at += n
    return dq.view(s["q"].shape), dk, dv
