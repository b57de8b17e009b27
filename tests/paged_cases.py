"""Paged caches for the tests: the pages of a dense cache [B][max_kv][Hkv][d] scattered over
a pool in no order, every slot that holds no key filled with NaN and every unused table
entry with -1, so that a read of either shows."""
import numpy as np
import torch


def make_pages(kc, vc, lens, page, seed, width=None, spare=2):
    """(kpool, vpool, table): page_size `page`, table of `width` entries per sequence."""
    B, _, Hkv, d = kc.shape
    rng = np.random.default_rng(seed)
    per = [-(-int(n) // page) for n in lens]
    width = max(1, max(per, default=0)) if width is None else width
    n_pages = sum(per) + spare
    order = rng.permutation(n_pages)
    kp = torch.full((n_pages, page, Hkv, d), float("nan"), dtype=torch.bfloat16)
    vp = kp.clone()
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        L = int(lens[b])
        for e in range(per[b]):
            g = int(order[at])
            at += 1
            table[b, e] = g
            n = min(page, L - e * page)
            kp[g, :n] = kc[b, e * page:e * page + n]
            vp[g, :n] = vc[b, e * page:e * page + n]
    return kp, vp, table


def gather(pool, table, b, n, page):
    """Keys 0..n-1 of sequence b: [n, Hkv, d]."""
    j = torch.arange(n)
    return pool[table[b, j // page].long(), j % page]


def admitted(Sq, L, causal, window=0, n_sink=0):
    """Mask [Sq, L] of the keys each new row admits (bottom-right)."""
    p = np.arange(Sq)[:, None] + L - Sq
    j = np.arange(L)[None]
    ok = np.ones((Sq, L), bool) if not causal else j <= p
    if window:
        ok &= (j > p - window) | (j < n_sink)
    return ok
