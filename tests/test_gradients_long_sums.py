"""Gradients that are sums of millions of terms of one sign.

The tensor cores' fp32 sums round towards zero, by up to 2^-23 of the sum for every 16 terms.  A
run of at most 32768 rows is summed so: 2^-12 of it at 2^-23 a step, and then in fp32 to nearest.  With q = 0 every
weight is 1 / keys, a power of two here, and the gradients are short products in fp64:
  dv_j = sum_i g_i / n,   dq_i = scale / n (g_i (sum_j v_j k_j^T) - D_i sum_j k_j),   dk = 0.
Beside that: 2^-20 for the weights, and dS rounded to bf16, whose errors of up to 2^-8 of a term, of
either sign, add up to under 2^-13 of a sum of 2^17 and more.  Last, each is rounded to bf16.  Rounding keeps
order, so a sum within a part b of the exact value lies, rounded, between the rounded (1 - b) and (1 + b)
times it: no allowance for the rounding itself, under which values that lie close together (as these do) could
hide a bias of half a step, 2^-8, or show one that is none."""
import math

import pytest
import torch

import attention_forward_tcgen05_gb300 as attn

PART = 2.0 ** -12 + 2.0 ** -13


def _check(got, want):
    """All of these sums are positive."""
    low, high = (want * (1 - PART)).bfloat16(), (want * (1 + PART)).bfloat16()
    off = int(((got < low) | (got > high)).sum())
    assert off == 0, f"{off} of {got.numel()}, the mean off by {((got.double() - want) / want).mean().item():.2e}"


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_a_key(d):
    """4.2 million rows of all heads for each of 16384 keys."""
    S, H, n = 65536, 64, 16384
    g = torch.Generator(device="cuda").manual_seed(1)
    do = (torch.rand(1, S, H, d, generator=g, device="cuda") + 0.5).bfloat16()
    zero = torch.zeros_like(do)
    k = torch.zeros(1, n, 1, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, H, S), math.log(n), device="cuda")
    dq, dk, dv = attn.prefill_backward(do, zero, k, k, zero, lse, causal=False)
    attn.sync_check()
    want = sum(x.double().sum((0, 1, 2)) for x in do.split(4096, 1)) / n
    _check(dv[0, :, 0], want.expand(n, d))
    assert (dq == 0).all() and (dk == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_keys_of_a_row(d):
    """524288 keys for each of 8192 rows."""
    S, H, n = 8192, 4, 524288
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: (torch.rand(*s, generator=g, device="cuda") + 0.5).bfloat16()
    do, k, v = rnd(1, S, H, d), rnd(1, n, 2, d), rnd(1, n, 2, d)
    zero = torch.zeros_like(do)
    lse = torch.full((1, H, S), math.log(n), device="cuda")
    dq, dk, dv = attn.prefill_backward(do, zero, k, v, zero, lse, causal=False)
    attn.sync_check()
    scale = 1 / math.sqrt(d)
    for h in range(H):
        m = v[0, :, h // 2].double().T @ k[0, :, h // 2].double()
        _check(dq[0, :, h], do[0, :, h].double() @ m * (scale / n))
    for h in range(2):
        _check(dv[0, :, h], (do[0, :, 2 * h:2 * h + 2].double().sum((0, 1)) / n).expand(n, d))
    assert (dk == 0).all()


@pytest.mark.gpu
def test_two_terms():
    """196608 rows of a group's heads for a sequence's only key: of two terms each (2^-17 of a weight left out),
    so twice the sums.  lse = 0.1, as whole numbers would be summed exactly."""
    B, S, H, G, d = 10, 24576, 128, 8, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    do = (torch.rand(B, S, H, d, generator=g, device="cuda") + 0.5).bfloat16()
    zero = torch.zeros_like(do)
    k = torch.zeros(B, 1, H // G, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H, S), 0.1, device="cuda")
    dq, dk, dv = attn.prefill_backward(do, zero, k, k, zero, lse, causal=False)
    attn.sync_check()
    want = sum(x.double().sum(1) for x in do.split(2048, 1)).unflatten(1, (H // G, G)).sum(2) * math.exp(-lse[0, 0, 0].item())
    _check(dv[:, 0], want)
    assert (dq == 0).all() and (dk == 0).all()
