"""Gradients that are sums of millions of terms of one sign.

The tensor cores' fp32 sums round towards zero, by up to 2^-23 of the sum for every 16 terms.  A
run of at most 32768 rows is summed so: 2^-12 of it at 2^-23 a step, and then in fp32 to nearest.  With q = 0 every
weight is 1 / keys, a power of two here, and the gradients are short products in fp64:
  dv_j = sum_i g_i / n,   dq_i = scale / n (g_i (sum_j v_j k_j^T) - D_i sum_j k_j),   dk = 0.
Beside that: 2^-8 of each for its rounding (half a step of bf16's 8 bits), 2^-20 for the weights, and dS
rounded to bf16, whose errors of up to 2^-8 of a term, of either sign, add up to under 2^-13 of a sum of
2^17 and more.

The errors' mean shows the sums' bias where a single rounding hides it.  Rounding to bf16 leaves
errors of a standard deviation of at most 2^-8 / sqrt(3), and so 2^-8 / sqrt(3 n) for the mean of n
values; four of that are allowed."""
import math

import pytest
import torch

import attention_forward_tcgen05_gb300 as attn

BIAS = 2.0 ** -12


def _check(got, want, n):
    """n: values of want that are not the same."""
    e = (got.double() - want) / want
    assert e.abs().max().item() <= 2.0 ** -8 + BIAS + 2.0 ** -12
    assert abs(e.mean().item()) <= BIAS + 4 * 2.0 ** -8 / math.sqrt(3 * n)


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
    _check(dv[0, :, 0], want.expand(n, d), d)
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
        _check(dq[0, :, h], do[0, :, h].double() @ m * (scale / n), S * d)
    for h in range(2):
        _check(dv[0, :, h], (do[0, :, 2 * h:2 * h + 2].double().sum((0, 1)) / n).expand(n, d), d)
    assert (dk == 0).all()
