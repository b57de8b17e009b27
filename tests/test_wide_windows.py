"""Windows and sinks past what a C int holds are as wide as the sequences, not what is left of their lower bits."""
import pytest
import torch

import attention_forward_tcgen05_gb300 as attn
from attention_forward_tcgen05_gb300._binding import _keys


def test_counts_of_keys():
    for n in (0, 1, 4096, 2 ** 31 - 1, -1):
        assert _keys(n) == n
    assert _keys(2 ** 31) == _keys(2 ** 32 + 3) == _keys(2 ** 63 - 1) == 2 ** 31 - 1
    assert _keys(-2 ** 32 + 5) < 0


WIDE = [dict(window=2 ** 32 + 3), dict(window=3, n_sink=2 ** 32 + 1), dict(window=2 ** 63 - 1, n_sink=2 ** 63 - 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("wide", WIDE, ids=["window", "sinks", "both"])
def test_wider_than_everything(wide):
    S, Hq, Hkv, d = 150, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    q, do, k, v = rnd(1, S, Hq, d), rnd(1, S, Hq, d), rnd(1, S, Hkv, d), rnd(1, S, Hkv, d)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    lens, cu, table = i32(S), i32(0, S), i32(*range(10))[None]
    all_keys = dict(window=S)
    pages = [torch.cat([x[0], torch.zeros(10, Hkv, d, dtype=torch.bfloat16, device="cuda")]).view(10, 16, Hkv, d) for x in (k, v)]

    def weights(lse, **w):
        x = torch.zeros(1, Hkv, 160, device="cuda")
        attn.key_weights(q[0], lse, pages[0], lens, x, page_table=table, cu_seqlens_q=cu, max_sq=S, **w)
        return x

    o, lse = attn.prefill_window(q, k, v, S)
    calls = [lambda **w: attn.prefill_window(q, k, v, w["window"], w.get("n_sink", 0)),
             lambda **w: attn.prefill_varlen(q[0], k, v, cu, lens, S, **w),
             lambda **w: attn.prefill_paged(q[0], *pages, table, cu, lens, S, **w),
             lambda **w: attn.decode_window(q[:, -1], k, v, lens, **w),
             lambda **w: attn.decode_window(q[:, -1], *pages, lens, page_table=table, **w),
             lambda **w: weights(lse[0], **w),
             lambda **w: attn.prefill_backward(do, q, k, v, o, lse, **w),
             lambda **w: attn.prefill_varlen_backward(do[0], q[0], k, v, o[0], lse[0], cu, lens, S, **w)]
    for i, call in enumerate(calls):
        got, want = call(**wide), call(**all_keys)
        for x, y in zip(got, want):
            assert torch.equal(x, y) or (x.double() - y.double()).abs().max() <= 2.0 ** -7 * y.abs().max(), i
    attn.sync_check()
