"""Windowed attention of single tokens against the fp64 oracle's decode over the admitted keys
alone, moved together.  O and LSE tolerances are those of the other decode calls
(tests/tolerances.py): the same products, sums and roundings.  Keys out of the window and the
sinks hold NaN, and pages without an admitted key have left the table: neither may be read."""
import numpy as np
import pytest
import torch

import oracle
import attention_forward_tcgen05_gb300 as attn
from attention_forward_tcgen05_gb300 import workloads as W
from tests.paged_cases import make_pages
from tests.tolerances import check_lse, check_o

pytestmark = pytest.mark.gpu

LENS = [0, 1, 15, 16, 17, 64, 65, 128, 129, 300, 1000, 47]


def admitted(L, window, sink):
    return [j for j in range(L) if j >= L - window or j < sink]


def _case(lens, Hq, Hkv, d, page, window, sink, seed, junk=-1, width=None):
    """(q, compact K and V of the admitted keys, their counts, lens, caches and table on the GPU)"""
    lens = torch.tensor(lens, dtype=torch.int32)
    B = len(lens)
    q, kc, vc = W.decode_inputs(B, Hq, Hkv, d, lens, seed)
    keep = [admitted(int(L), window, sink) for L in lens]
    n = torch.tensor([len(k) for k in keep], dtype=torch.int32)
    ck = torch.zeros(B, max(1, int(n.max())), Hkv, d, dtype=torch.bfloat16)
    cv = torch.zeros_like(ck)
    for b, k in enumerate(keep):
        ck[b, :len(k)], cv[b, :len(k)] = kc[b, k], vc[b, k]
        hide = torch.ones(kc.shape[1], dtype=torch.bool)
        hide[k] = False
        kc[b, hide], vc[b, hide] = float("nan"), float("nan")
    if page is None:
        return q, ck, cv, n, lens, kc.cuda(), vc.cuda(), None
    kp, vp, table = make_pages(kc, vc, lens, page, seed, width)
    for b, k in enumerate(keep):
        for e in range(table.shape[1]):
            if not any(e * page <= j < (e + 1) * page for j in k):
                table[b, e] = junk  # given back
    return q, ck, cv, n, lens, kp.cuda(), vp.cuda(), table.cuda()


def _check(o, lse, q, ck, cv, n, scale, bf16):
    attn.sync_check()
    ro, rl = oracle.decode(q, ck, cv, n, scale)
    check_o(o.float().cpu().numpy(), ro, bf16)
    check_lse(lse.cpu().numpy(), rl)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (14, 2), (8, 1), (12, 1), (40, 2), (128, 1), (67, 1)])
@pytest.mark.parametrize("page,window,sink", [(None, 64, 0), (1, 1, 0), (1, 100, 3), (16, 64, 4), (48, 50, 70), (256, 129, 1),
                                              (16, 5000, 9), (None, 17, 40)])
def test_against_the_oracle(d, Hq, Hkv, page, window, sink):
    q, ck, cv, n, lens, kc, vc, table = _case(LENS, Hq, Hkv, d, page, window, sink, 700 + d + window)
    scale = 1.0 / np.sqrt(d)
    for dt, kw in ((torch.float32, {}), (torch.bfloat16, {}), (torch.bfloat16, dict(n_splits=5, min_rows_per_split=33)),
                   (torch.float32, dict(n_splits=1))):
        o, lse = attn.decode_window(q.cuda(), kc, vc, lens.cuda(), window, sink, page_table=table, out_dtype=dt, **kw)
        _check(o, lse, q, ck, cv, n, scale, dt is torch.bfloat16)


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 16, 2), (128, 28, 4), (256, 9, 1), (128, 40, 2)])
def test_long_contexts(d, Hq, Hkv):
    """Few sequences far past their window, many splits; the table is junk between sinks and window."""
    q, ck, cv, n, lens, kp, vp, table = _case([20011, 9000, 4097], Hq, Hkv, d, 32, 4096, 5, 40 + d, junk=1 << 30)
    for dt in (torch.bfloat16, torch.float32):
        o, lse = attn.decode_window(q.cuda(), kp, vp, lens.cuda(), 4096, 5, page_table=table, out_dtype=dt)
        _check(o, lse, q, ck, cv, n, 1.0 / np.sqrt(d), dt is torch.bfloat16)


@pytest.mark.parametrize("Hq,Hkv,d", [(32, 2, 64), (24, 2, 256), (16, 1, 128), (7, 1, 128)])
def test_many_sequences(Hq, Hkv, d):
    rng = np.random.default_rng(9)
    lens = [int(x) for x in rng.integers(0, 400, 320 // Hkv)]
    q, ck, cv, n, lens, kp, vp, table = _case(lens, Hq, Hkv, d, 16, 90, 4, 330 + d)
    for n_splits in (0, 1, 3):
        o, lse = attn.decode_window(q.cuda(), kp, vp, lens.cuda(), 90, 4, page_table=table, n_splits=n_splits)
        _check(o, lse, q, ck, cv, n, 1.0 / np.sqrt(d), True)


def test_a_window_of_everything_is_decode_paged():
    """The same bits: the list of admitted keys is the sequence itself."""
    q, _, _, _, lens, kp, vp, table = _case(LENS, 14, 2, 128, 16, 5000, 0, 12)
    for dt in (torch.bfloat16, torch.float32):
        for n_splits in (1, 4):
            x = attn.decode_window(q.cuda(), kp, vp, lens.cuda(), 5000, 0, page_table=table, n_splits=n_splits, out_dtype=dt)
            y = attn.decode_paged(q.cuda(), kp, vp, table, lens.cuda(), n_splits=n_splits, out_dtype=dt)
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    attn.sync_check()


def test_partials_follow_the_list():
    """Splits cut the admitted keys: the partials of the compact dense cache's decode, to rounding."""
    window, sink, S = 200, 6, 3
    q, ck, cv, n, lens, kp, vp, table = _case([1000, 150, 0, 207], 8, 2, 64, 16, window, sink, 77)
    parts = [(torch.empty(4, 8, S, 64, device="cuda"), torch.empty(4, 8, S, device="cuda")) for _ in range(2)]
    attn.decode_window(q.cuda(), kp, vp, lens.cuda(), window, sink, page_table=table, n_splits=S, min_rows_per_split=50,
                       out_dtype=torch.float32, parts=parts[0])
    attn.decode(q.cuda(), ck.cuda(), cv.cuda(), n.cuda(), S, 50, out_dtype=torch.float32, parts=parts[1])
    attn.sync_check()
    for x, y in zip(*parts):
        x, y = x.double().cpu().numpy(), y.double().cpu().numpy()
        assert np.array_equal(np.isneginf(x), np.isneginf(y))
        fin = np.isfinite(x)
        # sums of up to 206 fp32 terms around 1 in another order, P to 2^-17: both sides below 1e-4
        assert abs(x[fin] - y[fin]).max() <= 2e-4


def test_a_used_entry_that_is_no_page_is_reported():
    q, ck, cv, n, lens, kp, vp, table = _case([300], 4, 2, 64, 16, 64, 4, 5)
    table[0, 0] = kp.shape[0]  # the sinks' page
    attn.decode_window(q.cuda(), kp, vp, lens.cuda(), 64, 4, page_table=table)
    with pytest.raises(attn.AttnError) as e:
        attn.sync_check()
    assert e.value.status == attn.ATTN_ERR_DEVICE_INPUT
    # and the next call is sound
    o, lse = attn.decode_window(q.cuda(), kp, vp, lens.cuda(), 64, 0, page_table=table, out_dtype=torch.float32)
    q, ck, cv, n, *_ = _case([300], 4, 2, 64, 16, 64, 0, 5)
    _check(o, lse, q, ck, cv, n, 0.125, False)


def test_given_outputs_streams_and_a_graph():
    q, ck, cv, n, lens, kp, vp, table = _case([2000, 700], 8, 2, 128, 16, 512, 4, 21)
    q2 = torch.flip(q, (1,)).contiguous()
    qs, ls = q.cuda(), lens.cuda()
    out = torch.empty_like(qs), torch.empty(2, 8, device="cuda")
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = attn.decode_window(qs, kp, vp, ls, 512, 4, page_table=table, stream=side, out=out, n_splits=3)
    assert got[0] is out[0]
    side.synchronize()
    _check(*out, q, ck, cv, n, 1 / np.sqrt(128), True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=other):
        o, lse = attn.decode_window(qs, kp, vp, ls, 512, 4, page_table=table, n_splits=3)
    for x in (q2, q):
        qs.copy_(x.cuda())
        # another call on another stream meanwhile, with a workspace of its own
        side.wait_stream(torch.cuda.current_stream())
        a, b = attn.decode_window(qs, kp, vp, ls, 512, 4, page_table=table, n_splits=3, stream=side)
        graph.replay()
        torch.cuda.synchronize()
        _check(o, lse, x, ck, cv, n, 1 / np.sqrt(128), True)
        assert torch.equal(a, o) and torch.equal(b, lse)
