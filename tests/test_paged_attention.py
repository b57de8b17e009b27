"""Attention of new tokens over a paged cache (chunks and single tokens) against the fp64
oracle.  O and LSE tolerances are those of the dense entry points (tests/tolerances.py):
the same products, sums and roundings."""
import numpy as np
import pytest
import torch

import oracle
import attention_forward_tcgen05_gb300 as attn
from attention_forward_tcgen05_gb300 import workloads as W
from tests.paged_cases import make_pages
from tests.tolerances import check_lse, check_o, log_parity

pytestmark = pytest.mark.gpu

LENS = [0, 1, 15, 16, 17, 63, 64, 65, 128, 300, 1000, 47]


def _decode_case(lens, Hq, Hkv, d, page, seed, width=None):
    lens = torch.tensor(lens, dtype=torch.int32)
    q, kc, vc = W.decode_inputs(len(lens), Hq, Hkv, d, lens, seed)
    kp, vp, table = make_pages(kc, vc, lens, page, seed, width)
    return q, kc, vc, lens, kp.cuda(), vp.cuda(), table.cuda()


def _check_decode(o, lse, q, kc, vc, lens, scale, bf16):
    attn.sync_check()
    ro, rl = oracle.decode(q, kc, vc, lens, scale)
    eo = check_o(o.float().cpu().numpy(), ro, bf16)
    el = check_lse(lse.cpu().numpy(), rl)
    return eo, el


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (14, 2), (8, 1), (12, 1), (40, 2), (128, 1), (67, 1)])
@pytest.mark.parametrize("page", [1, 16, 48, 256])
def test_decode(d, Hq, Hkv, page):
    q, kc, vc, lens, kp, vp, table = _decode_case(LENS, Hq, Hkv, d, page, 300 + d + page)
    scale = 1.0 / np.sqrt(d)
    for out_dtype, kw in ((torch.float32, {}), (torch.bfloat16, {}),
                          (torch.bfloat16, dict(n_splits=5, min_rows_per_split=33))):
        o, lse = attn.decode_paged(q.cuda(), kp, vp, table, lens.cuda(), scale=scale, out_dtype=out_dtype, **kw)
        _check_decode(o, lse, q, kc, vc, lens, scale, out_dtype == torch.bfloat16)


@pytest.mark.parametrize("Hq,Hkv,d", [(32, 2, 64), (12, 1, 128), (24, 2, 256), (16, 1, 128), (4, 2, 64), (7, 1, 128),
                                      (8, 1, 256)])
def test_decode_of_many_sequences(Hq, Hkv, d):
    """160 units: more CTAs than SMs, and than one wave of tiles holds for groups of 9 to 16."""
    rng = np.random.default_rng(9)
    lens = [int(x) for x in rng.integers(0, 200, 160 // Hkv)]
    q, kc, vc, lens, kp, vp, table = _decode_case(lens, Hq, Hkv, d, 16, 330 + d)
    for n_splits in (0, 1, 3):
        for dt in (torch.bfloat16, torch.float32):
            o, lse = attn.decode_paged(q.cuda(), kp, vp, table, lens.cuda(), n_splits, out_dtype=dt)
            _check_decode(o, lse, q, kc, vc, lens, 1.0 / np.sqrt(d), dt is torch.bfloat16)


@pytest.mark.parametrize("n_splits,min_rows", [(1, 0), (3, 100), (8, 1)])
def test_decode_splits_as_dense(n_splits, min_rows):
    """The split rule of the dense decode: its partials and results to rounding."""
    q, kc, vc, lens, kp, vp, table = _decode_case(LENS, 28, 4, 128, 16, 310)
    parts = [(torch.empty(len(LENS), 28, n_splits, 128, device="cuda"), torch.empty(len(LENS), 28, n_splits, device="cuda"))
             for _ in range(2)]
    o, lse = attn.decode_paged(q.cuda(), kp, vp, table, lens.cuda(), n_splits, min_rows, out_dtype=torch.float32,
                               parts=parts[0])
    o2, lse2 = attn.decode(q.cuda(), kc.cuda(), vc.cuda(), lens.cuda(), n_splits, min_rows, out_dtype=torch.float32,
                           parts=parts[1])
    attn.sync_check()
    pairs = [(o, o2), (lse, lse2)]
    if n_splits > 1:  # (one split is the result itself: no partials)
        pairs += [(parts[0][0], parts[1][0]), (parts[0][1], parts[1][1])]
    for x, y in pairs:
        x, y = x.double().cpu().numpy(), y.double().cpu().numpy()
        assert np.array_equal(np.isneginf(x), np.isneginf(y))
        fin = np.isfinite(x)
        # sums of up to 1000 fp32 terms around 1 in another order, P to 2^-17: both sides below 1e-4
        assert abs(x[fin] - y[fin]).max() <= 2e-4


def test_decode_ragged_workload():
    """The ragged 64-sequence batch from pages of 64."""
    s = W.RAGGED_DECODE
    q, kc, vc, lens = W.decode_inputs_for(s)
    kp, vp, table = make_pages(kc, vc, lens, 64, 311)
    o, lse = attn.decode_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), scale=s.scale)
    eo, el = _check_decode(o, lse, q, kc, vc, lens, s.scale, True)
    log_parity("decode_paged " + s.name, eo, el)


@pytest.mark.parametrize("d,Hq,Hkv,n_splits", [(64, 8, 1, 1), (128, 28, 4, 3), (256, 16, 1, 2)])
def test_decode_fp32_output(d, Hq, Hkv, n_splits):
    """An fp32 O is good to fp32 sums: off by at most 2^-18 of sum p |v|.  That holds the score's
    fp32 dot product (the mma's truncation, d 2^-23 of scale sum |q k| at most, on average the
    root of that), ex2 (2^-22), P's three terms (2^-25) and the sums' roundings."""
    lens = torch.tensor([3000, 1, 77, 1500], dtype=torch.int32)
    q, kc, vc = W.decode_inputs(4, Hq, Hkv, d, lens, 320 + d)
    kp, vp, table = make_pages(kc, vc, lens, 16, 320)
    o, _ = attn.decode_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), n_splits,
                             out_dtype=torch.float32)
    attn.sync_check()
    o = o.double().cpu()
    G = Hq // Hkv
    for b, L in enumerate(lens.tolist()):
        for h in range(Hq):
            k, v = kc[b, :L, h // G].double(), vc[b, :L, h // G].double()
            p = torch.softmax(q[b, h].double() @ k.T / np.sqrt(d), -1)
            assert ((o[b, h] - p @ v).abs() <= 2.0 ** -18 * (p @ v.abs())).all(), (b, h)


def test_decode_shared_pages():
    """Two sequences that share their first pages (a common prefix)."""
    lens = torch.tensor([200, 170], dtype=torch.int32)
    q, kc, vc = W.decode_inputs(2, 8, 2, 64, lens, 312)
    kc[1, :96], vc[1, :96] = kc[0, :96], vc[0, :96]
    kp, vp, table = make_pages(kc, vc, lens, 32, 312)
    table[1, :3] = table[0, :3]
    o, lse = attn.decode_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), lens.cuda(), out_dtype=torch.float32)
    _check_decode(o, lse, q, kc, vc, lens, 0.125, False)


def test_bad_page_is_reported():
    """A table entry in use that is no page of the pool: read as zeros and reported; the
    other sequences' outputs stand, and the next call is clean."""
    q, kc, vc, lens, kp, vp, table = _decode_case([100, 100], 8, 2, 128, 16, 313)
    good, _ = attn.decode_paged(q.cuda(), kp, vp, table, lens.cuda(), out_dtype=torch.float32)
    attn.sync_check()
    for bad in (-1, kp.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 3] = bad
        o, _ = attn.decode_paged(q.cuda(), kp, vp, t, lens.cuda(), out_dtype=torch.float32)
        with pytest.raises(attn.AttnError) as e:
            attn.sync_check()
        assert e.value.status == attn.ATTN_ERR_DEVICE_INPUT
        assert torch.equal(o[0], good[0])
        cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
        attn.prefill_paged(q.cuda(), kp, vp, t, cu, lens.cuda(), 1)
        with pytest.raises(attn.AttnError):
            attn.sync_check()
    o, _ = attn.decode_paged(q.cuda(), kp, vp, table, lens.cuda(), out_dtype=torch.float32)
    attn.sync_check()
    assert torch.equal(o, good)


def test_bad_page_of_whole_tiles_is_reported():
    """The same where whole tiles are copied by pages: the other sequence stands."""
    q, kc, vc, lens, kp, vp, table = _decode_case([500, 700], 8, 2, 128, 64, 314)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    good, _ = attn.prefill_paged(q.cuda(), kp, vp, table, cu, lens.cuda(), 1, out_dtype=torch.float32)
    attn.sync_check()
    for bad in (-1, kp.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 2] = bad
        o, _ = attn.prefill_paged(q.cuda(), kp, vp, t, cu, lens.cuda(), 1, out_dtype=torch.float32)
        with pytest.raises(attn.AttnError) as e:
            attn.sync_check()
        assert e.value.status == attn.ATTN_ERR_DEVICE_INPUT
        assert torch.equal(o[0], good[0])


# ------------------------------------------------------------------ chunks
MIXED = [(1, 1), (77, 300), (128, 128), (300, 1200), (0, 50), (200, 150), (129, 1000), (3, 0), (36, 36)]
SHORT = [(1, 1), (5, 300), (9, 9), (3, 1200), (0, 50), (8, 2), (4, 129)]


def _chunk_case(seqs, Hq, Hkv, d, page, seed):
    sq = torch.tensor([a for a, _ in seqs], dtype=torch.int32)
    kv = torch.tensor([b for _, b in seqs], dtype=torch.int32)
    q, kc, vc, cu = W.varlen_inputs(len(seqs), Hq, Hkv, d, sq, kv, seed)
    kp, vp, table = make_pages(kc, vc, kv, page, seed)
    return q, kc, vc, cu, kv, kp.cuda(), vp.cuda(), table.cuda(), int(sq.max())


def _run(case, **kw):
    q, kc, vc, cu, kv, kp, vp, table, max_sq = case
    o, lse = attn.prefill_paged(q.cuda(), kp, vp, table, cu.cuda(), kv.cuda(), max_sq, **kw)
    attn.sync_check()
    return o, lse


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,page", [(4, 2, 16), (7, 1, 48), (5, 5, 128), (2, 1, 8), (3, 1, 20), (1, 1, 1)])
@pytest.mark.parametrize("seqs", [MIXED, SHORT], ids=["mixed", "short"])
def test_chunks(d, causal, Hq, Hkv, page, seqs):
    case = _chunk_case(seqs, Hq, Hkv, d, page, 400 + d + page)
    q, kc, vc, cu, kv = case[:5]
    scale = 1.0 / np.sqrt(d)
    ro, rl = oracle.sdpa_varlen(q, kc, vc, cu, kv, causal, scale)
    for out_dtype, n_splits in ((torch.float32, 1), (torch.bfloat16, 1), (torch.bfloat16, 3), (torch.float32, 0)):
        o, lse = _run(case, causal=causal, scale=scale, out_dtype=out_dtype, n_splits=n_splits)
        check_o(o.float().cpu().numpy(), ro, out_dtype == torch.bfloat16, f"O, {n_splits} splits")
        check_lse(lse.cpu().numpy(), rl)


@pytest.mark.parametrize("d,seqs,n_splits", [(64, MIXED, 1), (128, MIXED, 3), (256, MIXED, 1), (128, SHORT, 1)])
def test_chunk_fp32_output(d, seqs, n_splits):
    """An fp32 O is off by at most 2^-15 of sum p |v|: P's two terms leave out 2^-17 of it, the
    mma's accumulation truncates 2^-24 in each of its L / 8 steps (2^-17 at 1200 keys), the
    score's dot product and ex2 are below 2^-18."""
    case = _chunk_case(seqs, 4, 2, d, 16, 440 + d)
    q, kc, vc, cu, kv = case[:5]
    scale = 1.0 / np.sqrt(d)
    o, _ = _run(case, scale=scale, out_dtype=torch.float32, n_splits=n_splits)
    o = o.double().cpu().numpy()
    from tests.paged_cases import admitted
    for b in range(len(seqs)):
        a, e, L = int(cu[b]), int(cu[b + 1]), int(kv[b])
        if L == 0 or a == e:
            assert not o[a:e].any()
            continue
        ok = admitted(e - a, L, True)
        for h in range(4):
            k, v = kc[b, :L, h // 2].double().numpy(), vc[b, :L, h // 2].double().numpy()
            s = np.where(ok, scale * (q[a:e, h].double().numpy() @ k.T), -np.inf)
            live = ok.any(1)
            p = np.zeros_like(s)
            p[live] = np.exp(s[live] - s[live].max(1, keepdims=True))
            p[live] /= p[live].sum(1, keepdims=True)
            assert (abs(o[a:e, h] - p @ v) <= 2.0 ** -15 * (p @ abs(v))).all(), (b, h)


@pytest.mark.parametrize("G", [1, 3, 9, 16, 24, 67, 100, 128, 150])
def test_chunk_head_groups(G):
    """Head groups that do and do not divide a tile, of one and of several tiles."""
    for seqs in ([(1, 200), (40, 140)], [(1, 90), (1, 1)]):
        case = _chunk_case(seqs, G, 1, 64, 32, 430 + G)
        q, kc, vc, cu, kv = case[:5]
        ro, rl = oracle.sdpa_varlen(q, kc, vc, cu, kv, True, 0.125)
        for out_dtype in (torch.float32, torch.bfloat16):
            o, lse = _run(case, scale=0.125, out_dtype=out_dtype)
            check_o(o.float().cpu().numpy(), ro, out_dtype == torch.bfloat16)
            check_lse(lse.cpu().numpy(), rl)


def test_splits_of_more_rows_than_any_sequence():
    """The largest min_rows_per_split an int holds: one split takes every key."""
    big = (1 << 31) - 1
    case = _chunk_case(MIXED, 4, 2, 128, 16, 445)
    q, kc, vc, cu, kv = case[:5]
    ro, rl = oracle.sdpa_varlen(q, kc, vc, cu, kv, True, 0.1)
    o, lse = _run(case, scale=0.1, out_dtype=torch.float32, n_splits=3, min_rows_per_split=big)
    check_o(o.cpu().numpy(), ro, False)
    check_lse(lse.cpu().numpy(), rl)
    for Hq in (4, 12, 20):
        q, kc, vc, lens, kp, vp, table = _decode_case(LENS, Hq, 1, 64, 16, 446)
        o, lse = attn.decode_paged(q.cuda(), kp, vp, table, lens.cuda(), 3, big, 0.125)
        _check_decode(o, lse, q, kc, vc, lens, 0.125, True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,n_sink", [(1, 0), (100, 4), (256, 130), (2000, 7)])
def test_chunk_window(d, window, n_sink):
    for seqs, page in ((MIXED, 16), (SHORT, 48), (MIXED, 20)):
        case = _chunk_case(seqs, 7, 1, d, page, 450 + d + window)
        q, kc, vc, cu, kv = case[:5]
        scale = 1.0 / np.sqrt(d)
        o, lse = _run(case, scale=scale, out_dtype=torch.float32, window=window, n_sink=n_sink)
        ro, rl = oracle.sdpa_varlen_window(q, kc, vc, cu, kv, window, n_sink, scale)
        check_o(o.cpu().numpy(), ro, False)
        check_lse(lse.cpu().numpy(), rl)


def test_chunk_workload():
    """The chunked prefill batch from pages of 64, with and without key splits."""
    s = W.CHUNKED_PREFILL
    q, kc, vc, cu, kv = W.varlen_inputs_for(s)
    kp, vp, table = make_pages(kc, vc, kv, 64, 460)
    ro, rl = oracle.sdpa_varlen(q, kc, vc, cu, kv, True, s.scale)
    for n in (1, 2):
        o, lse = attn.prefill_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), cu.cuda(), kv.cuda(),
                                    int((cu[1:] - cu[:-1]).max()), scale=s.scale, n_splits=n)
        attn.sync_check()
        eo, el = check_o(o.float().cpu().numpy(), ro, True), check_lse(lse.cpu().numpy(), rl)
        log_parity(f"prefill_paged {s.name} splits={n}", eo, el)


def test_chunk_rows_behind_the_last_sequence_stay():
    """A padded batch: cu_seqlens_q ends before total_q; the rows behind keep their bytes."""
    case = list(_chunk_case([(30, 100), (9, 20)], 4, 2, 128, 16, 470))
    q, kc, vc, cu, kv, kp, vp, table, max_sq = case
    pad = torch.full((50, 4, 128), float("nan"), dtype=torch.bfloat16)
    qp = torch.cat([q, pad]).cuda()
    for n_splits in (1, 2):
        for dt in (torch.bfloat16, torch.float32):
            o = torch.full((89, 4, 128), 7.0, dtype=dt, device="cuda")
            lse = torch.full((4, 89), 7.0, device="cuda")
            attn.prefill_paged(qp, kp, vp, table, cu.cuda(), kv.cuda(), max_sq, scale=0.1, n_splits=n_splits,
                               out=(o, lse))
            attn.sync_check()
            ro, rl = oracle.sdpa_varlen(q, kc, vc, cu, kv, True, 0.1)
            check_o(o[:39].float().cpu().numpy(), ro, dt == torch.bfloat16)
            check_lse(lse[:, :39].cpu().numpy(), rl)
            assert (o[39:] == 7).all() and (lse[:, 39:] == 7).all()


def test_long_cache_addresses():
    """A pool of more than 2^31 elements and a page behind that offset."""
    page, Hkv, d = 256, 8, 256
    n_pages = 2 ** 31 // (page * Hkv * d) + 8
    kp = torch.zeros(n_pages, page, Hkv, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    lens = torch.tensor([300, 77], dtype=torch.int32)
    q, kc, vc = W.decode_inputs(2, 8, Hkv, d, lens, 480)
    table = torch.tensor([[n_pages - 1, n_pages - 3], [2, -1]], dtype=torch.int32)
    for b in range(2):
        for e in range(-(-int(lens[b]) // page)):
            n = min(page, int(lens[b]) - e * page)
            kp[int(table[b, e]), :n] = kc[b, e * page:e * page + n].cuda()
            vp[int(table[b, e]), :n] = vc[b, e * page:e * page + n].cuda()
    scale = 1.0 / 16
    o, lse = attn.decode_paged(q.cuda(), kp, vp, table.cuda(), lens.cuda(), scale=scale, out_dtype=torch.float32)
    _check_decode(o, lse, q, kc, vc, lens, scale, False)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    o2, lse2 = attn.prefill_paged(q.cuda(), kp, vp, table.cuda(), cu, lens.cuda(), 1, scale=scale,
                                  out_dtype=torch.float32)
    _check_decode(o2, lse2.T.contiguous(), q, kc, vc, lens, scale, False)
