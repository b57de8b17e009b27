"""Calls of the paged serving functions at the edge of what they document: errors on one
stream beside work on another, arguments left out, the largest sizes."""
import math
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

import oracle
import attention_forward_tcgen05_gb300 as attn
from attention_forward_tcgen05_gb300 import _binding
from attention_forward_tcgen05_gb300 import build as attn_build
from attention_forward_tcgen05_gb300 import workloads as W
from tests.paged_cases import gather, make_pages
from tests.test_evict import lse_of, weights_ref
from tests.tolerances import check_lse, check_o, half_ulp_bf16


@pytest.fixture(scope="module", autouse=True)
def lib():
    attn_build.build()
    return attn.load()


# ------------------------------------------------------------------ sync_check
class _Buffer:
    """A stand-in for a counter buffer that notes when it is zeroed."""

    def __init__(self, device, log):
        self.device, self.log = device, log

    def zero_(self):
        self.log.append(("zero", self.device, _binding._launching.locked()))


def test_counters_are_zeroed_only_between_synchronisations(monkeypatch):
    """After a device error the shared counters are zeroed with every device that owns one
    idle: synchronised before (another stream may be counting on its buffer) and after (the
    next launch may be on any stream), and no split call launches in between."""
    log = []
    bufs = {("cuda", 0): _Buffer("cuda:0", log), (0, 77): _Buffer("cuda:0", log), (1, 5): _Buffer("cuda:1", log)}
    monkeypatch.setattr(_binding, "_counters", bufs)
    monkeypatch.setattr(_binding, "_stream_handle", lambda stream: None)
    monkeypatch.setattr(_binding, "attn_sync_check", lambda s: attn.ATTN_ERR_DEVICE_INPUT)
    monkeypatch.setattr(torch.cuda, "synchronize",
                        lambda device=None: log.append(("sync", str(device), _binding._launching.locked())))
    with pytest.raises(attn.AttnError):
        attn.sync_check()
    assert all(locked for _, _, locked in log)
    zeroed = [i for i, x in enumerate(log) if x[0] == "zero"]
    assert len(zeroed) == 3
    for device in ("cuda:0", "cuda:1"):
        synced = [i for i, x in enumerate(log) if x[:2] == ("sync", device)]
        mine = [i for i in zeroed if log[i][1] == device]
        assert min(synced) < min(mine) and max(synced) > max(mine)
    assert not _binding._launching.locked()


@pytest.mark.gpu
def test_an_error_on_one_stream_leaves_the_decodes_of_another():
    """A bad page is reported on one stream, again and again, while split decodes run on
    another: those, and the ones after, come out as alone."""
    B, Hq, Hkv, d, page = 32, 32, 8, 128, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    lens = torch.randint(2000, 4097, (B,), generator=g, device="cuda", dtype=torch.int32)
    table = torch.randperm(B * 64, generator=g, device="cuda").to(torch.int32).view(B, 64)
    kp, vp = (torch.randn(B * 64, page, Hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(B, Hq, d, generator=g, device="cuda").bfloat16()
    bad = torch.full((1, 1), -1, dtype=torch.int32, device="cuda")
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    busy = torch.cuda.Stream()
    outs = [(torch.empty(B, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(B, Hq, device="cuda"))
            for _ in range(40)]
    torch.cuda.synchronize()

    def decode(out=None):
        with torch.cuda.stream(busy):
            return attn.decode_paged(q, kp, vp, table, lens, 9, out=out)

    o, lse = decode()
    torch.cuda.synchronize()
    attn.sync_check()
    want = o.clone(), lse.clone()
    for i, out in enumerate(outs):
        out[0].fill_(float("nan"))
    torch.cuda.synchronize()
    reported = 0
    for i, out in enumerate(outs):
        decode(out)
        if i % 4 == 3:
            attn.decode_paged(q[:1], kp, vp, bad, one, 1)
            with pytest.raises(attn.AttnError) as e:
                attn.sync_check()
            assert e.value.status == attn.ATTN_ERR_DEVICE_INPUT
            reported += 1
    torch.cuda.synchronize()
    attn.sync_check()
    assert reported == 10
    for i, (o, lse) in enumerate(outs):
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), i


# ------------------------------------------------------------------ key weights
def test_key_weights_of_packed_rows_need_max_sq():
    """Left out, the launch would be sized for one row a sequence: refused, whatever else is
    wrong with the call."""
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    w, lens, cu = torch.zeros(2, 2, 16), torch.ones(2, dtype=torch.int32), torch.tensor([0, 2, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="max_sq"):
        attn.key_weights(x, w[:, 0, :4], c, lens, w, cu_seqlens_q=cu)
    with pytest.raises(TypeError):  # (given, the host tensors are what is wrong)
        attn.key_weights(x, w[:, 0, :4], c, lens, w, cu_seqlens_q=cu, max_sq=2)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [[3, 2], [40, 2], [2, 40]])
@pytest.mark.parametrize("G", [1, 4])
def test_key_weights_report_a_sequence_above_max_sq(rows, G):
    Hkv, d = 2, 64
    kv = torch.tensor([100, 100], dtype=torch.int32)
    q, kc, _, cu = W.varlen_inputs(2, G * Hkv, Hkv, d, torch.tensor(rows, dtype=torch.int32), kv, 31)
    lse = torch.zeros(G * Hkv, sum(rows), device="cuda")
    w = torch.zeros(2, Hkv, 100, device="cuda")

    def call(max_sq):
        attn.key_weights(q.cuda(), lse, kc.cuda(), kv.cuda(), w, cu_seqlens_q=cu.cuda(), max_sq=max_sq)
        attn.sync_check()

    call(max(rows))
    call(1000)
    with pytest.raises(attn.AttnError) as e:
        call(max(rows) - 1)
    assert e.value.status == attn.ATTN_ERR_DEVICE_INPUT
    call(max(rows))


# ------------------------------------------------------------------ rotary append
@pytest.mark.gpu
@pytest.mark.parametrize("long", [False, True], ids=["one_a_cta", "eight_a_cta"])
def test_append_clamps_cu_seqlens_as_attention_does(long):
    """cu_seqlens_q whose first entry lies below 0 and whose last one above total: the append
    counts a sequence's tokens within [0, total], as the attention calls do, so both put the
    same token at the same key."""
    n = [1500, 7, 1200] if long else [5, 7, 4]
    lens = [n[0] + 3, 20, n[2] + 9]
    T, Hkv, d, page = sum(n), 2, 64, 32
    cu = torch.tensor([-6, n[0], n[0] + n[1], T + 8], dtype=torch.int32)
    width = -(-max(lens) // page)
    table = torch.randperm(3 * width, generator=torch.Generator().manual_seed(2)).to(torch.int32).view(3, width)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(T, Hkv, d, generator=g).bfloat16() for _ in range(2))
    kp = torch.zeros(3 * width, page, Hkv, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    attn.rope_append(None, k.cuda(), v.cuda(), kp, vp, kv, None, page_table=table.cuda(), cu_seqlens_q=cu.cuda())
    attn.sync_check()
    want_k, want_v = torch.zeros_like(kp.cpu()), torch.zeros_like(kp.cpu())
    t = 0
    for b in range(3):
        for i in range(n[b]):
            j = lens[b] - n[b] + i
            want_k[table[b, j // page], j % page], want_v[table[b, j // page], j % page] = k[t], v[t]
            t += 1
    assert torch.equal(kp.cpu(), want_k) and torch.equal(vp.cpu(), want_v)


@pytest.mark.gpu
def test_append_to_more_sequences_than_half_an_int():
    """1.6e9 sequences, the tokens in the last one: the search for a token's sequence adds two
    of their numbers.  (19 GB of lengths, offsets and table.)"""
    B, Hkv, d = (1 << 30) + (1 << 29), 1, 64
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, cu, table = torch.zeros(B, **i32), torch.zeros(B + 1, **i32), torch.zeros(B, 1, **i32)
    lens[-1], cu[-1], table[-1] = 8, 8, 1
    k = torch.randn(8, Hkv, d, device="cuda").bfloat16()
    kp = torch.zeros(2, 8, Hkv, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    attn.rope_append(None, k, -k, kp, vp, lens, None, page_table=table, cu_seqlens_q=cu)
    attn.sync_check()
    assert torch.equal(kp[1], k) and torch.equal(vp[1], -k) and not kp[0].any()
    del lens, cu, table
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [1, -1])
def test_far_angles_of_either_sign(sign):
    """The angle itself, at positions above 2^30: with x = (1, 0) the second output is sin a,
    and near a multiple of pi bf16 resolves it to less than the angle's bound, which is
    |p f / 2 pi| 2^-52 + 2^-25 of a turn (times 2 pi in radians; sincospi and the product add
    2^-21 of the value)."""
    inv_2pi = Decimal("0.15915494309189533576888376337251436203445964574045644874766734405889679763")
    T, d = 32768, 64
    pos = np.random.default_rng(11).integers(2 ** 30, 2 ** 31 - 1, T).astype(np.int32)
    freq = sign * attn.rope_frequencies(d, device="cpu")[0]
    x = torch.zeros(T, 1, d, dtype=torch.bfloat16, device="cuda")
    x[..., :d // 2] = 1
    kp = torch.zeros(1, T, 1, d, dtype=torch.bfloat16, device="cuda")
    lens, cu = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([T], [0, T]))
    attn.rope_append(None, x, x, kp, torch.zeros_like(kp), lens, freq.cuda(), cu_seqlens_q=cu,
                     positions=torch.from_numpy(pos).cuda())
    attn.sync_check()
    got = kp[0, :, 0, d // 2:].double().cpu().numpy()
    checked = 0
    with localcontext() as ctx:
        ctx.prec = 60
        for m in range(d // 4, d // 2):  # f <= 0.01
            f = Decimal(float(freq[m])) * inv_2pi
            for t in np.flatnonzero(abs(got[:, m]) < 2.0 ** -11):
                turns = f * int(pos[t])
                a = 2 * np.pi * float(turns - turns.to_integral_value())
                want = math.sin(a)
                tol = 2 * np.pi * (float(abs(turns)) * 2.0 ** -52 + 2.0 ** -25) + abs(want) * 2.0 ** -21
                assert abs(got[t, m] - want) <= half_ulp_bf16(abs(want) + tol) + tol, (m, pos[t])
                checked += 1
    assert checked > 50


# ------------------------------------------------------------------ eviction
@pytest.mark.gpu
def test_evict_with_the_largest_budget():
    """A budget of 2^31 - 1 keys, with room for them in `kept`: every key stays, the rest of
    `kept` is -1 up to its end.  (8.6 GB.)"""
    L, d, budget = 5, 64, 2 ** 31 - 1
    kc = torch.randn(1, 16, 1, d, device="cuda").bfloat16()
    vc, w, lens = -kc, torch.rand(1, 1, 16, device="cuda"), torch.tensor([L], dtype=torch.int32, device="cuda")
    before = kc.clone()
    kept = torch.zeros(1, 1, budget, dtype=torch.int32, device="cuda")
    new = torch.empty_like(lens)
    attn.evict(w, kc, vc, lens, budget, out=(kept, new))
    attn.sync_check()
    assert new.item() == L and kept[0, 0, :L].tolist() == list(range(L))
    assert all((part == -1).all().item() for part in kept[0, 0, L:].split(1 << 28))
    assert torch.equal(kc, before)
    del kept
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [True, False], ids=["in_place", "pages"])
def test_evict_from_a_bad_page(in_place):
    """A table entry that is no page, under kept keys: reported; its keys' rows read as zeros
    in both forms, rows that would go to it are not written, and the others stand."""
    page, Hkv, d, L, budget = 16, 2, 64, 64, 24
    g = torch.Generator().manual_seed(4)
    kp = torch.randn(6, page, Hkv, d, generator=g).bfloat16()
    vp = torch.randn(6, page, Hkv, d, generator=g).bfloat16()
    table = torch.tensor([[4, 0, 5, 1]], dtype=torch.int32)
    w = torch.zeros(1, Hkv, L)
    heavy = list(range(8, 12)) + list(range(36, 56))  # keys that stay: of pages 0, 2 and 3
    w[:, :, heavy] = 1.0
    for entry in (2, 1):  # the page that is read, the page that is written
        t = table.clone()
        t[0, entry] = 77
        kg, vg = kp.cuda(), vp.cuda()
        kd, vd = (kg, vg) if in_place else (torch.full_like(kg, 3), torch.full_like(vg, 3))
        t2 = t if in_place else torch.tensor([[2, 77 if entry == 1 else 3]], dtype=torch.int32)
        kept, _ = attn.evict(w.cuda(), kg, vg, torch.tensor([L], dtype=torch.int32, device="cuda"), budget,
                             page_table=t.cuda(), dst=None if in_place else (kd, vd, t2.cuda(), None))
        with pytest.raises(attn.AttnError) as e:
            attn.sync_check()
        assert e.value.status == attn.ATTN_ERR_DEVICE_INPUT
        assert kept[0, 0].tolist() == heavy and kept[0, 1].tolist() == heavy
        for got, src, fill in ((kd, kp, kp), (vd, vp, vp)):
            want = fill.clone() if in_place else torch.full_like(fill, 3)
            for i, j in enumerate(heavy):
                to, frm = int(t2[0, i // page]), int(t[0, j // page])
                if to < 6:
                    want[to, i % page] = src[frm, j % page] if frm < 6 else 0
            assert torch.equal(got.cpu(), want), entry


# ------------------------------------------------------------------ sizes the kernels cannot index
def test_key_weights_refuse_more_units_than_an_int():
    """A CTA finds its (sequence, KV head) by their product: 2^31 of them are refused."""
    #  q lse kc table cu lens w stride B Hq Hkv total max_sq d max_pages page pages causal window sink scale acc stream
    def call(B, Hkv):
        return attn.attn_key_weights(16, 16, 16, 16, 16, 16, 16, 1, B, Hkv, Hkv, 7, 5, 64, 1, 1, 9, 1, 0, 0, 0.5, 1, None)
    assert call(1 << 28, 8) == attn.ATTN_ERR_INVALID_ARG
    assert call(1 << 30, 4) == attn.ATTN_ERR_INVALID_ARG


def test_slots_above_4_gb_are_refused():
    """The row gathers hold a slot's bytes, Hkv * d * 2, in 32 bits."""
    big = 1 << 23  # heads of 256 dims
    for Hkv, want in ((big, attn.ATTN_ERR_INVALID_ARG), (big - 1, attn.ATTN_OK)):
        # (B = 0: nothing is launched; the sizes are checked first)
        rc = [attn.attn_prefill_paged(16, 16, 16, 16, 16, 16, 16, 16, 0, Hkv, Hkv, 0, 0, 1, 1, 9, 256, 1, 0, 0, 0.5, 1,
                                      1, None, None, 0, None),
              attn.attn_decode_paged(16, 16, 16, 16, 16, 0, Hkv, Hkv, 256, 1, 1, 9, 0.5, 1, 1, None, None, 16, 16, 0,
                                     None, None),
              attn.attn_key_weights(16, 16, 16, 16, 16, 16, 16, 1, 0, Hkv, Hkv, 0, 0, 256, 1, 1, 9, 1, 0, 0, 0.5, 1,
                                    None)]
        assert rc == [want] * 3, (Hkv, rc)


# ------------------------------------------------------------------ forms beside the common ones
@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("mask", [(True, 0, 0), (False, 0, 0), (True, 150, 4)], ids=["causal", "full", "window"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (14, 1)])
def test_key_weights_of_eight_ctas_a_block(d, mask, Hq, Hkv):
    """Few key blocks and many query rows: clusters of eight share a block of keys, and every
    rank's sum counts once.  (At most 15 blocks, at least 16 query tiles; both ways of ending:
    set and accumulated.)"""
    causal, window, n_sink = mask
    sq, kv = torch.tensor([900], dtype=torch.int32), torch.tensor([1100], dtype=torch.int32)
    q, kc, _, cu = W.varlen_inputs(1, Hq, Hkv, d, sq, kv, 700 + d)
    scale = d ** -0.5
    lse = lse_of(q, kc, cu, kv, Hkv, scale, causal, window, n_sink)
    (ref, bound), = weights_ref(q, lse, kc, cu, kv, Hkv, scale, causal, window, n_sink)
    w0 = torch.rand(1, Hkv, 1100)
    for acc in (False, True):
        w = w0.cuda()
        attn.key_weights(q.cuda(), lse.cuda(), kc.cuda(), kv.cuda(), w, cu_seqlens_q=cu.cuda(), max_sq=900,
                         causal=causal, window=window, n_sink=n_sink, scale=scale, accumulate=acc)
        attn.sync_check()
        want = ref + (w0[0].double().numpy() if acc else 0)
        got = w[0].cpu().double().numpy()
        assert (abs(got - want) <= bound + (abs(want) * 2.0 ** -24 if acc else 0)).all()


def _bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [[1, 1, 1], [7, 300, 2]], ids=["tokens", "chunks"])
def test_a_table_wider_than_its_lengths(rows):
    """A table with room for 131,072 keys over sequences of up to 2,000: results as from the
    tight one (launch shapes follow the width, sums of key weights keep their order only within
    a split of the rows, attention its splits: compared to the tolerances of either)."""
    Hq, Hkv, d, page = 8, 2, 64, 32
    kv = torch.tensor([2000, 300, 77], dtype=torch.int32)
    q, kc, vc, cu = W.varlen_inputs(3, Hq, Hkv, d, torch.tensor(rows, dtype=torch.int32), kv, 710)
    kp, vp, tight = make_pages(kc, vc, kv, page, 710)
    wide = torch.full((3, 131072 // page), -1, dtype=torch.int32)
    wide[:, :tight.shape[1]] = tight
    ro, rl = oracle.sdpa_varlen(q, kc, vc, cu, kv, True, 0.125)
    one = max(rows) == 1
    lens, cug, qg = kv.cuda(), cu.cuda(), q.cuda()
    ref = kept0 = None
    for table in (tight, wide):
        cap = table.shape[1] * page
        tg, kg, vg = table.cuda(), kp.cuda(), vp.cuda()
        for max_kv in (None, 2000):
            if one:
                o, lse = attn.decode_paged(qg, kg, vg, tg, lens, scale=0.125, out_dtype=torch.float32, max_kv=max_kv)
                check_lse(lse.T.cpu().numpy(), rl)
            else:
                o, lse = attn.prefill_paged(qg, kg, vg, tg, cug, lens, max(rows), scale=0.125, out_dtype=torch.float32,
                                            max_kv=max_kv)
                check_lse(lse.cpu().numpy(), rl)
            attn.sync_check()
            check_o(o.cpu().numpy(), ro, False)
        w = torch.full((3, Hkv, cap), 5.0, device="cuda")
        attn.key_weights(qg, lse, kg, lens, w, page_table=tg, cu_seqlens_q=None if one else cug, max_sq=max(rows),
                         scale=0.125, accumulate=False)
        attn.sync_check()
        fp32_lse = (lse.T if one else lse).cpu()
        ref = weights_ref(q, fp32_lse, kc, cu, kv, Hkv, 0.125, True)
        for b, (want, bound) in enumerate(ref):
            L = int(kv[b])
            assert (abs(w[b, :, :L].cpu().double().numpy() - want) <= bound).all()
            assert (w[b, :, L:] == 5).all()
        score = torch.rand(3, Hkv, cap, generator=torch.Generator().manual_seed(1))
        score[:, :, :tight.shape[1] * page] = torch.rand(3, Hkv, tight.shape[1] * page,
                                                         generator=torch.Generator().manual_seed(2))
        kept, new = attn.evict(score.cuda(), kg, vg, lens, 128, 16, 4, page_table=tg)
        attn.sync_check()
        kept0 = kept if kept0 is None else kept0
        assert torch.equal(kept, kept0) and new.tolist() == [128, 128, 77]
        for b in range(3):
            n = min(128, int(kv[b]))
            for h in range(Hkv):
                idx = kept[b, h, :n].cpu().long()
                assert torch.equal(gather(kg.cpu(), tight, b, n, page)[:, h], kc[b, idx, h])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 20])
def test_windowed_chunks_with_bf16_outputs(d, page):
    rows, keys = [1, 77, 128, 300, 0, 200, 3], [1, 300, 128, 1200, 50, 150, 0]
    sq, kv = torch.tensor(rows, dtype=torch.int32), torch.tensor(keys, dtype=torch.int32)
    q, kc, vc, cu = W.varlen_inputs(len(rows), 7, 1, d, sq, kv, 720 + d)
    kp, vp, table = make_pages(kc, vc, kv, page, 720)
    scale = d ** -0.5
    for window, n_sink in ((1, 0), (100, 4), (2 ** 31 - 1, 2 ** 31 - 1)):
        o, lse = attn.prefill_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), cu.cuda(), kv.cuda(), max(rows),
                                    scale=scale, window=window, n_sink=n_sink)
        attn.sync_check()
        ro, rl = oracle.sdpa_varlen_window(q, kc, vc, cu, kv, min(window, 4096), min(n_sink, 4096), scale)
        check_o(o.float().cpu().numpy(), ro, True)
        check_lse(lse.cpu().numpy(), rl)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n_splits", [1, 3])
def test_chunks_of_many_sequences(causal, n_splits):
    """40 sequences: more than are ordered by their tiles."""
    rng = np.random.default_rng(8)
    sq = torch.from_numpy(rng.integers(0, 150, 40).astype(np.int32))
    kv = torch.from_numpy(rng.integers(0, 600, 40).astype(np.int32))
    q, kc, vc, cu = W.varlen_inputs(40, 4, 2, 64, sq, kv, 730)
    kp, vp, table = make_pages(kc, vc, kv, 16, 730)
    ro, rl = oracle.sdpa_varlen(q, kc, vc, cu, kv, causal, 0.125)
    for dt in (torch.bfloat16, torch.float32):
        o, lse = attn.prefill_paged(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), cu.cuda(), kv.cuda(), int(sq.max()),
                                    causal=causal, scale=0.125, out_dtype=dt, n_splits=n_splits)
        attn.sync_check()
        check_o(o.float().cpu().numpy(), ro, dt is torch.bfloat16)
        check_lse(lse.cpu().numpy(), rl)


@pytest.mark.gpu
def test_calls_repeat_their_bits():
    """The same call on the same inputs, other calls between: the same bits, splits or not."""
    q, kc, vc, cu = W.varlen_inputs(3, 8, 2, 128, torch.tensor([5, 200, 1]), torch.tensor([900, 700, 300]), 740)
    kv = torch.tensor([900, 700, 300], dtype=torch.int32)
    kp, vp, table = (x.cuda() for x in make_pages(kc, vc, kv, 16, 740))
    lens, cug, qg = kv.cuda(), cu.cuda(), q.cuda()
    first = {}
    for _ in range(4):
        for n in (1, 3):
            out = (*attn.prefill_paged(qg, kp, vp, table, cug, lens, 200, n_splits=n),
                   *attn.decode_paged(qg[:3].contiguous(), kp, vp, table, lens, n))
            attn.sync_check()
            for a, b in zip(out, first.setdefault(n, [t.clone() for t in out])):
                assert torch.equal(_bits(a), _bits(b))


# ------------------------------------------------------------------ streams
@pytest.mark.gpu
def test_inputs_dropped_after_a_call_on_another_stream():
    """The stream argument, with inputs that the caller lets go of right after the call while
    the stream is still busy with work before it: their memory is not handed out again before
    the call has read them."""
    B, Hq, Hkv, d, page, L = 4, 8, 2, 64, 16, 96
    g = torch.Generator(device="cuda").manual_seed(9)

    def bf16(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    pool = B * L // page, page, Hkv, d
    q, k, v, kc, vc = bf16(B, Hq, d), bf16(B, Hkv, d), bf16(B, Hkv, d), bf16(*pool), bf16(*pool)
    table = torch.arange(pool[0], dtype=torch.int32, device="cuda").view(B, -1)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    lse, w = torch.randn(B, Hq, generator=g, device="cuda") + 5, torch.rand(B, Hkv, L, generator=g, device="cuda")
    freq = attn.rope_frequencies(d)[0]
    calls = [  # inputs, and the call that is made with copies of them
        ((q, k, v, kc, vc, lens, freq, table), lambda a, s: attn.rope_append(*a, stream=s)),
        ((q, kc, vc, table, cu, lens), lambda a, s: attn.prefill_paged(*a, 1, n_splits=1, stream=s)[0]),
        ((q, kc, vc, table, lens), lambda a, s: attn.decode_paged(*a, 3, stream=s)[0]),
        ((q, lse, kc, lens, w, table), lambda a, s: attn.key_weights(*a, accumulate=False, stream=s)),
        ((w, kc, vc, lens, table), lambda a, s: attn.evict(*a[:4], 40, 4, 2, page_table=a[4], stream=s)[0]),
    ]
    busy, front = torch.cuda.Stream(), torch.zeros(1 << 28, device="cuda")
    for inputs, call in calls:
        want = call([t.clone() for t in inputs], None).clone()
        call([t.clone() for t in inputs], busy)
        torch.cuda.synchronize()
        with torch.cuda.stream(busy):
            for _ in range(20):  # some milliseconds
                front.add_(1)
        args = [t.clone() for t in inputs]
        busy.wait_stream(torch.cuda.current_stream())
        got = call(args, busy)
        if any(got is a for a in args):  # (the weights themselves: what else was given goes)
            args = [a for a in args if a is got]
        else:
            args = None
        others = [torch.full_like(t, -1) for t in inputs for _ in range(3)]  # of the same sizes
        torch.cuda.synchronize()
        attn.sync_check()
        assert torch.equal(_bits(got), _bits(want))
        del others, args
