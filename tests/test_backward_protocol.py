"""The barrier schedule of the prefill's gradients, modelled on the CPU.

A CTA of prefill_backward.cuh has two warps that issue the first products (S, dP), one for the
second products, one that fills the rings of Y1 and Y2, and eight of softmax.  They meet at
mbarriers, whose waits test a phase *parity*: a wait is sound only if the barrier can be
neither one phase short of what it takes for done nor one beyond it.

The model runs those roles as generators in random order, with an exact mbarrier, copies that
land at any time after they are issued, and products that each issuing warp's queue executes in
order, the warps' queues interleaved at random.  Every buffer carries the item it holds: a
product or a read must find its own item, a write must find the buffer's readers done.  The
same model shows that one slot fewer for the lse and D columns would be overwritten early.
"""
import random

import pytest


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0
        if self.pending == 0:
            self.phase += 1
            self.pending = self.count

    def done(self, n):
        """A wait for n completions: the parity test, and what it is to mean."""
        if (self.phase & 1) != (n & 1):
            return False
        assert self.phase == n, "a wait passed for another phase than its own"
        return True


CONFIGS = {  # dK/dV or dQ, rows of a Y tile, stages of Y1 and Y2
    "dkdv-128": dict(kv=True, sep=True, st1=5, st2=4),
    "dkdv-64": dict(kv=True, sep=False, st1=4, st2=4),
    "dq-128": dict(kv=False, sep=False, st1=3, st2=2),
    "dq-64": dict(kv=False, sep=False, st1=4, st2=4),
    # P and dS as two terms (where the sums are wide, in one buffer)
    "dkdv-128-fine": dict(kv=True, sep=True, st1=5, st2=4, one_p=True),
    "dkdv-64-fine": dict(kv=True, sep=True, st1=4, st2=4),
    "dq-128-fine": dict(kv=False, sep=True, st1=3, st2=2),
    "dq-64-fine": dict(kv=False, sep=True, st1=4, st2=4),
}


def simulate(kv, sep, st1, st2, runs, parts, seed, ext_slots=5, one_p=False):
    rng = random.Random(seed)
    nd, arrive = (1, 4) if sep else (2, 8)
    stages = (st1, st2)
    full = [[Bar(1) for _ in range(n)] for n in stages]
    empty = [[Bar(1) for _ in range(n)] for n in stages]
    full_f, empty_f = [Bar(1), Bar(1)], [Bar(1), Bar(1)]
    done = [[Bar(1), Bar(1)], [Bar(1), Bar(1)]]               # S and dP computed
    freed = [[Bar(arrive)], [Bar(arrive if sep else 1) for _ in range(nd)]]
    bar_p, bar_pr = [Bar(arrive), Bar(arrive)], [Bar(1), Bar(1)]
    acc, accr, go, out, last = Bar(1), Bar(8), Bar(1), Bar(8), Bar(1)
    n_items = sum(runs)
    executed = {k: set() for k in ("S", "dP", "2a", "2b")}    # items
    y = [[None] * n for n in stages]
    f = [None, None]
    ext = [[None] * ext_slots, [None] * ext_slots]
    s_buf, dp_buf, p_buf = [None], [None] * nd, [None, None]  # item, and who of the readers / writers is through
    s_read, dp_read, p_parts = {}, {}, {}
    sums, sums_read = None, {}
    landing, queues = [], {8: [], 9: [], 10: []}

    def read_done(item, k):
        """No product still has to read item's tile of Y1 (k = 0) or Y2."""
        if k == 0:
            return item in executed["S"] and item in executed["2b"]
        return item in executed["dP"] and (not kv or item in executed["2a"])

    def first(which):
        name, it = ("S", "dP")[which], 0
        warp, bufs = 8 + which, 1 if which == 0 else nd
        issued, landed = [0], [0]  # ext items on their way, and landed

        def load_ext():
            if not kv:
                return
            if issued[0] < n_items:
                old = issued[0] - ext_slots
                assert old < 0 or old in executed[name], "lse or D columns overwritten"
                ext[which][issued[0] % ext_slots] = None
            issued[0] += 1

        def next_ext():
            load_ext()
            while kv and landed[0] < issued[0] - 2:
                if landed[0] < n_items:
                    ext[which][landed[0] % ext_slots] = landed[0]
                landed[0] += 1

        load_ext()
        load_ext()
        next_ext()
        for r, n in enumerate(runs):
            yield lambda: empty_f[which].done(r)
            assert r == 0 or all(i in executed[name] for i in range(it)), "F overwritten"
            f[which] = None

            def land(r=r):
                f[which] = r
                full_f[which].arrive()
            landing.append(land)
            yield lambda: full_f[which].done(r + 1)
            if r > 0:
                yield lambda: go.done(r)
            for m in range(n):
                s, buf = it % stages[which], it % bufs
                yield lambda: freed[which][buf].done(it // bufs)
                yield lambda: full[which][s].done(it // stages[which] + 1)

                def product(it=it, r=r, s=s, buf=buf):
                    assert y[which][s] == it and f[which] == r
                    assert not kv or ext[which][it % ext_slots] == it
                    if which == 0:
                        assert s_buf[0] is None or s_read[s_buf[0]] == arrive, "S overwritten"
                        s_buf[0] = it
                    else:
                        old = dp_buf[buf]
                        if old is not None and sep:
                            assert dp_read[old] == arrive, "dP overwritten"
                        elif old is not None:  # P and dS lie over it
                            assert old in executed["2b"], "P or dS overwritten"
                        dp_buf[buf] = it
                    executed[name].add(it)
                queues[warp].append(product)
                queues[warp].append(done[which][it & 1].arrive)
                if not kv and which == 1:
                    queues[warp].append(empty[1][s].arrive)
                if m == n - 1:
                    queues[warp].append(empty_f[which].arrive)
                next_ext()
                it += 1
                yield lambda: True

    def second():
        nonlocal sums
        it = 0
        for r, n in enumerate(runs):
            if r > 0:
                yield lambda: accr.done(r)
            for m in range(n):
                buf = it & 1
                yield lambda: bar_p[buf].done(it // 2 + 1)

                def product(k, it=it, r=r, m=m, buf=buf):
                    nonlocal sums
                    assert p_buf[0 if one_p else buf] == it and p_parts[it] == arrive
                    assert y[0][it % st1] == it if k == "2b" else y[1][it % st2] == it
                    if m == 0 and r > 0:
                        assert sums_read.get(r - 1) == 8, "sums overwritten"
                    sums = r
                    executed[k].add(it)
                if kv:
                    queues[10].append(lambda it=it, p=product: p("2a"))
                    queues[10].append(empty[1][it % st2].arrive)
                queues[10].append(lambda p=product: p("2b"))
                queues[10].append((bar_pr[buf] if sep else freed[1][it % nd]).arrive)
                queues[10].append(empty[0][it % st1].arrive)
                if m == n - 1:
                    queues[10].append(acc.arrive)
                    go.arrive()
                it += 1
                yield lambda: True

    def copies(k):
        for it in range(n_items):
            s = it % stages[k]
            yield lambda: empty[k][s].done(it // stages[k])
            assert it < stages[k] or read_done(it - stages[k], k), "a tile overwritten"
            y[k][s] = None

            def land(it=it, s=s):
                y[k][s] = it
                full[k][s].arrive()
            landing.append(land)

    def softmax(warp):
        wg, it, n_part = warp >> 2, 0, 0
        for r, n in enumerate(runs):
            for m in range(n):
                if sep and (it & 1) != wg:
                    it += 1
                    continue
                bp, bd = it & 1, it % nd
                yield lambda: done[0][bp].done(it // 2 + 1)
                assert s_buf[0] == it
                s_read[it] = s_read.get(it, 0) + 1
                freed[0][0].arrive()
                yield lambda: done[1][bp].done(it // 2 + 1)
                assert dp_buf[bd] == it
                dp_read[it] = dp_read.get(it, 0) + 1
                if sep:
                    freed[1][0].arrive()
                    if one_p:
                        yield lambda: it == 0 or bar_pr[bp ^ 1].done((it - 1) // 2 + 1)
                    else:
                        yield lambda: bar_pr[bp].done(it // 2)
                last_p = it - (1 if one_p else 2)
                assert last_p < 0 or last_p in executed["2b"], "P or dS overwritten"
                # (where rows behind a sequence's last are cleared: both tiles are whole and read once)
                assert y[0][it % st1] == it and it in executed["S"] and it in executed["dP"]
                assert not kv or y[1][it % st2] == it
                p_buf[0 if one_p else bp] = it
                p_parts[it] = p_parts.get(it, 0) + 1
                bar_p[bp].arrive()
                it += 1
            yield lambda: acc.done(r + 1)
            assert sums == r and all(i in executed["2b"] for i in range(sum(runs[:r + 1])))
            sums_read[r] = sums_read.get(r, 0) + 1
            accr.arrive()
            if parts[r]:
                out.arrive()
                if warp == 0:
                    yield lambda: out.done(n_part + 1)
                    last.arrive()
                yield lambda: last.done(n_part + 1)
                n_part += 1

    roles = [first(0), first(1), second(), copies(0), copies(1)] + [softmax(w) for w in range(8)]
    waits = {}
    for g in roles:
        c = next(g, None)
        if c is not None:
            waits[g] = c
    while waits or landing or any(queues.values()):
        moves = [("land", i) for i in range(len(landing))]
        moves += [("run", q) for q, items in queues.items() if items]
        moves += [("role", g) for g, c in waits.items() if c()]
        assert moves, "deadlock"
        kind, x = rng.choice(moves)
        if kind == "land":
            landing.pop(x)()
        elif kind == "run":
            queues[x].pop(0)()
        else:
            c = next(x, None)
            if c is None:
                del waits[x]
            else:
                waits[x] = c
    assert len(executed["2b"]) == n_items and all(v == 8 for v in sums_read.values())


def _case(seed):
    rng = random.Random(seed)
    runs = [rng.choice((1, 1, 2, 3, 5, 8, 13)) for _ in range(rng.randint(1, 7))]
    return runs, [rng.random() < 0.4 for _ in runs]


@pytest.mark.parametrize("name", CONFIGS)
@pytest.mark.parametrize("seed", range(25))
def test_schedule(name, seed):
    runs, parts = _case(seed)
    simulate(**CONFIGS[name], runs=runs, parts=parts, seed=seed)


def test_four_slots_of_columns_are_too_few():
    """With two dP buffers an item's product may run while the columns three items on are
    brought."""
    lost = 0
    for seed in range(40):
        try:
            simulate(**CONFIGS["dkdv-64"], runs=[12, 9], parts=[False, True], seed=seed, ext_slots=4)
        except AssertionError as e:
            assert "columns overwritten" in str(e)
            lost += 1
    assert lost
