"""The lse and D columns of a run's rows in the gradients' dQ pass at d = 64, modelled on the CPU.

There either first-product warp keeps one slot of shared memory for its run's 128 rows (in the dK/dV
pass the columns belong to items and have rings: test_backward_protocol).  The warp writes the slot
itself, after the wait for the F tile's buffer: a run's products read both, and the commit behind the
last of them frees both.  The model runs the two warps, their queues of products, the softmax that frees
their accumulators and the second products' warp in random order; every product must find its own run's
tile and columns.  A slot written ahead of that wait is shown to be overwritten early."""
import random

import pytest

from tests.test_backward_protocol import Bar


def simulate(runs, seed, bufs, early=False):
    """bufs: accumulators of the two products (S, dP)."""
    rng = random.Random(seed)
    full_f, empty_f = [Bar(1), Bar(1)], [Bar(1), Bar(1)]
    done = [[Bar(1) for _ in range(2)] for _ in range(2)]
    freed = [[Bar(1) for _ in range(n)] for n in bufs]
    go = Bar(1)
    f, rows = [None, None], [None, None]                 # run whose tile, and whose columns, are there
    executed, n_items = [0, 0], sum(runs)
    landing, queues = [], [[], []]

    def first(w):
        it = 0
        for r, n in enumerate(runs):
            def write():
                assert executed[w] == it, "columns overwritten"
                rows[w] = r                              # (copied and waited for by the warp's own lanes)
            if early:
                write()
            yield lambda: empty_f[w].done(r)
            assert executed[w] == it, "F overwritten"
            f[w] = None

            def land(r=r):
                f[w] = r
                full_f[w].arrive()
            landing.append(land)
            if not early:
                write()
            yield lambda: full_f[w].done(r + 1)
            if r > 0:
                yield lambda: go.done(r)
            for m in range(n):
                buf = it % bufs[w]
                yield lambda: freed[w][buf].done(it // bufs[w])

                def product(r=r):
                    assert f[w] == r and rows[w] == r
                    executed[w] += 1
                queues[w] += [product, done[w][it & 1].arrive]
                if m == n - 1:
                    queues[w].append(empty_f[w].arrive)
                it += 1
                yield lambda: True

    def softmax():
        for it in range(n_items):
            for w in range(2):
                yield lambda: done[w][it & 1].done(it // 2 + 1)
                freed[w][it % bufs[w]].arrive()

    def second():
        it = 0
        for r, n in enumerate(runs):
            for _ in range(n):
                yield lambda: executed[0] > it and executed[1] > it
                it += 1
            go.arrive()
            yield lambda: True

    waits = {g: next(g) for g in (first(0), first(1), softmax(), second())}
    while waits or landing or any(queues):
        moves = [("land", i) for i in range(len(landing))] + [("run", w) for w in range(2) if queues[w]]
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
    assert executed == [n_items, n_items]


@pytest.mark.parametrize("bufs", [(1, 2), (1, 1)], ids=["one-term", "two-terms"])
@pytest.mark.parametrize("seed", range(40))
def test_columns_of_a_run(bufs, seed):
    rng = random.Random(seed)
    simulate([rng.choice((1, 1, 2, 3, 8)) for _ in range(rng.randint(1, 9))], seed, bufs)


@pytest.mark.parametrize("bufs", [(1, 2), (1, 1)], ids=["one-term", "two-terms"])
def test_columns_written_ahead_of_the_wait_are_lost(bufs):
    lost = 0
    for seed in range(40):
        try:
            simulate([3, 2, 4, 1], seed, bufs, early=True)
        except AssertionError as e:
            assert "columns overwritten" in str(e)
            lost += 1
    assert lost
