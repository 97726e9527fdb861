"""The barrier protocol of the decayed layer's tensor-core kernels
(csrc/decay_tc.cuh), run as a model under random schedules on the CPU.

Each role of a block is a generator of the waits, arrivals and asynchronous
operations that it makes, in the kernel's order.  Loads and MMA commits arrive
later, commits of one issuing thread in order.  A schedule picks any step that
can go on.  Checked: every role finishes; no barrier completes two phases past
one that a waiter still has to see (a parity wait would then wait for good);
no resource is written while something else may still use it."""
import random

import pytest


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.phase, self.want = count, count, 0, {}

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.phase += 1
            self.pending = self.count


class Block:
    """Runs the roles; `use`/`free` keep who holds a resource."""

    def __init__(self, seed):
        self.rng, self.roles, self.async_, self.held = random.Random(seed), [], [], {}

    def hold(self, what, by):
        assert what not in self.held, f"{by} writes {what}, still in use by {self.held[what]}"
        self.held[what] = by

    def drop(self, what):
        self.held.pop(what, None)

    def run(self):
        state = {i: next(r, None) for i, r in enumerate(self.roles)}
        queues = {}  # in-order completions of each issuer
        steps = 0
        while any(s is not None for s in state.values()) or any(queues.values()):
            steps += 1
            assert steps < 200000
            ready = []
            for i, s in state.items():
                if s is None:
                    continue
                if s[0] == "wait":
                    bar, n = s[1], s[2]
                    assert bar.phase <= n + 1, "a barrier ran two phases ahead of a waiter"
                    if bar.phase > n:
                        ready.append(("role", i))
                else:
                    ready.append(("role", i))
            ready += [("queue", q) for q, items in queues.items() if items]
            assert ready, "deadlock"
            kind, x = self.rng.choice(ready)
            if kind == "queue":
                queues[x].pop(0)()
                continue
            s = state[x]
            if s[0] == "arrive":
                s[1].arrive()
            elif s[0] == "later":  # issuer, completion
                queues.setdefault(s[1], []).append(s[2])
            state[x] = next(self.roles[x], None)


def outputs(nt, nst, nsb, ragged, seed, beside=False, warps=2):
    """The output kernel.  `ragged`: index of the tile that ends early, or -1;
    `beside`: K~'s second part has a place of its own."""
    k = Block(seed)
    arr = lambda n, c: [Bar(c) for _ in range(n)]  # noqa: E731
    full, fullv, free_qk, empty, sfull, pready = arr(nst, 1), arr(nst, 1), arr(nst, 2), arr(nst, 1), arr(2, 1), arr(2, warps)
    kready, qdone, dfull, wready, ofull, ofree, cut, sread = (Bar(c) for c in (warps, 1, 1, warps, 1, warps, warps, warps))

    def load():
        for i in range(nt):
            st = i % nst
            if i >= nst:
                yield "wait", free_qk[st], i // nst - 1
            if i == nst - 1:
                yield "wait", sread, 0
            k.hold(("QK", st), f"load {i}")
            yield "later", f"qk{st}", full[st].arrive
            if i >= nst:
                yield "wait", empty[st], i // nst - 1
            k.hold(("V", st), f"load {i}")
            yield "later", f"v{st}", fullv[st].arrive

    def mma_a():
        def scores(i):
            if i == ragged:
                yield "wait", cut, 0
            k.hold(("S", i % nsb), f"scores {i}")
            yield "later", "A", sfull[i & 1].arrive
        yield "wait", full[0], 0
        yield from scores(0)
        for i in range(nt):
            j = i + 1
            yield "wait", wready, i
            ahead = nsb == 2 and j < nt and j != ragged and full[j % nst].phase > j // nst
            if ahead:
                yield from scores(j)
            if i:
                yield "wait", ofree, i - 1
            k.hold("O", f"o2 {i}")

            def o2_done(i=i):
                qdone.arrive()
            yield "later", "A", o2_done

            def a_done(i=i):
                free_qk[i % nst].arrive()
                if free_qk[i % nst].pending == 2:
                    k.drop(("QK", i % nst))
            yield "later", "A", a_done
            yield "wait", fullv[i % nst], i // nst
            yield "wait", pready[i & 1], i // 2
            k.drop(("S", i % nsb))  # the next scores there follow this product in the pipe's order
            yield "later", "A", ofull.arrive
            if j < nt and not ahead:
                yield "wait", full[j % nst], j // nst
                yield from scores(j)

    def mma_d():
        for i in range(nt):
            if i + 1 < nt:
                yield "wait", fullv[i % nst], i // nst
                yield "wait", kready, i
                k.hold("D", f"d {i}")
                yield "later", "B", dfull.arrive

            def b_done(i=i):
                free_qk[i % nst].arrive()
                if free_qk[i % nst].pending == 2:
                    k.drop(("QK", i % nst))
            yield "later", "B", b_done

    def po(w):
        def p(i):
            yield "wait", sfull[i & 1], i // 2
            yield "arrive", pready[i & 1]

        def o(i):
            yield "wait", ofull, i
            yield "wait", free_qk[i % nst], i // nst
            done_o[i] = done_o.get(i, 0) + 1
            if done_o[i] == warps:
                k.drop("O")
            yield "arrive", ofree
            meet[i] = meet.get(i, 0) + 1  # the named barrier before the store
            while meet[i] < warps:
                yield "spin",
            if w == 0:
                def stored():
                    k.drop(("V", i % nst))
                    empty[i % nst].arrive()
                yield "later", "store", stored
        if nsb == 2:
            yield from p(0)
            for i in range(nt):
                if i + 1 < nt:
                    yield from p(i + 1)
                yield from o(i)
        else:
            for i in range(nt):
                yield from p(i)
                yield from o(i)

    def state(w):
        yield "arrive", sread
        yield "arrive", wready
        for i in range(nt):
            st = i % nst
            yield "wait", full[st], i // nst
            if i == ragged:
                yield "wait", fullv[st], i // nst
                yield "arrive", cut
            yield "wait", sfull[i & 1], i // 2
            if i + 1 < nt and not beside:
                yield "wait", qdone, i  # K~'s second part goes where Q was
            yield "arrive", kready
            if i + 1 == nt:
                return
            yield "wait", dfull, i
            read_d[i] = read_d.get(i, 0) + 1
            if read_d[i] == warps:
                k.drop("D")
            if beside:
                yield "wait", qdone, i
            yield "arrive", wready

    done_o, meet, read_d = {}, {}, {}
    k.roles = [load(), mma_a(), mma_d()] + [po(w) for w in range(warps)] + [state(w) for w in range(warps)]
    k.run()


def totals(nt, nst, seed, warps=2):
    k = Block(seed)
    arr = lambda n, c: [Bar(c) for _ in range(n)]  # noqa: E731
    full, ready, empty, dfull, lofree, dfree = arr(nst, 1), arr(nst, warps), arr(nst, 1), arr(2, 1), arr(2, 1), arr(2, warps)
    read = {}

    def load():
        for i in range(nt):
            if i >= nst:
                yield "wait", empty[i % nst], i // nst - 1
            k.hold(("KV", i % nst), f"load {i}")
            yield "later", f"kv{i % nst}", full[i % nst].arrive

    def mma():
        for i in range(nt):
            yield "wait", ready[i % nst], i // nst
            if i > 1:
                yield "wait", dfree[i & 1], i // 2 - 1
            k.hold(("D", i & 1), f"d {i}")

            def lo(i=i):
                k.drop(("lo", i & 1))
                lofree[i & 1].arrive()
            yield "later", "M", lo

            def done(i=i):
                k.drop(("KV", i % nst))
                empty[i % nst].arrive()
                dfull[i & 1].arrive()
            yield "later", "M", done

    def scale(w):
        for i in range(nt):
            yield "wait", full[i % nst], i // nst
            if i > 1:
                yield "wait", lofree[i & 1], i // 2 - 1
            if ("lo", i) not in read:
                k.hold(("lo", i & 1), f"scale {i}")
                read["lo", i] = 1
            yield "arrive", ready[i % nst]

    def add(w):
        for i in range(nt):
            yield "wait", dfull[i & 1], i // 2
            read[i] = read.get(i, 0) + 1
            if read[i] == warps:
                k.drop(("D", i & 1))
            yield "arrive", dfree[i & 1]

    k.roles = [load(), mma()] + [scale(w) for w in range(warps)] + [add(w) for w in range(warps)]
    k.run()


@pytest.mark.parametrize("nsb", [1, 2])
@pytest.mark.parametrize("nst", [2, 3, 4])
def test_outputs_protocol(nsb, nst):
    for nt in range(1, 10):
        for ragged in {-1, 0, nt - 1}:
            for seed in range(60):
                outputs(nt, nst, nsb, ragged, 1000 * nt + seed, beside=seed % 2 == 0)


@pytest.mark.parametrize("nst", [2, 3, 6])
def test_totals_protocol(nst):
    for nt in range(1, 12):
        for seed in range(60):
            totals(nt, nst, 1000 * nt + seed)
