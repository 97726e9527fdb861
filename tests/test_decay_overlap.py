"""The output kernel of the decayed layer (csrc/decay_tc.cuh), whose state is
read in two bf16 parts, starts before the launch before it has ended.  Its bounded waits are to measure the block's own
pipeline: however long that launch still runs, no role may stand in one that
only the launch's end can release.  Run as a model on the CPU like
test_decay_protocol, with the same checks of its barriers and resources; the
launch before ends when nothing else can go on."""
import pytest

from tests import test_decay_protocol as protocol


class Overlapped(protocol.Block):
    """A Block whose roles call wait_before where `at(index, roles)` says:
    "start", or ahead of their next wait after that many, or None: nowhere.
    Roles: 0 loads, 1 and 2 the MMAs, then as many for P and the outputs as
    for the state."""
    at = None

    def _gated(self, i, role):
        at, waits = self.at(i, len(self.roles)), 0
        if at == "start":
            yield "before",
        for step in role:
            if step[0] == "wait":
                if waits == at:
                    yield "before",
                waits += 1
            yield step

    def run(self):
        roles = [self._gated(i, r) for i, r in enumerate(self.roles)]
        state, queues, ended = {i: next(r, None) for i, r in enumerate(roles)}, {}, False
        while any(s is not None for s in state.values()) or any(queues.values()):
            ready = [("queue", q) for q, items in queues.items() if items]
            for i, s in state.items():
                if s is not None and s[0] != "spin" and (s[1].phase > s[2] if s[0] == "wait" else s[0] != "before" or ended):
                    ready.append(("role", i))
            spins = [("role", i) for i, s in state.items() if s is not None and s[0] == "spin"]
            if not ready and not ended:
                waiting = [i for i, s in state.items() if s is not None and s[0] in ("wait", "spin")]
                assert not waiting, f"roles {waiting} wait for the launch before under their limit"
                ended = True
                continue
            kind, x = self.rng.choice(ready + spins)
            if kind == "queue":
                queues[x].pop(0)()
                continue
            s = state[x]
            if s[0] == "arrive":
                s[1].arrive()
            elif s[0] == "later":
                queues.setdefault(s[1], []).append(s[2])
            state[x] = next(roles[x], None)


def outputs(nt, nst, nsb, ragged, seed, beside, block, warps=2):
    """test_decay_protocol.outputs with the state's two bf16 parts.  `beside`:
    the second parts of the state and of K~ have places of their own.  Else
    K~'s goes over the state's first part, and the state's over the Q of the
    tile before (first of all over the start state's buffer, the last stage),
    which is loaded anew when the product with it is complete."""
    k = block(seed)
    arr = lambda n, c: [protocol.Bar(c) for _ in range(n)]  # noqa: E731
    full, fullv, free_qk, empty, sfull, pready = arr(nst, 2), arr(nst, 1), arr(nst, 2), arr(nst, 1), arr(2, 1), arr(2, warps)
    wfree, kready = arr(nst, 1), arr(2, warps)
    qdone, dfull, wready, ofull, ofree, cut, sread = (protocol.Bar(c) for c in (1, 1, warps, 1, warps, warps, warps))
    if nt >= nst:
        for what in "QKV":
            k.hold((what, nst - 1), "the start state")

    def load():
        for i in range(nt):
            st = i % nst
            if i >= nst:
                yield "wait", free_qk[st], i // nst - 1
            if i == nst - 1:
                yield "wait", sread, 0
            k.hold(("K", st), f"load {i}")
            yield "later", f"k{st}", full[st].arrive
            if not beside and i >= nst - 1:
                yield "wait", wfree[st], i // nst if st == nst - 1 else i // nst - 1
            k.hold(("Q", st), f"load {i}")
            yield "later", f"q{st}", full[st].arrive
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
            j, st = i + 1, i % nst
            yield "wait", wready, i
            ahead = nsb == 2 and j < nt and j != ragged and full[j % nst].phase > j // nst
            if ahead:
                yield from scores(j)
            if i:
                yield "wait", ofree, i - 1
            k.hold("O", f"o2 {i}")

            def o2(i=i, st=st):
                k.drop(("W", 0))
                k.drop(("W", 1) if beside else ("Q", (i + nst - 1) % nst))
                k.drop(("Q", st))
                qdone.arrive()
                if not beside:
                    wfree[(i + nst - 1) % nst].arrive()
            yield "later", "A", o2

            def a_done(st=st):
                free_qk[st].arrive()
                if free_qk[st].pending == 2:
                    k.drop(("K", st))
            yield "later", "A", a_done
            yield "wait", fullv[st], i // nst
            yield "wait", pready[i & 1], i // 2
            k.drop(("S", i % nsb))
            yield "later", "A", ofull.arrive
            if j < nt and not ahead:
                yield "wait", full[j % nst], j // nst
                yield from scores(j)

    def mma_d():
        for i in range(nt):
            st = i % nst
            if i + 1 < nt:
                yield "wait", fullv[st], i // nst
                yield "wait", kready[0], i
                k.hold("D", f"d {i}")
                yield "wait", kready[1], i

                def d_done():
                    if not beside:
                        k.drop(("W", 0))
                    dfull.arrive()
                yield "later", "B", d_done

            def b_done(st=st):
                free_qk[st].arrive()
                if free_qk[st].pending == 2:
                    k.drop(("K", st))
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
            meet[i] = meet.get(i, 0) + 1
            while meet[i] < warps:
                yield "spin",
            if w == 0:
                def stored():
                    k.drop(("V", i % nst))
                    empty[i % nst].arrive()
                yield "later", "store", stored
        for i in range(nt + nsb - 1):
            if i < nt:
                yield from p(i)
            if i >= nsb - 1:
                yield from o(i - nsb + 1)

    def first_of(key):
        wrote[key] = wrote.get(key, 0) + 1
        return wrote[key] == 1

    def state(w):
        yield "spin",  # (any warp may come late)
        read["start"] = read.get("start", 0) + 1
        if read["start"] == warps:
            for what in "QKV":
                k.drop((what, nst - 1))
        yield "arrive", sread
        while not beside and read["start"] < warps:  # the named barrier behind the buffer's reads
            yield "spin",
        for i in range(nt):
            st = i % nst
            if first_of(("W", i)):
                k.hold(("W", 0), f"state {i}")
                k.hold(("W", 1) if beside else ("Q", (i + nst - 1) % nst), f"state {i}, second part")
            yield "arrive", wready
            yield "wait", full[st], i // nst
            if i == ragged:
                yield "wait", fullv[st], i // nst
                yield "arrive", cut
            yield "wait", sfull[i & 1], i // 2
            if i + 1 == nt:
                return
            if not beside:
                yield "wait", qdone, i
                if first_of(("K~", i)):
                    k.hold(("W", 0), f"K~ {i}, second part")
            yield "arrive", kready[0]
            yield "arrive", kready[1]
            yield "wait", dfull, i
            read_d[i] = read_d.get(i, 0) + 1
            if read_d[i] == warps:
                k.drop("D")
            if beside:
                yield "wait", qdone, i

    done_o, meet, read_d, wrote, read = {}, {}, {}, {}, {}
    k.roles = [load(), mma_a(), mma_d()] + [po(w) for w in range(warps)] + [state(w) for w in range(warps)]
    k.run()


def _kernel(ragged):
    """Where the kernel's roles call it."""
    def at(i, n):
        if i >= 3 + (n - 3) // 2 or i == 2:
            return "start"
        if i == 0:
            return 0                      # its waits are for places that the state or a tile's end frees
        if i == 1:
            return 1                      # behind the first tile's arrival
        return 0 if ragged == 0 else 1    # behind the first tile's scores, if no rows of it are cut first
    return at


def _run(at, nt, nst, nsb, ragged, seed):
    class Block(Overlapped):
        pass
    Block.at = staticmethod(at)
    outputs(nt, nst, nsb, ragged, seed, beside=seed % 2 == 0, block=Block)


@pytest.mark.parametrize("nsb", [1, 2])
@pytest.mark.parametrize("nst", [2, 3, 4])
def test_protocol(nsb, nst):
    for nt in range(1, 9):
        for ragged in {-1, 0, nt - 1}:
            for seed in range(40):
                outputs(nt, nst, nsb, ragged, 1000 * nt + seed, beside=seed % 2 == 0, block=protocol.Block)


@pytest.mark.parametrize("nsb", [1, 2])
@pytest.mark.parametrize("nst", [2, 3, 4])
def test_no_limit_runs_while_the_launch_before_does(nsb, nst):
    for nt in range(1, 8):
        for ragged in {-1, 0, nt - 1}:
            for seed in range(40):
                _run(_kernel(ragged), nt, nst, nsb, ragged, 100 * nt + seed)


@pytest.mark.parametrize("role", [0, 1, 2, 3])
def test_the_model_flags_a_role_that_waits_at_once(role):
    """Loads past the first stages, the MMAs and P without the call."""
    at = lambda i, n: None if i == role else _kernel(-1)(i, n)  # noqa: E731
    with pytest.raises(AssertionError, match="launch before"):
        _run(at, 4, 2, 1, -1, 0)
