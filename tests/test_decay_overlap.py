"""The output kernel of the decayed layer (csrc/decay_tc.cuh) starts before the
launch before it has ended.  Its bounded waits are to measure the block's own
pipeline: however long that launch still runs, no role may stand in one that
only the launch's end can release.  Run as a model on the CPU, on the roles of
test_decay_protocol: the launch before ends when nothing else can go on."""
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


def _run(monkeypatch, at, nt, nst, nsb, ragged, seed):
    class Block(Overlapped):
        pass
    Block.at = staticmethod(at)
    monkeypatch.setattr(protocol, "Block", Block)
    protocol.outputs(nt, nst, nsb, ragged, seed, beside=seed % 2 == 0)


@pytest.mark.parametrize("nsb", [1, 2])
@pytest.mark.parametrize("nst", [2, 3, 4])
def test_no_limit_runs_while_the_launch_before_does(monkeypatch, nsb, nst):
    for nt in range(1, 8):
        for ragged in {-1, 0, nt - 1}:
            for seed in range(40):
                _run(monkeypatch, _kernel(ragged), nt, nst, nsb, ragged, 100 * nt + seed)


@pytest.mark.parametrize("role", [0, 1, 2, 3])
def test_the_model_flags_a_role_that_waits_at_once(monkeypatch, role):
    """Loads past the first stages, the MMAs and P without the call."""
    at = lambda i, n: None if i == role else _kernel(-1)(i, n)  # noqa: E731
    with pytest.raises(AssertionError, match="launch before"):
        _run(monkeypatch, at, 4, 2, 1, -1, 0)
