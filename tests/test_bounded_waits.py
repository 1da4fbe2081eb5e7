"""What the recurrence and the block norm do when a device wait gives up (host-side checks:
no wait is made to run out on a GPU in the middle of a cluster's exchange).

Their CTAs store values into each other's shared memory, and copies land in it behind the
threads' backs.  A CTA whose wait gave up therefore may not simply leave or carry on: it sends
nothing more, waits for its own copies, and leaves once nothing is on its way to it any more.  A
model replays that rule with CTAs that stall at random; it also shows that leaving without it
lets a value arrive at a CTA that is gone.
"""
import random
import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "gated_delta_rule_118_b200" / "csrc"


@pytest.mark.parametrize("name", ["scan.cu", "block_norm.cu"])
def test_no_outcome_of_a_wait_is_dropped(name):
    """A call of a wait is never a statement of its own (but for the last waits before a CTA leaves,
    which say so with a cast), and kernels with clusters leave through the cluster's barrier."""
    text = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    dropped = re.findall(r"(?:[;{}]|\)\s)\s*(?:sm100::mbar_|ring\.)?wait\(", text)
    assert not dropped, dropped
    assert len(re.findall(r"\(void\)\s*(?:sm100::mbar_)?wait\(", text)) == 1
    assert "leave_cluster()" in text


class Cluster:
    """CTAs that exchange a value a step: each sends to all and waits for all, up to a limit."""
    LIMIT, FLIGHT, GRACE = 400, 8, 20

    def __init__(self, size, steps, seed, rule=True):
        self.rnd, self.size, self.steps, self.rule = random.Random(seed), size, steps, rule
        self.stall = {(self.rnd.randrange(size), self.rnd.randrange(steps)): self.rnd.choice((5, 200, 395, 405, 420, 900, 3000))
                      for _ in range(self.rnd.randrange(1, 4))}

    def run(self):
        size = self.size
        step, state, since = [0] * size, ["work"] * size, [0] * size
        busy = [self.stall.get((c, 0), 1) for c in range(size)]
        got = [[0] * size for _ in range(size)]   # [receiver][sender]: values landed
        flying = []                               # (arrival, receiver, sender)
        late = failed = 0
        for now in range(200000):
            for f in [f for f in flying if f[0] <= now]:
                flying.remove(f)
                late += state[f[1]] == "gone"
                got[f[1]][f[2]] += 1
            for c in range(size):
                if state[c] == "work":
                    busy[c] -= 1
                    if busy[c] <= 0:
                        flying += [(now + 1 + self.rnd.randrange(self.FLIGHT), r, c) for r in range(size)]
                        state[c], since[c] = "wait", now
                elif state[c] == "wait":
                    if min(got[c]) > step[c]:
                        step[c] += 1
                        state[c] = "gone" if step[c] == self.steps else "work"
                        busy[c] = self.stall.get((c, step[c]), 1)
                    elif now - since[c] > self.LIMIT:
                        failed += 1
                        state[c], since[c] = "barrier" if self.rule else "gone", now
                elif state[c] == "barrier" and all(s in ("barrier", "grace", "gone") for s in state):
                    state[c], since[c] = "grace", now
                elif state[c] == "grace" and now - since[c] > self.GRACE:
                    state[c] = "gone"
            if all(s == "gone" for s in state):
                return late + len(flying), failed
        raise AssertionError("the cluster does not end")


@pytest.mark.parametrize("size", [2, 4, 8])
def test_a_cluster_whose_waits_give_up_ends_without_a_late_value(size):
    failed = 0
    for seed in range(150):
        late, f = Cluster(size, 6, seed).run()
        assert late == 0, seed
        failed += f > 0
    assert failed > 20  # (the stalls do make waits give up)


def test_the_model_catches_a_cta_that_leaves_at_once():
    assert any(Cluster(4, 6, seed, rule=False).run()[0] for seed in range(150))
