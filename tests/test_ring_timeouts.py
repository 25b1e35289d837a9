"""A model of the few-token layer's ring of weight tiles (csrc/forward_few.cu) when waits run out.

On the GPU a wait ends without its phase only if copies take seconds, which no test may bring about.
The model has the kernel's parts: barriers that count arrivals and whose waits see only a phase's
parity; a producer, one of whose lanes waits and sends, and which after a wait that ran out goes on
without either; sixteen warps that take a slot every other stage and, after a wait that ran out, go
on without giving slots back; copies that land in any order and as late as they like.  Whatever
runs out when: a slot with a copy under way is not filled again, the producer's lanes take the same
way, every role comes to its end, and no copy lands after it.

`early`, `split` and `careless` are rules that were wrong: slots given back after a wait that ran
out, a producer whose lanes each wait and judge for themselves, and waiting for copies under way
only where the producer's own wait ran out."""
import random

import pytest

WARPS = 16


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left = self.count
            self.phase += 1

    def done(self, parity):
        return (self.phase & 1) != parity


class Broken(Exception):
    pass


def ring(steps, stages, units, seed, rules=(), timeouts=2):
    """One block's two passes over its units; raises Broken where an invariant does not hold."""
    rnd = random.Random(seed)
    full, empty = [Barrier(1) for _ in range(stages)], [Barrier(WARPS // 2) for _ in range(stages)]
    under_way = []          # slots with a copy
    abort = False
    budget = timeouts       # waits that may still run out of time
    total = steps * units
    slow = rnd.random() < 0.5   # copies that rather land late

    def filled(slot):
        if slot in under_way:
            raise Broken("a slot with a copy under way is filled again")
        under_way.append(slot)

    lanes = 2 if "split" in rules else 1
    warps = [dict(gives_back=True, stage=[u * steps + 2 * i + w // 8 for u in range(units) for i in range(steps // 2)], at=0) for w in range(WARPS)]
    sent, verdicts, gave_up = 0, [None] * lanes, False

    def outcome(barrier, parity):
        """True, False (ran out, or saw the flag) or None: still waiting."""
        nonlocal budget
        if barrier.done(parity):
            return True
        if abort and rnd.random() < 0.5:
            return False
        if budget and rnd.random() < 0.02:
            budget -= 1
            return False
        return None

    idle = 0
    while (sent < total and not gave_up) or any(w["at"] < len(w["stage"]) for w in warps):
        idle += 1
        if idle > 20000:
            raise Broken("a role does not come to its end")
        who = rnd.randrange(WARPS + 3)
        if who < WARPS:
            w = warps[who]
            if w["at"] == len(w["stage"]):
                continue
            stage = w["stage"][w["at"]]
            got = outcome(full[stage % stages], (stage // stages) & 1)
            if got is None:
                continue
            if not got:
                abort = True
                w["gives_back"] = "early" in rules
            w["at"] += 1
            if w["gives_back"]:
                empty[stage % stages].arrive()
        elif who == WARPS:
            if sent == total or gave_up:
                continue
            slot = sent % stages
            if sent >= stages:
                for lane in range(lanes):
                    if verdicts[lane] is None:
                        verdicts[lane] = outcome(empty[slot], (sent // stages & 1) ^ 1)
                if None in verdicts:
                    continue
                if len(set(verdicts)) > 1:
                    raise Broken("the producer's lanes take different ways")
                go, verdicts = verdicts[0], [None] * lanes
                if not go:
                    abort = gave_up = True
                    continue
            filled(slot)
            sent += 1
        elif under_way and not (slow and rnd.random() < 0.9):
            slot = under_way.pop(rnd.randrange(len(under_way)))
            full[slot].arrive()
            idle = 0
    # the grid has synchronised: every role is here
    if gave_up if "careless" in rules else abort:
        for slot in range(min(stages, sent)):
            parity = (sent - 1 - slot) // stages & 1
            while not full[slot].done(parity):
                if not under_way:
                    raise Broken("a wait for a copy that was not sent")
                full[under_way.pop(0)].arrive()
    if under_way:
        raise Broken("a copy lands after the block's end")
    return abort


SHAPES = [(2, 4, 7), (4, 6, 5), (6, 8, 4), (8, 12, 4), (14, 12, 3), (4, 12, 1)]


@pytest.mark.parametrize("steps,stages,units", SHAPES)
def test_holds_whatever_runs_out(steps, stages, units):
    assert not ring(steps, stages, units, 0, timeouts=0)
    assert any([ring(steps, stages, units, seed, timeouts=seed % 4) for seed in range(150)])


@pytest.mark.parametrize("rule,what", [("early", "filled again"), ("split", "different ways"), ("careless", "after the block's end")])
def test_the_model_sees_what_was_wrong(rule, what):
    seen = set()
    for steps, stages, units in SHAPES:
        for seed in range(150):
            try:
                ring(steps, stages, units, seed, rules=(rule,), timeouts=seed % 4)
            except Broken as e:
                seen.add(str(e))
    assert any(what in s for s in seen), seen
