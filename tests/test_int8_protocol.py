"""The weight ring of the int8 kernel for few tokens, on the CPU: one producer, three issuers, copies that land in any
order.  A parity wait passes when the barrier's current phase has the other parity, so it says nothing about two phases;
the model checks that every issuer multiplies the stage contents it means to, for random interleavings, and that it would
see the mistake that the kernel's rule avoids (stages that are another issuer's from turn to turn)."""
import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(__file__), "..", "bit_rotated_weight_b200", "csrc", "tq4_int8_stream.cu")


def constant(name):
    return int(re.search(rf"constexpr int {name} = (\d+);", open(SRC).read()).group(1))


class Barrier:
    def __init__(self):
        self.phase = 0                     # completed phases

    def passes(self, parity):
        return (self.phase & 1) != parity


def run(stages, issuers, tiles, steps, seed):
    """None if every multiplication saw the fill it was meant for, else what went wrong."""
    rng = random.Random(seed)
    total = tiles * steps
    full, empty = [Barrier() for _ in range(stages)], [Barrier() for _ in range(stages)]
    content = [None] * stages
    flying, sent = [], 0
    # an issuer's own turns: (number of the fill, its stage, its parity)
    todo = [[(li, li % stages, (li // stages) & 1) for li in range(total) if li % issuers == me] for me in range(issuers)]
    pending = []                            # MMAs whose commit has not arrived
    idle = 0
    while any(todo) or flying or pending or sent < total:
        act = rng.randrange(3 + issuers)
        idle += 1
        if act == 0 and sent < total:
            st, turn = sent % stages, sent // stages
            if sent < stages or empty[st].passes((turn & 1) ^ 1):
                flying.append(sent)
                sent += 1
                idle = 0
        elif act == 1 and flying:
            li = flying.pop(rng.randrange(len(flying)))
            content[li % stages] = li
            full[li % stages].phase += 1
            idle = 0
        elif act == 2 and pending:
            st = pending.pop(rng.randrange(len(pending)))
            empty[st].phase += 1
            idle = 0
        elif act >= 3 and todo[act - 3]:
            li, st, parity = todo[act - 3][0]
            if full[st].passes(parity):
                if content[st] != li:
                    return f"fill {li} read stage {st} holding {content[st]}"
                todo[act - 3].pop(0)
                pending.append(st)
                idle = 0
        if idle > 20000:
            return "stuck"
    return None


@pytest.mark.parametrize("stages", [3, 6, 9, 12])
@pytest.mark.parametrize("steps", [1, 2, 3, 7, 15, 21])
def test_ring_of_own_stages(stages, steps):
    issuers = constant("kIssuers")
    assert issuers == 3 and constant("kMaxStages") % issuers == 0
    for seed in range(40):
        assert run(stages, issuers, 5, steps, seed) is None


def test_the_model_sees_shared_stages():
    assert any(run(7, 3, 5, 21, seed) is not None for seed in range(200))


def test_launch_keeps_the_rule():
    # stages used again are a multiple of the issuers; else there is one for every step
    text = open(SRC).read()
    assert re.search(r"if \(a\.parts > 1 && stages >= part_steps\) stages = part_steps;.*\n\s*else stages -= stages % kIssuers;",
                     text)
    # and a tile's first k step is the issuer's whose turn it is
    assert text.count("turn3 = (turn3 + steps) % kIssuers;") == 2
