"""The barriers of the int8 kernels, on the CPU.

The weight ring of the kernel for few tokens: one producer, three issuers, copies that land in any
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


# ------------------------------------------------------------------ named barriers
def source(name):
    with open(os.path.join(os.path.dirname(SRC), name)) as f:
        return f.read()


def test_named_barriers_are_reached_by_as_many_threads_as_they_count():
    # bar.sync cannot time out.  In each kernel the roles are whole warps, and each barrier stands in one role's code.
    stream = source("tq4_int8_stream.cu")
    assert re.search(r"kThreads = 512, kQuantThreads = 256, kEpilogue = 128;", stream)
    # barrier 3: warps 1 to 7, before the roles; barrier 2: the quantizers, warps 8 to 15
    assert "if (warp >= 1 && warp < 8) {" in stream and "named_bar_sync(3, 7 * 32);" in stream
    quant = stream[stream.index("} else if (warp >= 8) {"):stream.index("// ---- epilogue")]
    assert quant.count("named_bar_sync(2, kQuantThreads);") == 2 == stream.count("named_bar_sync(2,")
    assert stream.count("named_bar_sync(") == 3
    # every iteration of the quantizers reaches both: nothing leaves the loop early
    loop = quant[quant.index("for (int32_t s = seg0"):]
    assert "break;" not in loop and "return" not in loop and "continue" not in loop
    gemm = source("tq4_int8_gemm.cu")
    assert "kThreads = 128 + kEpilogue" in gemm and "kEpilogue = 128 * kParts" in gemm
    assert re.search(r"kPairThreads = 384, kPairEpilogue = 256;", gemm)
    cut = gemm.index("- pairs\n")
    single, pair = gemm[:cut], gemm[cut:]
    for text, count in ((single, "S::kEpilogue"), (pair, "kPairEpilogue")):
        role = text[text.index("} else if (warp >= 4) {"):]
        assert role.count(f"named_bar_sync(1, {count});") == 1 == text.count("named_bar_sync(")
        # the threads of the role agree on leaving: it is decided by one of them, before the barrier
        assert re.search(r"named_bar_sync\(1, [\w:]+\);\s+if \(!sh\.epi_ok\[db\]\) break;", role)


# ------------------------------------------------------------------ the ring of a pair of CTAs
def run_pair(stages, total, seed):
    """Two producers, one issuer: a stage's barrier counts one arrival and the bytes of both CTAs' copies."""
    rng = random.Random(seed)
    arrived, landed = [0] * stages, [0] * stages          # of the current phase: arrival, pieces (2 a CTA)
    full = [Barrier() for _ in range(stages)]
    empty = [[Barrier() for _ in range(stages)] for _ in range(2)]
    content = [[None] * stages for _ in range(2)]
    sent, flying, issued, commits, idle = [0, 0], [], 0, [], 0

    def settle(st):
        if arrived[st] == 1 and landed[st] == 4:
            full[st].phase += 1
            arrived[st] = landed[st] = 0

    while issued < total or flying or commits:
        act = rng.randrange(5)
        idle += 1
        if act < 2 and sent[act] < total:
            li = sent[act]
            st, turn = li % stages, li // stages
            if li < stages or empty[act][st].passes((turn & 1) ^ 1):
                if act == 0:                              # the first CTA's producer says how many bytes there will be
                    if arrived[st]:
                        return "a second arrival in one phase"
                    arrived[st] = 1
                    settle(st)
                flying += [(act, li), (act, li)]
                sent[act] += 1
                idle = 0
        elif act == 2 and flying:
            cta, li = flying.pop(rng.randrange(len(flying)))
            content[cta][li % stages] = li
            landed[li % stages] += 1
            if landed[li % stages] > 4:
                return "bytes of two turns in one phase"
            settle(li % stages)
            idle = 0
        elif act == 3 and issued < total:
            st = issued % stages
            if full[st].passes((issued // stages) & 1):
                if content[0][st] != issued or content[1][st] != issued:
                    return f"turn {issued} read {content[0][st]} and {content[1][st]}"
                commits.append(issued)
                issued += 1
                idle = 0
        elif act == 4 and commits:                        # commits complete in order, at both CTAs
            st = commits.pop(0) % stages
            for cta in range(2):
                empty[cta][st].phase += 1
            idle = 0
        if idle > 20000:
            return "stuck"
    return None


@pytest.mark.parametrize("stages", [1, 2, 6])
def test_ring_of_a_pair(stages):
    for seed in range(60):
        assert run_pair(stages, 40, seed) is None
