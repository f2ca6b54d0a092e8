"""How the int8 kernels end when a wait runs out, on the CPU.

No CTA may leave while something is still on its way into its shared memory: copies of its own, and what other CTAs
send.  The models run the roles in random order; a role gives up at a random moment, as a wait that runs out does, and
the others learn of it at their next wait that does not pass.

On the GPU a hook withholds one report and shortens the limit of every wait to 2 ms: the call has to end, to report
TQ_DEV_TIMEOUT, and to leave the context and the next calls as they were."""
import os
import random
import time

import pytest
import torch

import bit_rotated_weight_b200 as tq

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
CSRC = os.path.join(os.path.dirname(__file__), "..", "bit_rotated_weight_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


# ------------------------------------------------------------------ copies of the CTA itself
def one_cta(stages, issuers, total, seed, at_end):
    """Copies in flight when the CTA leaves.  `at_end`: where someone gave up, the last copies are waited for when every
    role has ended; else by the producer, when it has sent the last."""
    rng = random.Random(seed)
    give_up = rng.randrange(4 * total)                     # events until the epilogue gives up
    full, empty = [0] * stages, [0] * stages               # completed phases
    flying, pending = [], []
    sent, aborted, wait_for = 0, False, None
    turn = list(range(issuers))                            # each issuer's next fill
    producing, left = True, list(range(issuers))
    events = 0
    while True:
        events += 1
        assert events < 100000
        aborted = aborted or events >= give_up
        act = rng.randrange(issuers + 3)
        if act == 0 and flying and rng.random() < 0.3:
            full[flying.pop(rng.randrange(len(flying))) % stages] += 1
        elif act == 1 and pending:
            empty[pending.pop(0)] += 1
        elif act == 2 and producing:
            if wait_for is None:
                free = sent < stages or empty[sent % stages] >= sent // stages
                if sent == total or (not free and aborted):
                    wait_for = list(range(max(0, sent - stages), sent)) if aborted and not at_end else []
                elif free:
                    flying.append(sent)
                    sent += 1
            else:
                producing = not all(full[li % stages] > li // stages for li in wait_for)
        elif act >= 3 and act - 3 in left:
            me = act - 3
            if turn[me] >= total:
                left.remove(me)
            elif full[turn[me] % stages] > turn[me] // stages:
                pending.append(turn[me] % stages)
                turn[me] += issuers
            elif aborted:
                left.remove(me)
        if aborted and not producing and not left and not (
                at_end and any(full[li % stages] <= li // stages for li in range(max(0, sent - stages), sent))):
            return flying


@pytest.mark.parametrize("name,issuers", [("tq4_int8_stream.cu", 3), ("tq4_int8_gemm.cu", 1)])
@pytest.mark.parametrize("stages,total", [(3, 3), (3, 2), (6, 5), (6, 21), (12, 40)])
def test_own_copies_have_landed(name, issuers, stages, total):
    # where the source waits for them: behind the block's last barrier?
    kernel = source(name).split("// ---", 1)[0] if "gemm" in name else source(name)
    waits = max(kernel.rfind("int8_land_copies("), kernel.rfind("int8_drain_wait(&sh.full["))
    for seed in range(200):
        assert one_cta(stages, issuers, total, seed, waits > kernel.rindex("  __syncthreads();")) == []


def test_the_model_sees_copies_left_behind():
    assert any(one_cta(6, 1, 5, seed, False) for seed in range(200))


# ------------------------------------------------------------------ the tokens' codes
class Counted:
    """A barrier of so many arrivals a phase.  One operation of several threads must not run past the end of a phase."""

    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self, n=1):
        assert n <= self.pending, f"{n} arrivals at a phase with {self.pending} pending"
        self.pending -= n
        if self.pending == 0:
            self.phase, self.pending = self.phase + 1, self.count


def few_tokens(segments, withheld, seed, stop):
    """The roles that share the tokens' codes: 8 warps of quantizers (`withheld` threads of the first do not report the
    first segment), 3 issuers and 4 warps of the epilogue.  `stop`: quantizers whose wait ran out report no more."""
    rng = random.Random(seed)
    bfull, bempty, dfull = Counted(256), Counted(3 + 128), [Counted(3) for _ in range(segments)]
    give_up = rng.randrange(200, 800)                      # waits that began with the call run out from here on
    aborted = False
    turn = {("q", i): 0 for i in range(8)}
    turn.update({("i", i): 0 for i in range(3)})
    turn.update({("e", i): 0 for i in range(4)})
    inside = {("e", i): False for i in range(4)}           # has passed the wait for the codes
    at = {("q", i): "wait" for i in range(8)}              # for the last segment's readers, then the named barriers
    quit_ = False
    running = set(turn)
    for event in range(200000):
        if not running:
            return
        r = rng.choice(sorted(running))
        kind, t = r[0], turn[r]
        late = aborted or (event > give_up and rng.random() < 0.1)
        if t == segments:
            running.discard(r)
        elif kind == "q":
            if at[r] == "wait":
                free = bempty.phase >= t
                if free or late:
                    aborted |= not free
                    quit_ |= stop and not free
                    at[r] = "barrier"
                if all(v == "barrier" for v in at.values()):
                    at = dict.fromkeys(at, "left" if quit_ else "report")
            elif at[r] == "left":
                running.discard(r)
            elif at[r] == "report":
                n = 32 - (withheld if r[1] == 0 and t == 0 else 0)
                if n:
                    bfull.arrive(n)
                turn[r], at[r] = t + 1, "wait"
        elif kind == "i":
            if bfull.phase > t:
                dfull[t].arrive()
                bempty.arrive()
                turn[r] += 1
            elif late:
                aborted = True
                running.discard(r)
        else:
            if not inside[r] and bfull.phase > t:
                inside[r] = True
            elif inside[r] and dfull[t].phase:
                bempty.arrive(32)
                inside[r] = False
                turn[r] += 1
            elif late:
                aborted = True
                running.discard(r)
    raise AssertionError("stuck")


@pytest.mark.parametrize("withheld", [0, 1, 32])
@pytest.mark.parametrize("segments", [1, 2, 5])
def test_reports_stay_in_their_phase(segments, withheld):
    # do the quantizers leave their loop where a wait ran out?
    loop = source("tq4_int8_stream.cu").split("for (int32_t s = seg0", 1)[1].split("{", 1)[0]
    for seed in range(300):
        few_tokens(segments, withheld, seed, "go &&" in loop)


def test_the_model_sees_reports_that_run_over():
    def overruns(withheld):
        n = 0
        for seed in range(300):
            try:
                few_tokens(3, withheld, seed, False)
            except AssertionError as e:
                assert "pending" in str(e)
                n += 1
        return n

    assert overruns(1) > 0 and overruns(32) == 0


# ------------------------------------------------------------------ what other CTAs send
def cluster(parts, seed, barrier):
    """CTAs that exchange maxima, then sums, by stores that land some time after they are sent.  A CTA may be slow, and
    its waits run out.  None may be written to after it left.  `barrier`: the CTAs end together, and one whose wait ran
    out then waits for what was sent."""
    rng = random.Random(seed)
    speed = [rng.choice([1.0, 0.3, 0.02]) for _ in range(parts)]
    patience = rng.randrange(20, 400)
    step = ["send maxima"] * parts
    since = [0] * parts
    landed = [{"maxima": 0, "sums": 0} for _ in range(parts)]
    sent = [{"maxima": 0, "sums": 0} for _ in range(parts)]       # to this CTA
    flying, gone, gave_up = [], set(), set()
    for now in range(1000000):
        if len(gone) == parts and not flying:
            return gave_up
        if flying and rng.random() < 0.4:
            to, what = flying.pop(rng.randrange(len(flying)))
            assert to not in gone, "written to after its end"
            landed[to][what] += 1
        c = rng.randrange(parts)
        if c in gone or rng.random() > speed[c]:
            continue
        verb, _, what = step[c].partition(" ")
        if verb == "send":
            for to in range(parts):
                assert to not in gone, "written to after its end"
                flying.append((to, what))
                sent[to][what] += 1
            step[c], since[c] = "await " + what, now
        elif verb == "await":
            if landed[c][what] < parts:
                if now - since[c] < patience:
                    continue
                gave_up.add(c)
            step[c] = "send sums" if what == "maxima" else "end"
        elif not barrier:
            gone.add(c)
        elif all(s == "end" for i, s in enumerate(step)) and (c not in gave_up or landed[c] == sent[c]):
            gone.add(c)
    raise AssertionError("stuck")


@pytest.mark.parametrize("parts", [2, 4, 8])
def test_a_cluster_ends_together(parts):
    tail = source("tq4_int8_stream.cu")
    tail = tail[tail.rindex("mbar_arrive(&sh.bempty);"):tail.rindex("tmem_dealloc(")]
    runs = [cluster(parts, seed, tail.count("cluster_wait();") == 2) for seed in range(200)]
    assert any(runs) and not all(runs)                      # with waits that ran out, and without


def test_the_model_sees_a_cta_that_leaves_early():
    with pytest.raises(AssertionError, match="after its end"):
        for seed in range(200):
            cluster(4, seed, False)


# ------------------------------------------------------------------ two CTAs on one tile
def pair(stages, total, seed, both, last):
    """The ring of a pair, whose roles give up at random moments (the second CTA's at others).  A copy's bytes and the
    arrival that expects them are counted by the first CTA; commits arrive at both, at different times.
    `both`: at the end the first CTA waits for the copies of both, else for those of the stages that it sent itself, if
    it saw by then that it gave up.  `last`: the second CTA stays for its last arrival."""
    rng = random.Random(seed)
    give_up = [rng.randrange(6 * total), rng.randrange(12 * total)]
    aborted = [False, False]
    pending, tx = [1] * stages, [0] * stages               # of the first CTA's barriers
    full = [0] * stages
    empty = [[0] * stages for _ in range(2)]
    flying, arrivals = [], []                              # (cta, fill); (cta, stage or "done")
    sent, producing, issuing, issued = [0, 0], [True, True], True, 0
    seen = None                                            # what the first producer saw when it ended
    done = [False, False]

    def settle(s):
        if pending[s] == 0 and tx[s] == 0:
            full[s], pending[s] = full[s] + 1, 1

    def land():
        cta, li = flying.pop(rng.randrange(len(flying)))
        tx[li % stages] -= 1
        settle(li % stages)

    def arrive():
        cta, what = arrivals.pop(rng.randrange(min(2, len(arrivals))))
        if what == "done":
            done[cta] = True
        else:
            empty[cta][what] += 1

    for event in range(100000):
        for c in range(2):
            aborted[c] |= event >= give_up[c]
        act = rng.randrange(5)
        if act == 0 and flying and rng.random() < 0.3:
            land()
        elif act == 1 and arrivals:
            arrive()
        elif act in (2, 3) and producing[act - 2]:
            c, li = act - 2, sent[act - 2]
            free = li < stages or empty[c][li % stages] >= li // stages
            if li == total or (not free and aborted[c]):
                producing[c] = False
                if c == 0:
                    seen = aborted[0]
            elif free:
                if c == 0:
                    pending[li % stages] -= 1
                    tx[li % stages] += 2
                    settle(li % stages)
                flying.append((c, li))
                sent[c] += 1
        elif act == 4 and issuing:
            if issued < total and full[issued % stages] > issued // stages:
                arrivals += [(0, issued % stages), (1, issued % stages)]
                issued += 1
            elif issued == total or aborted[0]:
                arrivals += [(0, "done"), (1, "done")]
                issuing = False
        if not any(producing) and not issuing and done[0] and all(aborted):
            break                                           # both CTAs are at the cluster barrier
    else:
        raise AssertionError("stuck")
    own, other = sent
    most = max(own, other) if both else own if seen else 0
    for i in range(max(0, most - stages), most):
        s = i % stages
        if both and i >= own:
            pending[s] -= 1
            tx[s] += 1
            settle(s)
        elif both and i >= other:
            tx[s] -= 1
            settle(s)
        while full[s] <= i // stages and flying:
            land()
        if both:
            assert full[s] > i // stages
    while last and not done[1]:
        arrive()
    return flying, [a for a in arrivals if a[1] == "done"]


@pytest.mark.parametrize("stages,total", [(6, 4), (6, 30), (2, 9)])
def test_a_pair_ends_with_nothing_on_its_way(stages, total):
    text = source("tq4_int8_gemm.cu")
    text = text[text.index("int8_pair_kernel("):text.index("cudaError_t launch_pair")]
    end = text[text.rindex("__syncthreads();"):]
    for seed in range(300):
        assert pair(stages, total, seed, "land_pair(sh)" in end, "int8_drain_wait(&sh.mma_done, 0)" in end) == ([], [])


def test_the_model_sees_what_a_pair_leaves_behind():
    runs = [pair(6, 30, seed, False, False) for seed in range(300)]
    assert any(flying for flying, _ in runs) and any(late for _, late in runs)


# ------------------------------------------------------------------ on the GPU
@pytest.fixture
def hooks():
    tq.tq4_1s_get_status()
    yield
    tq.tq4_1s_debug_hook(tq.TQ_HOOK_FAIL_NEXT_CALLS, 0)
    tq.tq4_1s_debug_hook(tq.TQ_HOOK_WITHHOLD_ARRIVAL, 0)
    tq.tq4_1s_debug_hook(tq.TQ_HOOK_WAIT_NS, 0)


def runs_out(call):
    """`call` with a report withheld, between two that are whole."""
    want = call()
    torch.cuda.synchronize()
    assert tq.tq4_1s_get_status() == 0
    tq.tq4_1s_debug_hook(tq.TQ_HOOK_WAIT_NS, 2_000_000)
    tq.tq4_1s_debug_hook(tq.TQ_HOOK_WITHHOLD_ARRIVAL, 1)
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    tq.tq4_1s_debug_hook(tq.TQ_HOOK_WITHHOLD_ARRIVAL, 0)
    tq.tq4_1s_debug_hook(tq.TQ_HOOK_WAIT_NS, 0)
    assert tq.tq4_1s_get_status() & tq.TQ_DEV_TIMEOUT
    assert elapsed < 1.0
    for _ in range(3):
        assert torch.equal(call().view(torch.uint8), want.view(torch.uint8))
    assert tq.tq4_1s_get_status() == 0


def linear(m, n, k, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(m + n + k)
    w = tq.tq4_1s_int8_quantize(torch.randn(n, k, generator=g).to(DEV))
    x = torch.randn(m, k, generator=g).to(dtype).to(DEV)
    return lambda: tq.tq4_1s_linear_int8(x, w)


def moe(m, E, topk, H, I):
    g = torch.Generator().manual_seed(m + E)
    up = tq.tq4_1s_int8_quantize(torch.randn(E, I, H, generator=g).to(DEV))
    down = tq.tq4_1s_int8_quantize(torch.randn(E, H, I, generator=g).to(DEV))
    x = (0.1 * torch.randn(m, H, generator=g)).to(torch.bfloat16).to(DEV)
    ids = torch.randn(m, E, generator=g).argsort(1)[:, :topk].to(torch.int32).to(DEV)
    tw = torch.rand(m, topk, generator=g).to(DEV)
    return lambda: tq.tq4_1s_moe_int8(x, ids, tw, up, down)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(9, 40000, 256), (3, 20000, 4096), (40, 300, 64), (300, 4096, 1024),
                                   (100, 40000, 512)])
def test_linear_winds_down(hooks, m, n, k):
    # few tokens, many row tiles a block; one tile a block, and several
    runs_out(linear(m, n, k))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(2400, 4360, 416), (5000, 8192, 1024), (2304, 4096, 32)])
def test_pairs_wind_down(hooks, m, n, k):
    runs_out(linear(m, n, k))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k,dtype", [(1, 4096, 2688, torch.float16), (16, 4096, 4096, torch.bfloat16),
                                         (5, 300, 9216, torch.float32), (3, 7000, 4096, torch.bfloat16)])
def test_clusters_wind_down(hooks, m, n, k, dtype):
    # a row tile's k over 4, 4, 8 and 2 blocks, with stages used again in the last
    runs_out(linear(m, n, k, dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("m,E,topk,H,I", [(2, 16, 4, 256, 128), (90, 300, 3, 160, 96), (300, 8, 2, 512, 288)])
def test_moe_winds_down(hooks, m, E, topk, H, I):
    # slots sorted in the product, a segment a block; segments from a kernel of their own, several a block; tiles
    runs_out(moe(m, E, topk, H, I))


@pytest.mark.gpu
def test_failed_launches_are_reported_and_launch_nothing(hooks):
    W, z = torch.randn(64, 96, generator=torch.Generator().manual_seed(1)).to(DEV), torch.randn(5, 8, device=DEV)
    w = tq.tq4_1s_int8_quantize(W)
    few, many, pairs = linear(3, 300, 256), linear(40, 300, 256), linear(2304, 4096, 32)
    experts, prompt = moe(2, 16, 4, 256, 128), moe(300, 8, 2, 512, 288)
    for call in (lambda: tq.tq4_1s_int8_quantize(W).q, lambda: tq.tq4_1s_int8_dequantize(w), few, many, pairs, experts,
                 prompt, lambda: tq.tq4_1s_router_scored(z, 2)[1]):
        want = call()
        torch.cuda.synchronize()
        tq.tq4_1s_debug_hook(tq.TQ_HOOK_FAIL_NEXT_CALLS, 1)
        before = tq.tq4_1s_launch_count()
        with pytest.raises(tq.TQ4Error) as e:
            call()
        assert e.value.code == 5 and tq.tq4_1s_launch_count() == before
        assert torch.equal(call(), want) and tq.tq4_1s_launch_count() > before
    assert tq.tq4_1s_get_status() == 0
