"""The scored expert router: softmax or sigmoid scores, a balance bias, groups, top-k, renormalised weights.

Ids are compared with a plain fp64 implementation exactly.  Weights: with fp32 arithmetic an exponential is off by at most
2 units in the last place (2^-22), each other step by half a unit (2^-24); a weight takes its own score (exp, add, divide),
a sum of at most 1024 positive scores of which a lane adds 32 in a row and 5 across lanes, one of at most 32 chosen scores,
two divisions and the scale: (4 + 2) + 37 + 37 + 3 < 90 units of 2^-24, and for softmax the rounding of z - max z,
|z - max z| <= 20 here, up to 20 more each in the numerator and the sum: 130 * 2^-24 < 8e-6 relative."""
import ctypes
import gc

import numpy as np
import pytest
import torch

import bit_rotated_weight_b200 as tq

REL = 8e-6
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None


def reference(z, topk, bias, score, groups, keep, group_score, renorm, scale):
    z = np.asarray(z, np.float64)
    m, E = z.shape
    ids = np.full((m, topk), -1, np.int64)
    w = np.zeros((m, topk))
    for t in range(m):
        number = ~np.isnan(z[t])
        zt = np.where(number, z[t], -np.inf)
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                s = np.where(number, 1.0 / (1.0 + np.exp(-zt)), 0.0)
        else:
            top = zt.max()
            with np.errstate(invalid="ignore"):
                s = np.where(zt == top, 1.0, np.exp(zt - top)) if top > -np.inf else np.zeros(E)
            s = s / s.sum() if s.sum() > 0 else s
        can = number.copy()
        if bias is None:
            c = zt.copy()
            ranked = s if group_score == "top2" else c
        else:
            b = np.asarray(bias, np.float64)
            can &= b < np.inf
            c = s + np.where(can, b, 0.0)
            ranked = c
        if keep < groups:
            per = np.sort(np.where(can, ranked, -np.inf).reshape(groups, -1), axis=1)[:, ::-1]
            rank = per[:, 0] + per[:, 1] if group_score == "top2" else per[:, 0]
            best = np.argsort(-rank, kind="stable")[:keep]
            can &= np.isin(np.arange(E) // (E // groups), best)
        order = [e for e in np.argsort(-np.where(can, c, -np.inf), kind="stable") if can[e]][:topk]
        ids[t, :len(order)] = order
        w[t, :len(order)] = s[order]
    if renorm:
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return ids, w * scale


def check(z, topk, bias=None, score="sigmoid", groups=1, keep=1, group_score="top2", renorm=True, scale=1.0, **kw):
    b = None if bias is None else torch.as_tensor(bias, dtype=torch.float32, device=DEV)
    ids, w = tq.tq4_1s_router_scored(z, topk, bias=b, score=score, num_groups=groups, topk_groups=keep,
                                     group_score=group_score, renormalize=renorm, scale=scale, **kw)
    ids_ref, w_ref = reference(z.float().cpu().numpy(), topk, None if bias is None else b.cpu().numpy(), score, groups,
                               keep, group_score, renorm, scale)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    assert np.array_equal(ids.cpu().numpy(), ids_ref)
    got = w.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - w_ref) <= REL * np.abs(w_ref) + 1e-37), np.max(np.abs(got - w_ref) / (np.abs(w_ref) + 1e-37))
    return ids, w


@pytest.fixture(autouse=True)
def _clear_status():
    if torch.cuda.is_available():
        tq.tq4_1s_get_status()
    yield


def logits(m, E, seed, dtype=torch.float32, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(m, E, generator=g)).to(dtype).to(DEV)


def bias_of(E, seed):
    return 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(seed))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("m,E,topk,groups,keep,group_score,with_bias,renorm,scale", [
    (1, 128, 6, 1, 1, "max", True, True, 1.0),
    (16, 128, 6, 1, 1, "max", False, True, 1.0),
    (37, 128, 6, 8, 4, "max", False, False, 1.0),
    (33, 256, 8, 8, 4, "top2", True, True, 2.5),
    (5, 7, 7, 1, 1, "max", True, True, 0.5),          # every expert, fewer than a warp
    (3, 1, 1, 1, 1, "max", False, True, 1.0),         # one expert
    (6, 33, 3, 11, 1, "top2", True, False, 1.0),      # groups of 3 over a warp's edge
    (9, 1000, 12, 20, 3, "top2", False, True, 1.0),   # groups of 50, no bias
    (4, 1024, 32, 32, 32, "max", True, True, 1.0),    # the limits; every group kept
    (4, 1024, 32, 32, 1, "top2", True, True, 1.0),    # topk is the whole group
    (257, 64, 2, 32, 5, "top2", True, True, 1.0),     # groups of 2
    (300, 96, 5, 32, 7, "max", True, True, 1.0),      # groups of 3, by the best
])
def test_matches_plain(m, E, topk, groups, keep, group_score, with_bias, renorm, scale, score, dtype):
    check(logits(m, E, m * 1000 + E, dtype), topk, bias_of(E, E) if with_bias else None, score, groups, keep,
          group_score, renorm, scale)
    assert tq.tq4_1s_get_status() == 0


@pytest.mark.gpu
def test_near_ties_are_decided_in_64_bits():
    # scores plus biases that fp32 cannot tell apart: pairs of experts whose choice differs by 2^-30 .. 2^-40
    E, m = 64, 50
    rng = np.random.default_rng(5)
    z = rng.standard_normal((m, E)).astype(np.float32)
    zt = torch.from_numpy(z).to(DEV)
    # the same logit and biases that differ in their last bit, around values where fp32(s + b) rounds both alike
    z[:, 1::2] = z[:, 0::2]
    b = (0.01 * rng.standard_normal(E)).astype(np.float32)
    b[1::2] = np.nextafter(b[0::2], np.float32(np.inf))
    zt = torch.from_numpy(z).to(DEV)
    for score in ("softmax", "sigmoid"):
        check(zt, 8, torch.from_numpy(b), score)
        check(zt, 8, torch.from_numpy(b), score, 8, 3, "top2")
        check(zt, 8, torch.from_numpy(b), score, 8, 3, "max")
    # logits one unit apart, no bias
    z[:, 1::2] = np.nextafter(z[:, 0::2], np.float32(np.inf))
    for score in ("softmax", "sigmoid"):
        check(torch.from_numpy(z).to(DEV), 8, None, score, 8, 3, "max")
        check(torch.from_numpy(z).to(DEV), 8, None, score, 8, 3, "top2")


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_and_saturation(score):
    z = torch.zeros(3, 64, device=DEV)
    check(z, 5, None, score)                                       # all equal: the lowest ids
    check(z, 5, torch.zeros(64), score, 8, 3, "top2")
    z = torch.full((2, 64), 60.0, device=DEV)                      # saturated sigmoids keep the order of the logits
    z[:, 40:] = 61.0
    check(z, 6, None, score)
    z = logits(4, 64, 1, spread=1.0)
    z[1] = -200.0                                                  # scores far below 1
    z[2] += 300.0
    check(z, 6, bias_of(64, 3), score)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups,keep,group_score", [(1, 1, "max"), (8, 2, "top2"), (8, 2, "max")])
def test_infinities_and_nan(score, with_bias, groups, keep, group_score):
    z = logits(8, 64, 21)
    z[0, 5:] = -np.inf                          # fewer finite logits than topk
    z[1] = -np.inf                              # a row that leaves nothing
    z[2, 7] = np.inf
    z[2, 50] = np.inf
    b = bias_of(64, 22) if with_bias else None
    check(z, 8, b, score, groups, keep, group_score)
    check(z, 8, b, score, groups, keep, group_score, renorm=False)
    assert tq.tq4_1s_get_status() == 0
    z[3, 3] = np.nan
    z[4] = np.nan                               # nothing to choose: ids -1, weights 0
    z[5, :60] = np.nan                          # four left
    ids, w = check(z, 8, b, score, groups, keep, group_score)
    assert bool((ids[4] == -1).all()) and bool((w[4] == 0).all())
    assert tq.tq4_1s_get_status() == tq.TQ_DEV_NONFINITE


@pytest.mark.gpu
def test_bias_can_shut_experts():
    z = logits(16, 64, 31)
    b = bias_of(64, 32)
    b[10:20] = -np.inf
    check(z, 6, b, "sigmoid")
    check(z, 6, b, "softmax", 8, 3, "top2")
    assert tq.tq4_1s_get_status() == 0
    b[3] = np.nan
    b[4] = np.inf
    ids, _ = check(z, 6, b, "sigmoid")
    assert not bool(((ids == 3) | (ids == 4)).any())
    assert tq.tq4_1s_get_status() == tq.TQ_DEV_NONFINITE


@pytest.mark.gpu
def test_strides_streams_graph_and_empty():
    z = logits(40, 200, 41)
    b = bias_of(128, 42)
    view = z[:, 3:131]                                             # rows 200 apart, off alignment
    check(view, 6, b)
    check(z.t()[:128, :32].t(), 6, b)                              # column-major
    ids, w = tq.tq4_1s_router_scored(z[:0, :128].contiguous(), 6)
    assert ids.shape == (0, 6) and w.shape == (0, 6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = tq.tq4_1s_router_scored(view, 6, bias=b.to(DEV), score="sigmoid")
    s.synchronize()
    zin = z[:, :128].contiguous()
    bd = b.to(DEV)
    g = torch.cuda.CUDAGraph()
    gc.collect()                                                   # (a graph freed during a capture ends it)
    with torch.cuda.graph(g):
        out = tq.tq4_1s_router_scored(zin, 6, bias=bd, score="sigmoid")
    zin.copy_(view)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], a[0]) and torch.equal(out[1], a[1])


@pytest.mark.gpu
def test_many_rows_and_rows_behind_untouched():
    z = logits(70001, 40, 51, torch.bfloat16)
    check(z[:300], 4, bias_of(40, 52), "sigmoid", 5, 2, "top2")
    ids, w = tq.tq4_1s_router_scored(z, 4, score="sigmoid")
    top = torch.sort(z.float(), dim=1, descending=True, stable=True).indices[:, :4]
    assert torch.equal(ids.long(), top)
    # through the C entry, with guard values around the outputs
    lib = tq.load_library()
    cfg = tq._Router(40, 4, 1, 1, 1, 0, 1, 1.0)
    gi = torch.full((18, 4), -7, dtype=torch.int32, device=DEV)
    gw = torch.full((18, 4), -7.0, device=DEV)
    rc = lib.tq4_1s_router_scored(z.data_ptr(), 1, 16, ctypes.byref(cfg), 0, gi[1].data_ptr(), gw[1].data_ptr(),
                                  torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.equal(gi[1:17].long(), top[:16]) and torch.equal(gw[1:17], w[:16])
    assert bool((gi[[0, 17]] == -7).all()) and bool((gw[[0, 17]] == -7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("m,E,topk,groups,keep,group_score,with_bias,renorm", [
    (2048, 256, 8, 8, 4, "top2", True, True),
    (2079, 256, 8, 8, 4, "top2", False, False),
    (2081, 128, 6, 1, 1, "max", True, True),
    (2049, 128, 6, 1, 1, "max", False, True),
    (2500, 64, 3, 8, 2, "max", False, True),         # groups of 8, logits alone
    (2100, 512, 8, 32, 1, "top2", True, False),      # the widest bf16 row; one group of 16
    (2100, 24, 1, 1, 1, "max", True, True),
    (2100, 64, 8, 8, 8, "max", True, True),          # every group kept
])
def test_many_rows_match_plain(m, E, topk, groups, keep, group_score, with_bias, renorm, score, dtype):
    z = logits(m, E, m + E, dtype)
    z[5] = 0.0                                       # all equal
    z[6, ::2] = -0.0                                 # zeros of both signs are equal
    z[6, 1::2] = 0.0
    z[7] *= 100.0
    z[40] -= 300.0
    z[41, E // 2:] = -np.inf
    b = bias_of(E, E) if with_bias else None
    check(z, topk, b, score, groups, keep, group_score, renorm, 2.5)
    assert tq.tq4_1s_get_status() == 0
    z[m - 1, E - 1] = np.nan                         # in a group that may be left out
    z[100, 0] = np.inf
    check(z, topk, b, score, groups, keep, group_score, renorm)
    assert tq.tq4_1s_get_status() == tq.TQ_DEV_NONFINITE
    if with_bias:                                    # equal biases: ties by id wherever logits are equal
        check(z[:m - 1], topk, torch.zeros(E), score, groups, keep, group_score, renorm)
        b[3], b[5] = -np.inf, np.nan
        check(z[:m - 1], topk, b, score, groups, keep, group_score, renorm)


@pytest.mark.gpu
def test_zeros_of_both_signs_are_equal():
    z = torch.zeros(4, 64, device=DEV)
    z[0, ::2] = -0.0
    z[1, 1::3] = -0.0
    z[2, :] = -0.0
    for score in ("softmax", "sigmoid"):
        check(z, 9, None, score)
        check(z, 9, None, score, 8, 3, "max")
        check(z, 9, torch.zeros(64), score, 8, 3, "top2")


def test_refusals():
    lib = tq.load_library()
    good, null = 4096, None

    def call(logits=good, dtype=0, m=4, E=128, topk=6, score=1, groups=8, keep=4, gs=1, renorm=1, scale=1.0, bias=good,
             ids=good, w=good):
        cfg = tq._Router(E, topk, score, groups, keep, gs, renorm, scale)
        return lib.tq4_1s_router_scored(logits, dtype, m, ctypes.byref(cfg), bias, ids, w, null)

    assert call(m=0) == 0
    for bad in (dict(dtype=2), dict(dtype=-1), dict(m=-1), dict(E=0), dict(E=1025, groups=1, keep=1), dict(topk=0),
                dict(topk=33), dict(groups=0), dict(groups=3), dict(keep=0), dict(keep=9), dict(topk=17, keep=1),
                dict(score=2), dict(gs=2), dict(renorm=2), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(logits=null), dict(ids=null), dict(w=null), dict(E=8, groups=8, topk=4),
                dict(E=1024, groups=64, keep=64)):
        assert call(**bad) == 1, bad
    assert call(logits=4098) == 2 and call(logits=4097, dtype=1) == 2
    assert call(bias=4098) == 2 and call(ids=4098) == 2 and call(w=4097) == 2
    assert lib.tq4_1s_router_scored(good, 0, 4, None, null, good, good, null) == 1
    if not torch.cuda.is_available():
        assert call() == 3
    z = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        tq.tq4_1s_router_scored(z, 2)                              # not on a GPU


@pytest.mark.gpu
def test_refusals_of_the_binding():
    z = logits(4, 64, 61)
    for kw in (dict(score="tanh"), dict(group_score="sum"), dict(bias=torch.zeros(64)),
               dict(bias=torch.zeros(63, device=DEV)), dict(bias=torch.zeros(64, device=DEV, dtype=torch.float16))):
        with pytest.raises(ValueError):
            tq.tq4_1s_router_scored(z, 4, **kw)
    with pytest.raises(ValueError):
        tq.tq4_1s_router_scored(z.half(), 4)
    with pytest.raises(ValueError):
        tq.tq4_1s_router_scored(z[0], 4)
    for kw in (dict(topk=0), dict(topk=65), dict(topk=4, num_groups=3), dict(topk=9, num_groups=8, topk_groups=1)):
        with pytest.raises(tq.TQ4Error):
            tq.tq4_1s_router_scored(z, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [60, 3000])
@pytest.mark.parametrize("topk", [1, 5, 7, 8])
def test_near_ties_of_many_rows(m, topk):
    # logits on a coarse grid and biases that differ by 2^-20 .. 2^-26: most rows have neighbours that fp32 cannot order
    E = 64
    rng = np.random.default_rng(m + topk)
    z = (rng.integers(-6, 7, (m, E)) / 4).astype(np.float32)
    b = (rng.integers(0, 3, E) * 0.125 + rng.integers(-8, 9, E) * 2.0 ** -rng.integers(20, 27, E)).astype(np.float32)
    zt = torch.from_numpy(z).to(DEV)
    for score in ("sigmoid", "softmax"):
        check(zt, topk, torch.from_numpy(b), score)
        check(zt, topk, torch.from_numpy(b), score, 8, 3, "top2")
        check(zt.bfloat16(), topk, torch.from_numpy(b), score, 4, 2, "max")
    # logits alone, a unit or two apart
    z = (z.view(np.int32) + rng.integers(0, 3, z.shape).astype(np.int32) * (z != 0)).view(np.float32)
    check(torch.from_numpy(z).to(DEV), topk, None, "sigmoid", 8, 3, "max")
    check(torch.from_numpy(z).to(DEV), topk, None, "softmax")


@pytest.mark.gpu
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("m", [40, 1500])
def test_near_ties_of_groups(m, group_score):
    # groups made of the same few logits and of biases that differ by 2^-22 .. 2^-30: their ranks are near, or equal
    E, G = 128, 8
    rng = np.random.default_rng(m)
    z = np.tile((rng.integers(-4, 5, (m, 1, 16)) / 4), (1, G, 1)).reshape(m, E).astype(np.float32)
    b = np.tile(rng.integers(0, 3, 16) * 0.125, G) + np.repeat(rng.integers(0, 2, G) * 2.0 ** -rng.integers(22, 31, G), 16)
    b = torch.from_numpy(b.astype(np.float32))
    for score in ("sigmoid", "softmax"):
        for keep in (1, 4, 7):
            check(torch.from_numpy(z).to(DEV), 6, b, score, G, keep, group_score)
            check(torch.from_numpy(z).to(DEV), 6, None, score, G, keep, group_score)
    # two of the groups only
    z[:, 32:] -= rng.random((m, E - 32)).astype(np.float32) + 2
    for score in ("sigmoid", "softmax"):
        check(torch.from_numpy(z).to(DEV), 6, b, score, G, 1, group_score)


@pytest.mark.gpu
@pytest.mark.parametrize("E", [128, 256, 512])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("edge", [2.5, 3.0, 4.0])
def test_largest_biases_of_many_rows(E, score, edge):
    # choice values next to 4, and biases next to where the keys in fixed point end
    m = 300
    z = logits(m, E, E, torch.bfloat16)
    z[:, 5], z[:, E // 2] = 39.0, 4.0
    b = torch.zeros(E)
    b[5] = float(np.nextafter(np.float32(edge), np.float32(0)))
    b[9] = -b[5]
    check(z, 8, b, score)
    check(z, 8, b, score, 4, 2, "top2")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("m,E,topk,groups,keep,group_score,with_bias,renorm", [
    (301, 250, 7, 1, 1, "max", False, True),         # rows that are no whole number of 16 bytes
    (300, 245, 8, 1, 1, "max", True, True),
    (1025, 200, 8, 8, 5, "top2", True, False),       # groups of 25
    (515, 200, 3, 8, 5, "top2", False, True),
    (270, 148, 6, 2, 1, "top2", True, True),         # groups of 74
    (270, 60, 5, 4, 3, "max", True, True),           # groups of 15
    (270, 36, 8, 12, 5, "top2", True, True),         # groups of 3
    (270, 58, 2, 29, 1, "max", False, True),         # groups of 2, one kept, fewer than three
    (400, 317, 4, 1, 1, "max", True, False),
    (400, 511, 8, 7, 6, "max", True, True),          # as wide as they come: 7 x 80 places do not fit
    (400, 497, 8, 7, 6, "top2", True, True),         # 7 x 72 do
    (2048, 15, 8, 1, 1, "max", True, True),
    (2048, 9, 8, 1, 1, "max", False, True),          # all but one
    (256, 7, 6, 1, 1, "max", True, True),
    (260, 2, 1, 1, 1, "max", True, True),
])
def test_many_rows_of_odd_sizes(m, E, topk, groups, keep, group_score, with_bias, renorm, score, dtype):
    z = logits(m + 1, E, m + E, dtype)[1:] if E % 2 else logits(m, E, m + E, dtype)   # (off 16 bytes)
    b = bias_of(E, E) if with_bias else None
    check(z, topk, b, score, groups, keep, group_score, renorm, 2.5)
    z[3] = 0.0
    z[4] = -39.0
    z[5] = 41.0
    z[6, : E // 2] = -np.inf
    z[m - 9] *= 30.0
    check(z, topk, b, score, groups, keep, group_score, renorm)
    assert tq.tq4_1s_get_status() == 0
    if with_bias:
        b[0], b[E - 1] = -2.5, 2.5
        check(z, topk, b, score, groups, keep, group_score, renorm)
    z[m - 1, E - 1] = np.nan
    check(z, topk, b, score, groups, keep, group_score, renorm)
    assert tq.tq4_1s_get_status() == tq.TQ_DEV_NONFINITE


@pytest.mark.gpu
def test_equal_bf16_logits_at_the_last_place():
    # three and more equal logits around the last place: the lower ids, in either variant
    for m in (30, 300):
        z = logits(m, 250, m, torch.bfloat16)
        z[:, 10::20] = 2.5
        for topk in (1, 4, 8, 12):
            check(z, topk, None, "softmax")
            check(z, topk, None, "sigmoid", 5, 2, "max")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("m,E,topk,groups,keep,group_score,with_bias,renorm", [
    (300, 256, 9, 8, 4, "top2", True, True),
    (1031, 256, 16, 8, 4, "top2", True, True),       # as many as a thread keeps
    (300, 128, 12, 1, 1, "max", False, True),
    (300, 17, 16, 1, 1, "max", True, True),          # all but one
    (300, 24, 15, 4, 3, "max", True, False),
    (300, 500, 13, 1, 1, "max", True, True),
    (300, 96, 11, 12, 2, "top2", False, False),
    (300, 64, 17, 1, 1, "max", True, True),          # one more than that form takes
])
def test_many_rows_of_many_choices(m, E, topk, groups, keep, group_score, with_bias, renorm, score, dtype):
    z = logits(m, E, m + E + topk, dtype)
    b = bias_of(E, E) if with_bias else None
    check(z, topk, b, score, groups, keep, group_score, renorm, 2.5)
    z[3], z[4], z[5] = 0.0, -39.0, 41.0
    z[6, : E // 2] = -np.inf
    check(z, topk, b, score, groups, keep, group_score, renorm)
    # the same bits as in the form of few rows
    few = tq.tq4_1s_router_scored(z[:200].contiguous(), topk, bias=None if b is None else b.to(DEV), score=score,
                                  num_groups=groups, topk_groups=keep, group_score=group_score, renormalize=renorm)
    many = tq.tq4_1s_router_scored(z, topk, bias=None if b is None else b.to(DEV), score=score,
                                   num_groups=groups, topk_groups=keep, group_score=group_score, renormalize=renorm)
    assert torch.equal(few[0], many[0][:200])
    if score == "sigmoid":                           # (softmax sums its row in another order)
        assert torch.equal(few[1][7:], many[1][7:200])


@pytest.mark.gpu
@pytest.mark.parametrize("topk", [9, 12, 15, 16])
def test_near_ties_of_many_choices(topk):
    E, m = 64, 2000
    rng = np.random.default_rng(topk)
    z = (rng.integers(-6, 7, (m, E)) / 4).astype(np.float32)
    b = (rng.integers(0, 3, E) * 0.125 + rng.integers(-8, 9, E) * 2.0 ** -rng.integers(20, 27, E)).astype(np.float32)
    b[::2] += rng.random(32).astype(np.float32)      # single pairs too
    zt = torch.from_numpy(z).to(DEV)
    for score in ("sigmoid", "softmax"):
        check(zt, topk, torch.from_numpy(b), score)
        check(zt, topk, torch.from_numpy(b), score, 8, 3, "top2")
    z = (z.view(np.int32) + rng.integers(0, 3, z.shape).astype(np.int32) * (z != 0)).view(np.float32)
    check(torch.from_numpy(z).to(DEV), topk, None, "sigmoid", 8, 3, "max")
    check(torch.from_numpy(z).to(DEV), topk, None, "softmax")
