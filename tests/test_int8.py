"""The int8 format, its linear layer and its MoE.

Codes and scales are compared exactly with the definition in 64 bits.  Products: the integer sums are exact, so the result
is compared bit for bit with the same fp32 steps in numpy (fp32 of the sum, times the token's scale, times the row's, one
rounding to the output's type), and with the formula in 64 bits within those roundings: three of 2^-24 and half a unit of
the output's type."""
import contextlib
import ctypes
import gc
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import bit_rotated_weight_b200 as tq

DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _clear_status():
    if torch.cuda.is_available():
        tq.tq4_1s_get_status()
    yield


def gen(seed):
    return torch.Generator().manual_seed(seed)


def ref_rows(x):
    """(codes, fp32 scales) of the rows of x, from the definition in 64 bits.  127 x is exact there, and a quotient that is
    no tie is at least 2^-25 away from one (x and max|x| have 24 bits), far above the division's rounding."""
    x = x.detach().cpu().double().numpy()
    top = np.abs(x).max(axis=-1)
    q = np.rint(np.divide(127.0 * x, top[..., None], out=np.zeros_like(x), where=top[..., None] > 0)).astype(np.int64)
    return q, (top.astype(np.float32) / np.float32(127.0)).astype(np.float32)


def ref_fp32(acc, sx, sw):
    """The kernel's fp32 steps on exact sums."""
    return (acc.astype(np.float32) * sx[:, None].astype(np.float32)).astype(np.float32) * sw[None, :].astype(np.float32)


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32).cpu()


def weight(n, k, seed, E=1):
    W = 0.02 * torch.randn(E, n, k, generator=gen(seed))
    q, s = ref_rows(W)
    return tq.Int8Weight(torch.from_numpy(q.astype(np.int8)).to(DEV), torch.from_numpy(s).to(DEV), n, k, E), q, s


@contextlib.contextmanager
def capture(graph):
    """torch.cuda.graph with the collector at rest: a graph of an earlier test that is freed during a capture ends it."""
    gc.collect()
    gc.disable()
    try:
        with torch.cuda.graph(graph):
            yield
    finally:
        gc.enable()


# ------------------------------------------------------------------ the quantizer
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n,k", [(1, 32), (3, 64), (7, 96), (130, 160), (5, 1024), (33, 2688), (64, 4096), (9, 4128),
                                 (3, 8224), (2, 16416), (2, 131072), (1000, 32)])
def test_quantize_matches_definition(n, k, dtype):
    W = torch.randn(n, k, generator=gen(n * 7 + k)).to(dtype)
    w = tq.tq4_1s_int8_quantize(W.to(DEV))
    q, s = ref_rows(W)
    assert np.array_equal(w.q[0].cpu().numpy(), q)
    assert np.array_equal(w.wscale[0].cpu().numpy(), s)
    back = tq.tq4_1s_int8_dequantize(w)[0].cpu().numpy()
    assert np.array_equal(back, q.astype(np.float32) * s[:, None])
    assert tq.tq4_1s_get_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_quantize_borders(dtype):
    # halves of the largest value (63.5), every border (c + 1/2) / 127 of it and its neighbours, at several sizes
    rows = []
    for top in (1.0, 0.75, 127.0, 254.0, 3.0, 1.9921875, 0.001):
        t = torch.tensor(top, dtype=dtype).double()
        c = torch.arange(0, 127, dtype=torch.float64) + 0.5
        x = (c * t / 127.0).to(dtype)
        near = torch.nextafter(x, torch.tensor(float("inf"), dtype=dtype)), torch.nextafter(x, torch.zeros_like(x))
        row = torch.cat([t.to(dtype).view(1), (t / 2).to(dtype).view(1), (-t / 2).to(dtype).view(1), x, -x, *near])
        rows.append(torch.nn.functional.pad(row, (0, 640 - row.numel())))
    W = torch.stack(rows)
    w = tq.tq4_1s_int8_quantize(W.to(DEV))
    q, s = ref_rows(W)
    assert np.array_equal(w.q[0].cpu().numpy(), q) and np.array_equal(w.wscale[0].cpu().numpy(), s)


@pytest.mark.gpu
def test_quantize_random_fp32_borders():
    # fp32 values within a few units of a border of their row: the quotient's rounding decides
    rng = np.random.default_rng(3)
    top = rng.uniform(0.5, 2.0, (200, 1)).astype(np.float32)
    x = ((rng.integers(0, 127, (200, 512)) + 0.5) * top / 127.0).astype(np.float32)
    x = (x.view(np.int32) + rng.integers(-3, 4, x.shape).astype(np.int32)).view(np.float32)
    x[:, 0] = top[:, 0]
    x *= np.where(rng.random(x.shape) < 0.5, -1, 1).astype(np.float32)
    W = torch.from_numpy(np.clip(x, -top, top))
    w = tq.tq4_1s_int8_quantize(W.to(DEV))
    q, s = ref_rows(W)
    assert np.array_equal(w.q[0].cpu().numpy(), q) and np.array_equal(w.wscale[0].cpu().numpy(), s)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,sizes", [(F32, (1e-45, 1e-40, 1e-37, 1e-18, 1e-17, 1e18, 3e38)),
                                         (BF16, (1e-40, 1e-37, 1e-18, 3e38)), (F16, (6e-8, 1e-5, 6e4))])
def test_quantize_extreme_sizes(dtype, sizes):
    base = torch.randn(len(sizes), 256, generator=gen(8)).clamp(-1, 1)
    W = (base.double() * torch.tensor(sizes, dtype=torch.float64)[:, None]).to(dtype)
    W = torch.cat([W, torch.zeros(1, 256, dtype=dtype), -torch.zeros(1, 256, dtype=dtype)])
    w = tq.tq4_1s_int8_quantize(W.to(DEV))
    q, s = ref_rows(W)
    assert np.array_equal(w.q[0].cpu().numpy(), q) and np.array_equal(w.wscale[0].cpu().numpy(), s)
    assert tq.tq4_1s_get_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_quantize_nonfinite_rows(dtype):
    W = torch.randn(6, 320, generator=gen(9)).to(dtype)
    W[1, 7] = float("nan")
    W[3, 319] = float("inf")
    W[4, 0] = -float("inf")
    w = tq.tq4_1s_int8_quantize(W.to(DEV))
    assert tq.tq4_1s_get_status() == tq.TQ_DEV_NONFINITE
    q, s = ref_rows(W[[0, 2, 5]])
    assert np.array_equal(w.q[0].cpu().numpy()[[0, 2, 5]], q) and np.array_equal(w.wscale[0].cpu().numpy()[[0, 2, 5]], s)
    assert bool((w.q[0, [1, 3, 4]] == 0).all()) and bool(w.wscale[0, [1, 3, 4]].isnan().all())


@pytest.mark.gpu
def test_quantize_a_stack_and_a_strided_weight():
    W = torch.randn(3, 40, 64, generator=gen(10))
    w = tq.tq4_1s_int8_quantize(W.to(DEV))
    q, s = ref_rows(W)
    assert (w.num_experts, w.n, w.k) == (3, 40, 64)
    assert np.array_equal(w.q.cpu().numpy(), q) and np.array_equal(w.wscale.cpu().numpy(), s)
    wt = tq.tq4_1s_int8_quantize(W[0].to(DEV).t()[:, :32])
    q, s = ref_rows(W[0].t()[:, :32])
    assert np.array_equal(wt.q[0].cpu().numpy(), q) and np.array_equal(wt.wscale[0].cpu().numpy(), s)


# ------------------------------------------------------------------ the linear layer
def check_linear(x, w, q, s, **kw):
    y = tq.tq4_1s_linear_int8(x.to(DEV), w, **kw)
    xq, xs = ref_rows(x)
    acc = torch.from_numpy(xq.astype(np.float64)) @ torch.from_numpy(q[0].astype(np.float64)).t()   # exact: < 2^31
    acc = acc.numpy()
    want = torch.from_numpy(ref_fp32(acc, xs, s[0])).to(x.dtype)
    assert y.dtype == x.dtype and y.shape == want.shape
    assert torch.equal(bits(y), bits(want))
    exact = acc * xs[:, None].astype(np.float64) * s[0][None, :].astype(np.float64)
    room = 3 * 2.0 ** -24 + torch.finfo(x.dtype).eps / 2 * (1 + 2.0 ** -20)
    assert np.all(np.abs(y.cpu().double().numpy() - exact) <= room * np.abs(exact) + torch.finfo(x.dtype).tiny)
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k,dtype", [
    (1, 1, 32, F32), (1, 64, 96, BF16), (1, 4096, 2688, F16), (2, 130, 160, BF16), (3, 127, 128, F32),
    (5, 4096, 4096, BF16), (15, 1000, 2688, BF16), (16, 4096, 4096, BF16), (16, 129, 32, F16), (17, 256, 1024, BF16),
    (31, 1857, 2688, F32), (32, 2688, 4096, BF16), (33, 77, 224, F16), (64, 1856, 2688, BF16), (65, 300, 512, BF16),
    (100, 4097, 1024, F32), (128, 2688, 1856, BF16), (129, 513, 640, BF16), (200, 4096, 4096, BF16),
    (255, 128, 8192, F16), (256, 1024, 256, BF16), (257, 1857, 2688, F32), (333, 300, 4096, BF16),
    (1000, 1000, 992, F16), (2049, 384, 128, BF16), (7, 33000, 64, BF16), (513, 14336, 96, BF16), (4, 48, 40000, BF16),
])
def test_linear_matches_plain(m, n, k, dtype):
    w, q, s = weight(n, k, n + k)
    x = torch.randn(m, k, generator=gen(m + k)).to(dtype)
    if m > 2:
        x[m // 2] = 0
        x[-1] *= 100
    check_linear(x, w, q, s)
    assert tq.tq4_1s_get_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k,dtype", [
    (2304, 4096, 32, BF16), (2309, 4097, 160, BF16), (2500, 4099, 96, F32), (2400, 4360, 416, F16),
    (5000, 2561, 64, BF16), (9000, 1100, 1024, BF16),
])
def test_linear_many_tokens(m, n, k, dtype):
    # tiles shared by two blocks: ragged ends of tokens, rows and k
    w, q, s = weight(n, k, n + k)
    check_linear(torch.randn(m, k, generator=gen(m + k)).to(dtype), w, q, s)
    assert tq.tq4_1s_get_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 40])
def test_linear_largest_sums(m):
    # every product 127 * 127 at the largest k: the int32 sums reach 2.11e9
    k = 131072
    q = np.full((1, 5, k), 127, np.int64)
    q[0, 1] = -127
    s = np.full((1, 5), 0.5, np.float32)
    w = tq.Int8Weight(torch.from_numpy(q.astype(np.int8)).to(DEV), torch.from_numpy(s).to(DEV), 5, k, 1)
    check_linear(torch.full((m, k), 2.0), w, q, s)


@pytest.mark.gpu
def test_linear_codes_of_minus_128():
    # a weight from elsewhere may hold -128
    w, q, s = weight(70, 96, 4)
    q[0, ::3, ::5] = -128
    w.q.copy_(torch.from_numpy(q.astype(np.int8)))
    check_linear(torch.randn(9, 96, generator=gen(1)), w, q, s)


@pytest.mark.gpu
def test_linear_rows_do_not_depend_on_the_batch():
    w, _, _ = weight(1000, 1184, 12)
    x = torch.randn(700, 1184, generator=gen(13)).to(BF16).to(DEV)
    whole = tq.tq4_1s_linear_int8(x, w)
    for lo, hi in ((0, 1), (5, 21), (21, 53), (100, 164), (164, 292), (292, 549), (699, 700)):
        assert torch.equal(bits(tq.tq4_1s_linear_int8(x[lo:hi], w)), bits(whole[lo:hi])), (lo, hi)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_linear_strided_rows(dtype):
    w, q, s = weight(200, 320, 14)
    buf = torch.randn(50, 700, generator=gen(15)).to(dtype)
    dev = buf.to(DEV)
    for view in (lambda b: b[:, :320], lambda b: b[:, 1:321], lambda b: b[::3, 8:328], lambda b: b[3:4, 7:327],
                 lambda b: b[:320].t()[:60, :50].t().repeat(1, 6)[:, :320], lambda b: b[:1, :320].expand(9, 320),
                 lambda b: b[:, :640:2]):
        y = check_linear(view(buf), w, q, s)
        assert torch.equal(bits(tq.tq4_1s_linear_int8(view(dev), w)), bits(y))


@pytest.mark.gpu
def test_linear_nonfinite_rows_stay_their_own():
    w, q, s = weight(300, 256, 16)
    x = torch.randn(40, 256, generator=gen(17)).to(BF16)
    clean = tq.tq4_1s_linear_int8(x.to(DEV), w)
    x[3, 5] = float("nan")
    x[39, 0] = float("inf")
    y = tq.tq4_1s_linear_int8(x.to(DEV), w)
    assert tq.tq4_1s_get_status() == tq.TQ_DEV_NONFINITE
    rest = [i for i in range(40) if i not in (3, 39)]
    assert bool(y[[3, 39]].isnan().all()) and torch.equal(bits(y[rest]), bits(clean[rest]))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(5, 129), (40, 300), (300, 257)])
def test_linear_writes_its_rows_only(m, n):
    w, q, s = weight(n, 160, 18)
    x = torch.randn(m, 160, generator=gen(19)).to(BF16).to(DEV)
    buf = torch.full(((m + 16) * n + 64,), 7.0, dtype=BF16, device=DEV)
    lo = 8 * n + (-8 * n) % 8                  # a 16-byte boundary after eight rows
    out = buf[lo:lo + m * n].view(m, n)
    assert tq.tq4_1s_linear_int8(x, w, out=out) is out
    assert torch.equal(bits(out), bits(tq.tq4_1s_linear_int8(x, w)))
    assert bool((buf[:lo] == 7).all()) and bool((buf[lo + m * n:] == 7).all())


@pytest.mark.gpu
def test_linear_streams_graphs_and_workspaces():
    w, q, s = weight(1856, 2688, 20)
    xs = [torch.randn(m, 2688, generator=gen(21 + m)).to(BF16).to(DEV) for m in (1, 16, 100, 300)]
    want = [tq.tq4_1s_linear_int8(x, w) for x in xs]
    # one workspace for calls that follow one another, with anything in it
    ws = torch.full((max(tq.tq4_1s_linear_int8_workspace(x.shape[0], w) for x in xs),), 0xA5, dtype=torch.uint8,
                    device=DEV)
    for _ in range(3):
        for x, y in zip(xs, want):
            assert torch.equal(bits(tq.tq4_1s_linear_int8(x, w, workspace=ws)), bits(y))
    # four streams at once, each call with its own
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        got = []
        for st, x in zip(streams, xs):
            with torch.cuda.stream(st):
                got.append(tq.tq4_1s_linear_int8(x, w))
    torch.cuda.synchronize()
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want))
    # two captured graphs, replayed in turn over new inputs
    graphs = []
    for x in xs[1:3]:
        xin = x.clone()
        g = torch.cuda.CUDAGraph()
        with capture(g):
            y = tq.tq4_1s_linear_int8(xin, w)
        graphs.append((g, xin, y, x))
    for r in range(6):
        for g, xin, y, x in graphs:
            xin.copy_(x * (r + 1))
            g.replay()
    torch.cuda.synchronize()
    for g, xin, y, x in graphs:
        assert torch.equal(bits(y), bits(tq.tq4_1s_linear_int8(x * 6, w)))
    with pytest.raises(tq.TQ4Error, match=r"code 4\)"):
        tq.tq4_1s_linear_int8(xs[3], w, workspace=ws[:100])
    assert tq.tq4_1s_get_status() == 0


@pytest.mark.gpu
def test_linear_offsets_past_32_bits():
    # 2.2e9 outputs: the last rows of a batch against the same rows on their own
    w, q, s = weight(33000, 32, 90)
    x = torch.randn(66000, 32, generator=gen(91)).half().to(DEV)
    y = tq.tq4_1s_linear_int8(x, w)
    for rows in (slice(0, 9), slice(65000, 65009), slice(65990, 66000), slice(65000, 65300)):
        assert torch.equal(bits(y[rows]), bits(tq.tq4_1s_linear_int8(x[rows], w)))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 100])
def test_linear_refuses_an_output_over_its_input(m):
    w, _, _ = weight(64, 64, 92)
    buf = torch.zeros(2 * m * 64, dtype=BF16, device=DEV)
    x = buf[:m * 64].view(m, 64)
    for out in (x, buf[8:8 + m * 64].view(m, 64)):
        with pytest.raises(tq.TQ4Error, match=r"code 1\)"):
            tq.tq4_1s_linear_int8(x, w, out=out)
    assert tq.tq4_1s_linear_int8(x, w, out=buf[m * 64:].view(m, 64)).shape == (m, 64)


@pytest.mark.gpu
def test_linear_right_after_its_weight_is_written():
    # the weight's quantizer, the product and the next weight's quantizer into the same planes, back to back
    x = torch.randn(16, 1024, generator=gen(30)).to(BF16).to(DEV)
    Ws = [torch.randn(2048, 1024, generator=gen(31 + i)).to(DEV) for i in range(3)]
    want = [tq.tq4_1s_linear_int8(x, tq.tq4_1s_int8_quantize(W)) for W in Ws]
    torch.cuda.synchronize()
    w = tq.tq4_1s_int8_quantize(Ws[0])
    lib, st = tq.load_library(), torch.cuda.current_stream().cuda_stream
    for _ in range(10):
        got = []
        for W in Ws:
            c = w.c_struct()
            assert lib.tq4_1s_int8_quantize(W.data_ptr(), 0, ctypes.byref(c), st) == 0
            got.append(tq.tq4_1s_linear_int8(x, w))
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want))


# ------------------------------------------------------------------ the MoE
def ref_moe(x, ids, tw, up, down):
    """The kernel's steps in numpy (fp32 where it uses fp32, exact sums), and the formula in 64 bits on the same codes."""
    (qu, su), (qd, sd) = up, down
    m, topk = ids.shape
    E, H = qu.shape[0], qd.shape[1]
    xq, xs = ref_rows(x)
    y32, y64 = np.zeros((m, H), np.float32), np.zeros((m, H))
    z = np.zeros((m, topk, H), np.float32)
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        u = ref_fp32(xq[t].astype(np.float64) @ qu[e].T.astype(np.float64), xs[t], su[e])
        h = torch.from_numpy(np.maximum(u, 0) * np.maximum(u, 0)).to(BF16)
        hq, hs = ref_rows(h)
        acc = hq.astype(np.float64) @ qd[e].T.astype(np.float64)
        z[t, j] = ref_fp32(acc, hs, sd[e]) * tw[t, j][:, None].astype(np.float32)
        np.add.at(y64, t, acc * hs[:, None].astype(np.float64) * sd[e][None].astype(np.float64) * tw[t, j][:, None])
    for j in range(topk):
        ok = (ids[:, j] >= 0) & (ids[:, j] < E)
        y32[ok] += z[ok, j]
    return y32, y64, np.abs(z).sum(1)


def moe_weights(E, H, I, seed):
    up, qu, su = weight(I, H, seed, E)
    down, qd, sd = weight(H, I, seed + 1, E)
    return up, down, (qu, su), (qd, sd)


def check_moe(x, ids, tw, up, down, ru, rd, **kw):
    y = tq.tq4_1s_moe_int8(x.to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(tw).to(DEV), up, down, **kw)
    y32, y64, size = ref_moe(x, ids, tw, ru, rd)
    assert y.dtype == x.dtype
    assert torch.equal(bits(y), bits(torch.from_numpy(y32).to(x.dtype)))
    # four roundings per term, topk - 1 in the sum (relative to the terms' sizes), one to the output's type
    room = (4 + ids.shape[1]) * 2.0 ** -24 * size + torch.finfo(x.dtype).eps / 2 * 1.001 * np.abs(y64)
    assert np.all(np.abs(y.cpu().double().numpy() - y64) <= room + torch.finfo(x.dtype).tiny)
    return y


def routing(m, E, topk, seed):
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.standard_normal((m, E)), axis=1)[:, :topk].astype(np.int32)
    tw = rng.random((m, topk)).astype(np.float32)
    return ids, tw / tw.sum(1, keepdims=True)


@pytest.mark.gpu
@pytest.mark.parametrize("m,E,topk,H,I,dtype", [
    (1, 8, 2, 256, 128, BF16), (1, 128, 6, 160, 96, BF16), (4, 1, 1, 64, 32, F16), (16, 32, 6, 512, 256, BF16),
    (33, 8, 3, 96, 416, F16), (64, 4, 4, 288, 160, BF16), (200, 8, 2, 256, 224, BF16), (500, 5, 3, 128, 192, F16),
    (1500, 4, 2, 64, 320, BF16), (3, 300, 64, 64, 64, BF16), (40, 1100, 4, 32, 64, BF16), (2, 8, 2, 9248, 64, BF16),
])
def test_moe_matches_plain(m, E, topk, H, I, dtype):
    up, down, ru, rd = moe_weights(E, H, I, m + E)
    ids, tw = routing(m, E, topk, m)
    x = torch.randn(m, H, generator=gen(m)).to(dtype)
    if m > 3:
        x[2] = 0
    check_moe(x, ids, tw, up, down, ru, rd)
    assert tq.tq4_1s_get_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 17, 130, 600])
def test_moe_all_tokens_at_one_expert_and_repeated_ids(m):
    up, down, ru, rd = moe_weights(6, 96, 160, 40)
    x = torch.randn(m, 96, generator=gen(m)).to(BF16)
    ids = np.full((m, 2), 3, np.int32)                     # the same expert twice
    tw = np.random.default_rng(m).standard_normal((m, 2)).astype(np.float32)
    check_moe(x, ids, tw, up, down, ru, rd)
    ids[:, 1] = 5
    check_moe(x, ids, tw, up, down, ru, rd)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [40, 64, 300])
def test_moe_many_experts_and_all_tokens_at_one(m):
    # few rows an expert on the mean, and all of them at one: segments of 16 of its rows
    up, down, ru, rd = moe_weights(700, 64, 96, 41)
    x = torch.randn(m, 64, generator=gen(m)).to(BF16)
    ids = np.full((m, 2), 699, np.int32)
    tw = np.random.default_rng(m).standard_normal((m, 2)).astype(np.float32)
    check_moe(x, ids, tw, up, down, ru, rd)
    ids[::3, 0] = 0
    ids[1::5, 1] = -1
    check_moe(x, ids, tw, up, down, ru, rd)


@pytest.mark.gpu
def test_moe_bad_ids_are_skipped_and_flagged():
    up, down, ru, rd = moe_weights(8, 128, 96, 42)
    ids, tw = routing(30, 8, 3, 43)
    ids[0] = -1                                            # a token with no expert: a row of zeros
    ids[5, 1] = 8
    ids[29, 2] = 2 ** 31 - 1
    x = torch.randn(30, 128, generator=gen(44)).to(BF16)
    y = check_moe(x, ids, tw, up, down, ru, rd)
    assert bool((y[0] == 0).all())
    assert tq.tq4_1s_get_status() == tq.TQ_DEV_BAD_ROUTING
    y = tq.tq4_1s_moe_int8(x.to(DEV), torch.full((30, 3), -1, dtype=torch.int32, device=DEV),
                           torch.from_numpy(tw).to(DEV), up, down)
    assert bool((y == 0).all()) and tq.tq4_1s_get_status() == tq.TQ_DEV_BAD_ROUTING


@pytest.mark.gpu
@pytest.mark.parametrize("m,E", [(2, 32), (30, 200), (60, 8)])
def test_moe_tokens_and_routing_off_alignment(m, E):
    # slices that start at odd places, ids as int64, a token's ids in a wider matrix
    up, down, ru, rd = moe_weights(E, 96, 64, 93)
    ids, tw = routing(m, E, 3, 94)
    x = torch.randn(m, 96, generator=gen(95)).to(BF16)
    buf = torch.zeros(m * 96 + 3, dtype=BF16, device=DEV)
    view = buf[3:].view(m, 96)
    view.copy_(x)
    wide = torch.zeros(m, 5, dtype=torch.int64, device=DEV)
    wide[:, 1:4] = torch.from_numpy(ids).to(DEV)
    tbuf = torch.zeros(m * 3 + 1, device=DEV)
    tbuf[1:] = torch.from_numpy(tw).to(DEV).flatten()
    y = tq.tq4_1s_moe_int8(view, wide[:, 1:4], tbuf[1:].view(m, 3), up, down)
    y32, _, _ = ref_moe(x, ids, tw, ru, rd)
    assert torch.equal(bits(y), bits(torch.from_numpy(y32).to(BF16)))


@pytest.mark.gpu
def test_moe_in_place():
    up, down, ru, rd = moe_weights(8, 128, 96, 96)
    for m in (2, 40):                                      # x is read before y is written
        ids, tw = routing(m, 8, 2, 97)
        x = torch.randn(m, 128, generator=gen(98)).to(BF16)
        want = check_moe(x, ids, tw, up, down, ru, rd)
        xd = x.to(DEV)
        tq.tq4_1s_moe_int8(xd, torch.from_numpy(ids).to(DEV), torch.from_numpy(tw).to(DEV), up, down, out=xd)
        assert torch.equal(bits(xd), bits(want))


@pytest.mark.gpu
def test_first_calls_of_a_process_may_be_captured():
    code = """
import torch, bit_rotated_weight_b200 as tq
d = 'cuda'
w = tq.Int8Weight(torch.ones(1, 4096, 64, dtype=torch.int8, device=d), torch.ones(1, 4096, device=d), 4096, 64, 1)
up = tq.Int8Weight(torch.ones(4, 64, 96, dtype=torch.int8, device=d), torch.full((4, 64), 1e-3, device=d), 64, 96, 4)
dn = tq.Int8Weight(torch.ones(4, 96, 64, dtype=torch.int8, device=d), torch.full((4, 96), 1e-3, device=d), 96, 64, 4)
xs = [torch.ones(m, 64, device=d) for m in (4, 100, 2500)]
xm = [torch.ones(m, 96, device=d, dtype=torch.bfloat16) for m in (1, 40, 600)]
z = [torch.randn(m, 4, device=d) for m in (1, 40, 600)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    ys = [tq.tq4_1s_linear_int8(x, w) for x in xs]
    rs = [tq.tq4_1s_router_scored(t, 2, score='sigmoid') for t in z]
    ms = [tq.tq4_1s_moe_int8(x, i, t, up, dn) for x, (i, t) in zip(xm, rs)]
    q = tq.tq4_1s_int8_dequantize(tq.tq4_1s_int8_quantize(xs[1]))
g.replay()
torch.cuda.synchronize()
assert all(bool((y == 64.0).all()) for y in ys), [float(y.flatten()[0]) for y in ys]
for x, (i, t), y, zz in zip(xm, rs, ms, z):
    assert torch.equal(y, tq.tq4_1s_moe_int8(x, i, t, up, dn))
    assert all(torch.equal(a, b) for a, b in zip((i, t), tq.tq4_1s_router_scored(zz, 2, score='sigmoid')))
assert bool((q == 1.0).all())
print('captured')
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.gpu
def test_moe_nonfinite_tokens_stay_their_own():
    up, down, ru, rd = moe_weights(8, 128, 96, 45)
    ids, tw = routing(50, 8, 3, 46)
    x = torch.randn(50, 128, generator=gen(47)).to(BF16)
    d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    clean = tq.tq4_1s_moe_int8(x.to(DEV), d(ids), d(tw), up, down)
    x[7, 3] = float("nan")
    y = tq.tq4_1s_moe_int8(x.to(DEV), d(ids), d(tw), up, down)
    assert tq.tq4_1s_get_status() == tq.TQ_DEV_NONFINITE
    rest = [i for i in range(50) if i != 7]
    assert bool(y[7].isnan().all()) and torch.equal(bits(y[rest]), bits(clean[rest]))


@pytest.mark.gpu
def test_moe_streams_graphs_and_workspaces():
    up, down, ru, rd = moe_weights(16, 256, 320, 48)
    d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    calls = []
    for m in (1, 16, 300):
        ids, tw = routing(m, 16, 4, 49 + m)
        calls.append((torch.randn(m, 256, generator=gen(m)).to(BF16).to(DEV), d(ids), d(tw)))
    want = [tq.tq4_1s_moe_int8(*c, up, down) for c in calls]
    ws = torch.full((max(tq.tq4_1s_moe_int8_workspace(c[0].shape[0], 4, up, down) for c in calls),), 0xA5,
                    dtype=torch.uint8, device=DEV)
    for _ in range(3):
        for c, y in zip(calls, want):
            assert torch.equal(bits(tq.tq4_1s_moe_int8(*c, up, down, workspace=ws)), bits(y))
    streams = [torch.cuda.Stream() for _ in calls]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        got = []
        for st, c in zip(streams, calls):
            with torch.cuda.stream(st):
                got.append(tq.tq4_1s_moe_int8(*c, up, down))
    torch.cuda.synchronize()
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want))
    xin, iin, win = (t.clone() for t in calls[1])
    g = torch.cuda.CUDAGraph()
    with capture(g):
        y = tq.tq4_1s_moe_int8(xin, iin, win, up, down)
    ids, tw = routing(16, 16, 4, 77)
    iin.copy_(d(ids))
    win.copy_(d(tw))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(y), bits(tq.tq4_1s_moe_int8(xin, iin, win, up, down)))
    assert tq.tq4_1s_get_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 16, 250])
def test_layer_router_experts_and_projection(m):
    """As a decode or prefill step runs them: quantize a checkpoint's weights, project, route by the scored router, run the
    experts in int8, once eagerly and once from a graph."""
    E, H, I, topk = 16, 256, 192, 4
    g = gen(60 + m)
    Wg, Wp = torch.randn(E, H, generator=g), 0.05 * torch.randn(H, 512, generator=g).to(BF16)
    Wu, Wd = 0.05 * torch.randn(E, I, H, generator=g).to(BF16), 0.05 * torch.randn(E, H, I, generator=g).to(BF16)
    bias = 0.1 * torch.randn(E, generator=g)
    a = torch.randn(m, 512, generator=g).to(BF16)
    p, up, down = (tq.tq4_1s_int8_quantize(W.to(DEV)) for W in (Wp, Wu, Wd))
    z = (torch.randn(m, E, generator=g)).to(DEV)
    kw = dict(bias=bias.to(DEV), score="sigmoid", num_groups=4, topk_groups=2, group_score="top2", scale=2.5)

    def layer(a):
        x = tq.tq4_1s_linear_int8(a, p)
        ids, w = tq.tq4_1s_router_scored(z, topk, **kw)
        return x, ids, w, tq.tq4_1s_moe_int8(x, ids, w, up, down)

    ain = a.to(DEV)
    x, ids, w, y = layer(ain)
    graph = torch.cuda.CUDAGraph()
    with capture(graph):
        again = layer(ain)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip((x, ids, w, y), again))
    qp, sp = ref_rows(Wp)
    aq, sa = ref_rows(a)
    xr = torch.from_numpy(ref_fp32(aq.astype(np.float64) @ qp.T.astype(np.float64), sa, sp)).to(BF16)
    assert torch.equal(bits(x), bits(xr))
    y32, _, _ = ref_moe(xr, ids.cpu().numpy(), w.cpu().numpy(), ref_rows(Wu), ref_rows(Wd))
    assert torch.equal(bits(y), bits(torch.from_numpy(y32).to(BF16)))
    # the same routing drives the TQ4_1S experts
    pu, pd = tq.tq4_1s_quantize(Wu.to(DEV), seed=1), tq.tq4_1s_quantize(Wd.to(DEV), seed=2)
    y4 = tq.tq4_1s_moe(x, ids, w, pu, pd).float()
    yf = y.float()
    # both formats stand for the same layer: 4-bit codes are off by about 10 %, the int8 ones by about 1 %
    assert float((y4 - yf).norm() / yf.norm()) < 0.5
    assert tq.tq4_1s_get_status() == 0


# ------------------------------------------------------------------ refusals
def _w(n=64, k=64, e=1, q=16, scale=16, reserved=0):
    return tq._Int8Weight(n, k, e, reserved, q, scale)


def test_refusals():
    lib = tq.load_library()
    good, r = 4096, ctypes.byref
    for bad, code in ((dict(n=0), 1), (dict(k=0), 1), (dict(k=48), 1), (dict(k=131104), 1), (dict(e=0), 1),
                      (dict(e=4097), 1), (dict(q=0), 1), (dict(scale=0), 1), (dict(q=24), 2), (dict(scale=8), 2),
                      (dict(reserved=1), 1)):
        assert lib.tq4_1s_int8_quantize(good, 0, r(_w(**bad)), None) == code, bad
        assert lib.tq4_1s_int8_dequantize(r(_w(**bad)), good, None) == code, bad
        assert lib.tq4_1s_linear_int8(good, 0, 4, 1 << 20, r(_w(**bad)), good, good, 1 << 30, None) == code, bad
    assert lib.tq4_1s_int8_quantize(good, 3, r(_w()), None) == 1
    assert lib.tq4_1s_int8_quantize(None, 0, r(_w()), None) == 1
    assert lib.tq4_1s_int8_quantize(4104, 0, r(_w()), None) == 2
    assert lib.tq4_1s_int8_dequantize(r(_w()), None, None) == 1
    assert lib.tq4_1s_int8_dequantize(r(_w()), 4104, None) == 2
    lin = lambda x=good, dt=1, m=4, ld=64, w=_w(), y=good: lib.tq4_1s_linear_int8(x, dt, m, ld, r(w), y, good, 1 << 30, None)  # noqa: E731
    assert lin(m=0) == 0 and lin(x=None) == 1 and lin(y=None) == 1 and lin(m=-1) == 1 and lin(m=(1 << 24) + 1) == 1
    assert lin(ld=63) == 1 and lin(dt=3) == 1 and lin(w=_w(e=2)) == 1
    assert lin(x=4097) == 2 and lin(x=4098, dt=0) == 2 and lin(y=4104) == 2
    assert lib.tq4_1s_linear_int8_workspace(17, r(_w(n=4096, k=4096))) >= 17 * 4096
    assert lib.tq4_1s_linear_int8_workspace(16, r(_w(n=4096, k=4096))) == 0        # few tokens: none needed
    assert lib.tq4_1s_linear_int8_workspace(16, r(_w(n=4096, k=16384))) > 0        # rows too long to stay on chip
    for m, w in ((0, _w()), (-1, _w()), (16, _w(k=48)), (16, _w(e=2))):
        assert lib.tq4_1s_linear_int8_workspace(m, r(w)) == 0
    up, dn = _w(n=96, k=64, e=4), _w(n=64, k=96, e=4)
    moe = lambda x=good, dt=1, m=4, ids=good, tw=good, topk=2, u=up, d=dn, y=good: lib.tq4_1s_moe_int8(  # noqa: E731
        x, dt, m, ids, tw, topk, r(u), r(d), y, good, 1 << 30, None)
    assert moe(m=0) == 0
    for bad in (dict(dt=0), dict(dt=3), dict(m=-1), dict(topk=0), dict(topk=65), dict(u=_w(n=96, k=64, e=3)),
                dict(u=_w(n=128, k=64, e=4)), dict(d=_w(n=32, k=96, e=4)), dict(x=None), dict(ids=None), dict(tw=None),
                dict(y=None), dict(m=1 << 26, topk=2)):
        assert moe(**bad) == 1, bad
    assert moe(x=4097) == 2 and moe(ids=4098) == 2 and moe(tw=4097) == 2 and moe(y=4100) == 2
    assert lib.tq4_1s_moe_int8_workspace(4, 2, r(up), r(dn)) > 0
    assert lib.tq4_1s_moe_int8_workspace(0, 2, r(up), r(dn)) == 0
    assert lib.tq4_1s_moe_int8_workspace(4, 2, r(up), r(up)) == 0
    if not torch.cuda.is_available():
        assert lin() == 3 and moe() == 3
        assert lib.tq4_1s_int8_quantize(good, 0, r(_w()), None) == 3
        assert lib.tq4_1s_int8_dequantize(r(_w()), good, None) == 3


def test_refusals_of_the_binding_on_cpu_tensors():
    w = tq.Int8Weight(torch.zeros(1, 4, 32, dtype=torch.int8), torch.zeros(1, 4), 4, 32, 1)
    for call in (lambda: tq.tq4_1s_int8_quantize(torch.zeros(4, 32)), lambda: tq.tq4_1s_int8_dequantize(w),
                 lambda: tq.tq4_1s_linear_int8(torch.zeros(2, 32), w),
                 lambda: tq.tq4_1s_moe_int8(torch.zeros(2, 32, dtype=BF16), torch.zeros(2, 1), torch.zeros(2, 1), w, w)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_refusals_of_the_binding():
    w, _, _ = weight(64, 96, 70)
    x = torch.zeros(4, 96, dtype=BF16, device=DEV)
    up, down, _, _ = moe_weights(4, 64, 96, 71)
    xm = torch.zeros(3, 64, dtype=BF16, device=DEV)
    ids, tw = torch.zeros(3, 2, dtype=torch.int32, device=DEV), torch.zeros(3, 2, device=DEV)
    bad_q = tq.Int8Weight(w.q[:, :63], w.wscale, 64, 96, 1)
    bad_s = tq.Int8Weight(w.q, w.wscale.double(), 64, 96, 1)
    bad_t = tq.Int8Weight(w.q.float(), w.wscale, 64, 96, 1)
    for call in (
            lambda: tq.tq4_1s_linear_int8(x[:, :64], w), lambda: tq.tq4_1s_linear_int8(x[0], w),
            lambda: tq.tq4_1s_linear_int8(x.double(), w), lambda: tq.tq4_1s_linear_int8(x, bad_q),
            lambda: tq.tq4_1s_linear_int8(x, bad_s), lambda: tq.tq4_1s_linear_int8(x, bad_t),
            lambda: tq.tq4_1s_linear_int8(x, w, out=torch.empty(4, 64, device=DEV)),
            lambda: tq.tq4_1s_linear_int8(x, w, out=torch.empty(64, 4, dtype=BF16, device=DEV).t()),
            lambda: tq.tq4_1s_linear_int8(x, w, workspace=torch.empty(1 << 20, dtype=torch.uint8)),
            lambda: tq.tq4_1s_moe_int8(xm.float(), ids, tw, up, down), lambda: tq.tq4_1s_moe_int8(xm, ids[:2], tw, up, down),
            lambda: tq.tq4_1s_moe_int8(xm, ids.cpu(), tw, up, down), lambda: tq.tq4_1s_moe_int8(xm[:, :32], ids, tw, up, down),
            lambda: tq.tq4_1s_int8_quantize(x.double()), lambda: tq.tq4_1s_int8_quantize(x[0])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(tq.TQ4Error):
        tq.tq4_1s_moe_int8(xm, ids, tw, up, up)
    with pytest.raises(tq.TQ4Error):
        tq.tq4_1s_int8_quantize(torch.zeros(4, 48, device=DEV))
    assert tq.tq4_1s_linear_int8(x[:0], w).shape == (0, 64)
    assert tq.tq4_1s_moe_int8(xm[:0], ids[:0], tw[:0], up, down).shape == (0, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("E,topk,H,I,m,calls", [
    (128, 6, 288, 1184, 16, 40),     # several row tiles of two segments a block, calls back to back
    (12, 4, 2688, 160, 24, 20),      # rows of 21 k steps, up to nine tokens a segment
    (200, 3, 96, 96, 350, 20),       # more segments than blocks: four or five of them a block
])
def test_moe_few_rows_an_expert_back_to_back(E, topk, H, I, m, calls):
    up, down, ru, rd = moe_weights(E, H, I, 80)
    ids, tw = routing(m, E, topk, 81)
    x = torch.randn(m, H, generator=gen(82)).to(BF16)
    y = check_moe(x, ids, tw, up, down, ru, rd)
    args = x.to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(tw).to(DEV), up, down
    ys = [tq.tq4_1s_moe_int8(*args) for _ in range(calls)]
    assert all(torch.equal(bits(a), bits(y)) for a in ys)
    assert tq.tq4_1s_get_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(16, 40000, 2688), (1, 20000, 4096), (7, 2048, 8192), (16, 256, 9216),
                                   (16, 19200, 9216), (9, 19000, 32)])
def test_linear_few_tokens_back_to_back(m, n, k):
    w, q, s = weight(n, k, 83) if n * k < 1 << 25 else (None, None, None)
    if w is None:                                       # too large for numpy: three row blocks are compared
        q = torch.randint(-127, 128, (1, n, k), generator=gen(84), dtype=torch.int8)
        s = torch.rand(1, n, generator=gen(85)) + 0.5
        w = tq.Int8Weight(q.to(DEV), s.to(DEV), n, k, 1)
        rows = torch.cat([torch.arange(0, 140), torch.arange(n // 2, n // 2 + 140), torch.arange(n - 140, n)])
        q, s = q[:, rows].numpy().astype(np.int64), s[:, rows].numpy()
    else:
        rows = torch.arange(n)
    x = torch.randn(m, k, generator=gen(86)).to(BF16)
    xd = x.to(DEV)
    ys = [tq.tq4_1s_linear_int8(xd, w) for _ in range(30)]
    xq, xs = ref_rows(x)
    acc = xq.astype(np.float64) @ q[0].T.astype(np.float64)
    want = torch.from_numpy(ref_fp32(acc, xs, s[0])).to(BF16)
    assert all(torch.equal(bits(y[:, rows.to(DEV)]), bits(want)) for y in ys)
    assert tq.tq4_1s_get_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("m", [4, 16, 40, 300, 2400])
def test_calls_read_what_the_call_before_wrote(m):
    # each kernel may be set up while the one before it still runs: chains of calls without a pause, against calls that
    # wait for the GPU, with fresh inputs in the same buffers
    E = 128
    w1 = tq.tq4_1s_int8_quantize(torch.randn(512, 256, generator=gen(m)).to(DEV))
    w2 = tq.tq4_1s_int8_quantize(torch.randn(E, 512, generator=gen(m + 1)).to(DEV))
    up = tq.tq4_1s_int8_quantize(torch.randn(E, 64, 256, generator=gen(m + 2)).to(DEV))
    dn = tq.tq4_1s_int8_quantize(torch.randn(E, 256, 64, generator=gen(m + 3)).to(DEV))
    x = torch.empty(m, 256, dtype=BF16, device=DEV)
    bias = torch.randn(E, generator=gen(m + 4)).to(DEV)

    def chain(wait):
        pause = torch.cuda.synchronize if wait else (lambda: None)
        h = tq.tq4_1s_linear_int8(x, w1)
        pause()
        z = tq.tq4_1s_linear_int8(h.float(), w2)
        pause()
        z2 = tq.tq4_1s_linear_int8(tq.tq4_1s_linear_int8(x, w1), w2)
        pause()
        ids, tw = tq.tq4_1s_router_scored(z2, 4, bias=bias, score="sigmoid", num_groups=8, topk_groups=3,
                                          group_score="top2")
        pause()
        y = tq.tq4_1s_moe_int8(x, ids, tw, up, dn)
        pause()
        q = tq.tq4_1s_int8_quantize(y)
        pause()
        back = tq.tq4_1s_int8_dequantize(q)
        pause()
        last = tq.tq4_1s_linear_int8(y, tq.tq4_1s_int8_quantize(back.to(BF16)[0]))
        pause()
        return z, z2, ids, tw, y, q.q, q.wscale, back, last

    g = gen(m + 5)
    for _ in range(6):
        fresh = torch.randn(m, 256, generator=g).to(BF16).to(DEV)
        torch.cuda.synchronize()
        x.copy_(fresh)
        got = chain(False)
        torch.cuda.synchronize()
        want = chain(True)
        for a, b in zip(got, want):
            assert torch.equal(bits(a) if a.is_floating_point() else a, bits(b) if b.is_floating_point() else b)


@pytest.mark.gpu
@pytest.mark.parametrize("m,E,topk", [(100, 8, 3), (256, 8, 8), (257, 8, 8), (900, 1100, 2), (33, 40, 64)])
def test_moe_bad_ids_of_more_tokens(m, E, topk):
    # slots that are counted by the rows themselves (up to 2048), by a kernel of their own, of more experts than threads
    up, down, ru, rd = moe_weights(E, 64, 96, 46)
    ids, tw = routing(m, E, topk, 47) if topk <= E else (np.random.default_rng(5).integers(0, E, (m, topk)).astype(np.int32),
                                                         np.random.default_rng(6).random((m, topk)).astype(np.float32))
    ids[0] = -1
    ids[1] = ids[2]                                        # two tokens alike
    ids[5, 1] = E
    ids[m - 1, topk - 1] = 2 ** 31 - 1
    ids[7, 0] = -(2 ** 31)
    x = torch.randn(m, 64, generator=gen(48)).to(BF16)
    y = check_moe(x, ids, tw, up, down, ru, rd)
    assert bool((y[0] == 0).all()) and tq.tq4_1s_get_status() == tq.TQ_DEV_BAD_ROUTING
    tq.tq4_1s_moe_int8(x.to(DEV), torch.full((m, topk), -1, dtype=torch.int32, device=DEV), torch.from_numpy(tw).to(DEV),
                       up, down, out=y)
    assert bool((y == 0).all())
