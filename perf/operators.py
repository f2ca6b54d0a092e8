"""Cases of the scored expert router and of the 8-bit integer layers, with their plain forms.

Four operators: the router that scores experts by softmax or sigmoid, with a balance bias, groups and renormalised
weights; the row quantizer of the int8 format (and its way back); the dense layer with int8 weights and activations; and
the mixture of experts with int8 experts.  `listed()` and `draw()` give the sizes, `run()` one pass.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one token of a decode loop: 128 experts, top-6, sigmoid scores with a balance bias; latency alone
        dict(name="router_1x128", op="router", m=1, e=128, topk=6, score="sigmoid", bias=True, groups=1, keep=1,
             group_score="top2", renorm=True, scale=1.0, dtype="f32"),
        # 32 blocks of 16 tokens of a denoise step, softmax scores, half of 8 groups kept by their best expert
        dict(name="router_512x128_groups", op="router", m=512, e=128, topk=6, score="softmax", bias=False, groups=8,
             keep=4, group_score="max", renorm=False, scale=1.0, dtype="f32"),
        # a long prompt batch: bf16 logits of 256 experts, groups by the sum of their two best, bias, scaled weights
        dict(name="router_65536x256_bias", op="router", m=65536, e=256, topk=8, score="sigmoid", bias=True, groups=8,
             keep=4, group_score="top2", renorm=True, scale=2.5, dtype="bf16"),
        # the decode layer's weight from fp32, once per load
        dict(name="quantize_4096x4096_f32", op="quantize", n=4096, k=4096, dtype="f32"),
        # the prefill layer's weight from a bf16 checkpoint
        dict(name="quantize_14336x4096_bf16", op="quantize", n=14336, k=4096, dtype="bf16"),
        # a single token through a dense projection of the denoise sweep
        dict(name="linear_1x4096x2688_f16", op="linear", m=1, n=4096, k=2688, dtype="f16"),
        # the decode block: 16 tokens through a 4096 x 4096 layer
        dict(name="linear_16x4096x4096_bf16", op="linear", m=16, n=4096, k=4096, dtype="bf16"),
        # a ragged batch, an odd number of outputs, fp32 in and out
        dict(name="linear_333x1857x2688_f32", op="linear", m=333, n=1857, k=2688, dtype="f32"),
        # the prefill layer
        dict(name="linear_8192x14336x4096_bf16", op="linear", m=8192, n=14336, k=4096, dtype="bf16"),
        # one token through 6 of 128 experts: the weights of those six are the work
        dict(name="moe_1x128", op="moe", m=1, e=128, topk=6, h=2688, i=1856, dtype="bf16"),
        # a block of 16 tokens, top-6: two thirds of the experts are read, each for a row or two
        dict(name="moe_16x128", op="moe", m=16, e=128, topk=6, h=2688, i=1856, dtype="bf16"),
        # a prompt batch: every expert has about 200 rows
        dict(name="moe_4096x128", op="moe", m=4096, e=128, topk=6, h=2688, i=1856, dtype="bf16"),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["router", "quantize", "linear", "linear", "moe"])
    if op == "router":
        groups = rng.choice([1, 1, 2, 4, 8])
        e = groups * _log(rng, 8, 1024 // groups // 2)
        keep = rng.randint(1, groups)
        return dict(op=op, m=_log(rng, 1, 65536 * 256 // max(e, 256)), e=e, topk=rng.randint(1, min(12, keep * (e // groups))),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, groups=groups, keep=keep,
                    group_score=rng.choice(["max", "top2"]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5, 0.5]), dtype=rng.choice(["f32", "bf16"]))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quantize":
        return dict(op=op, n=_log(rng, 64, 14336), k=_log(rng, 64, 8192, 32), dtype=dtype)
    if op == "linear":
        return dict(op=op, m=_log(rng, 1, 4096), n=_log(rng, 64, 14336), k=_log(rng, 64, 8192, 32), dtype=dtype)
    e = _log(rng, 4, 128)
    return dict(op=op, m=_log(rng, 1, 2048), e=e, topk=rng.randint(1, min(8, e)), h=_log(rng, 128, 2688, 32),
                i=_log(rng, 64, 2048, 32), dtype=rng.choice(["bf16", "bf16", "f16"]))


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(m, k, g, dtype):
    """Gaussian tokens of different sizes with a few strong channels; of more than four tokens the last is padding (zeros)."""
    x = torch.randn(m, k, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(m, 1, generator=g, device="cuda"))
    x *= 1.0 + 9.0 * (torch.rand(k, generator=g, device="cuda") < 0.01)
    if m > 4:
        x[-1] = 0
    return x.to(dtype)


def _int8_weight(shape, g):
    """Int8 codes and row scales of a Gaussian weight."""
    w = torch.randn(shape, generator=g, device="cuda").mul_(0.02)
    scale = w.abs().amax(-1) / 127.0
    return w.div_(scale.unsqueeze(-1)).round_().to(torch.int8), scale


def _inputs(case, seed):
    g, s = _gen(seed), {"case": case}
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "router":
        s["logits"] = (1.5 * torch.randn(case["m"], case["e"], generator=g, device="cuda")).to(dtype)
        s["bias"] = 0.1 * torch.randn(case["e"], generator=g, device="cuda") if case["bias"] else None
    elif case["op"] == "quantize":
        s["w"] = torch.randn(case["n"], case["k"], generator=g, device="cuda").mul_(0.02).to(dtype)
    elif case["op"] == "linear":
        s["x"] = _activations(case["m"], case["k"], g, dtype)
        s["q"], s["scale"] = _int8_weight((case["n"], case["k"]), g)
    else:
        m, e, topk, h, i = case["m"], case["e"], case["topk"], case["h"], case["i"]
        s["x"] = _activations(m, h, g, dtype)
        s["qu"], s["su"] = _int8_weight((e, i, h), g)
        s["qd"], s["sd"] = _int8_weight((e, h, i), g)
        z, ids = torch.sort(torch.randn(m, e, generator=g, device="cuda"), dim=1, descending=True)
        s["ids"] = ids[:, :topk].to(torch.int32).contiguous()
        s["tw"] = torch.softmax(z[:, :topk], dim=1)
        s["most"] = int(torch.bincount(s["ids"].flatten(), minlength=e).max())  # rows of the fullest expert
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import bit_rotated_weight_b200 as tq
        s["tq"] = tq
        if case["op"] == "linear":
            s["weight"] = tq.Int8Weight(s["q"].unsqueeze(0), s["scale"].unsqueeze(0), case["n"], case["k"], 1)
        elif case["op"] == "moe":
            s["up"] = tq.Int8Weight(s["qu"], s["su"], case["i"], case["h"], case["e"])
            s["down"] = tq.Int8Weight(s["qd"], s["sd"], case["h"], case["i"], case["e"])
    return s


# ---------------------------------------------------------------- plain forms
def _quantize_rows(x):
    """Codes (as fp32 whole numbers) and row scales: q = round(127 x / max|x|), ties to even, taken in 64 bits because
    half the largest value of a row lies on a border."""
    top = x.abs().amax(-1, keepdim=True)
    q = torch.round(x.double() * 127.0 / torch.where(top > 0, top, 1.0).double())
    return q.float(), top.float() / 127.0


def _router(s):
    c, z, bias = s["case"], s["logits"].double(), s["bias"]
    m, e = z.shape
    score = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.exp(z - z.amax(1, keepdim=True))
    if c["score"] == "softmax":
        score = score / score.sum(1, keepdim=True)
    choice = score + bias.double() if bias is not None else score
    if c["groups"] > 1:
        per = torch.sort(choice.view(m, c["groups"], -1), dim=2, descending=True).values
        rank = per[..., :2].sum(2) if c["group_score"] == "top2" else per[..., 0]
        kept = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        open_ = torch.zeros(m, c["groups"], dtype=torch.bool, device=z.device).scatter_(1, kept, True)
        choice = torch.where(open_.repeat_interleave(e // c["groups"], 1), choice, -math.inf)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :c["topk"]]
    w = torch.gather(score, 1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.to(torch.int32), (w * c["scale"]).float()


def _linear(s):
    q, sx = _quantize_rows(s["x"])
    return ((q @ s["q"].float().t()) * sx * s["scale"]).to(s["x"].dtype)


def _moe(s):
    ids, (m, topk), e = s["ids"].long().flatten(), s["ids"].shape, s["case"]["e"]
    q, sx = _quantize_rows(s["x"])
    if ids.numel() < e:  # few pairs: the weights of each pair's expert
        token = torch.arange(ids.numel(), device=ids.device) // topk
        xq, xs = q[token].unsqueeze(1), sx[token].unsqueeze(1)
        qu, su, qd, sd = s["qu"][ids], s["su"][ids], s["qd"][ids], s["sd"][ids]
        place = None
    else:  # every expert once, over its rows
        order = torch.argsort(ids, stable=True)
        count = torch.bincount(ids, minlength=e)
        nth = torch.arange(ids.numel(), device=ids.device) - (count.cumsum(0) - count)[ids[order]]
        place = torch.empty_like(order)
        place[order] = ids[order] * s["most"] + nth
        xq = q.new_zeros(e * s["most"], q.shape[1]).index_copy_(0, place, q.repeat_interleave(topk, 0)).view(e, s["most"], -1)
        xs = q.new_zeros(e * s["most"], 1).index_copy_(0, place, sx.repeat_interleave(topk, 0)).view(e, s["most"], 1)
        qu, su, qd, sd = s["qu"], s["su"], s["qd"], s["sd"]
    u = torch.bmm(xq, qu.float().transpose(1, 2)) * xs * su.unsqueeze(1)
    hq, hs = _quantize_rows(torch.relu(u).square().to(torch.bfloat16))
    z = (torch.bmm(hq, qd.float().transpose(1, 2)) * hs * sd.unsqueeze(1)).flatten(0, 1)
    z = z if place is None else z[place]
    return (z.view(m, topk, -1) * s["tw"].unsqueeze(2)).sum(1).to(s["x"].dtype)


def run(state):
    c = state["case"]
    if own:
        tq = state["tq"]
        if c["op"] == "router":
            return tq.tq4_1s_router_scored(state["logits"], c["topk"], bias=state["bias"], score=c["score"],
                                           num_groups=c["groups"], topk_groups=c["keep"], group_score=c["group_score"],
                                           renormalize=c["renorm"], scale=c["scale"])
        if c["op"] == "quantize":
            w = tq.tq4_1s_int8_quantize(state["w"])
            return tq.tq4_1s_int8_dequantize(w)[0], w.wscale[0]
        if c["op"] == "linear":
            return tq.tq4_1s_linear_int8(state["x"], state["weight"])
        return tq.tq4_1s_moe_int8(state["x"], state["ids"], state["tw"], state["up"], state["down"])
    if c["op"] == "router":
        return _router(state)
    if c["op"] == "quantize":
        q, scale = _quantize_rows(state["w"])
        return q * scale, scale[:, 0]
    return _linear(state) if c["op"] == "linear" else _moe(state)


def work(case):
    """Bytes read and written once, and operations (a multiply-add is two)."""
    b = BYTES[case["dtype"]]
    if case["op"] == "router":
        m, e, k = case["m"], case["e"], case["topk"]
        return {"bytes": m * e * b + m * k * 8 + (4 * e if case["bias"] else 0), "flops": 4 * m * e}
    if case["op"] == "quantize":  # to codes, and from the codes to the fp32 values
        n, k = case["n"], case["k"]
        return {"bytes": n * k * (b + 1) + 4 * n + n * k * 5 + 4 * n, "flops": 4 * n * k}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k * b + n * k + 4 * n + m * n * b, "flops": 2 * m * n * k}
    m, e, k, h, i = case["m"], case["e"], case["topk"], case["h"], case["i"]
    read = e * (1 - (1 - k / e) ** m)  # experts that at least one token names
    return {"bytes": read * (2 * h * i + 4 * (h + i)) + 2 * m * h * b + m * k * 8, "flops": 4 * m * k * h * i}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "router":
        return _exact_router(case, s["logits"].double().cpu(), None if s["bias"] is None else s["bias"].double().cpu())
    if case["op"] == "quantize":
        w = s["w"].double()
        a = w.abs().max(dim=1).values
        return torch.round(127.0 * w / a[:, None]) * (a / 127.0)[:, None], a / 127.0
    if case["op"] == "linear":
        return _exact_product(s["x"].double(), s["q"], s["scale"])
    y = torch.zeros(case["m"], case["h"], dtype=torch.float64, device="cuda")
    x = s["x"].double()
    for e in torch.unique(s["ids"]).tolist():
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        u = _exact_product(x[t], s["qu"][e], s["su"][e])
        h = torch.clamp(u, min=0).pow(2).to(torch.bfloat16).double()
        z = _exact_product(h, s["qd"][e], s["sd"][e])
        y.index_add_(0, t, z * s["tw"][t, j].double()[:, None])
    return y


def _exact_product(x, q, scale):
    """x quantized by rows, times the weight that (q, scale) stand for."""
    a = x.abs().max(dim=1).values
    unit = torch.where(a > 0, a, torch.ones_like(a))
    near = torch.round(127.0 * x / unit[:, None])  # (127 x is exact, so halves of the largest value stay on their border)
    return torch.matmul(near, q.double().T) * (a / 127.0)[:, None] * scale.double()[None, :]


def _exact_router(case, z, bias):
    m, e = z.shape
    if case["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-z))
    else:
        score = torch.softmax(z, dim=1)
    choice = score if bias is None else score + bias
    size = e // case["groups"]
    best = choice.reshape(m, case["groups"], size)
    first = best.max(dim=2).values
    if case["group_score"] == "top2":
        first = first + torch.topk(best, 2, dim=2).values[:, :, 1]
    shut = torch.argsort(first, dim=1, descending=True, stable=True)[:, case["keep"]:]
    for column in range(shut.shape[1]):
        group = torch.arange(e)[None, :] // size
        choice = choice.masked_fill(group == shut[:, column:column + 1], -math.inf)
    ids = torch.argsort(choice, dim=1, descending=True, stable=True)[:, :case["topk"]]
    w = score.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), w * case["scale"]
