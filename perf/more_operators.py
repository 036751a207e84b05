"""Operators around 8-bit expert products, as measured cases.

Four groups of operators that one step through a mixture of experts uses in turn: routing by scores
(softmax or sigmoid, a bias for balance, groups of experts, renormalised weights) and its gradient;
8-bit floating point (e4m3) with a scale for each block of 128, of tokens along their rows and of
weights in squares; the grouped product of such rows with such expert weights; and the gated
activation between two products, with its gradient, to values or straight to 8 bits.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits; scores that
decide a choice in 64), or, where ``own`` is true, through the package's entry points.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ELEMENT = {"f16": 2, "bf16": 2, "f32": 4}
BLOCK = 128
E4M3_MAX = 448.0
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases
def listed():
    def route(name, T, E, k, dtype, score, bias=False, groups=1, kept=1, best=1, normalize=True, scale=1.0,
              padded=0, backward=False):
        return dict(name=name, op="route_backward" if backward else "route", T=T, E=E, k=k, dtype=dtype, score=score,
                    bias=bias, groups=groups, kept=kept, best=best, normalize=normalize, scale=scale, padded=padded)

    def product(name, T, k, E, K, N, dtype, gather, skew=0.0, scales="two"):
        return dict(name=name, op="matmul", T=T, k=k, E=E, K=K, N=N, dtype=dtype, gather=gather, skew=skew,
                    scales=scales)

    def gate(name, rows, I, dtype, activation, halves=False, to8=False, backward=False):
        return dict(name=name, op="activate_backward" if backward else "activate", rows=rows, I=I, dtype=dtype,
                    activation=activation, halves=halves, to8=to8)

    return [
        # six decode tokens over 512 experts, top-10: the smallest choice, all latency
        route("route_decode", 6, 512, 10, "f32", "softmax"),
        # a large prefill's tokens: sigmoid scores, a bias for balance, four of eight groups
        route("route_groups", 4096, 256, 8, "f32", "sigmoid", bias=True, groups=8, kept=4, best=2, scale=2.0),
        # a training step's gradient to the router's logits: weights that are not renormalised reach every expert
        route("route_grad", 8191, 60, 4, "bf16", "softmax", normalize=False, padded=5, backward=True),
        # a prefill's activations to 8 bits and the values they stand for
        dict(name="fp8_tokens", op="quantize", E=1, rows=4096, K=4096, dtype="bf16", form="rows"),
        # weights of eight experts in squares, transposed for the gradient's product
        dict(name="fp8_weights_t", op="quantize", E=8, rows=2048, K=2048, dtype="f16", form="transposed"),
        # one decode token through its two experts: a plain read of two experts' weights
        product("fp8_matmul_token", 1, 2, 8, 2048, 4096, "f16", True),
        # six decode tokens over 512 experts, top-10: about 57 experts of one or two rows each
        product("fp8_matmul_many_experts", 6, 10, 512, 2048, 1536, "bf16", True),
        # a 512-token prefill of the 8-expert layer, weights with the scales of a checkpoint
        product("fp8_matmul_prefill", 512, 2, 8, 2048, 4096, "f16", True, scales="any"),
        # the large skewed prefill's first projection
        product("fp8_matmul_skewed", 4096, 2, 8, 4096, 28672, "bf16", True, skew=2.0),
        # eight decode tokens' first projection, activated
        gate("activate_decode", 16, 2048, "f16", "geglu"),
        # the large prefill's first projection, activated straight to the 8 bits of the second
        gate("activate_to_fp8", 8192, 14336, "bf16", "swiglu", to8=True),
        # the gradient of that step, to the first projection's outputs
        gate("activate_grad", 8192, 14336, "bf16", "swiglu", backward=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "quantize", "quantize", "matmul", "matmul", "matmul",
                     "activate", "activate", "activate_backward"])
    dtype = rng.choice(["f16", "bf16", "bf16", "f32"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = _log(rng, 2 * groups, 1024) // groups * groups
        kept = rng.randint(1, groups)
        k = rng.randint(1, min(16, E // groups * kept))
        T = min(_log(rng, 1, 65536), (1 << 24) // E)
        # one expert's renormalised weight is 1 whatever its logit: its gradient says nothing
        normalize = rng.random() < 0.6 and (op == "route" or k > 1)
        return dict(op=op, T=T, E=E, k=k, dtype=rng.choice(["f32", dtype]), score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, kept=kept, best=rng.choice([1, 2]),
                    normalize=normalize, scale=rng.choice([1.0, 1.5]), padded=rng.choice([0, 0, 20]))
    if op == "quantize":
        form = rng.choice(["rows", "rows", "squares", "transposed"])
        E = 1 if form == "rows" else _log(rng, 1, 8)
        rows, K = _log(rng, 1, 16384), _log(rng, 16, 8192)
        if form == "transposed":
            rows = max(16, rows // 16 * 16)
        else:
            K = K // 16 * 16
        while E * rows * K > 1 << 25:
            rows = rows // 2 if form != "transposed" else max(16, rows // 32 * 16)
        return dict(op=op, E=E, rows=rows, K=K, dtype=dtype, form=form)
    if op in ("activate", "activate_backward"):
        rows, I = _log(rng, 1, 16384), _log(rng, 16, 16384)
        to8 = dtype != "f32" and op == "activate" and rng.random() < 0.5
        if to8:
            I = I // 16 * 16
        while rows * I > 1 << 26:
            rows //= 2
        return dict(op=op, rows=rows, I=I, dtype=dtype, activation=rng.choice(["swiglu", "swiglu", "geglu"]),
                    halves=rng.random() < 0.4, to8=to8)
    E = _log(rng, 1, 512)
    k = rng.randint(1, min(E, 10))
    K = _log(rng, 32, 8192) // 16 * 16
    N = _log(rng, 16, 16384)
    if rng.random() < 0.7:
        N = (N + 15) // 16 * 16
    while E * N * K > 1 << 30:
        E = max(1, E // 2)
    k = min(k, E)
    T = _log(rng, 1, 8192)
    while T > 1 and T * k * N * K > 1 << 39:
        T //= 2
    # 16-bit outputs: sums of 8-bit products on matrix units are not float32's
    return dict(op=op, T=T, k=k, E=E, K=K, N=N, dtype=rng.choice(["f16", "bf16"]), gather=rng.random() < 0.7,
                skew=rng.choice([0.0, 0.0, 2.0]), scales=rng.choice(["two", "any"]))


# ---------------------------------------------------------------- plain pieces
def _scores(logits, score):
    return torch.sigmoid(logits) if score == "sigmoid" else torch.softmax(logits, 1)


def _choose(case, logits, bias):
    """Ids [T, k] (int32, -1 where no expert is left) by the scores in 64 bits; ties to the lowest index."""
    T, E = logits.shape
    # a row without any expert has scores of NaN, which the mask below replaces
    choice = _scores(logits.double(), case["score"])
    if bias is not None:
        choice = choice + bias.double()
    choice = torch.where(torch.isneginf(logits), -math.inf, choice)
    G, kept = case["groups"], case["kept"]
    if kept < G:
        top = choice.view(T, G, E // G).topk(min(case["best"], E // G), 2).values
        rank = torch.where(torch.isneginf(top[..., :1]), -math.inf, torch.where(torch.isneginf(top), 0.0, top).sum(2, keepdim=True))
        order = torch.sort(rank[..., 0], dim=1, descending=True, stable=True).indices[:, :kept]
        lost = torch.ones(T, G, dtype=torch.bool, device=logits.device).scatter_(1, order, False)
        choice = torch.where(lost.repeat_interleave(E // G, 1), -math.inf, choice)
    top, ids = torch.sort(choice, dim=1, descending=True, stable=True)
    top, ids = top[:, :case["k"]], ids[:, :case["k"]]
    return torch.where(torch.isneginf(top), -1, ids).int().contiguous()


def _weights(case, logits, ids):
    """Scores of the chosen experts, over their sum where they are renormalised, times the scale."""
    s = _scores(logits.float(), case["score"]).gather(1, ids.long().clamp(min=0))
    s = torch.where(ids >= 0, s, 0.0)
    if case["normalize"]:
        total = s.sum(1, keepdim=True)
        s = s / torch.where(total > 0, total, 1.0)
    return s * case["scale"]


def _route_grad(case, logits, ids, grad):
    """The gradient of the weights with respect to the logits."""
    s = _scores(logits.float(), case["score"])
    at = ids.long().clamp(min=0)
    kept = ids >= 0
    chosen = torch.where(kept, s.gather(1, at), 0.0)
    grad = torch.where(kept, grad * case["scale"], 0.0)
    if case["normalize"]:
        total = chosen.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        grad = (grad - (grad * chosen).sum(1, keepdim=True) / total) / total
        grad = torch.where(kept, grad, 0.0)
    full = torch.zeros_like(s).scatter_add_(1, at, grad)  # experts are chosen once; lost slots add 0
    if case["score"] == "sigmoid":
        out = full * s * (1.0 - s)
    else:
        out = s * (full - (grad * chosen).sum(1, keepdim=True))
    # a row without any expert has no scores
    return torch.where(torch.isneginf(logits), 0.0, out).to(logits.dtype)


def _exponent(top):
    """The least e with top <= 448 * 2^e, at least -126."""
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(top == 0, -126, e).clamp(min=-126).int()


def _power(e):
    return ((e + 127) << 23).view(torch.float32)


def _blocks(x):
    """[..., K] as [..., K/128 rounded up, 128], filled up with zeros."""
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % BLOCK)).unflatten(-1, (-1, BLOCK))


def _quantise_rows(x):
    """Codes (e4m3) of x [..., K] and scales [..., K/128 rounded up]: blocks of 128 along the last axis."""
    b = _blocks(x.float())
    top = b.abs().amax(-1)
    finite = torch.isfinite(top)
    e = _exponent(torch.where(finite, top, 0.0))
    code = torch.where(finite[..., None], b, 0.0) * _power(-e)[..., None]
    return code.flatten(-2)[..., :x.shape[-1]].to(E4M3), torch.where(finite, _power(e), float("nan"))


def _squares(x):
    """[..., R, C] as [..., R/128, C/128, 128, 128], filled up with zeros."""
    x = torch.nn.functional.pad(x, (0, -x.shape[-1] % BLOCK, 0, -x.shape[-2] % BLOCK))
    return x.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK)).transpose(-3, -2)


def _quantise_squares(x, two=True):
    """Codes of x [..., R, C] and scales [..., R/128, C/128 rounded up], blocks of 128 x 128.  Scales that
    are no powers of two (the largest value over 448) come with a checkpoint."""
    R, C = x.shape[-2:]
    b = _squares(x.float())
    top = b.abs().amax((-1, -2))
    if two:
        e = _exponent(top)
        scale, code = _power(e), b * _power(-e)[..., None, None]
    else:
        scale = torch.where(top > 0, top / torch.full_like(top, E4M3_MAX), 1.0)
        code = (b / scale[..., None, None]).clamp(-E4M3_MAX, E4M3_MAX)
    code = code.transpose(-3, -2).flatten(-2).flatten(-3, -2)
    return code[..., :R, :C].to(E4M3).contiguous(), scale


def _row_values(codes, scales):
    """What codes [..., K] with scales [..., K/128 rounded up] stand for, in 32 bits."""
    return codes.float() * scales.repeat_interleave(BLOCK, -1)[..., :codes.shape[-1]]


def _square_values(codes, scales):
    R, C = codes.shape[-2:]
    s = scales.repeat_interleave(BLOCK, -1)[..., :C].repeat_interleave(BLOCK, -2)[..., :R, :]
    return codes.float() * s


def _product(a, ws, offsets, rows, N, dtype):
    """out[r] = a[r] . w_e^T for the rows of each expert; rows behind the last expert's are 0."""
    out = torch.zeros(rows, N, dtype=dtype, device=a.device)
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            out[lo:hi] = (a[lo:hi] @ ws(e).T).to(dtype)
    return out


def _gate_up(case, y):
    I = case["I"]
    return (y[:, :I], y[:, I:]) if case["halves"] else (y[:, 0::2], y[:, 1::2])


def _sigmoid_of(case, g):
    """The gate is g * sigmoid(z): z = g, or twice the argument of GELU's tanh; and dz/dg."""
    if case["activation"] == "swiglu":
        return torch.sigmoid(g), 1.0
    c = 2.0 * math.sqrt(2.0 / math.pi)
    return torch.sigmoid(c * (g + 0.044715 * g * g * g)), c * (1.0 + 3 * 0.044715 * g * g)


def _activated(case, y):
    g, u = _gate_up(case, y)
    g, u = g.float(), u.float()
    return g * _sigmoid_of(case, g)[0] * u


# ---------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(DTYPES[dtype])


def _sorted_routes(case, g):
    """Offsets [E + 1] and routes sorted by expert of router logits N(0, 2), busier experts with `skew`."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = torch.randn(T, E, generator=g, device="cuda") * 2.0
    logits += torch.linspace(0.0, case["skew"], E, device="cuda")
    flat = torch.topk(logits, k, dim=1).indices.reshape(-1)
    order = torch.argsort(flat, stable=True)
    offsets = torch.searchsorted(flat[order], torch.arange(E + 1, device="cuda"))
    return offsets.int(), order.int()


def prepare(case, seed):
    g = _generator(seed)
    state = dict(case=dict(case))
    op = case["op"]
    if op in ("route", "route_backward"):
        T, E = case["T"], case["E"]
        logits = _normal(g, (T, E), case["dtype"], 2.0)
        # padding tokens: no expert is left to them
        lost = torch.rand(T, 1, generator=g, device="cuda") * 100 < case["padded"]
        state["logits"] = torch.where(lost, -math.inf, logits)
        state["bias"] = torch.randn(E, generator=g, device="cuda") * 0.1 if case["bias"] else None
        if op == "route_backward":
            state["ids"] = _choose(case, state["logits"], state["bias"])
            state["grad"] = torch.randn(T, case["k"], generator=g, device="cuda")
    elif op == "quantize":
        shape = (case["E"], case["rows"], case["K"])
        state["x"] = _normal(g, shape[1:] if case["form"] == "rows" else shape, case["dtype"])
    elif op == "matmul":
        T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
        offsets, order = _sorted_routes(case, g)
        rows = torch.randn(T if case["gather"] else T * k, K, generator=g, device="cuda")
        state["a_codes"], state["a_scales"] = _quantise_rows(rows)
        state["w_codes"] = torch.empty(E, N, K, dtype=E4M3, device="cuda")
        state["w_scales"] = torch.empty(E, -(-N // BLOCK), -(-K // BLOCK), device="cuda")
        step = max(1, min(E, (1 << 26) // (N * K)))
        for e in range(0, E, step):
            n = min(step, E - e)
            w = torch.randn(n, N, K, generator=g, device="cuda") * K ** -0.5
            state["w_codes"][e:e + n], state["w_scales"][e:e + n] = _quantise_squares(w, case["scales"] == "two")
        state["offsets"] = offsets
        state["order"] = order if case["gather"] else None
        state["offsets_host"] = offsets.tolist()  # what the plain form's loop over experts goes by
    else:
        state["y"] = _normal(g, (case["rows"], 2 * case["I"]), case["dtype"])
        if op == "activate_backward":
            state["grad"] = _normal(g, (case["rows"], case["I"]), case["dtype"])
    return state


# ---------------------------------------------------------------- one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import quantized_mixture_experts_route_amd as qm
    case = state["case"]
    op = case["op"]
    dtype = DTYPES[case["dtype"]]
    if op in ("route", "route_backward"):
        score = qm.SCORE_SIGMOID if case["score"] == "sigmoid" else qm.SCORE_SOFTMAX
        if op == "route_backward":
            return qm.route_scores_backward(state["grad"], state["logits"], state["ids"], score=score,
                                            normalize=case["normalize"], scale=case["scale"])
        return qm.route_scores(state["logits"], case["k"], score=score, bias=state["bias"], n_groups=case["groups"],
                               top_groups=case["kept"], group_top=case["best"], normalize=case["normalize"],
                               scale=case["scale"])
    if op == "quantize":
        if case["form"] == "rows":
            codes, scales = qm.fp8_quantize(state["x"])
            return qm.fp8_dequantize(codes, scales, dtype)
        codes, scales = qm.fp8_quantize_weights(state["x"], transpose=case["form"] == "transposed")
        return qm.fp8_dequantize_weights(codes, scales, dtype)
    if op == "matmul":
        return qm.fp8_matmul(state["a_codes"], state["a_scales"], state["w_codes"], state["w_scales"],
                             state["offsets"], sorted_routes=state["order"],
                             top_k=case["k"] if case["gather"] else None, dtype=dtype)
    activation = qm.ACT_SWIGLU if case["activation"] == "swiglu" else qm.ACT_GEGLU
    layout = qm.SWIGLU_HALVES if case["halves"] else qm.SWIGLU_INTERLEAVED
    if op == "activate_backward":
        return qm.activate_backward(state["grad"], state["y"], activation=activation, swiglu_fusion=layout)
    if case["to8"]:
        codes, scales = qm.activate_fp8(state["y"], activation=activation, swiglu_fusion=layout)
        return qm.fp8_dequantize(codes, scales, dtype)
    return qm.activate(state["y"], activation=activation, swiglu_fusion=layout)


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    dtype = DTYPES[case["dtype"]]
    if op == "route":
        ids = _choose(case, state["logits"], state["bias"])
        return ids, _weights(case, state["logits"], ids)
    if op == "route_backward":
        return _route_grad(case, state["logits"], state["ids"], state["grad"])
    if op == "quantize":
        if case["form"] == "rows":
            return _row_values(*_quantise_rows(state["x"])).to(dtype)
        x = state["x"].transpose(1, 2) if case["form"] == "transposed" else state["x"]
        return _square_values(*_quantise_squares(x)).to(dtype)
    if op == "matmul":
        a = _row_values(state["a_codes"], state["a_scales"])
        if state["order"] is not None:
            a = a[state["order"].long() // case["k"]]
        return _product(a, lambda e: _square_values(state["w_codes"][e], state["w_scales"][e]),
                        state["offsets_host"], case["T"] * case["k"], case["N"], dtype)
    if op == "activate":
        a = _activated(case, state["y"])
        return _row_values(*_quantise_rows(a)).to(dtype) if case["to8"] else a.to(dtype)
    g, u = _gate_up(case, state["y"])
    g, u, d = g.float(), u.float(), state["grad"].float()
    s, slope = _sigmoid_of(case, g)
    out = torch.empty_like(state["y"])
    to_gate, to_up = _gate_up(case, out)
    to_gate.copy_(d * u * (s + g * s * (1.0 - s) * slope))
    to_up.copy_(d * g * s)
    return out


# ---------------------------------------------------------------- what a pass cannot do without
def _selected(case):
    """Experts that the routes reach, as expected from T independent draws of k out of E."""
    return case["E"] * (1.0 - (1.0 - case["k"] / case["E"]) ** case["T"])


def work(case):
    op = case["op"]
    size = ELEMENT[case["dtype"]]
    if op in ("route", "route_backward"):
        T, E, k = case["T"], case["E"], case["k"]
        n = 8 * T * k + (4 * E if case["bias"] else 0)
        return {"bytes": T * E * size * (2 if op == "route_backward" else 1) + n, "flops": 4 * T * E}
    if op == "quantize":
        n = case["E"] * case["rows"] * case["K"]
        return {"bytes": 2 * n * size, "flops": 2 * n}  # values in, what their codes stand for out
    if op == "matmul":
        R = case["T"] * case["k"]
        K, N = case["K"], case["N"]
        kb, nb = -(-K // BLOCK), -(-N // BLOCK)
        a_rows = case["T"] if case["gather"] else R
        return {"bytes": int(_selected(case) * (N * K + 4 * nb * kb) + a_rows * (K + 4 * kb) + R * N * size
                             + 4 * (case["E"] + 1) + (4 * R if case["gather"] else 0)),
                "flops": 2 * R * N * K}
    n = case["rows"] * case["I"]
    return {"bytes": (5 if op == "activate_backward" else 3) * n * size, "flops": 8 * n}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_scores(case, logits):
    x = logits.double()
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.max(1, keepdim=True).values
    p = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(1, keepdim=True)
    return p / torch.where(total > 0, total, 1.0)


def _exact_choice(case, logits, bias):
    """One expert after another: each round takes the first of the largest that are left."""
    T, E = logits.shape
    left = _exact_scores(case, logits) + (0.0 if bias is None else bias.double())
    left[torch.isneginf(logits)] = -math.inf
    G, size = case["groups"], E // case["groups"]
    if case["kept"] < G:
        rank = torch.zeros(T, G, dtype=torch.float64, device=logits.device)
        for n in range(G):
            members = torch.sort(left[:, n * size:(n + 1) * size], 1).values
            rank[:, n] = members[:, -1]
            if case["best"] == 2 and size > 1:
                second = members[:, -2]
                rank[:, n] += torch.where(torch.isneginf(second), 0.0, second)
        open_ = torch.zeros(T, G, dtype=torch.bool, device=logits.device)
        for _ in range(case["kept"]):
            top = rank.max(1, keepdim=True).values
            first = ((rank == top) & ~open_).int().argmax(1, keepdim=True)
            open_.scatter_(1, first, True)
            rank.scatter_(1, first, -math.inf)
        for n in range(G):
            left[:, n * size:(n + 1) * size][~open_[:, n]] = -math.inf
    ids = torch.empty(T, case["k"], dtype=torch.int32, device=logits.device)
    for s in range(case["k"]):
        top = left.max(1, keepdim=True).values
        first = (left == top).int().argmax(1, keepdim=True)
        ids[:, s:s + 1] = torch.where(torch.isneginf(top), -1, first).int()
        left.scatter_(1, first, -math.inf)
    return ids


def _exact_e4m3(m):
    """Nearest e4m3 value to m (|m| <= 448), ties to even: the spacing is 2^(floor(log2 |m|) - 3), at least 2^-9."""
    power = torch.frexp(m)[1] - 1
    gap = torch.exp2((power - 3).clamp(min=-9).double())
    return torch.round(m / gap) * gap


def _exact_blocks(x, rows, cols):
    """Every block of rows x cols of the last two axes over its scale, rounded, times the scale."""
    out = torch.empty_like(x)
    for i in range(0, x.shape[-2], rows):
        for j in range(0, x.shape[-1], cols):
            b = x[..., i:i + rows, j:j + cols]
            top = b.abs().amax((-1, -2) if rows > 1 else -1, keepdim=True)
            e = torch.frexp(top / E4M3_MAX)
            e = torch.where(e.mantissa == 0.5, e.exponent - 1, e.exponent)  # ceil(log2(top / 448))
            scale = torch.exp2(torch.where(top > 0, e, -126).clamp(min=-126).double())
            out[..., i:i + rows, j:j + cols] = _exact_e4m3(b / scale) * scale
    return out


def _exact_rows(x):
    """Blocks of 128 of each row on its own."""
    K = x.shape[-1]
    full = torch.zeros(x.shape[0], -(-K // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    full[:, :K] = x
    return _exact_blocks(full[:, None, :].view(x.shape[0], -1, 1, BLOCK), 1, BLOCK).view(x.shape[0], -1)[:, :K]


def _exact_gate(case, g):
    """The gate's value and slope in 64 bits, GELU by its tanh."""
    if case["activation"] == "swiglu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "route":
        ids = _exact_choice(case, state["logits"], state["bias"])
        p = _exact_scores(case, state["logits"])
        w = torch.zeros(ids.shape, dtype=torch.float64, device="cuda")
        for s in range(case["k"]):
            at = ids[:, s:s + 1].long()
            w[:, s:s + 1] = torch.where(at < 0, 0.0, p.gather(1, at.clamp(min=0)))
        if case["normalize"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        return ids, w * case["scale"]
    if op == "route_backward":
        p, ids = _exact_scores(case, state["logits"]), state["ids"].long()
        T, E = p.shape
        picked = torch.zeros(T, E + 1, dtype=torch.float64, device="cuda")
        grad = torch.zeros_like(picked)
        at = torch.where(ids < 0, E, ids)
        picked.scatter_(1, at, 1.0)
        grad.scatter_(1, at, state["grad"].double() * case["scale"])
        picked, grad = picked[:, :E], grad[:, :E]
        # through the scores: w = p / sum of the picked, or p itself
        if case["normalize"]:
            total = (p * picked).sum(1, keepdim=True).clamp(min=1e-100)
            to_p = picked * (grad / total - (grad * p).sum(1, keepdim=True) / total ** 2)
        else:
            to_p = grad
        return to_p * p * (1 - p) if case["score"] == "sigmoid" else p * to_p - p * (p * to_p).sum(1, keepdim=True)
    if op == "quantize":
        x = state["x"].double()
        if case["form"] == "rows":
            return _exact_rows(x)
        return _exact_blocks(x.transpose(1, 2).contiguous() if case["form"] == "transposed" else x, BLOCK, BLOCK)
    if op == "matmul":
        R, K, N = case["T"] * case["k"], case["K"], case["N"]
        row_of = torch.arange(R, device="cuda") if state["order"] is None else state["order"].long() // case["k"]
        block = torch.arange(K, device="cuda") // BLOCK
        a = (state["a_codes"].double() * state["a_scales"].double()[:, block])[row_of]
        out = torch.zeros(R, N, dtype=torch.float64, device="cuda")
        bounds = state["offsets_host"]
        for e in range(case["E"]):
            if bounds[e + 1] > bounds[e]:
                scale = state["w_scales"][e].double()[torch.arange(N, device="cuda") // BLOCK][:, block]
                w = state["w_codes"][e].double() * scale
                out[bounds[e]:bounds[e + 1]] = torch.mm(a[bounds[e]:bounds[e + 1]], w.t().contiguous())
        return out
    y = state["y"].double()
    n = case["I"]
    g, u = (y[:, :n], y[:, n:]) if case["halves"] else (y[:, 0::2], y[:, 1::2])
    value, slope = _exact_gate(case, g)
    if op == "activate":
        return _exact_rows(value * u) if case["to8"] else value * u
    d = state["grad"].double()
    parts = (d * u * slope, d * value)
    return torch.cat(parts, 1) if case["halves"] else torch.stack(parts, 2).flatten(1)
