"""Operators of the expert path, as measured cases.

Two groups of operators: tokens sorted by expert and brought back with their
routing weights (and the gradients of both), and microscaled 4-bit floating
point (blocks of 32 e2m1 values sharing one power-of-two scale): quantisation
and the product of quantised rows with quantised expert weights.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits), or, where ``own`` is true, through the package's entry points.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ELEMENT = {"f16": 2, "bf16": 2, "f32": 4}
BLOCK = 32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases
def listed():
    def move(name, op, T, H, E, k, dtype, skew=0.0, dropped=0):
        return dict(name=name, op=op, T=T, H=H, E=E, k=k, dtype=dtype, skew=skew, dropped=dropped)

    def product(name, T, k, E, K, N, dtype, gather, skew=0.0):
        return dict(name=name, op="mx_matmul", T=T, k=k, E=E, K=K, N=N, dtype=dtype, gather=gather,
                    skew=skew)

    return [
        # six decode tokens over 512 experts, top-10: the smallest sort, all latency
        move("permute_decode", "permute", 6, 2048, 512, 10, "bf16"),
        # the large skewed prefill's tokens, sorted for its experts
        move("permute_prefill", "permute", 4096, 4096, 8, 2, "bf16", skew=2.0),
        # a training step's gradient back through the sort: odd width, some routes over capacity
        move("permute_grad_odd", "permute_backward", 1023, 1001, 60, 6, "f16", dropped=10),
        # one decode step's expert outputs back to its eight tokens
        move("unpermute_decode", "unpermute", 8, 2048, 8, 2, "f16"),
        # the large skewed prefill's expert outputs back to its tokens
        move("unpermute_prefill", "unpermute", 4096, 4096, 8, 2, "bf16", skew=2.0),
        # the gradient of the same step: to the expert outputs and to the routing weights
        move("unpermute_grad", "unpermute_backward", 4096, 4096, 8, 2, "bf16", skew=2.0, dropped=5),
        # a prefill's activations to 4 bits and the values they stand for
        dict(name="mx_quantize_tokens", op="mx_quantize", E=1, rows=4096, K=4096, dtype="bf16",
             transpose=False),
        # weights of eight experts quantised along the other axis, as the gradient's product takes them
        dict(name="mx_quantize_weights_t", op="mx_quantize", E=8, rows=2048, K=2048, dtype="f16",
             transpose=True),
        # one decode token through its two experts: a plain read of two experts' weights
        product("mx_matmul_token", 1, 2, 8, 2048, 4096, "f16", True),
        # six decode tokens over 512 experts, top-10: about 57 experts of one or two rows each
        product("mx_matmul_many_experts", 6, 10, 512, 2048, 1536, "bf16", True),
        # a 512-token prefill of the 8-expert layer
        product("mx_matmul_prefill", 512, 2, 8, 2048, 4096, "f16", True),
        # the large skewed prefill's first projection
        product("mx_matmul_skewed", 4096, 2, 8, 4096, 28672, "bf16", True, skew=2.0),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["permute", "permute_backward", "unpermute", "unpermute_backward",
                     "mx_quantize", "mx_quantize", "mx_matmul", "mx_matmul", "mx_matmul",
                     "mx_matmul"])
    dtype = rng.choice(["f16", "bf16", "bf16", "f32"])
    if op == "mx_quantize":
        transpose = rng.random() < 0.4
        rows = _log(rng, 1, 16384)
        K = _log(rng, 1 if transpose else 32, 8192)
        if transpose:
            rows = max(32, rows // BLOCK * BLOCK)
        else:
            K = K // BLOCK * BLOCK
        E = _log(rng, 1, 8) if transpose else 1
        while E * rows * K > 1 << 25:
            if transpose:
                rows = max(32, rows // 2 // BLOCK * BLOCK)
            else:
                rows = rows // 2
        return dict(op=op, E=E, rows=rows, K=K, dtype=dtype, transpose=transpose)
    E = _log(rng, 1, 512)
    k = rng.randint(1, min(E, 10))
    skew = rng.choice([0.0, 0.0, 2.0])
    if op == "mx_matmul":
        K = _log(rng, 64, 8192) // BLOCK * BLOCK
        N = _log(rng, 16, 16384)
        if rng.random() < 0.7:
            N = (N + 15) // 16 * 16
        while E * N * K > 1 << 30:
            E = max(1, E // 2)
        k = min(k, E)
        T = _log(rng, 1, 8192)
        while T > 1 and T * k * N * K > 1 << 39:
            T //= 2
        return dict(op=op, T=T, k=k, E=E, K=K, N=N, dtype=dtype, gather=rng.random() < 0.7, skew=skew)
    H = _log(rng, 64, 8192)
    if rng.random() < 0.7:
        H = H // 8 * 8
    T = _log(rng, 1, 16384)
    while T > 1 and T * k * H > 1 << 25:
        T //= 2
    return dict(op=op, T=T, H=H, E=E, k=k, dtype=dtype, skew=skew,
                dropped=rng.choice([0, 0, 0, 10, 50]))


# ---------------------------------------------------------------- plain pieces
def _sort(ids, E):
    """Stable sort of the routes by expert, dropped routes (ids outside [0, E)) last:
    offsets [E + 1], sorted_routes [R], route_rows [T, k] (-1 - row for a dropped route)."""
    flat = ids.reshape(-1).long()
    valid = (flat >= 0) & (flat < E)
    key = torch.where(valid, flat, E)
    order = torch.argsort(key, stable=True)
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=ids.device))
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=ids.device)
    row = torch.where(valid, row, -1 - row)
    return offsets.int(), order.int(), row.int().reshape(ids.shape)


def _scatter_back(rows, route_rows, weights):
    """sum over slots of weight * row; dropped routes add nothing."""
    j = route_rows.long()
    v = rows[j.clamp(min=0)].float()
    if weights is not None:
        v = v * weights[..., None]
    return torch.where((j >= 0)[..., None], v, 0.0).sum(1).to(rows.dtype)


def _quantise(x):
    """Blocks of 32 along the last axis: e2m1 codes [..., K] (uint8, sign in bit 3) and scale
    bytes [..., K/32]: 2^(byte - 127) with exponent floor(log2 max|x|) - 2."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1)
    exponent = torch.frexp(top)[1].int() - 3
    exponent = torch.where(top == 0, -127, exponent).clamp(-127, 127)
    finite = torch.isfinite(b).all(-1)
    step = ((127 - exponent) << 23).view(torch.float32)  # 2^-exponent, from its bits
    m = b.abs() * step[..., None]
    # the borders between neighbouring values; a value on a border takes the even code
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5)
            + (m >= 3.5) + (m > 5.0))
    code |= torch.signbit(b).to(torch.uint8) << 3
    code = torch.where(finite[..., None], code, 0)
    scale = torch.where(finite, exponent + 127, 255).to(torch.uint8)
    return code.flatten(-2), scale


def _pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _values(codes, scales):
    """What packed codes [..., K/2] with scale bytes [..., K/32] stand for, in 32 bits."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    e = scales.int()
    # 2^(e - 127) from its bits; 2^-127 is subnormal, 255 stands for NaN
    step = torch.where(e == 0, 1 << 22, e << 23).view(torch.float32)
    step = torch.where(e == 255, float("nan"), step)
    v = table[code.int()].unflatten(-1, (-1, BLOCK)) * step[..., None]
    return v.flatten(-2)


def _product(a, ws, offsets, rows, N, dtype):
    """out[r] = a[r] . w_e^T for the rows of each expert; rows behind the last expert's are 0."""
    out = torch.zeros(rows, N, dtype=dtype, device=a.device)
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            out[lo:hi] = (a[lo:hi] @ ws(e).T).to(dtype)
    return out


# ---------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _routing(case, g):
    """Top-k ids and softmax weights of router logits N(0, 2), busier experts with `skew`."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = torch.randn(T, E, generator=g, device="cuda") * 2.0
    logits += torch.linspace(0.0, case["skew"], E, device="cuda")
    top, ids = torch.topk(logits, k, dim=1)
    ids = ids.int()
    if case.get("dropped"):
        lost = torch.rand(T, k, generator=g, device="cuda") * 100 < case["dropped"]
        ids = torch.where(lost, -1, ids)
    return ids.contiguous(), torch.softmax(top, 1).contiguous()


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(DTYPES[dtype])


def prepare(case, seed):
    g = _generator(seed)
    state = dict(case=dict(case))
    op = case["op"]
    if op == "mx_quantize":
        shape = (case["E"], case["rows"], case["K"])
        state["x"] = _normal(g, shape if case["transpose"] else shape[1:], case["dtype"])
    elif op == "mx_matmul":
        T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
        ids, _ = _routing(case, g)
        offsets, order, _ = _sort(ids, E)
        code, scale = _quantise(torch.randn(T if case["gather"] else T * k, K, generator=g, device="cuda"))
        state["a_codes"], state["a_scales"] = _pack(code), scale
        state["w_codes"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
        state["w_scales"] = torch.empty(E, N, K // BLOCK, dtype=torch.uint8, device="cuda")
        step = max(1, min(E, (1 << 26) // (N * K)))
        for e in range(0, E, step):
            n = min(step, E - e)
            code, scale = _quantise(torch.randn(n, N, K, generator=g, device="cuda") * K ** -0.5)
            state["w_codes"][e:e + n], state["w_scales"][e:e + n] = _pack(code), scale
        state["offsets"] = offsets
        state["order"] = order if case["gather"] else None
        state["offsets_host"] = offsets.tolist()  # what the plain form's loop over experts goes by
    else:
        T, k, E, H = (case[n] for n in ("T", "k", "E", "H"))
        state["ids"], state["weights"] = _routing(case, g)
        if op == "permute":
            state["hidden"] = _normal(g, (T, H), case["dtype"])
        else:
            state["route_rows"] = _sort(state["ids"], E)[2]
            state["rows"] = _normal(g, (T * k, H), case["dtype"])
            if op == "unpermute_backward":
                state["grad_out"] = _normal(g, (T, H), case["dtype"])
    return state


# ---------------------------------------------------------------- one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import quantized_mixture_experts_route_amd as qm
    case = state["case"]
    op = case["op"]
    if op == "permute":
        return qm.permute(state["hidden"], state["ids"], case["E"])
    if op == "permute_backward":
        return qm.permute_backward(state["rows"], state["route_rows"])
    if op == "unpermute":
        return qm.unpermute(state["rows"], state["route_rows"], state["weights"])
    if op == "unpermute_backward":
        return qm.unpermute_backward(state["grad_out"], state["rows"], state["route_rows"], state["weights"])
    if op == "mx_quantize":
        codes, scales = qm.mx_quantize(state["x"], transpose=case["transpose"])
        return qm.mx_dequantize(codes, scales, DTYPES[case["dtype"]])
    return qm.mx_matmul(state["a_codes"], state["a_scales"], state["w_codes"], state["w_scales"],
                        state["offsets"], sorted_routes=state["order"], top_k=case["k"],
                        dtype=DTYPES[case["dtype"]])


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    if op == "permute":
        E, k = case["E"], case["k"]
        ids = state["ids"]
        offsets, order, route_rows = _sort(ids, E)
        rows = state["hidden"][order.long() // k]
        kept = torch.arange(order.numel(), device=rows.device) < offsets[E]
        rows = torch.where(kept[:, None], rows, 0)
        return rows, offsets, order, route_rows
    if op == "permute_backward":
        return _scatter_back(state["rows"], state["route_rows"], None)
    if op == "unpermute":
        return _scatter_back(state["rows"], state["route_rows"], state["weights"])
    if op == "unpermute_backward":
        rows, weights, route_rows = state["rows"], state["weights"], state["route_rows"]
        T, k = route_rows.shape
        j = route_rows.reshape(-1).long()
        kept = j >= 0
        at = torch.where(kept, j, -1 - j)
        grad = state["grad_out"].float()[torch.arange(T * k, device=rows.device) // k]
        grad_rows = torch.empty_like(rows)
        grad_rows[at] = torch.where(kept[:, None], weights.reshape(-1, 1) * grad, 0.0).to(rows.dtype)
        dots = (grad * rows[at].float()).sum(1)
        return grad_rows, torch.where(kept, dots, 0.0).reshape(T, k)
    if op == "mx_quantize":
        x = state["x"].transpose(1, 2) if case["transpose"] else state["x"]
        code, scale = _quantise(x)
        return _values(_pack(code), scale).to(DTYPES[case["dtype"]])
    a = _values(state["a_codes"], state["a_scales"])
    if state["order"] is not None:
        a = a[state["order"].long() // case["k"]]
    return _product(a, lambda e: _values(state["w_codes"][e], state["w_scales"][e]),
                    state["offsets_host"], case["T"] * case["k"], case["N"], DTYPES[case["dtype"]])


# ---------------------------------------------------------------- what a pass cannot do without
def _selected(case):
    """Experts that the routes reach, as expected from T independent draws of k out of E."""
    return case["E"] * (1.0 - (1.0 - case["k"] / case["E"]) ** case["T"])


def work(case):
    op = case["op"]
    size = ELEMENT[case["dtype"]]
    if op == "mx_quantize":
        n = case["E"] * case["rows"] * case["K"]
        return {"bytes": 2 * n * size, "flops": 2 * n}  # values in, what their codes stand for out
    R = case["T"] * case["k"]
    if op == "mx_matmul":
        K, N = case["K"], case["N"]
        packed = K / 2 + K / BLOCK
        a_rows = case["T"] if case["gather"] else R
        return {"bytes": int(_selected(case) * N * packed + a_rows * packed + R * N * size
                             + 4 * (case["E"] + 1) + (4 * R if case["gather"] else 0)),
                "flops": 2 * R * N * K}
    T, H, E = case["T"], case["H"], case["E"]
    if op == "permute":
        return {"bytes": (T + R) * H * size + 12 * R + 4 * (E + 1), "flops": 0}
    if op == "permute_backward":
        return {"bytes": (T + R) * H * size + 4 * R, "flops": R * H}
    if op == "unpermute":
        return {"bytes": (T + R) * H * size + 8 * R, "flops": 2 * R * H}
    return {"bytes": (T + 2 * R) * H * size + 12 * R, "flops": 3 * R * H}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_rows(ids, E):
    """Row of every route (T * k of them) by counting, and whether the route is kept."""
    flat = ids.reshape(-1).tolist()
    kept = [0 <= e < E for e in flat]
    count = [0] * (E + 1)
    for e, ok in zip(flat, kept):
        count[e if ok else E] += 1
    start, total = [], 0
    for c in count:
        start.append(total)
        total += c
    offsets = list(start)
    row = []
    for e, ok in zip(flat, kept):
        e = e if ok else E
        row.append(start[e])
        start[e] += 1
    return row, kept, offsets


def _exact_quantised(x):
    """Nearest e2m1 value (ties to the even code) of x / 2^(floor(log2 max) - 2), times it."""
    b = x.double().reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    top = b.abs().max(-1, keepdim=True).values
    power = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    # log2 rounds: put the power right where it lands beside a whole number
    power = torch.where(torch.exp2(power) > top, power - 1, power)
    power = torch.where(torch.exp2(power + 1) <= top, power + 1, power)
    scale = torch.exp2(torch.clamp(torch.where(top > 0, power - 2, -127.0), -127.0, 127.0))
    m = b.abs() / scale
    # the spacing of e2m1 is 0.5 below 2, 1 below 4, 2 from there; round() takes ties to even
    gap = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    q = torch.clamp(torch.round(m / gap) * gap, max=6.0)
    return (torch.copysign(q, b) * scale).reshape(x.shape)


def _exact_values(codes, scales):
    """Sign, exponent and mantissa of each code: s * 2^(e - 1) * (1 + m/2), or s * m/2 at e = 0."""
    c = torch.stack((codes % 16, codes // 16), -1).reshape(*codes.shape[:-1], -1).double()
    sign = torch.where(c >= 8, -1.0, 1.0)
    c = torch.remainder(c, 8)
    e, m = torch.floor(c / 2), torch.remainder(c, 2)
    v = sign * torch.where(e == 0, m / 2, torch.exp2(e - 1) * (1 + m / 2))
    power = torch.exp2(scales.double() - 127)
    power = torch.where(scales == 255, float("nan"), power)
    return v * power.repeat_interleave(BLOCK, -1)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "mx_quantize":
        x = state["x"]
        return _exact_quantised(x.permute(0, 2, 1).contiguous() if case["transpose"] else x)
    if op == "mx_matmul":
        R = case["T"] * case["k"]
        row_of = torch.arange(R, device="cuda") if state["order"] is None else state["order"].long() // case["k"]
        a = _exact_values(state["a_codes"], state["a_scales"])[row_of]
        out = torch.zeros(R, case["N"], dtype=torch.float64, device="cuda")
        bounds = state["offsets_host"]
        for e in range(case["E"]):
            if bounds[e + 1] > bounds[e]:
                w = _exact_values(state["w_codes"][e], state["w_scales"][e])
                out[bounds[e]:bounds[e + 1]] = torch.mm(a[bounds[e]:bounds[e + 1]], w.t().contiguous())
        return out
    k = case["k"]
    row, kept, offsets = _exact_rows(state["ids"], case["E"])
    row = torch.tensor(row, device="cuda")
    kept = torch.tensor(kept, device="cuda")
    token = torch.arange(row.numel(), device="cuda") // k
    if op == "permute":
        out = torch.zeros(row.numel(), case["H"], dtype=torch.float64, device="cuda")
        out[row[kept]] = state["hidden"].double()[token[kept]]
        order = torch.empty_like(row)
        order[row] = torch.arange(row.numel(), device="cuda")
        route_rows = torch.where(kept, row, -1 - row).int().reshape(case["T"], k)
        return out, torch.tensor(offsets, device="cuda").int(), order.int(), route_rows
    rows = state["rows"].double()
    weights = state["weights"].double().reshape(-1)
    if op in ("permute_backward", "unpermute"):
        out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
        for s in range(k):
            part = rows[row[s::k]] * kept[s::k, None]
            out += part if op == "permute_backward" else part * weights[s::k, None]
        return out
    grad = state["grad_out"].double()
    grad_rows = torch.zeros_like(rows)
    grad_weights = torch.zeros(row.numel(), dtype=torch.float64, device="cuda")
    for s in range(k):
        j, ok = row[s::k], kept[s::k, None]
        grad_rows[j] = grad * weights[s::k, None] * ok
        grad_weights[s::k] = ((grad * rows[j]).sum(1) * kept[s::k])
    return grad_rows, grad_weights.reshape(case["T"], k)
