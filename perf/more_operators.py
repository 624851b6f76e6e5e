"""Measured cases of the operators between the MoE block's routed experts.

  route    expert choice from router logits: softmax or sigmoid scores, a bias
           that balances the choice, groups of experts, top-k, renormalised
           and scaled weights
  norm     the norm after a block, its gate and scale, the residual addition
           and the norm before the next block, in one pass; rows in bf16, as
           MXFP8 codes with UE8M0 scales, or both
  dense    a matrix product with bias, activation and residual in its epilogue:
           router logits in FP32, the shared expert's SiLU(gate) * up and its
           way back onto the residual stream

`run` computes them in elementary torch operations in 32 bits (the choice of
experts, which compares scores that may lie close, in 64), or, with `own` set,
through the framework's public calls. MXFP8 outputs are returned as their E4M3
elements and UE8M0 scales in torch's 8-bit floating types.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
INF = float("inf")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of a decode step, scores balanced by a bias, in groups
        _route("route one token", 1, 8, 256, "fp32", "sigmoid", True, 8, 4, "top2", 0, 0),
        # a decode batch in a bucket of 96, two experts switched off
        _route("route padded decode batch", 96, 6, 160, "bf16", "softmax", False, 8, 3, "max", 2, 19),
        # a prefill batch's routing
        _route("route prefill", 16384, 8, 256, "fp32", "sigmoid", True, 8, 4, "top2", 0, 0),
        # one token between two layers: a scale per channel on the block's way back
        _norm("norms one token", 1, 2048, True, "channel", None, "both"),
        # a prompt chunk: a gate per token; bf16 rows for the router, MXFP8 rows for the experts
        _norm("norms prompt chunk", 4096, 2048, True, "row", "sigmoid", "both"),
        # the wide model's whole prefill batch, no gate, rows for dense products
        _norm("norms wide prefill", 8191, 7168, True, None, None, "bf16"),
        # a decode batch's router logits
        _dense("router decode batch", 8, 2048, 128, False, None, False, "fp32"),
        # the wide model's, of a prefill batch
        _dense("router prefill", 8191, 7168, 256, False, None, False, "fp32"),
        # a decode batch through a shared expert's gate and up projections
        _dense("shared gate/up decode", 16, 7168, 4096, False, "silu_mul", False, "bf16"),
        # an odd prompt chunk through a projection with bias and activation
        _dense("projection odd chunk", 1001, 2080, 2056, True, "gelu_tanh", True, "bf16"),
        # the shared expert's way back onto the residual stream, at prefill
        _dense("shared down prefill", 8192, 2048, 7168, False, None, True, "bf16"),
        # and its gate and up projections
        _dense("shared gate/up prefill", 8192, 7168, 4096, False, "silu_mul", False, "bf16"),
    ]


def _route(name, T, k, E, dtype, score, bias, groups, top, group_score, masked, padded):
    return {"name": name, "op": "route", "T": T, "k": k, "E": E, "dtype": dtype, "score": score,
            "bias": bias, "groups": groups, "top_groups": top, "group_score": group_score,
            "masked": masked, "padded": padded}


def _norm(name, T, H, post, gate, gate_fn, out):
    return {"name": name, "op": "norm", "T": T, "H": H, "post": post,
            "gate": gate or "none", "gate_fn": gate_fn or "none", "out": out}


def _dense(name, R, K, N, bias, act, residual, dtype):
    return {"name": name, "op": "dense", "R": R, "K": K, "N": N, "bias": bias, "act": act or "none",
            "residual": residual, "dtype": dtype}


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(max(int(round(v / step)) * step, lo), hi)


def draw(rng):
    op = rng.choice(["route", "route", "norm", "norm", "dense", "dense", "dense"])
    if op == "route":
        groups, per = rng.choice([(1, 8), (1, 60), (1, 128), (1, 256), (4, 32), (8, 20), (8, 32),
                                  (4, 15), (8, 16)])
        top = groups if groups == 1 else rng.randint(2, groups - 1)
        T = _log(rng, 1, 16384)
        k = rng.choice([1, 2, 4, 6, 8])
        c = _route("", T, k, groups * per, rng.choice(["fp32", "bf16"]),
                   rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6, groups, top,
                   rng.choice(["max", "top2"]), rng.choice([0, 0, 1, 3]),
                   rng.choice([0, rng.randint(0, T - 1)]))
    elif op == "norm":
        H = _log(rng, 256, 7168, 32)
        gate = rng.choice([None, "channel", "row", "full"])
        c = _norm("", _log(rng, 1, min(16384, 8191 * 7168 // (2 * H))), H, rng.random() < 0.8, gate,
                  rng.choice([None, "sigmoid", "tanh"]) if gate else None,
                  rng.choice(["bf16", "mxfp8", "both", "sum"]))
    else:
        K = _log(rng, 256, 7168, 8)
        act = rng.choice([None, "relu", "silu", "gelu", "gelu_tanh", "silu_mul", "silu_mul"])
        N = _log(rng, 60, 8192, 2 if act == "silu_mul" else 1)
        R = _log(rng, 1, 8192)
        while R > 1 and R * K * N > 8192 * 7168 * 4096:
            R //= 2
        c = _dense("", R, K, N, rng.random() < 0.5, act, act != "silu_mul" and rng.random() < 0.5,
                   rng.choice(["bf16", "bf16", "fp32"]))
    del c["name"]
    return c


def work(case):
    op = case["op"]
    if op == "route":
        T, k, E = case["T"], case["k"], case["E"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": T * E * size + T * k * 8 + (4 * E if case["bias"] else 0),
                "flops": 6 * T * E}
    if op == "norm":
        T, H = case["T"], case["H"]
        b = T * H * (2 + 2 + 2) + {"none": 0, "channel": 2 * H, "row": 2 * T, "full": 2 * T * H}[
            case["gate"]]
        if case["post"]:
            b += 2 * H
        if case["out"] != "sum":
            b += 2 * H
        if case["out"] in ("bf16", "both"):
            b += 2 * T * H
        if case["out"] in ("mxfp8", "both"):
            b += T * H + T * (H // 32)
        return {"bytes": b, "flops": 12 * T * H}
    R, K, N = case["R"], case["K"], case["N"]
    cols = N // 2 if case["act"] == "silu_mul" else N
    b = 2 * R * K + 2 * N * K + R * cols * (4 if case["dtype"] == "fp32" else 2)
    b += 2 * N if case["bias"] else 0
    b += 2 * R * cols if case["residual"] else 0
    return {"bytes": b, "flops": 2 * R * K * N}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g, op = torch.Generator(device=DEV).manual_seed(seed), case["op"]

    def randn(*shape):
        return torch.randn(*shape, device=DEV, generator=g)

    s = {"case": case}
    if op == "route":
        T, E = case["T"], case["E"]
        # a trained router: some experts preferred, a few logits far from the rest
        z = 0.5 * randn(E) + randn(T, E) * (1 + 0.5 * torch.rand(T, 1, device=DEV, generator=g))
        off = torch.randperm(E, device=DEV, generator=g)[:case["masked"]]
        z[:, off] = -INF                           # experts that are switched off
        z[T - case["padded"]:] = -INF              # rows behind the batch's last token
        s["logits"] = z if case["dtype"] == "fp32" else z.to(torch.bfloat16)
        # a balancing bias: steps of a thousandth that have added up
        spread = 0.1 if case["score"] == "sigmoid" else 2 / E
        s["bias"] = (randn(E) * spread * 1000).round() / 1000 if case["bias"] else None
    elif op == "norm":
        T, H = case["T"], case["H"]
        # a residual stream: some channels far larger than the rest
        loud = 1 + 15 * (torch.rand(H, device=DEV, generator=g) < 0.01)
        s["x"] = (0.5 * randn(T, H) * (1 + randn(T, 1).abs())).to(torch.bfloat16)
        s["residual"] = (2 * loud * randn(T, H)).to(torch.bfloat16)
        s["post"] = (0.5 + 0.1 * randn(H)).to(torch.bfloat16) if case["post"] else None
        s["pre"] = (1 + 0.1 * randn(H)).to(torch.bfloat16) if case["out"] != "sum" else None
        shape = {"none": None, "channel": (H,), "row": (T, 1), "full": (T, H)}[case["gate"]]
        s["gate"] = None if shape is None else (0.5 + randn(*shape)).to(torch.bfloat16)
        s["scale"] = 0.875
    else:
        R, K, N = case["R"], case["K"], case["N"]
        s["x"] = randn(R, K).to(torch.bfloat16)
        s["weight"] = (randn(N, K) * K ** -0.5).to(torch.bfloat16)
        s["bias"] = (0.5 * randn(N)).to(torch.bfloat16) if case["bias"] else None
        s["residual"] = (2 * randn(R, N)).to(torch.bfloat16) if case["residual"] else None
        if own:                                    # the handle that a program keeps with its weights
            from sparse_expert_gemv_gb300 import DenseProduct
            s["product"] = DenseProduct(s["weight"], s["bias"], activation=_or_none(case["act"]))
    return s


def _or_none(name):
    return None if name == "none" else name


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


ROUTE_SCALE = 2.5


def _run_own(s):
    import sparse_expert_gemv_gb300 as moe
    case, op = s["case"], s["case"]["op"]
    if op == "route":
        return list(moe.route_experts(
            s["logits"], case["k"], score=case["score"], bias=s["bias"], groups=case["groups"],
            top_groups=case["top_groups"], group_score=case["group_score"], scale=ROUTE_SCALE))
    if op == "norm":
        out = case["out"]
        n = moe.norm_add_norm(s["x"], s["residual"], s["post"], s["pre"], gate=s["gate"],
                              gate_fn=_or_none(case["gate_fn"]), scale=s["scale"], eps=EPS,
                              bf16=out in ("bf16", "both"), mxfp8=out in ("mxfp8", "both"))
        got = [n.sum] + ([] if n.y is None else [n.y])
        if n.codes is not None:
            got += [n.codes.view(torch.float8_e4m3fn), n.scales.view(torch.float8_e8m0fnu)]
        return got
    return [s["product"](s["x"], s["residual"], float32=case["dtype"] == "fp32")]


def _run_plain(s):
    return {"route": _route_plain, "norm": _norm_plain, "dense": _dense_plain}[s["case"]["op"]](s)


def _route_plain(s):
    case, E, G = s["case"], s["case"]["E"], s["case"]["groups"]
    logits = s["logits"].double()
    left = logits > -INF
    if case["score"] == "softmax":
        top = torch.where(left, logits, -INF).amax(1, keepdim=True)
        e = torch.where(left, torch.exp(logits - top), 0.0)
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-logits))
    choice = score if s["bias"] is None else score + s["bias"].double()
    choice = torch.where(left, choice, -INF)
    if G > 1:
        per = choice.view(-1, G, E // G).sort(dim=-1, descending=True).values
        group = per[..., 0]
        if case["group_score"] == "top2" and E > G:
            group = torch.where(per[..., 1] > -INF, group + per[..., 1], group)
        rank = group.sort(dim=1, descending=True, stable=True).indices.argsort(1)
        kept = (rank < case["top_groups"]).repeat_interleave(E // G, dim=1)
        choice = torch.where(kept, choice, -INF)
    value, ids = choice.sort(dim=1, descending=True, stable=True)
    value, ids = value[:, :case["k"]], ids[:, :case["k"]]
    w = torch.where(value > -INF, score.gather(1, ids), 0.0).float()
    total = w.sum(1, keepdim=True)
    w = torch.where(total > 0, w / total, 0.0) * ROUTE_SCALE
    return [torch.where(value > -INF, ids, -1).to(torch.int32), w]


def _norm_plain(s):
    case = s["case"]
    p = s["x"].float()
    if case["post"]:
        p = p * torch.rsqrt((p * p).mean(-1, keepdim=True) + EPS) * s["post"].float()
    if s["gate"] is not None:
        gate = s["gate"].float()
        if case["gate_fn"] == "sigmoid":
            gate = 1 / (1 + torch.exp(-gate))
        elif case["gate_fn"] == "tanh":
            gate = torch.tanh(gate)
        p = p * gate
    total = (s["residual"].float() + s["scale"] * p).to(torch.bfloat16)
    out = [total]
    if case["out"] != "sum":
        v = total.float()
        v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * s["pre"].float()
        if case["out"] != "mxfp8":
            out.append(v.to(torch.bfloat16))
        if case["out"] != "bf16":
            out += _mxfp8(v)
    return out


def _mxfp8(v):
    """Blocks of 32 over the last axis, each divided by the power of two that
    brings its largest magnitude to [256, 512), saturated to 448 and rounded
    to E4M3; the powers as UE8M0."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 9, 0).clamp(-127, 127)
    q = torch.ldexp(b, -e.unsqueeze(-1)).clamp(-448, 448)
    return [q.flatten(-2).to(torch.float8_e4m3fn),
            (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)]


def _dense_plain(s):
    case, act = s["case"], s["case"]["act"]
    y = s["x"].float() @ s["weight"].float().T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if act == "relu":
        y = y.clamp(min=0)
    elif act == "silu":
        y = y / (1 + torch.exp(-y))
    elif act == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * 0.5 ** 0.5))
    elif act == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh((2 / math.pi) ** 0.5 * (y + 0.044715 * y * y * y)))
    elif act == "silu_mul":
        gate, up = y.chunk(2, dim=1)
        y = gate / (1 + torch.exp(-gate)) * up
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y if case["dtype"] == "fp32" else y.to(torch.bfloat16)]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _route_exact, "norm": _norm_exact, "dense": _dense_exact}[case["op"]](s)


def _route_exact(s):
    case = s["case"]
    T, E, G, k = case["T"], case["E"], case["groups"], case["k"]
    z = s["logits"].double()
    z = z.masked_fill(z.isnan(), -INF)
    score = torch.sigmoid(z)
    if case["score"] == "softmax":
        score = (z - z.logsumexp(1, keepdim=True)).exp().nan_to_num(0.0)
    c = score + (s["bias"].double() if case["bias"] else 0)
    c = c.masked_fill(z == -INF, -INF)
    rows, index = torch.arange(T, device=DEV), torch.arange(E, device=DEV)

    def best(v):                  # the largest of each row, of equals the first
        top = v.max(1, keepdim=True).values
        return torch.where(v == top, torch.arange(v.shape[1], device=DEV), v.shape[1]).min(1).values

    if G > 1:
        first = c.view(T, G, -1)
        group = first.max(-1).values
        if case["group_score"] == "top2" and E > G:
            second = first.topk(2, dim=-1).values[..., 1]
            group = torch.where(second == -INF, group, group + second)
        keep = torch.zeros(T, G, dtype=torch.bool, device=DEV)
        for _ in range(case["top_groups"]):
            at = best(group.masked_fill(keep, -INF))
            # (a row of which nothing is left marks its first group again)
            keep[rows, at] = True
        c = c.masked_fill(~keep[:, index // (E // G)], -INF)
    ids = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    w = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    for j in range(k):
        at = best(c)
        some = c[rows, at] > -INF
        ids[:, j] = torch.where(some, at, -1).to(torch.int32)
        w[:, j] = torch.where(some, score[rows, at], 0.0)
        c[rows, at] = -INF
    return [ids, (w / w.sum(1, keepdim=True)).nan_to_num(0.0) * ROUTE_SCALE]


def _norm_exact(s):
    case, H = s["case"], s["case"]["H"]
    p = s["x"].double()
    if case["post"]:
        p = p / (p.square().sum(-1, keepdim=True) / H + EPS).sqrt() * s["post"].double()
    if s["gate"] is not None:
        gate = s["gate"].double()
        gate = {"none": lambda v: v, "sigmoid": torch.sigmoid, "tanh": torch.tanh}[
            case["gate_fn"]](gate)
        p = p * gate
    t = s["residual"].double() + s["scale"] * p
    out = [t]
    if case["out"] != "sum":
        # the stream is kept in bf16, and what is kept is normalised
        kept = _round(t, 8, -133)
        n = kept / (kept.square().sum(-1, keepdim=True) / H + EPS).sqrt() * s["pre"].double()
        if case["out"] != "mxfp8":
            out.append(n)
        if case["out"] != "bf16":
            out += _mxfp8_exact(n)
    return out


def _round(v, bits, least):
    """To `bits` significant bits, half to even, in steps of 2^least or more."""
    step = torch.exp2(torch.clamp(torch.frexp(v).exponent - bits, min=least).double())
    return torch.round(v / step) * step


def _mxfp8_exact(v):
    b = v.reshape(*v.shape[:-1], v.shape[-1] // 32, 32)
    amax = b.abs().max(-1).values
    e = (torch.frexp(amax).exponent.double() - 9).clamp(-127, 127)
    scale = torch.exp2(torch.where(amax > 0, e, torch.zeros_like(e)))
    q = _round(b / scale.unsqueeze(-1), 4, -9).clamp(-448, 448)
    return [q.reshape(v.shape), scale]


def _dense_exact(s):
    case, act = s["case"], s["case"]["act"]
    y = s["x"].double() @ s["weight"].double().T
    if case["bias"]:
        y += s["bias"].double()
    if act == "relu":
        y = torch.where(y > 0, y, 0.0)
    elif act == "silu":
        y = y * torch.sigmoid(y)
    elif act == "gelu":
        y = y * torch.erfc(-y / math.sqrt(2)) / 2
    elif act == "gelu_tanh":
        # (1 + tanh(z)) / 2 = sigmoid(2 z)
        y = y * torch.sigmoid(math.sqrt(8 / math.pi) * (y + 0.044715 * y ** 3))
    elif act == "silu_mul":
        half = case["N"] // 2
        y = y[:, :half] * torch.sigmoid(y[:, :half]) * y[:, half:]
    if case["residual"]:
        y = y + s["residual"].double()
    return [y]
