"""Measured cases of the MoE block's prompt operators.

Four operators that a layer with many tokens needs around its routed experts:

  norm     residual addition and root-mean-square norm, with the normalised
           rows in bf16, as MXFP8 codes with UE8M0 scales, or both
  group    the grouping of routed (token, slot) pairs by expert
  product  the ragged matrix products of the groups with their experts'
           MXFP8 or MXFP4 weights: plain rows in bf16, or the gate/up pair
           finished to SiLU(gate) * up and requantised to MXFP8
  combine  the routing-weighted sum of a token's expert rows, with the
           residual stream added

`run` computes them in elementary torch operations in 32 bits, or, with `own`
set, through the framework's public calls. MXFP8 outputs are returned as their
E4M3 elements and UE8M0 scales in torch's 8-bit floating types.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token between two layers of a decode step
        _norm("norm one token", 1, 2048, "both"),
        # a prompt chunk: bf16 rows for the router, MXFP8 rows for the experts
        _norm("norm prompt chunk", 4096, 2048, "both"),
        # the wide model's whole prefill batch, rows for the experts alone
        _norm("norm wide prefill", 8191, 7168, "mxfp8"),
        # a skewed decode batch's routing
        _group("group decode batch", 32, 8, 128, True, 0),
        # a prefill batch's routing, its bucket's tail of unused slots empty
        _group("group prefill", 16384, 8, 256, False, 37),
        # a decode batch: most experts idle, one or two rows in the others
        _product("gate/up decode batch", 8, 8, 128, 2048, 768, "mxfp8", True, False),
        # a prompt chunk over the 128-expert layer, both projections
        _product("gate/up prompt chunk", 4096, 8, 128, 2048, 768, "mxfp8", True, False),
        _product("down odd skewed chunk", 1001, 8, 128, 2048, 768, "mxfp8", False, True),
        # the same layer with 4-bit weights
        _product("gate/up 4-bit chunk", 2048, 8, 128, 2048, 768, "mxfp4", True, False),
        # one device's share of the large experts at prefill
        _product("down large experts", 4096, 8, 32, 7168, 2048, "mxfp8", False, False),
        # a short prompt's rows back in token order
        _combine("combine short prompt", 77, 8, 2048, 5),
        # a prefill batch's
        _combine("combine prefill", 8192, 8, 2048, 0),
    ]


def _norm(name, T, H, out):
    return {"name": name, "op": "norm", "T": T, "H": H, "out": out}


def _group(name, T, k, E, skew, unused):
    return {"name": name, "op": "group", "T": T, "k": k, "E": E, "skew": skew, "unused": unused}


def _product(name, T, k, E, H, I, fmt, gate_up, skew):
    return {"name": name, "op": "product", "T": T, "k": k, "E": E, "H": H, "I": I, "fmt": fmt,
            "gate_up": gate_up, "skew": skew}


def _combine(name, T, k, H, unused):
    return {"name": name, "op": "combine", "T": T, "k": k, "H": H, "unused": unused}


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(max(int(round(v / step)) * step, lo), hi)


def draw(rng):
    op = rng.choice(["norm", "group", "product", "product", "product", "combine"])
    if op == "norm":
        H = _log(rng, 256, 7168, 32)
        c = _norm("", _log(rng, 1, min(16384, 8191 * 7168 // H)), H,
                  rng.choice(["bf16", "mxfp8", "both"]))
    elif op == "group":
        E = rng.choice([8, 60, 128, 160, 256])
        T = _log(rng, 1, 16384)
        c = _group("", T, rng.choice([1, 2, 4, 6, 8]), E, rng.random() < 0.5,
                   rng.choice([0, rng.randint(0, T)]))
    elif op == "product":
        fmt = rng.choice(["mxfp8", "mxfp8", "mxfp4"])
        step = 128 if fmt == "mxfp4" else 32
        k = rng.choice([1, 2, 4, 6, 8])
        E = rng.choice([8, 16, 60, 128])
        H = _log(rng, 256, 4096, step)
        I = _log(rng, 128, 2048, step)
        while E * 3 * H * I > 640e6:        # weights of a layer that is loaded quickly
            E //= 2
        T = _log(rng, 1, 8192)
        while T > 1 and T * k * H * I > 4096 * 8 * 7168 * 2048 / 4:
            T //= 2
        c = _product("", T, min(k, E), E, H, I, fmt, rng.random() < 0.5, rng.random() < 0.5)
    else:
        H = _log(rng, 256, 7168, 32)
        k = rng.choice([1, 2, 4, 6, 8])
        T = _log(rng, 1, max(1, 8192 * 8 * 2048 // (k * H)))
        T = min(T, 16384)
        c = _combine("", T, k, H, rng.choice([0, rng.randint(0, T)]))
    del c["name"]
    return c


def work(case):
    op, T = case["op"], case["T"]
    if op == "norm":
        H = case["H"]
        b = T * H * (2 + 2 + 2) + 2 * H
        if case["out"] != "mxfp8":
            b += 2 * T * H
        if case["out"] != "bf16":
            b += T * H + T * (H // 32)
        return {"bytes": b, "flops": 5 * T * H}
    if op == "group":
        S = T * case["k"]
        return {"bytes": 4 * S + 4 * S + 4 * S + 4 * (case["E"] + 1), "flops": S}
    if op == "product":
        k, E, H, I = case["k"], case["E"], case["H"], case["I"]
        R = T * k
        code = 1.0 if case["fmt"] == "mxfp8" else 0.5
        # experts that some row is routed to; all of them beyond a few rows each
        used = E * (1 - (1 - k / E) ** T) if not case["skew"] else min(E, R)
        if case["gate_up"]:
            N, K, rows_in = 2 * I, H, T
            out = R * I * (1 + 1 / 32)
        else:
            N, K, rows_in = H, I, R
            out = R * N * 2
        b = used * N * K * (code + 1 / 32) + rows_in * K * (1 + 1 / 32) + out + 4 * (E + 1)
        if case["gate_up"]:
            b += 4 * R
        return {"bytes": b, "flops": 2 * R * N * K}
    k, H = case["k"], case["H"]
    used = T - case["unused"]
    return {"bytes": used * k * H * 2 + 8 * T * k + T * H * 2 * 2, "flops": 2 * used * k * H}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def _route(g, T, k, E, skew):
    """Top-k ids and renormalised weights of random router logits; a skewed
    router prefers some experts as a Zipf(1.1) popularity does."""
    z = _randn(g, T, E)
    if skew:
        rank = 1 + torch.randperm(E, device=DEV, generator=g).float()
        z = z - 1.1 * rank.log()
    top, ids = z.topk(k, dim=1)
    return ids.to(torch.int32).contiguous(), torch.softmax(top, dim=1).contiguous()


def _grouping(ids, E):
    """offsets[E + 1], rows[S] and slots like ids, in the order of slots."""
    flat = ids.reshape(-1).long()
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    slots = torch.empty_like(flat)
    slots[order] = torch.arange(flat.numel(), device=DEV)
    slots = torch.where(flat < 0, -1, slots).to(torch.int32).view(ids.shape)
    rows = (order // ids.shape[1]).to(torch.int32)
    return offsets, rows, slots, int(counts.max())


def _encode_fp8(v):
    """MXFP8 of the last axis: E4M3 codes and UE8M0 scale codes, both uint8."""
    codes, e = _mxfp8(v)
    return codes.view(torch.uint8), e.view(torch.uint8)


def _encode_fp4(v):
    """MXFP4: packed E2M1 codes (even element in the low nibble), scales."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, 0).clamp(-127, 127)
    q = torch.ldexp(b, -e.unsqueeze(-1)).abs().clamp(max=6.0)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    code = torch.bucketize(q, mids) | (torch.signbit(b).int() << 3)
    code = code.flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def prepare(case, seed):
    g, op, T = _gen(seed), case["op"], case["T"]
    s = {"case": case}
    if op == "norm":
        H = case["H"]
        # a residual stream: some channels far larger than the rest
        loud = 1 + 15 * (torch.rand(H, device=DEV, generator=g) < 0.01)
        s["x"] = _randn(g, T, H).to(torch.bfloat16)
        s["residual"] = (2 * loud * _randn(g, T, H)).to(torch.bfloat16)
        s["weight"] = (1 + 0.1 * _randn(g, H)).to(torch.bfloat16)
    elif op == "group":
        s["ids"] = _route(g, T, case["k"], case["E"], case["skew"])[0]
        s["ids"][T - case["unused"]:] = -1
    elif op == "product":
        E, H, I, k = case["E"], case["H"], case["I"], case["k"]
        ids, _ = _route(g, T, k, E, case["skew"])
        s["offsets"], rows, _, s["most"] = _grouping(ids, E)
        N, K = (2 * I, H) if case["gate_up"] else (H, I)
        s["rows"] = rows if case["gate_up"] else None
        a = _randn(g, T if case["gate_up"] else T * k, K)
        s["a"], s["a_scales"] = _encode_fp8(a if case["gate_up"] else a * torch.sigmoid(a))
        encode = _encode_fp8 if case["fmt"] == "mxfp8" else _encode_fp4
        w = [encode(0.02 * _randn(g, N, K)) for _ in range(E)]
        s["w"], s["w_scales"] = torch.stack([c for c, _ in w]), torch.stack([z for _, z in w])
        if own:                              # the handle that a program keeps with its weights
            from sparse_expert_gemv_gb300 import GroupedProduct
            s["product"] = GroupedProduct(s["w"], s["w_scales"], fmt=case["fmt"],
                                          silu_mul=case["gate_up"])
    else:
        k, H = case["k"], case["H"]
        E = 8 * k
        ids, s["weights"] = _route(g, T, k, E, False)
        ids[T - case["unused"]:] = -1
        _, _, s["slots"], _ = _grouping(ids, E)
        s["y"] = _randn(g, T * k, H).to(torch.bfloat16)
        s["residual"] = (2 * _randn(g, T, H)).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sparse_expert_gemv_gb300 as moe
    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        out = case["out"]
        n = moe.add_rms_norm(s["x"], s["weight"], s["residual"], eps=EPS,
                             bf16=out != "mxfp8", mxfp8=out != "bf16")
        q = () if n.codes is None else _as_floats(n.codes, n.scales)
        return [n.sum] + ([] if n.y is None else [n.y]) + list(q)
    if op == "group":
        return list(moe.group_by_expert(s["ids"], case["E"]))
    if op == "product":
        got = s["product"](s["a"], s["a_scales"], s["offsets"], rows=s["rows"])
        return list(_as_floats(*got)) if case["gate_up"] else [got]
    return [moe.combine(s["y"], s["slots"], s["weights"], residual=s["residual"])]


def _as_floats(codes, scales):
    return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        total = (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
        v = total.float()
        v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * s["weight"].float()
        out = [total]
        if case["out"] != "mxfp8":
            out.append(v.to(torch.bfloat16))
        if case["out"] != "bf16":
            out += _mxfp8(v)
        return out
    if op == "group":
        ids, E, k = s["ids"].reshape(-1).long(), case["E"], case["k"]
        hit = ids == torch.arange(E, device=DEV).unsqueeze(1)
        seen = hit.cumsum(1, dtype=torch.int32)
        offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        offsets[1:] = seen[:, -1].cumsum(0)
        rank = seen.gather(0, ids.clamp(min=0).unsqueeze(0)).squeeze(0) - 1
        slots = torch.where(ids < 0, -1, offsets[ids.clamp(min=0)] + rank).to(torch.int32)
        # unused slots write past the end, where nothing is read
        rows = torch.full((ids.numel() + 1,), -1, dtype=torch.int32, device=DEV)
        at = torch.where(ids < 0, ids.numel(), slots.long())
        token = torch.arange(ids.numel(), device=DEV, dtype=torch.int32) // k
        rows[at] = torch.where(ids < 0, -1, token)
        return [offsets, rows[:-1], slots.view(s["ids"].shape)]
    if op == "product":
        w = _decode(s["w"], s["w_scales"], case["fmt"])
        a = _decode(s["a"], s["a_scales"], "mxfp8")
        R = case["T"] * case["k"]
        off = s["offsets"].long()
        r = torch.arange(R, device=DEV)
        e = (r.unsqueeze(1) >= off[1:]).sum(1)           # the group of every row
        at = e * s["most"] + (r - off[e])                # its place among padded groups
        padded = torch.zeros(case["E"] * s["most"], a.shape[1], device=DEV)
        padded[at] = a if s["rows"] is None else a[s["rows"].long()]
        y = torch.bmm(padded.view(case["E"], s["most"], -1), w.transpose(1, 2)).flatten(0, 1)[at]
        if not case["gate_up"]:
            return [y.to(torch.bfloat16)]
        gate, up = y.chunk(2, dim=1)
        return list(_mxfp8(gate / (1 + torch.exp(-gate)) * up))
    rows = s["y"].float()[s["slots"].clamp(min=0).long()]
    w = torch.where(s["slots"] < 0, 0.0, s["weights"])
    y = (rows * w.unsqueeze(-1)).sum(1) + s["residual"].float()
    return [y.to(torch.bfloat16)]


def _mxfp8(v):
    """Blocks of 32 over the last axis, each divided by the power of two that
    brings its largest magnitude to [256, 512), saturated to 448 and rounded
    to E4M3; the powers as UE8M0."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 9, 0).clamp(-127, 127)
    q = torch.ldexp(b, -e.unsqueeze(-1)).clamp(-448, 448)
    return (q.flatten(-2).to(torch.float8_e4m3fn),
            (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu))


def _decode(codes, scales, fmt):
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                            device=DEV)
        v = grid[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    power = torch.exp2(scales.float() - 127)
    return (v.unflatten(-1, (-1, 32)) * power.unsqueeze(-1)).flatten(-2)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op == "group":                        # whole numbers alone
        return None
    s = prepare(case, seed)
    if op == "norm":
        t = s["x"].double() + s["residual"].double()
        # the stream is kept in bf16, and what is kept is normalised
        kept = _round(t, 8, -133)
        n = kept / (kept.square().sum(-1, keepdim=True) / case["H"] + EPS).sqrt()
        n = n * s["weight"].double()
        out = [kept]
        if case["out"] != "mxfp8":
            out.append(n)
        if case["out"] != "bf16":
            out += _mxfp8_exact(n)
        return out
    if op == "product":
        off = s["offsets"].tolist()
        a = _values(s["a"], s["a_scales"], "mxfp8")
        y = torch.zeros(off[-1], s["w"].shape[1], dtype=torch.float64, device=DEV)
        for e in range(case["E"]):
            lo, hi = off[e], off[e + 1]
            if hi > lo:
                x = a[lo:hi] if s["rows"] is None else a[s["rows"][lo:hi].long()]
                y[lo:hi] = x @ _values(s["w"][e], s["w_scales"][e], case["fmt"]).T
        if not case["gate_up"]:
            return [y]
        I = case["I"]
        return _mxfp8_exact(y[:, :I] * torch.sigmoid(y[:, :I]) * y[:, I:])
    total = s["residual"].double()
    for j in range(case["k"]):
        at = s["slots"][:, j].long()
        term = s["weights"][:, j:j + 1].double() * s["y"].double()[at.clamp(min=0)]
        total = total + torch.where(at.unsqueeze(1) < 0, 0.0, term)
    return [total]


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


def _values(codes, scales, fmt):
    if fmt == "mxfp8":
        c = codes.int()
        field, frac = (c >> 3) & 15, (c & 7).double()
        mag = torch.where(field > 0, (8 + frac) * torch.exp2(field.double() - 10), frac / 512)
        v = torch.where(c > 127, -mag, mag)
    else:
        c = torch.stack([codes % 16, codes // 16], dim=-1).reshape(*codes.shape[:-1], -1).int()
        field, frac = (c >> 1) & 3, (c & 1).double()
        mag = torch.where(field > 0, (2 + frac) * torch.exp2(field.double() - 2), frac / 2)
        v = torch.where(c > 7, -mag, mag)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=-1)
