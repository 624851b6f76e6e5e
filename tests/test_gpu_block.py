"""GPU parity of the block operators (include/moe_block.h) with the float64
oracle, at the sizes and masks where they can go wrong.

Tolerances, from the formats and the FP32 steps (u = 2^-24, half a step at 1):

  * expert ids are equal, whatever lies how close.
  * weights: an exponential is off by 4 u and by u |argument| from rounding the
    difference of two logits; numerator and denominator each, a sum of up to
    1024 of them in pieces (a lane adds 32 in turn, then five steps), two
    divisions and the scale: u (2 range + 64).
  * bf16 outputs: with the FP32 value known to +-delta, the result lies between
    the roundings of value - delta and value + delta.
  * a norm's FP32 chain: below 2^-18 of the result (a sum of H squares in pieces,
    at most 16 a thread in turn and two five-step butterflies, a reciprocal
    square root of 2 units and four more operations). A gate's function adds
    8 u of its value, the two scalings and the addition 3 u of their terms.
  * a product's FP32 sum of K exact products in steps of 16 on the tensor cores:
    each step aligns 17 terms to the largest magnitude seen, at most 17 * u of
    the sum S of magnitudes, K / 16 steps (+ one for the bias): u S (1.1 K + 17).
    Activations have slopes below 1.13 and add 2^-20 of |value| of their own
    (GELU's sum cancels: 2^-20 of its argument), the residual u of both terms.
"""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import tensor_to_f64
from oracle import block as ref
from test_gpu_prompt import NORM_EPS32, assert_bf16, assert_mxfp8, bf16, dev, on, rng  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF = float("inf")


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------

def check_route(dev, logits, k, bias=None, rows=slice(None), **kw):  # noqa: F811
    """logits: a torch tensor on the CPU (its values decide); `rows` are compared."""
    from sparse_expert_gemv_gb300 import route_experts
    b = None if bias is None else torch.from_numpy(np.asarray(bias, dtype=np.float32)).to(dev)
    ids, w = route_experts(logits.to(dev), k, bias=b, **kw)
    ids, w = ids[rows], w[rows]
    z = logits[rows].double().numpy()
    want_ids, want_w = ref.route_experts(z, k, bias=None if bias is None else np.float32(bias), **kw)
    got = ids.cpu().numpy()
    assert np.array_equal(got, want_ids), np.flatnonzero((got != want_ids).any(1))[:5]
    fin = np.where(np.isfinite(z), z, 0.0)
    span = np.abs(fin).max(1, keepdims=True) * 2 if z.size else 0.0
    w = w.cpu().numpy().astype(np.float64)
    # (values below FP32's normal range round in steps of 2^-149)
    assert (np.abs(w - want_w) <= U * (2 * span + 64) * want_w + 2.0 ** -148).all()
    return ids, w


def logits_of(T, E, dtype, seed, masked=0, padded=0):
    r = rng(seed, T, E)
    z = r.standard_normal((T, E)) * (1 + r.random((T, 1))) + 0.5 * r.standard_normal(E)
    z[:, r.permutation(E)[:masked]] = -INF
    z[T - padded:] = -INF
    return torch.from_numpy(z.astype(np.float32)).to(dtype)


ROUTES = [
    # T, E, k, groups, top, group score
    (1, 1, 1, 1, 1, "max"), (3, 8, 8, 1, 1, "max"), (1, 256, 8, 8, 4, "top2"), (5, 33, 4, 1, 1, "max"),
    (65, 60, 6, 4, 2, "max"), (9, 60, 4, 4, 3, "top2"), (130, 128, 8, 1, 1, "max"),
    (77, 160, 6, 8, 3, "max"), (31, 160, 6, 8, 3, "top2"), (300, 256, 8, 8, 4, "top2"),
    (40, 256, 32, 32, 8, "top2"), (17, 257, 5, 1, 1, "max"), (6, 1000, 32, 25, 3, "top2"),
    (7, 1024, 10, 16, 2, "max"), (12, 1024, 8, 32, 1, "top2"), (4, 24, 3, 24, 5, "top2"),
    (11, 512, 8, 8, 8, "top2"), (21, 64, 1, 2, 1, "max"), (8, 128, 7, 16, 5, "top2")]


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,top,group_score", ROUTES)
def test_route(dev, T, E, k, groups, top, group_score, score, bias):  # noqa: F811
    for dtype in (torch.float32, torch.bfloat16):
        b = rng(1, E).standard_normal(E) * (0.1 if score == "sigmoid" else 2 / E) if bias else None
        check_route(dev, logits_of(T, E, dtype, 2), k, b, score=score, groups=groups, top_groups=top,
                    group_score=group_score, renormalize=E % 2 == 0, scale=2.5)


PACKED = [
    # E, k, groups, top: several tokens a warp (from 4096 on)
    (64, 6, 1, 1), (64, 8, 2, 1), (128, 8, 1, 1), (128, 5, 4, 2), (128, 8, 2, 1), (256, 8, 1, 1),
    (256, 8, 8, 4), (256, 1, 4, 3), (64, 2, 2, 2)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,top", PACKED)
def test_route_many_tokens(dev, E, k, groups, top, score):  # noqa: F811
    # ordinary rows, ties, masked experts, far and infinite logits, NaN, near ties; an
    # odd number of tokens, the last ones padding
    T = 4103
    r = rng(14, E)
    z = logits_of(T, E, torch.float32, 15, masked=3, padded=9).numpy()
    z[:60] = r.integers(0, 3, (60, E))
    base = np.float32(1 + 3 * r.random((60, 1)))
    z[60:120] = base + r.integers(-4, 5, (60, E)) * np.spacing(base)
    z[120:150] *= 40
    z[150:170] = np.where(r.random((20, E)) < 0.9, -INF, z[150:170])
    z[170, :], z[171, 5], z[172, :], z[173, 7:9], z[174, 3] = np.nan, np.nan, INF, INF, INF
    z[175:178] = 0.0
    z[178:182] = -70 - r.random((4, E))
    z[182, ::2] = -0.0
    z[182, 1::2] = 0.0
    rows = np.concatenate([np.arange(183), r.choice(T, 60), np.arange(T - 12, T)])
    for dtype in (torch.float32, torch.bfloat16):
        for bias in (None, np.round(r.standard_normal(E) * 100) / 1000, 3 * r.standard_normal(E)):
            for group_score in ("max", "top2") if groups > 1 else ("max",):
                check_route(dev, torch.from_numpy(z).to(dtype), k, bias, rows, score=score, groups=groups,
                            top_groups=top, group_score=group_score, renormalize=k != 5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_route_masked_and_padded_rows(dev, score, group_score):  # noqa: F811
    # so many experts off that slots stay empty; rows of which nothing is left
    for masked in (3, 36, 38, 40):
        for bias in (None, rng(3).standard_normal(40) * 0.05):
            z = logits_of(23, 40, torch.float32, 4, masked, padded=6)
            ids, w = check_route(dev, z, 4, bias, score=score, groups=8, top_groups=3,
                                 group_score=group_score)
            assert ids[17:].eq(-1).all() and (w[17:] == 0).all()


def test_route_switched_off_by_the_bias(dev):  # noqa: F811
    bias = rng(5).standard_normal(32) * 0.1
    bias[[0, 7, 8, 9, 31]] = -INF
    bias[12] = np.nan
    bias[20] = INF                        # always chosen, first
    for group_score in ("max", "top2"):
        ids, _ = check_route(dev, logits_of(50, 32, torch.float32, 6), 5, bias, score="sigmoid",
                             groups=4, top_groups=2, group_score=group_score)
        assert ids[:, 0].eq(20).all()
    check_route(dev, logits_of(50, 32, torch.float32, 6), 5, bias, score="softmax", renormalize=False)


def test_route_nan_and_infinite_logits(dev):  # noqa: F811
    z = logits_of(8, 48, torch.float32, 7)
    z[0, 5], z[1, :], z[2, 9], z[3, 10:13], z[4, :] = float("nan"), float("nan"), INF, INF, INF
    z[5, ::2], z[6, 1:] = -INF, -INF
    for dtype in (torch.float32, torch.bfloat16):
        for score in ("softmax", "sigmoid"):
            for bias in (None, rng(8).standard_normal(48) * 0.02):
                check_route(dev, z.to(dtype), 4, bias, score=score)
                check_route(dev, z.to(dtype), 4, bias, score=score, groups=6, top_groups=2,
                            group_score="top2", renormalize=False)


@pytest.mark.parametrize("E,groups,top", [(64, 1, 1), (64, 8, 3), (160, 8, 2), (256, 8, 4), (1024, 16, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties(dev, E, groups, top, score):  # noqa: F811
    # whole numbers, few values, zeros: the lower index wins, of groups too
    r = rng(9, E)
    for hi in (1, 2, 5):
        z = torch.from_numpy(r.integers(0, hi, (40, E)).astype(np.float32))
        for bias in (None, np.zeros(E), r.integers(0, 3, E) / 4):
            for group_score in ("max", "top2"):
                for dtype in (torch.float32, torch.bfloat16):
                    check_route(dev, z.to(dtype), 8, bias, score=score, groups=groups, top_groups=top,
                                group_score=group_score)


@pytest.mark.parametrize("groups,top", [(1, 1), (8, 3)])
def test_route_scores_too_close_for_fp32(dev, groups, top):  # noqa: F811
    # logits a few FP32 steps apart, and biases that make up for their scores:
    # differences of 1e-12 to 1e-7 decide
    E, T = 128, 64
    r = rng(10)
    base = np.float32(1 + 3 * r.random((T, 1)))
    z = (base + r.integers(-4, 5, (T, E)) * np.spacing(base)).astype(np.float32)
    check_route(dev, torch.from_numpy(z), 8, None, score="softmax", groups=groups, top_groups=top)
    for score in ("sigmoid", "softmax"):
        check_route(dev, torch.from_numpy(z), 8, None, score=score, groups=groups, top_groups=top,
                    group_score="top2")
        for bias in (np.zeros(E), r.integers(-1, 2, E) * 2.0 ** -26):
            for group_score in ("max", "top2"):
                check_route(dev, torch.from_numpy(z), 8, bias, score=score, groups=groups,
                            top_groups=top, group_score=group_score)
    z = np.float32(r.standard_normal((1, E)) * 2)
    bias = np.float32(1 - ref.sigmoid(z[0]))
    check_route(dev, torch.from_numpy(np.repeat(z, T, 0)), 8, bias, score="sigmoid", groups=groups,
                top_groups=top, group_score="top2")


def test_route_far_logits(dev):  # noqa: F811
    # sigmoids that are all one or all zero in FP32: logits still tell experts apart
    z = torch.from_numpy(np.float32(30 + 5 * rng(11).random((9, 64))))
    check_route(dev, z, 6, score="sigmoid")
    check_route(dev, -z, 6, score="sigmoid", renormalize=False)
    check_route(dev, 2 * z, 6, score="softmax")


def test_route_into_buffers_and_none(dev):  # noqa: F811
    from sparse_expert_gemv_gb300 import route_experts
    z = logits_of(10, 64, torch.float32, 12).to(dev)
    ids, w = route_experts(z, 4)
    out = (torch.full((10, 4), 7, dtype=torch.int32, device=dev), torch.zeros(10, 4, device=dev))
    got = route_experts(z, 4, ids=out[0], w=out[1])
    assert got[0] is out[0] or got[0].data_ptr() == out[0].data_ptr()
    assert torch.equal(out[0], ids) and torch.equal(out[1], w)
    empty = route_experts(z[:0], 4)
    assert empty[0].shape == (0, 4) and empty[1].shape == (0, 4)


@pytest.mark.parametrize("E", [30, 61, 127, 250])
def test_route_rows_off_the_vector_alignment(dev, E):  # noqa: F811
    flat = torch.zeros(33 * E + 1)
    z = flat[1:].view(33, E)
    z.copy_(logits_of(33, E, torch.float32, 13))
    for dtype in (torch.float32, torch.bfloat16):
        from sparse_expert_gemv_gb300 import route_experts
        on_dev = flat.to(dtype).to(dev)[1:].view(33, E)
        ids, _ = route_experts(on_dev, 6, score="sigmoid")
        want, _ = ref.route_experts(on_dev.double().cpu().numpy(), 6, score="sigmoid")
        assert np.array_equal(ids.cpu().numpy(), want)


# ---------------------------------------------------------------------------
# norms around a block's end
# ---------------------------------------------------------------------------

class Norms:
    def __init__(self, T, H, post=True, gate=None, seed=20):
        r = rng(seed, T, H)
        self.x = oracle.bf16_rne(r.standard_normal((T, H)) * np.exp2(r.integers(-2, 3, (T, 1))))
        self.res = oracle.bf16_rne(3 * r.standard_normal((T, H)))
        self.res[:, ::7] *= 64
        self.post = oracle.bf16_rne(0.5 + 0.2 * r.standard_normal(H)) if post else None
        self.pre = oracle.bf16_rne(1 + 0.2 * r.standard_normal(H))
        shape = {None: None, "channel": (H,), "row": (T, 1), "full": (T, H)}[gate]
        self.gate = None if shape is None else oracle.bf16_rne(0.5 + r.standard_normal(shape))

    def args(self, dev):  # noqa: F811
        return [None if a is None else bf16(a, dev) for a in (self.x, self.res, self.post, self.pre)]

    def check(self, got, *, gate_fn=None, scale=1.0, residual_scale=1.0, eps=1e-6, unit_offset=False):
        t, p = ref.norm_add(self.x, self.res, self.post, self.gate, gate_fn, np.float32(scale),
                            np.float32(residual_scale), eps, unit_offset)
        d = (NORM_EPS32 + 8 * U) * np.abs(p) + 3 * U * (np.abs(p) + np.abs(self.res * residual_scale))
        assert_bf16(got.sum, t, d, "sum")
        # the norm is that of the stream as it is kept
        s = tensor_to_f64(got.sum)
        n = ref.norm(s, self.pre, eps, 1.0 if unit_offset else 0.0)
        if got.y is not None:
            assert_bf16(got.y, n, NORM_EPS32 * np.abs(n), "y")
        if got.codes is not None:
            assert_mxfp8(got.codes, got.scales, n, NORM_EPS32 * np.abs(n), "MXFP8")


@pytest.mark.parametrize("gate,gate_fn", [(None, None), ("channel", None), ("row", "sigmoid"),
                                          ("full", "tanh"), ("row", None), ("channel", "sigmoid"),
                                          ("full", None), ("row", "tanh")])
@pytest.mark.parametrize("T,H,post", [
    (1, 32, True), (3, 64, False), (33, 256, True), (1, 2048, True), (5, 2080, True),
    (2, 7168, True), (3, 8224, False), (2, 16384, True), (2100, 1056, True)])
def test_norms(dev, T, H, post, gate, gate_fn):  # noqa: F811
    from sparse_expert_gemv_gb300 import norm_add_norm
    c = Norms(T, H, post, gate)
    kw = dict(gate_fn=gate_fn, scale=0.6, residual_scale=1.25 if T % 2 else 1.0, eps=1e-5)
    g = None if c.gate is None else bf16(c.gate, dev)
    c.check(norm_add_norm(*c.args(dev), gate=g, mxfp8=True, **kw), **kw)


@pytest.mark.parametrize("gate", [None, "channel", "row", "full"])
@pytest.mark.parametrize("T,H", [(1, 1), (2, 7), (3, 100), (2, 1032), (2, 4099), (1, 9999), (1, 16383),
                                 (2500, 130)])
def test_norms_of_odd_rows(dev, T, H, gate):  # noqa: F811
    from sparse_expert_gemv_gb300 import norm_add_norm
    c = Norms(T, H, True, gate, seed=21)
    g = None if c.gate is None else bf16(c.gate, dev)
    c.check(norm_add_norm(*c.args(dev), gate=g, unit_offset=True), unit_offset=True)


@pytest.mark.parametrize("which", range(5))
def test_norms_unaligned_rows_take_the_narrow_form(dev, which):  # noqa: F811
    from sparse_expert_gemv_gb300 import norm_add_norm
    c = Norms(3, 64, True, "full", seed=22)
    args = c.args(dev) + [bf16(c.gate, dev)]
    flat = torch.zeros(args[which].numel() + 1, dtype=torch.bfloat16, device=dev)
    flat[1:] = args[which].reshape(-1)
    args[which] = flat[1:].view(args[which].shape)
    c.check(norm_add_norm(*args[:4], gate=args[4], gate_fn="sigmoid", mxfp8=True), gate_fn="sigmoid")


def test_norms_in_place_alone_and_without_the_second_norm(dev):  # noqa: F811
    from sparse_expert_gemv_gb300 import norm_add_norm
    c = Norms(9, 512, True, "row", seed=23)
    x, res, post, pre = c.args(dev)
    g = bf16(c.gate, dev)
    both = norm_add_norm(x, res, post, pre, gate=g, mxfp8=True)
    stream = norm_add_norm(x, res, post, gate=g)
    assert stream.y is None and stream.codes is None and torch.equal(stream.sum, both.sum)
    for buf in ("x", "res"):
        a = {"x": x.clone(), "res": res.clone()}
        got = norm_add_norm(a["x"], a["res"], post, pre, gate=g, bf16=False, mxfp8=True, sum=a[buf])
        assert got.y is None and got.sum.data_ptr() == a[buf].data_ptr()
        for u, v in [(got.sum, both.sum), (got.codes, both.codes), (got.scales, both.scales)]:
            assert torch.equal(u, v)
    empty = norm_add_norm(x[:0], res[:0], post, pre, gate=g[:0], mxfp8=True)
    assert empty.sum.shape == (0, 512) and empty.scales.shape == (0, 16)


def test_norms_zero_rows_and_non_finite_values(dev):  # noqa: F811
    from sparse_expert_gemv_gb300 import norm_add_norm
    H = 96
    x = torch.zeros(4, H, dtype=torch.bfloat16, device=dev)
    res = torch.zeros_like(x)
    x[1, 40], res[2, 70], x[3, 3] = float("nan"), float("inf"), float("inf")
    w = torch.ones(H, dtype=torch.bfloat16, device=dev)
    n = norm_add_norm(x, res, w, w, mxfp8=True)
    assert n.sum[0].eq(0).all() and n.y[0].eq(0).all() and n.scales[0].eq(127).all()
    assert n.sum[1].isnan().all() and n.y[1].isnan().all() and n.scales[1].eq(255).all()
    # an infinity makes the norm infinite: zeros, and NaN where it stood
    assert n.sum[2, 70].isinf() and n.y[2, :70].eq(0).all() and n.y[2, 70].isnan()
    assert n.scales[2, 2] == 255 and n.codes[2, 64:].bitwise_and(0x7F).eq(0x7F).all()
    assert n.sum[3, 3].isnan() and n.sum[3, :3].eq(0).all() and n.y[3].isnan().all()


# ---------------------------------------------------------------------------
# dense products
# ---------------------------------------------------------------------------

class Dense:
    def __init__(self, R, K, N, bias=False, act=None, residual=False, seed=30):
        r = rng(seed, R, K, N)
        self.M = N // 2 if act == "silu_mul" else N
        self.x = oracle.bf16_rne(r.standard_normal((R, K)) * np.exp2(r.integers(-2, 3, (R, 1))))
        self.w = oracle.bf16_rne(r.standard_normal((N, K)) * K ** -0.5)
        self.b = oracle.bf16_rne(r.standard_normal(N)) if bias else None
        self.res = oracle.bf16_rne(3 * r.standard_normal((R, self.M))) if residual else None
        self.act = act

    def handle(self, dev):  # noqa: F811
        from sparse_expert_gemv_gb300 import DenseProduct
        return DenseProduct(bf16(self.w, dev), None if self.b is None else bf16(self.b, dev),
                            activation=self.act)

    def run(self, dev, p=None, **kw):  # noqa: F811
        p = p or self.handle(dev)
        return p(bf16(self.x, dev), None if self.res is None else bf16(self.res, dev), **kw)

    def check(self, got):
        out, Y, S = ref.dense(self.x, self.w, self.b, self.act, self.res)
        K = self.w.shape[1]
        dY = U * S * (1.1 * K + 17)
        if self.act == "silu_mul":
            I = self.M
            g, u, dg, du = np.abs(Y[:, :I]), np.abs(Y[:, I:]), dY[:, :I], dY[:, I:]
            d = 1.13 * dg * (u + du) + (g + dg) * du + 2.0 ** -20 * (1 + g) * np.abs(g * u)
        else:
            d = 1.13 * dY + 2.0 ** -20 * np.abs(Y)
        if self.res is not None:
            d = d + U * (np.abs(out) + np.abs(self.res))
        assert got.shape == out.shape
        if got.dtype == torch.float32:
            assert (np.abs(got.double().cpu().numpy() - out) <= d + U * np.abs(out)).all()
        else:
            assert_bf16(got, out, d, f"dense {self.act}")


ACTS = [None, "relu", "silu", "gelu", "gelu_tanh", "silu_mul"]
DENSE = [
    # R, K, N
    (1, 8, 1), (1, 2048, 128), (2, 64, 2), (3, 72, 60), (7, 256, 130), (8, 2048, 128), (16, 1024, 384),
    (17, 200, 128), (31, 4096, 96), (33, 64, 514), (64, 520, 256), (65, 128, 1000), (100, 264, 258),
    (127, 64, 64), (129, 328, 640), (256, 512, 512), (300, 1032, 776), (513, 96, 130), (1000, 80, 1030),
    (1, 7168, 256), (5, 7168, 34), (12, 8, 4100), (2000, 192, 2600), (3001, 136, 1544), (700, 448, 5000),
    (4100, 64, 514)]


@pytest.mark.parametrize("R,K,N", DENSE)
def test_dense(dev, R, K, N):  # noqa: F811
    for i, act in enumerate(ACTS):
        if act == "silu_mul" and N % 2:
            continue
        c = Dense(R, K, N, bias=i % 2 == 1, act=act, residual=i % 3 != 0)
        p = c.handle(dev)
        c.check(c.run(dev, p))
        c.check(c.run(dev, p, float32=True))
        assert p.get_error() == 0


def test_dense_in_place_residual_and_buffers(dev):  # noqa: F811
    c = Dense(40, 256, 384, True, "gelu", True)
    p = c.handle(dev)
    want = c.run(dev, p)
    x, res = bf16(c.x, dev), bf16(c.res, dev)
    got = p(x, res, out=res)
    assert got.data_ptr() == res.data_ptr() and torch.equal(res, want)
    wide = torch.full((42, 384), 7.0, dtype=torch.bfloat16, device=dev)
    p(x, bf16(c.res, dev), out=wide[1:41])
    assert torch.equal(wide[1:41], want) and wide[0].eq(7).all() and wide[41].eq(7).all()
    assert p(x[:0]).shape == (0, 384)


@pytest.mark.parametrize("N", [64, 61])
@pytest.mark.parametrize("float32", [False, True])
def test_dense_outputs_off_the_vector_alignment(dev, N, float32):  # noqa: F811
    c = Dense(37, 128, N, True, None, True)
    p = c.handle(dev)
    want = c.run(dev, p, float32=float32)
    c.check(want)
    for skew_res, skew_out in ((1, 0), (0, 1), (1, 1)):
        res = torch.zeros(37 * N + 8, dtype=torch.bfloat16, device=dev)
        out = torch.full((37 * N + 8,), 7.0, dtype=want.dtype, device=dev)
        rv, ov = res[skew_res:][:37 * N].view(37, N), out[skew_out:][:37 * N].view(37, N)
        rv.copy_(bf16(c.res, dev))
        p(bf16(c.x, dev), rv, out=ov, float32=float32)
        assert torch.equal(ov, want)
        assert out[:skew_out].eq(7).all() and out[skew_out + 37 * N:].eq(7).all()


@pytest.mark.parametrize("R,K,N,act", [(1301, 264, 2120, None), (2900, 136, 1208, "gelu_tanh"),
                                       (1301, 264, 4240, "silu_mul"), (2900, 136, 2288, "silu_mul"),
                                       (9000, 64, 8, None), (9000, 64, 16, "silu_mul")])
def test_dense_of_many_rows_in_place_and_off_the_alignment(dev, R, K, N, act):  # noqa: F811
    import ctypes
    from sparse_expert_gemv_gb300._lib import MoEDenseConfig, MoEDensePlan, lib
    plan = MoEDensePlan()
    config = MoEDenseConfig(N, K, 5 if act == "silu_mul" else 4 if act else 0)
    assert lib.moe_dense_plan(ctypes.byref(config), R, 0, 152, ctypes.byref(plan)) == 0 and not plan.split
    c = Dense(R, K, N, True, act, True, seed=35)
    p, M = c.handle(dev), c.M
    x, res = bf16(c.x, dev), bf16(c.res, dev)
    want = p(x, res)
    c.check(want)
    for skew_res, skew_out in ((0, 0), (0, 8), (8, 0), (1, 0), (0, 1), (3, 5)):
        r = torch.full((R * M + 16,), 7.0, dtype=torch.bfloat16, device=dev)
        out = torch.full((R * M + 16,), 7.0, dtype=torch.bfloat16, device=dev)
        rv, ov = r[skew_res:][:R * M].view(R, M), out[skew_out:][:R * M].view(R, M)
        rv.copy_(res)
        p(x, rv, out=ov)
        assert torch.equal(ov, want) and torch.equal(rv, res)
        assert out[:skew_out].eq(7).all() and out[skew_out + R * M:].eq(7).all()
        p(x, rv, out=rv)
        assert torch.equal(rv, want)
        assert r[:skew_res].eq(7).all() and r[skew_res + R * M:].eq(7).all()
    p(x[:-3], res[:-3], out=out[:(R - 3) * M].view(R - 3, M))
    assert torch.equal(out[:(R - 3) * M].view(R - 3, M), want[:-3])
    assert p.get_error() == 0


@pytest.mark.parametrize("act", [None, "silu_mul"])
@pytest.mark.parametrize("R,K,N", [(2, 64, 128), (5, 2048, 384), (40, 1024, 4096), (600, 512, 2048),
                                   (3000, 256, 2048)])
def test_dense_winds_down_when_its_waits_give_up(dev, R, K, N, act):  # noqa: F811
    # failure detection without a fault: the MMAs' bounded wait runs out (for an
    # arrival that nothing makes), and then every other role's; the launch ends, the
    # handle reports it once, and the next runs are right
    from sparse_expert_gemv_gb300 import MOE_DEVICE_TIMEOUT
    c = Dense(R, K, N, True, act, True, seed=33)
    p = c.handle(dev)
    want = c.run(dev, p)
    assert p.get_error() == 0
    for _ in range(3):
        p.arm_timeout()
        p(bf16(c.x[:0], dev))                     # launches nothing
        assert p.get_error() == 0
        c.run(dev, p)
        assert p.get_error() == MOE_DEVICE_TIMEOUT
        assert p.get_error() == 0
        assert torch.equal(c.run(dev, p), want)
        assert p.get_error() == 0


def test_dense_of_exact_sums(dev):  # noqa: F811
    # whole numbers: every sum is exact, so every bit is
    r = rng(31)
    for R, K, N in ((5, 640, 200), (200, 1536, 328), (700, 128, 512)):
        x, w = r.integers(-3, 4, (R, K)).astype(float), r.integers(-3, 4, (N, K)).astype(float)
        from sparse_expert_gemv_gb300 import DenseProduct
        got = DenseProduct(bf16(w, dev))(bf16(x, dev), float32=True)
        assert np.array_equal(got.double().cpu().numpy(), x @ w.T)


def test_dense_non_finite_values_stay_in_their_row_and_column(dev):  # noqa: F811
    from sparse_expert_gemv_gb300 import DenseProduct
    r = rng(32)
    R, K, N = 150, 256, 300
    x, w = bf16(r.standard_normal((R, K)), dev), bf16(r.standard_normal((N, K)), dev)
    x[3, 7], x[100, 0] = float("inf"), float("nan")
    w[11, 9] = float("nan")
    got = DenseProduct(w)(x, float32=True)
    bad = torch.zeros(R, N, dtype=torch.bool, device=dev)
    bad[3], bad[100], bad[:, 11] = True, True, True
    assert torch.equal(~got.isfinite(), bad)
    assert got[100].isnan().all() and got[:, 11].isnan().all()
    act = DenseProduct(w, activation="relu")(x)
    assert act[100].isnan().all() and act[3].isnan().sum() == 1


def test_dense_far_gates(dev):  # noqa: F811
    # one-hot weights: SiLU and GELU of values whose exponentials overflow
    from sparse_expert_gemv_gb300 import DenseProduct
    v = np.array([-200.0, -89.0, -88.0, -20.0, -1.0, -0.0, 1.0, 20.0, 89.0, 200.0, 3.0e38, -3.0e38])
    v = oracle.bf16_rne(v)
    n = len(v)
    x = np.zeros((n, 16))
    x[:, 0] = v
    x[:, 1] = 1.0
    w = np.zeros((2, 16))
    w[0, 0], w[1, 1] = 1.0, 1.0
    for act in ("silu", "gelu", "gelu_tanh"):
        got = DenseProduct(bf16(w[:1], dev), activation=act)(bf16(x, dev), float32=True)
        with np.errstate(over="ignore"):
            want = ref.activate(v[:, None], act)
        assert got.isfinite().all()
        err, m = np.abs(got.double().cpu().numpy() - want), np.abs(v[:, None])
        # SiLU keeps its relative accuracy, GELU that of its cancelling sum
        assert (err <= (2.0 ** -20 * (1 + np.minimum(m, 100)) * np.abs(want) + 2.0 ** -126
                        if act == "silu" else 2.0 ** -20 * np.where(m > 50, np.abs(want), m))).all(), act
    got = DenseProduct(bf16(w, dev), activation="silu_mul")(bf16(x, dev), float32=True)
    err, want = np.abs(got.double().cpu().numpy()[:, 0] - v * ref.sigmoid(v)), np.abs(v * ref.sigmoid(v))
    assert (err <= 2.0 ** -20 * (1 + np.minimum(np.abs(v), 100)) * want + 2.0 ** -126).all()


# ---------------------------------------------------------------------------
# buffers and streams
# ---------------------------------------------------------------------------

def calls(dev):  # noqa: F811
    """Each operator as a call of its keyword arguments, and its buffers' names."""
    from sparse_expert_gemv_gb300 import norm_add_norm, route_experts
    z = logits_of(64, 32, torch.float32, 50).to(dev)
    n = Norms(64, 512, True, "row", seed=51)
    args, gate = n.args(dev), bf16(n.gate, dev)
    d = Dense(64, 512, 384, True, "silu", True)
    p, few = d.handle(dev), Dense(3, 512, 384, True, "silu", True)
    x, res, fx, fres = (bf16(a, dev) for a in (d.x, d.res, few.x, few.res))
    return {"route": (lambda **kw: route_experts(z, 4, **kw), ["ids", "w"]),
            "norms": (lambda **kw: norm_add_norm(*args, gate=gate, mxfp8=True, **kw),
                      ["sum", "y", "codes", "scales"]),
            "dense": (lambda **kw: p(x, res, **kw), ["out"]),
            "dense few": (lambda **kw: p(fx, fres, **kw), ["out"])}


def listed(out):
    return [out] if isinstance(out, torch.Tensor) else list(out)


@pytest.mark.parametrize("op", ["route", "norms", "dense", "dense few"])
def test_outputs_on_a_given_stream_are_of_its_memory(dev, op):  # noqa: F811
    call, _ = calls(dev)[op]
    want = [t.clone() for t in listed(call())]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    # blocks of the outputs' sizes that the current stream has just let go of, with
    # work on them still queued there
    freed = [torch.full_like(t, 3) for t in want for _ in range(4)]
    blocks = {f.data_ptr() for f in freed}
    kept = [torch.empty_like(f) for f in freed]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    for k, f in zip(kept, freed):
        k.copy_(f)
    del freed, f
    got = listed(call(stream=side))
    assert not blocks & {t.data_ptr() for t in got}
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    for k in kept:
        assert k.eq(3).all()


def test_wrong_buffers_and_streams_are_refused(dev):  # noqa: F811
    from test_prompt_devices_cpu import fake
    for call, names in calls(dev).values():
        want = listed(call())
        for name, t in zip(names, want):
            with pytest.raises(ValueError, match=f"{name}: expected a tensor on cuda:0, got one on cuda:1"):
                call(**{name: fake(t.shape, t.dtype, 1)})
            with pytest.raises(ValueError, match=f"{name}: expected shape"):
                call(**{name: t[:-1]})
            with pytest.raises(TypeError, match=f"{name}: expected torch"):
                call(**{name: t.to(torch.float64)})
        with pytest.raises(TypeError, match="stream must be"):
            call(stream=torch.cuda.Stream().cuda_stream)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

class Block:
    """One block of a small model with a shared expert, on the framework's calls."""

    def __init__(self, dev, T, fmt="mxfp8"):  # noqa: F811
        import workloads as wl
        from sparse_expert_gemv_gb300 import DenseProduct, MoEDecode
        E, k, H, I = 16, 4, 256, 128
        self.k = k
        w = wl.Workload(92, "block", E, k, H, I, max(T, 1), 0.05)
        experts = wl.make_experts(w, 40, range(E), fmt=fmt)
        stack = [torch.from_numpy(np.stack([experts[e][i] for e in range(E)])).to(dev) for i in range(4)]
        self.layer = MoEDecode(*stack, k=k, max_T=max(T, 1), fmt=fmt)
        r = rng(41, T)
        self.x, self.res = bf16(r.standard_normal((T, H)), dev), bf16(2 * r.standard_normal((T, H)), dev)
        self.post, self.pre = (bf16(1 + 0.1 * r.standard_normal(H), dev) for _ in range(2))
        self.bias = torch.from_numpy(np.float32(0.1 * r.standard_normal(E))).to(dev)
        self.wr, self.wgu, self.wd = (bf16(r.standard_normal(s) * s[1] ** -0.5, dev)
                                      for s in ((E, H), (2 * I, H), (H, I)))
        self.router = DenseProduct(self.wr)
        self.gate_up = DenseProduct(self.wgu, activation="silu_mul")
        self.down = DenseProduct(self.wd)

    def __call__(self):
        from sparse_expert_gemv_gb300 import norm_add_norm, route_experts
        n = norm_add_norm(self.x, self.res, self.post, self.pre, mxfp8=True)
        logits = self.router(n.y, float32=True)
        ids, w = route_experts(logits, self.k, score="sigmoid", bias=self.bias, groups=4, top_groups=2,
                               group_score="top2", scale=1.5)
        shared = self.down(self.gate_up(n.y), n.sum)
        out = self.layer.prompt(n.codes, n.scales, ids, w, residual=shared)
        return [*n, logits, ids, w, shared, out]


@pytest.mark.parametrize("T", [1, 5, 33, 200])
def test_a_block(dev, T):  # noqa: F811
    b = Block(dev, T)
    s, y, codes, scales, logits, ids, w, shared, out = b()
    f = tensor_to_f64
    x, res, post, pre = map(f, (b.x, b.res, b.post, b.pre))
    t, p = ref.norm_add(x, res, post)
    assert_bf16(s, t, NORM_EPS32 * np.abs(p) + 3 * U * (np.abs(p) + np.abs(res)), "sum")
    # each operator against its definition on what the ones before it gave
    want, _, S = ref.dense(f(y), f(b.wr))
    assert (np.abs(f(logits) - want) <= U * S * (1.1 * 256 + 17)).all()
    want_ids, want_w = ref.route_experts(f(logits), b.k, "sigmoid", b.bias.cpu().numpy(), 4, 2, "top2",
                                         scale=1.5)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert (np.abs(f(w) - want_w) <= U * 100 * want_w).all()
    # h rounded to bf16 once (2^-8), then a sum of 128 such
    h, _, _ = ref.dense(f(y), f(b.wgu), activation="silu_mul")
    want, _, _ = ref.dense(h, f(b.wd), residual=f(s))
    err = np.abs(f(shared) - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * (np.abs(h) @ np.abs(f(b.wd)).T)).all()
    routed = b.layer.prompt(codes, scales, ids, w)
    both = f(shared) + f(routed)
    assert (np.abs(f(out) - both) <= 2.0 ** -8 * (np.abs(both) + np.abs(f(routed)))).all()
    assert b.layer.get_error() == 0 and b.router.get_error() == 0


def test_a_block_replayed_and_on_another_stream(dev):  # noqa: F811
    b = Block(dev, 40)
    want = [t.clone() for t in b()]
    for got in (b(),):
        for u, v in zip(got, want):
            assert torch.equal(u, v)               # bit for bit, call after call
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = b()
    side.synchronize()
    for u, v in zip(got, want):
        assert torch.equal(u, v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = b()
    other = b.x.clone()
    b.x.neg_()
    g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(got[0], want[0])
    b.x.copy_(other)
    g.replay()
    torch.cuda.synchronize()
    for u, v in zip(got, want):
        assert torch.equal(u, v)
    assert b.router.get_error() == 0


def test_the_layers_router_takes_the_options(dev):  # noqa: F811
    from sparse_expert_gemv_gb300 import route_experts
    b = Block(dev, 30)
    z = logits_of(30, 16, torch.float32, 60).to(dev)
    plain = b.layer.route(z)
    want = ref.route_experts(z.double().cpu().numpy(), 4)
    assert np.array_equal(plain[0].cpu().numpy(), want[0])
    # the operator without options is the layer's own router
    same = route_experts(z, 4)
    assert torch.equal(same[0], plain[0]) and torch.allclose(same[1], plain[1], rtol=1e-6)
    kw = dict(score="sigmoid", bias=b.bias, groups=4, top_groups=2, group_score="top2", scale=1.5)
    for got, like in zip(b.layer.route(z.bfloat16(), **kw), route_experts(z.bfloat16(), 4, **kw)):
        assert torch.equal(got, like)
    ids = torch.empty(30, 4, dtype=torch.int32, device=dev)
    assert b.layer.route(z, ids=ids, **kw)[0].data_ptr() == ids.data_ptr()
    with pytest.raises(ValueError, match="expected 16 experts"):
        b.layer.route(z[:, :8].contiguous(), **kw)


def test_example_with_a_shared_expert(dev, capsys):  # noqa: F811
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "prompt_block.py")
    spec = importlib.util.spec_from_file_location("prompt_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    assert ex.main(["--tokens", "70", "--experts", "16", "--topk", "2", "--hidden", "256",
                    "--intermediate", "128", "--shared"]) > 0
    assert "shared expert" in capsys.readouterr().out
    b = Block(dev, 33)
    block = ex.SharedBlock(b.layer, b.post, b.pre, b.wr, b.bias, b.wgu, b.wd, groups=4, top_groups=2,
                           scale=1.5)
    assert torch.equal(block(b.x, b.res), b()[-1])


# ---------------------------------------------------------------------------
# one handle from several places, long tensors
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("R,K,N,act", [(5, 2048, 256, None), (40, 1024, 2048, "silu_mul"),
                                       (700, 512, 1024, "gelu"), (3000, 256, 2048, "silu_mul")])
def test_dense_on_two_streams_at_once(dev, R, K, N, act):  # noqa: F811
    # one handle, calls side by side on two streams and in two graphs replayed side by
    # side: calls share nothing but the weight
    c, d = Dense(R, K, N, True, act, True, seed=70), Dense(R, K, N, True, act, True, seed=71)
    p = c.handle(dev)
    d.w, d.b = c.w, c.b
    args = [(bf16(k.x, dev), bf16(k.res, dev)) for k in (c, d)]
    want = [p(*a) for a in args]
    c.check(want[0])
    outs = [[torch.empty_like(want[0]) for _ in range(20)] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for s, a, o in zip(streams, args, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for t in o:
                p(*a, out=t)
        graphs.append(g)
    for run in ("calls", "graphs"):
        for o in outs[0] + outs[1]:
            o.fill_(7)
        torch.cuda.synchronize()
        for i in range(20):
            for s, a, o, g in zip(streams, args, outs, graphs):
                with torch.cuda.stream(s):
                    if run == "calls":
                        p(*a, out=o[i])
                    elif i == 0:
                        g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(t, w) for t in o)
    assert p.get_error() == 0


def test_dense_offsets_past_32_bits(dev):  # noqa: F811
    from sparse_expert_gemv_gb300 import DenseProduct
    R, K, N = 1_100_003, 64, 2056
    g = torch.Generator(device=dev).manual_seed(72)
    x = torch.randn(R, K, device=dev, generator=g).bfloat16()
    w, b = torch.randn(N, K, device=dev, generator=g).bfloat16(), torch.randn(N, device=dev).bfloat16()
    res = torch.full((R, N), 0.5, dtype=torch.bfloat16, device=dev)
    rows = torch.tensor([0, 1_044_461, 1_044_500, R - 1], device=dev)
    p = DenseProduct(w, b)
    want = x[rows].double() @ w.double().T + b.double() + 0.5
    for float32 in (False, True):
        got = p(x, res, float32=float32)[rows].double()
        assert torch.allclose(got, want, rtol=1e-5 if float32 else 2.0 ** -8, atol=1e-4)
        del got
    assert p.get_error() == 0


def test_norms_and_routing_offsets_past_32_bits(dev):  # noqa: F811
    from sparse_expert_gemv_gb300 import norm_add_norm, route_experts
    T, H = 300_001, 7168
    g = torch.Generator(device=dev).manual_seed(73)
    x = torch.randn(T, H, device=dev, generator=g, dtype=torch.bfloat16)
    res = torch.randn(T, H, device=dev, generator=g, dtype=torch.bfloat16)
    w = (1 + 0.1 * torch.randn(H, device=dev, generator=g)).bfloat16()
    n = norm_add_norm(x, res, w, w, gate=x, gate_fn="sigmoid", mxfp8=True)
    rows = [0, 2 ** 31 // H, 2 ** 31 // H + 1, T - 1]
    few = norm_add_norm(x[rows], res[rows], w, w, gate=x[rows], gate_fn="sigmoid", mxfp8=True)
    for a, b in zip(n, few):
        assert torch.equal(a[rows], b)
    del n, x, res
    T, E = 8_400_007, 256
    z = torch.randn(T, E, device=dev, generator=g)
    bias = 0.1 * torch.randn(E, device=dev, generator=g)
    rows = [0, 2 ** 31 // E, 2 ** 31 // E + 1, T - 1]
    for kw in (dict(score="sigmoid", bias=bias, groups=8, top_groups=4, group_score="top2"), {}):
        ids, wt = route_experts(z, 8, **kw)
        few = route_experts(z[rows], 8, **kw)
        assert torch.equal(ids[rows], few[0]) and torch.allclose(wt[rows], few[1], rtol=1e-6)
