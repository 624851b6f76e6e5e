"""GPU parity of the prompt operators (include/moe_prompt.h) with the float64
oracle, at the sizes and masks where they can go wrong.

Tolerances, from the formats and the FP32 sums:

  * bf16 outputs: with the FP32 value known to +-delta, the result lies between
    the roundings of value - delta and value + delta.
  * the norm's FP32 chain: a sum of H squares in pieces (a thread adds at most
    16 in turn, then two five-step butterflies), a reciprocal square root of 2
    units and four more operations, each 2^-24 of its result: below 2^-18.
  * a product's FP32 sum of K exact products in steps of 32 on the tensor
    cores: each step aligns 33 terms to the largest magnitude seen, at most
    33 * 2^-24 of the sum S of magnitudes, K / 32 steps: K 2^-24 1.1 S (+ 2^-24 S).
  * SiLU(g) u: |SiLU'| < 1.1, |SiLU(g)| <= |g|, and 2^-20 for its own FP32
    steps (the exponential's error grows with its argument: 2^-23 (2 + |g|)).
  * MXFP8 outputs: with the value known to +-delta, the scale code lies between
    those of the smallest and the largest possible block maximum, and every
    code between the roundings of value - delta and value + delta.
"""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from gpu_util import tensor_to_f64
from oracle import prompt as ref

pytestmark = pytest.mark.gpu

NORM_EPS32 = 2.0 ** -18


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def rng(*seed):
    return np.random.default_rng(list(seed))


def bf16(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).to(dev)


def on(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def assert_bf16(got, want, extra, what):
    g = tensor_to_f64(got)
    assert g.shape == want.shape, what
    bad = ~((g >= oracle.bf16_rne(want - extra)) & (g <= oracle.bf16_rne(want + extra)))
    assert not bad.any(), f"{what}: {np.count_nonzero(bad)} of {bad.size} outside their interval"


def assert_mxfp8(codes, scales, v, delta, what):
    """codes, scales against float64 values v known to +-delta."""
    codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
    assert codes.shape == v.shape and scales.shape == (v.shape[0], v.shape[1] // 32), what
    lo = ref.mx_exponent(np.maximum(np.abs(v) - delta, 0.0))
    hi = ref.mx_exponent(np.abs(v) + delta)
    e = scales.astype(np.int64) - 127
    # a block that may be all zeros has exponent 0 by definition
    fine = ((e >= lo) & (e <= hi)) | ((e == 0) & (lo == 0))
    assert fine.all(), f"{what}: {np.count_nonzero(~fine)} scale codes"
    unit = -np.repeat(e, 32, axis=1)
    q = oracle.E4M3[codes]
    low, high = ref.e4m3_rne(np.ldexp(v - delta, unit)), ref.e4m3_rne(np.ldexp(v + delta, unit))
    bad = ~((q >= low) & (q <= high))
    assert not bad.any(), f"{what}: {np.count_nonzero(bad)} codes outside their interval"


# ---------------------------------------------------------------------------
# residual norm
# ---------------------------------------------------------------------------

def norm_case(T, H, seed, residual=True, loud=False):
    r = rng(seed, T, H)
    x = oracle.bf16_rne(r.standard_normal((T, H)))
    res = oracle.bf16_rne(3 * r.standard_normal((T, H))) if residual else None
    if loud and residual:
        res[:, ::7] *= 64
    w = oracle.bf16_rne(1 + 0.2 * r.standard_normal(H))
    return x, res, w


@pytest.mark.parametrize("T,H,residual,mx", [
    (1, 32, True, True), (3, 64, False, True), (2, 96, True, True), (33, 256, True, True),
    (1, 2048, True, True), (5, 2080, True, True), (2, 7168, False, True), (3, 8224, True, True),
    (2, 16384, True, True),
    (1, 1, True, False), (2, 7, False, False), (3, 100, True, False), (2, 1032, True, False),
    (2, 4099, True, False), (1, 9999, True, False), (1, 16383, False, False)])
def test_norm(dev, T, H, residual, mx):
    from sparse_expert_gemv_gb300 import add_rms_norm
    x, res, w = norm_case(T, H, 1, residual, loud=True)
    n = add_rms_norm(bf16(x, dev), bf16(w, dev), None if res is None else bf16(res, dev), eps=1e-5,
                     bf16=True, mxfp8=mx)
    s, want = ref.add_rms_norm(x, w, res, 1e-5)
    if residual:
        # an exact sum of two bf16 values, rounded once
        assert np.array_equal(tensor_to_f64(n.sum), s)
    else:
        assert n.sum is None
    assert_bf16(n.y, want, NORM_EPS32 * np.abs(want), "y")
    if mx:
        assert_mxfp8(n.codes, n.scales, want, NORM_EPS32 * np.abs(want), "MXFP8")
    else:
        assert n.codes is None and n.scales is None


@pytest.mark.parametrize("H", [64, 4096])
def test_norm_unaligned_rows_take_the_narrow_form(dev, H):
    from sparse_expert_gemv_gb300 import add_rms_norm
    T = 3
    x, res, w = norm_case(T, H, 2)
    flat = torch.zeros(T * H + 1, dtype=torch.bfloat16, device=dev)
    xv = flat[1:].view(T, H)
    xv.copy_(bf16(x, dev))
    a = add_rms_norm(xv, bf16(w, dev), bf16(res, dev), mxfp8=True)
    s, want = ref.add_rms_norm(x, w, res, 1e-6)
    assert np.array_equal(tensor_to_f64(a.sum), s)
    assert_bf16(a.y, want, NORM_EPS32 * np.abs(want), "y")
    assert_mxfp8(a.codes, a.scales, want, NORM_EPS32 * np.abs(want), "MXFP8")


def test_norm_in_place_sum_and_mxfp8_alone(dev):
    from sparse_expert_gemv_gb300 import add_rms_norm
    x, res, w = norm_case(9, 512, 3)
    xt, rt, wt = bf16(x, dev), bf16(res, dev), bf16(w, dev)
    both = add_rms_norm(xt, wt, rt, mxfp8=True)
    alone = add_rms_norm(xt, wt, rt, bf16=False, mxfp8=True, sum=rt)
    assert alone.y is None and alone.sum.data_ptr() == rt.data_ptr()
    for a, b in [(rt, both.sum), (alone.codes, both.codes), (alone.scales, both.scales)]:
        assert torch.equal(a, b)


def test_norm_zero_rows_and_non_finite_values(dev):
    from sparse_expert_gemv_gb300 import add_rms_norm
    H = 96
    x = torch.zeros(4, H, dtype=torch.bfloat16, device=dev)
    x[1, 40] = float("nan")
    x[2, 70] = float("inf")
    x[3] = 2.0 ** -130        # subnormal: its square is zero, eps decides
    w = torch.ones(H, dtype=torch.bfloat16, device=dev)
    n = add_rms_norm(x, w, mxfp8=True)
    assert torch.equal(n.y[0], torch.zeros_like(n.y[0]))
    assert n.codes[0].eq(0).all() and n.scales[0].eq(127).all()
    assert n.y[1].isnan().all()
    assert n.codes[1].bitwise_and(0x7F).eq(0x7F).all() and n.scales[1].eq(255).all()
    # an infinity makes the norm infinite: zeros, and NaN where it stood
    assert n.y[2, :70].eq(0).all() and n.y[2, 70].isnan()
    assert n.scales[2, :2].eq(127).all() and n.scales[2, 2] == 255
    assert n.codes[2, 64:].bitwise_and(0x7F).eq(0x7F).all()
    _, want = ref.add_rms_norm(np.full((1, H), 2.0 ** -130), np.ones(H))
    assert_mxfp8(n.codes[3:], n.scales[3:], want, NORM_EPS32 * np.abs(want), "subnormal row")


def test_norm_tiny_and_huge_scales(dev):
    # weights near bf16's ends: the scale code reaches 0, and its upper part
    from sparse_expert_gemv_gb300 import add_rms_norm
    H = 128
    x = oracle.bf16_rne(rng(4).standard_normal((2, H)))
    w = np.repeat([2.0 ** -126, 2.0 ** -123, 2.0 ** 126, 1.0], 32)
    n = add_rms_norm(bf16(x, dev), bf16(w, dev), mxfp8=True)
    _, want = ref.add_rms_norm(x, w)
    assert_mxfp8(n.codes, n.scales, want, NORM_EPS32 * np.abs(want) + 2.0 ** -149, "extremes")
    assert n.scales[:, 0].eq(0).all()


# ---------------------------------------------------------------------------
# grouping
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,k,E,bad", [
    (1, 1, 1, 0.0), (1, 8, 128, 0.0), (3, 2, 5, 0.3), (32, 8, 128, 0.0), (33, 4, 60, 0.2),
    (200, 8, 1024, 0.1), (257, 8, 8, 0.0), (1000, 6, 160, 0.05), (5000, 8, 256, 0.0),
    (40, 3, 7, 1.0), (20000, 6, 300, 0.1), (40000, 8, 128, 0.02)])
def test_group(dev, T, k, E, bad):
    from sparse_expert_gemv_gb300 import group_by_expert
    r = rng(5, T, k, E)
    # a few experts take most slots
    ids = np.minimum(r.integers(0, E, (T, k)), r.integers(0, E, (T, k))).astype(np.int32)
    out = r.random((T, k)) < bad
    ids[out] = r.choice([-1, E, -2 ** 31, 2 ** 31 - 1], out.sum())
    got = group_by_expert(on(ids, dev), E)
    for g, want, name in zip(got, ref.group(ids, E), ("offsets", "rows", "slots")):
        assert np.array_equal(g.cpu().numpy(), want), name


def test_group_one_expert_and_none(dev):
    from sparse_expert_gemv_gb300 import group_by_expert
    ids = torch.full((700, 4), 3, dtype=torch.int32, device=dev)
    off, rows, slots = group_by_expert(ids, 9)
    assert off.tolist() == [0, 0, 0, 0] + [2800] * 6
    assert torch.equal(slots.view(-1), torch.arange(2800, dtype=torch.int32, device=dev))
    off, rows, slots = group_by_expert(ids[:0], 9)
    assert off.tolist() == [0] * 10 and rows.numel() == 0 and slots.shape == (0, 4)


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

class Products:
    """Seeded weights and grouped rows with the given group sizes."""

    def __init__(self, dev, fmt, N, K, counts, seed, gather=False, sigma=0.05, lead=0, tail=0):
        r = rng(6, seed, N, K)
        E = len(counts)
        enc = wl.FORMATS[fmt]
        ws = [enc((sigma * r.standard_normal((N, K))).astype(np.float32)) for _ in range(E)]
        self.w, self.ws = np.stack([c for c, _ in ws]), np.stack([s for _, s in ws])
        self.offsets = (lead + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
        self.R = int(self.offsets[-1]) + tail
        self.rows, A = None, self.R
        if gather:
            A = max(1, self.R // 3)
            self.rows = r.integers(0, A, self.R).astype(np.int32)
        a = r.standard_normal((A, K)) * np.exp2(r.integers(-3, 4, (A, 1)))
        self.a, self.as_ = wl.encode_mxfp8(a.astype(np.float32))
        self.fmt, self.N, self.K, self.dev = fmt, N, K, dev

    def handle(self, silu):
        from sparse_expert_gemv_gb300 import GroupedProduct
        return GroupedProduct(on(self.w, self.dev), on(self.ws, self.dev), fmt=self.fmt,
                              silu_mul=silu)

    def args(self):
        rows = None if self.rows is None else on(self.rows, self.dev)
        return on(self.a, self.dev), on(self.as_, self.dev), on(self.offsets, self.dev), rows

    def check(self, silu, got):
        Y, S = ref.product(self.w, self.ws, self.a, self.as_, self.offsets, self.rows, self.fmt)
        lo, hi = int(self.offsets[0]), int(self.offsets[-1])
        Y, S = Y[lo:hi], S[lo:hi]
        dY = (1.1 * self.K + 1) * 2.0 ** -24 * S
        if not silu:
            assert_bf16(got[lo:hi], Y, dY, "rows")
            return
        I = self.N // 2
        g, u, dg, du = Y[:, :I], Y[:, I:], dY[:, :I], dY[:, I:]
        h = ref.silu_mul(Y)
        own = (2.0 ** -20 + 2.0 ** -23 * (2 + np.abs(g))) * np.abs(h)
        delta = 1.1 * dg * (np.abs(u) + du) + (np.abs(g) + dg) * du + own
        assert_mxfp8(got[0][lo:hi], got[1][lo:hi], h, delta, "h")


SIZES = [
    # counts, N (plain), K
    ([1], 8, 32), ([3], 128, 128), ([0, 0, 5, 0], 136, 96), ([16, 15, 17, 0, 33], 256, 512),
    ([224, 225, 1], 128, 256), ([449, 0, 128, 129], 200, 160), ([1000], 24, 1056),
    ([2] * 40, 384, 2048), ([0, 0], 64, 64)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,N,K", SIZES)
def test_plain_product(dev, counts, N, K, gather):
    c = Products(dev, "mxfp8", N, K, counts, 1, gather)
    a, s, off, rows = c.args()
    p = c.handle(False)
    out = torch.full((c.R, N), 7.0, dtype=torch.bfloat16, device=dev)
    c.check(False, p(a, s, off, rows, out=out))
    assert p.get_error() == 0


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,N,K", [(c, max(64, n // 64 * 64), k) for c, n, k in SIZES] +
                         [([70, 300], 320, 768)])
def test_silu_product(dev, counts, N, K, gather):
    c = Products(dev, "mxfp8", N, K, counts, 2, gather)
    a, s, off, rows = c.args()
    p = c.handle(True)
    c.check(True, p(a, s, off, rows))
    assert p.get_error() == 0


@pytest.mark.parametrize("silu,counts,N,K,gather", [
    (False, [3], 128, 128, False), (False, [0, 40, 1, 225], 200, 384, True),
    (True, [5, 0, 231], 192, 256, True), (True, [17], 64, 1152, False)])
def test_mxfp4_product(dev, silu, counts, N, K, gather):
    c = Products(dev, "mxfp4", N, K, counts, 3, gather)
    a, s, off, rows = c.args()
    p = c.handle(silu)
    c.check(silu, p(a, s, off, rows))
    assert p.get_error() == 0


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("counts", [
    # wide pieces one after another on the same SMs, whose accumulators overlap
    # in tensor memory, with narrow ones and splits between them
    [256, 255, 256, 250, 225, 256, 31, 256, 224, 300, 256, 1, 256],
    # few tiles: the groups are cut finer
    [200, 0, 190], [33, 64, 65]])
def test_wide_and_cut_pieces(dev, counts, silu):
    c = Products(dev, "mxfp8", 3200, 288, counts, 9, gather=silu)
    a, s, off, rows = c.args()
    p = c.handle(silu)
    c.check(silu, p(a, s, off, rows))
    assert p.get_error() == 0


def test_every_e2m1_and_e4m3_code_through_one_hot_rows(dev):
    # a one-hot row picks one weight column: exact products, so exact bf16
    from sparse_expert_gemv_gb300 import GroupedProduct
    N, K = 256, 128
    a = np.zeros((K, K), dtype=np.uint8)
    np.fill_diagonal(a, 0x38)                      # E4M3 1.0
    s = np.full((K, K // 32), 127, dtype=np.uint8)
    off = np.array([0, K], dtype=np.int32)
    codes = np.arange(N * K, dtype=np.int64).reshape(N, K) * 5 % 256
    codes[codes % 128 == 127] = 0                  # no NaN codes
    w8 = codes.astype(np.uint8)[None]
    sw = np.full((1, N, K // 32), 127, dtype=np.uint8)
    sw[0, :, 1], sw[0, ::3, 2] = 90, 150
    y = GroupedProduct(on(w8, dev), on(sw, dev))(on(a, dev), on(s, dev), on(off, dev))
    assert np.array_equal(tensor_to_f64(y), oracle.dequantize(w8[0], sw[0]).T)
    w4 = (np.arange(N * K // 2, dtype=np.int64).reshape(1, N, K // 2) * 7 % 256).astype(np.uint8)
    y = GroupedProduct(on(w4, dev), on(sw, dev), fmt="mxfp4")(on(a, dev), on(s, dev), on(off, dev))
    assert np.array_equal(tensor_to_f64(y), oracle.dequantize_mxfp4(w4[0], sw[0]).T)


def test_silu_of_far_gates_under_large_ups(dev):
    # one-hot weights: every neuron's gate and up are a row's two values, exactly.
    # exp(-gate) overflows or comes near it while the product is a normal number.
    from sparse_expert_gemv_gb300 import GroupedProduct
    gates = np.array([-72.0, -80.0, -88.0, -96.0, -104.0, 72.0, 104.0, -0.0])
    K, N, R = 64, 64, gates.size
    w = np.zeros((1, N, K), dtype=np.uint8)
    w[0, :32, 0] = w[0, 32:, 32] = 0x38                  # E4M3 1.0
    a, s = np.zeros((R, K), dtype=np.uint8), np.full((R, 2), 127, dtype=np.uint8)
    unit = [int(np.flatnonzero(oracle.E4M3 == g)[0]) for g in gates]
    a[:, 0], a[:, 32], s[:, 1] = unit, 0x38, 127 + 40    # ups 2^40
    p = GroupedProduct(on(w, dev), on(np.full((1, N, 2), 127, dtype=np.uint8), dev), silu_mul=True)
    got = p(on(a, dev), on(s, dev), on(np.array([0, R], dtype=np.int32), dev))
    Y = np.concatenate([np.repeat(gates[:, None], 32, 1), np.full((R, 32), 2.0 ** 40)], 1)
    h = ref.silu_mul(Y)
    g = np.abs(Y[:, :32])
    # the usual error and, where exp or its product is subnormal, a unit of each
    delta = (2.0 ** -20 + 2.0 ** -23 * (2 + g)) * np.abs(h) + 2.0 ** 40 * 2.0 ** -149 * (g + 3)
    assert_mxfp8(got[0], got[1], h, delta, "h")


def test_rows_outside_the_groups_stay_as_they_are(dev):
    c = Products(dev, "mxfp8", 128, 256, [10, 0, 30], 4, lead=5, tail=50)
    # what lies outside the groups is poison: NaN codes and NaN scales
    c.a[:5], c.a[45:], c.as_[:5], c.as_[45:] = 0x7F, 0x7F, 0xFF, 0xFF
    a, s, off, _ = c.args()
    out = torch.full((c.R, 128), -3.0, dtype=torch.bfloat16, device=dev)
    c.handle(False)(a, s, off, out=out)
    c.check(False, out)
    assert out[:5].eq(-3).all() and out[45:].eq(-3).all()
    codes = torch.full((c.R, 64), 9, dtype=torch.uint8, device=dev)
    scales = torch.full((c.R, 2), 9, dtype=torch.uint8, device=dev)
    c.handle(True)(a, s, off, out=codes, out_scales=scales)
    c.check(True, (codes, scales))
    for t in (codes, scales):
        assert t[:5].eq(9).all() and t[45:].eq(9).all()


def test_offsets_out_of_range_are_clamped(dev):
    c = Products(dev, "mxfp8", 64, 128, [20, 20], 5)
    a, s, _, _ = c.args()
    p = c.handle(False)
    want = p(a, s, on(c.offsets, dev))
    wild = on(np.array([-7, 20, 2 ** 31 - 1], dtype=np.int32), dev)
    assert torch.equal(p(a, s, wild), want)
    # descending offsets: the groups are empty
    out = torch.full((40, 64), 2.0, dtype=torch.bfloat16, device=dev)
    p(a, s, on(np.array([40, 20, 0], dtype=np.int32), dev), out=out)
    assert out.eq(2).all() and p.get_error() == 0


def test_nan_in_one_group_stays_there(dev):
    c = Products(dev, "mxfp8", 128, 128, [40, 40, 40], 6)
    a, s, off, _ = c.args()
    p = c.handle(True)
    clean = p(a, s, off)
    a[50, 3] = 0x7F
    got = p(a, s, off)
    keep = torch.arange(120, device=dev) != 50
    assert torch.equal(got[0][keep], clean[0][keep]) and torch.equal(got[1][keep], clean[1][keep])
    assert got[1][50].eq(255).all() and got[0][50].bitwise_and(0x7F).eq(0x7F).all()


@pytest.mark.parametrize("K,shift", [(2048, 4), (2048, 1), (256, 2)])
def test_row_scales_at_any_alignment(dev, K, shift):
    c = Products(dev, "mxfp8", 128, K, [100, 200], 7, gather=True)
    a, s, off, rows = c.args()
    flat = torch.zeros(s.numel() + shift, dtype=torch.uint8, device=dev)
    view = flat[shift:].view_as(s)
    view.copy_(s)
    p = c.handle(False)
    assert torch.equal(p(a, view, off, rows), p(a, s, off, rows))


def test_product_repeats_streams_and_graphs(dev):
    c = Products(dev, "mxfp8", 256, 512, [100, 3, 0, 250], 8, gather=True)
    a, s, off, rows = c.args()
    p = c.handle(True)
    want = p(a, s, off, rows)
    c.check(True, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = p(a, s, off, rows)
    torch.cuda.current_stream().wait_stream(side)
    out = tuple(torch.zeros_like(t) for t in want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p(a, s, off, rows, out=out[0], out_scales=out[1])
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(want, other, out):
        assert torch.equal(x, y) and torch.equal(x, z)


# ---------------------------------------------------------------------------
# combination
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,k,H,R,residual", [
    (1, 1, 8, 1, True), (1, 8, 2048, 8, True), (5, 2, 100, 6, False), (3, 32, 64, 40, True),
    (77, 8, 4104, 500, True), (9, 6, 33, 30, True), (2, 3, 16, 0, True)])
def test_combine(dev, T, k, H, R, residual):
    from sparse_expert_gemv_gb300 import combine
    r = rng(9, T, k, H)
    y = oracle.bf16_rne(r.standard_normal((R, H)))
    slots = r.integers(-2, R + 2, (T, k)).astype(np.int32)     # some outside [0, R)
    w = r.random((T, k)).astype(np.float32)
    w[(slots < 0) | (slots >= R)] = np.nan                     # their weights count for nothing
    res = oracle.bf16_rne(r.standard_normal((T, H))) if residual else None
    rt = None if res is None else bf16(res, dev)
    got = combine(bf16(y, dev), on(slots, dev), on(w, dev), residual=rt)
    want, mag = ref.combine(y, slots, w, res)
    assert_bf16(got, want, (k + 2) * 2.0 ** -24 * mag, "out")
    if residual:
        assert torch.equal(combine(bf16(y, dev), on(slots, dev), on(w, dev), residual=rt, out=rt), got)


# ---------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt,T,E,k,H,I", [
    ("mxfp8", 1, 8, 2, 256, 128), ("mxfp8", 50, 8, 2, 256, 96), ("mxfp4", 300, 16, 4, 512, 256)])
def test_prompt_layer(dev, fmt, T, E, k, H, I):
    """The composed layer equals its operators call by call, and the layer in
    float64 within the noise of the two MXFP8 roundings: each is at most 2^-4
    of a value, evenly spread 2^-4 / sqrt(3) = 0.036 rms; x's passes the SiLU
    product (slope below 1.1 in each factor), h's adds: below 0.0625 of the
    output's norm."""
    from sparse_expert_gemv_gb300 import (GroupedProduct, MoEDecode, add_rms_norm, combine,
                                          group_by_expert)
    w = wl.Workload(90, "prompt", E, k, H, I, T, 0.05)
    experts = wl.make_experts(w, 17, range(E), fmt=fmt)
    stack = [on(np.stack([experts[e][i] for e in range(E)]), dev) for i in range(4)]
    layer = MoEDecode(*stack, k=k, max_T=4, fmt=fmt)
    x, res, nw = norm_case(T, H, 18)
    n = add_rms_norm(bf16(x, dev), bf16(nw, dev), bf16(res, dev), mxfp8=True)
    ids_np, tw = oracle.route(wl.make_logits(w, 19, T), k)
    ids_np = ids_np.copy()
    ids_np[T // 2, 0] = -1                                     # one unused slot
    ids, wt = on(ids_np, dev), on(tw, dev)
    got = layer.prompt(n.codes, n.scales, ids, wt, residual=n.sum)
    off, rows, slots = group_by_expert(ids, E)
    hc, hs = GroupedProduct(stack[0], stack[1], fmt=fmt, silu_mul=True)(n.codes, n.scales, off, rows)
    y = GroupedProduct(stack[2], stack[3], fmt=fmt)(hc, hs, off)
    assert torch.equal(got, combine(y, slots, wt, residual=n.sum))
    _, v = ref.add_rms_norm(x, nw, res)
    full = oracle.layer(v, ids_np, tw, experts, E, H, I, fmt=fmt)["y_pure"]
    mine = tensor_to_f64(got) - tensor_to_f64(n.sum)
    # what the bf16 sum with the residual rounds away: half a step, 2^-8 at most
    room = 0.0625 * np.linalg.norm(full) + 2.0 ** -8 * np.linalg.norm(tensor_to_f64(got))
    assert np.linalg.norm(mine - full) <= room
    assert layer.get_error() == 0


def test_refusals_of_the_python_calls(dev):
    from sparse_expert_gemv_gb300 import (GroupedProduct, MoEError, add_rms_norm, combine,
                                          group_by_expert)
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device=dev)  # noqa: E731
    u8, i32 = torch.uint8, torch.int32
    with pytest.raises(TypeError):
        add_rms_norm(z(2, 32, t=torch.float32), z(32))
    with pytest.raises(ValueError):
        add_rms_norm(z(2, 32), z(31))
    with pytest.raises(ValueError):
        add_rms_norm(z(2, 32), z(32), z(3, 32))
    with pytest.raises(ValueError):
        add_rms_norm(z(2, 64)[:, ::2], z(32))
    with pytest.raises(ValueError):
        add_rms_norm(z(2, 32), z(32), bf16=False)
    with pytest.raises(MoEError):
        add_rms_norm(z(2, 40), z(40), mxfp8=True)
    with pytest.raises(MoEError):
        add_rms_norm(z(1, 16385), z(16385))
    with pytest.raises(TypeError):
        group_by_expert(z(2, 2, t=torch.int64), 4)
    with pytest.raises(MoEError):
        group_by_expert(z(2, 2, t=i32), 1025)
    with pytest.raises(ValueError):
        combine(z(4, 8), z(2, 2, t=i32), z(2, 3, t=torch.float32))
    with pytest.raises(ValueError):
        GroupedProduct(z(2, 8, 32, t=u8), z(2, 8, 1, t=u8), fmt="int8")
    with pytest.raises(MoEError):
        GroupedProduct(z(2, 12, 32, t=u8), z(2, 12, 1, t=u8))
    with pytest.raises(MoEError):                     # MXFP4 rows come in whole 128s
        GroupedProduct(z(2, 8, 32, t=u8), z(2, 8, 2, t=u8), fmt="mxfp4")
    p = GroupedProduct(z(2, 64, 64, t=u8), z(2, 64, 2, t=u8), silu_mul=True)
    with pytest.raises(ValueError):
        p(z(4, 32, t=u8), z(4, 1, t=u8), z(3, t=i32))
    with pytest.raises(ValueError):
        p(z(4, 64, t=u8), z(4, 2, t=u8), z(2, t=i32))
    with pytest.raises(ValueError):
        p(z(4, 64, t=u8), z(4, 2, t=u8), z(3, t=i32), out=z(4, 64, t=u8))
    empty = p(z(0, 64, t=u8), z(0, 2, t=u8), z(3, t=i32))
    assert empty[0].shape == (0, 32) and empty[1].shape == (0, 1)


def test_example_block(dev, capsys):
    """The example runs, and its block is its operators: the stream after it is
    the sum of the norm's stream and the routed experts."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "prompt_block.py")
    spec = importlib.util.spec_from_file_location("prompt_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    assert ex.main(["--tokens", "70", "--experts", "8", "--topk", "2", "--hidden", "256",
                    "--intermediate", "128"]) > 0
    assert "tokens a us" in capsys.readouterr().out
    from sparse_expert_gemv_gb300 import add_rms_norm
    layer = ex.random_layer(8, 2, 256, 128, "mxfp4", max_T=40)
    x, res, nw = norm_case(40, 256, 20)
    r = bf16(rng(21).standard_normal((8, 256)) / 16, dev)
    block = ex.PromptBlock(layer, bf16(nw, dev), r)
    n = add_rms_norm(bf16(x, dev), bf16(nw, dev), bf16(res, dev), mxfp8=True)
    ids, w = layer.route((n.y @ r.T).float())
    want = layer.prompt(n.codes, n.scales, ids, w, residual=n.sum)
    assert torch.equal(block(bf16(x, dev), bf16(res, dev)), want)
    # a stream of zeros before the block: the same without a residual
    zeros = torch.zeros(40, 256, dtype=torch.bfloat16, device=dev)
    assert torch.equal(block(bf16(x, dev), None), block(bf16(x, dev), zeros))
