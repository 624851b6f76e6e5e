"""Every path of the dense products, by shapes whose cut is asserted: tiles whose
sums are added up over several parts of K and whose ring turns many times, several
tiles a pair, splits into one to eight parts with narrow and wide tiles.

Whole numbers make every sum exact, so every bit is checked (FP32 outputs) or the
one rounding to bf16. SiLU(gate) * up of whole numbers, with u = 2^-24: the short
exponential is off by 2 + 1.173 |g| units of 2^-23, the short division by two, three
more operations by u each: u (2.4 |g| + 11), and what lies below 2^-126 may be 0.

On random values the tensor cores cut a sum off at each of its steps of 16 K, on
average by half a unit in its last place. Over a binade a unit is 0.72 * 2^-23 of the
value, and the sum on its way 2/3 of its end, as the way of a random sum is: 0.48 u a
step, 15.4 u over the 512 K of a part, always towards zero. The K / 512 parts are
then added up in FP32, each addition off by a third of a unit of a sum that is on
its way: 0.42 u sqrt(K / 512), and the result is rounded: u. This is a relative
2-norm over the outputs; without the parts it would be 0.48 u K / 16 (at K = 7168
1.3e-5).
"""
import ctypes

import numpy as np
import pytest
import torch

from test_gpu_prompt import assert_bf16, dev  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
CODES = {None: 0, "relu": 1, "silu_mul": 5}


def cut(dev, R, K, N, act, float32):  # noqa: F811
    from sparse_expert_gemv_gb300._lib import MoEDenseConfig, MoEDensePlan, lib
    p, sms = MoEDensePlan(), torch.cuda.get_device_properties(dev).multi_processor_count
    config = MoEDenseConfig(N, K, CODES[act])
    assert lib.moe_dense_plan(ctypes.byref(config), R, float32, sms, ctypes.byref(p)) == 0
    return p


TILES, S1, S2, S4, S8 = "tiles", "split 1", "split 2", "split 4", "split 8"


def name(p):
    return f"split {p.parts}" if p.split else TILES


PATHS = [
    # R, K, N, the path of bf16 outputs, of FP32 ones
    (2600, 576, 2600, TILES, TILES), (3001, 1024, 1544, TILES, TILES), (5000, 1088, 1030, TILES, TILES),
    (1500, 7168, 4100, TILES, TILES), (9000, 7168, 520, TILES, TILES), (500, 7168, 1024, S4, TILES),
    (3370, 280, 66, S1, S1), (3656, 280, 282, S1, S1), (90, 1024, 2000, S2, S2), (141, 1552, 3942, S2, S2),
    (1213, 4040, 320, S4, S4), (606, 5792, 478, S4, S8), (128, 7168, 2048, S4, S8), (100, 7168, 512, S8, S8),
    (64, 8192, 640, S8, S8), (100, 28672, 1024, S4, S8), (5, 65536, 256, S8, TILES)]


def whole(g, *shape, hi=3):
    return torch.randint(-hi, hi + 1, shape, device=g.device, generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("act", [None, "relu", "silu_mul"])
@pytest.mark.parametrize("R,K,N,narrow,wide", PATHS)
def test_whole_numbers(dev, R, K, N, narrow, wide, act):  # noqa: F811
    from sparse_expert_gemv_gb300 import DenseProduct
    g = torch.Generator(device=dev).manual_seed(R + K + N)
    silu = act == "silu_mul"
    M = N // 2 if silu else N
    x, w, b = whole(g, R, K), whole(g, N, K), whole(g, N, hi=100)
    if silu:                                       # gates of a few units, as gates are
        w[:M] = torch.where(torch.rand(M, K, device=dev, generator=g) < 8 / K, w[:M].float(), 0.0).bfloat16()
        b[:M] = whole(g, M, hi=4)
    res = whole(g, R, M, hi=100)
    y = x.double() @ w.double().T + b.double()     # whole numbers: exact
    p = DenseProduct(w, b, activation=act)
    if silu:
        gate, up = y[:, :M], y[:, M:]
        silus = gate * torch.sigmoid(gate) * up
        d = (U * (2.4 * gate.abs() + 11) * silus.abs() + 2.0 ** -126 * (gate * up).abs()).cpu().numpy()
        d_res = d + (U * (silus.abs() + 2 * res.abs().double())).cpu().numpy()
    want = silus if silu else y.clamp(min=0) if act else y
    for float32, path in ((False, narrow), (True, wide)):
        assert name(cut(dev, R, K, N, act, float32)) == path
        for r in (None, res):
            got = p(x, r, float32=float32)
            exact = want if r is None else want + r.double()
            if not silu:
                assert torch.equal(got, exact.float() if float32 else exact.bfloat16())
                continue
            e, bound = exact.cpu().numpy(), d if r is None else d_res
            if float32:
                assert (np.abs(got.double().cpu().numpy() - e) <= bound + U * np.abs(e)).all()
            else:
                assert_bf16(got, e, bound, path)
    assert p.get_error() == 0


@pytest.mark.parametrize("R,K,N", [(2600, 576, 2600), (3000, 7168, 256), (9000, 7168, 512), (500, 7168, 1024),
                                   (8, 7168, 256), (100, 7168, 512), (128, 7168, 2048), (606, 5792, 478),
                                   (64, 8192, 640), (100, 28672, 1024), (128, 28672, 1024), (5, 65536, 256),
                                   (300, 65536, 384)])
def test_fp32_outputs_keep_fp32_accuracy(dev, R, K, N):  # noqa: F811
    from sparse_expert_gemv_gb300 import DenseProduct
    g = torch.Generator(device=dev).manual_seed(K)
    x = torch.randn(R, K, device=dev, generator=g).bfloat16()
    w = (torch.randn(N, K, device=dev, generator=g) * K ** -0.5).bfloat16()
    want = x.double() @ w.double().T
    got = DenseProduct(w)(x, float32=True).double()
    error = ((got - want).norm() / want.norm()).item()
    assert error <= U * (15.4 + 0.42 * (K / 512) ** 0.5 + 1), error


@pytest.mark.parametrize("act", [None, "silu_mul"])
@pytest.mark.parametrize("R,K,N,path", [(2600, 576, 2600, TILES), (500, 7168, 1024, TILES), (128, 7168, 2048, S8),
                                        (3656, 280, 282, S1)])
def test_runs_with_fp32_outputs_wind_down(dev, R, K, N, path, act):  # noqa: F811
    # as test_dense_winds_down_when_its_waits_give_up, where sums are added up over parts
    from sparse_expert_gemv_gb300 import MOE_DEVICE_TIMEOUT, DenseProduct
    g = torch.Generator(device=dev).manual_seed(R)
    assert name(cut(dev, R, K, N, act, True)) == path
    x, w = whole(g, R, K), whole(g, N, K)
    p = DenseProduct(w, activation=act)
    want = p(x, float32=True)
    assert p.get_error() == 0
    for _ in range(2):
        p.arm_timeout()
        p(x, float32=True)
        assert p.get_error() == MOE_DEVICE_TIMEOUT
        assert torch.equal(p(x, float32=True), want)
        assert p.get_error() == 0
