"""GPU parity of a dense product's GELUs where their value is small beside their
argument: one-hot weights hand every value of the rows to the activation as it
is, and the bounds are relative to the result.

With u = 2^-24 (half a step of FP32 at 1):

  * GELU, v erfc(z) / 2 with z = -v / sqrt 2: z is off by u for its rounding and
    u / 2 for its constant, which erfc makes 2 z^2 + 1 = v^2 + 1 times larger at
    most; erfc by 4 units of 2^-23, the product by u: u (1.5 v^2 + 11).
  * tanh-GELU, v sigmoid(y) with y = sqrt(8 / pi) (v + 0.044715 v^3): y is off by
    six roundings (two constants, four operations), the short exponential by
    2 + 1.173 |y| units of 2^-23 and the short division by two, two more
    operations by u each: u (8.4 |y| + 10).

Exponentials below 2^-126 are 0, and erfc below it rounds in steps of 2^-149.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import block as ref
from test_gpu_prompt import assert_bf16, bf16, dev  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
VALUES = np.unique(oracle.bf16_rne(np.concatenate([np.linspace(-14, 14, 1800), [-30.0, -100.0, -3e38, 3e38]])))


def is_split(R, K, N, act, float32):
    from sparse_expert_gemv_gb300._lib import MoEDenseConfig, MoEDensePlan, lib
    p = MoEDensePlan()
    code = {"gelu": 3, "gelu_tanh": 4}[act]
    assert lib.moe_dense_plan(ctypes.byref(MoEDenseConfig(N, K, code)), R, float32, 152, ctypes.byref(p)) == 0
    return p.split == 1


# few rows with a long K (moe_dense_split), many rows (moe_dense_tiles)
@pytest.mark.parametrize("R,K,N", [(16, 2048, 256), (4000, 64, 8)])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh"])
def test_small_values_keep_their_relative_accuracy(dev, act, R, K, N):  # noqa: F811
    from sparse_expert_gemv_gb300 import DenseProduct
    per = min(N, -(-len(VALUES) // R))          # value j of row r is v[r, j], its column j
    v = np.resize(VALUES, (R, per))
    assert set(VALUES) <= set(v.ravel())
    x, w = np.zeros((R, K)), np.zeros((N, K))
    x[:, :per] = v
    w[:per, :per] = np.eye(per)
    with np.errstate(over="ignore"):
        want = ref.activate(v, act)
        y = np.abs(np.sqrt(8 / np.pi) * (v + 0.044715 * v ** 3))
    m = np.abs(v)
    units = np.minimum(1.5 * v ** 2 + 11 if act == "gelu" else 8.4 * y + 10, 2.0 ** 24)
    bound = U * units * np.abs(want) + m * (2.0 ** -147 if act == "gelu" else 2.0 ** -126)
    p = DenseProduct(bf16(w, dev), activation=act)
    for float32 in (True, False):
        assert is_split(R, K, N, act, float32) == (K == 2048)
        got = p(bf16(x, dev), float32=float32)[:, :per]
        if float32:
            err = np.abs(got.double().cpu().numpy() - want)
            assert (err <= bound).all(), (v[err > bound][:5], (err / bound).max())
        else:
            assert_bf16(got, want, bound, act)
    assert p.get_error() == 0


@pytest.mark.parametrize("R", [3, 4000])
def test_gelu_of_infinity_and_nan(dev, R):  # noqa: F811
    from sparse_expert_gemv_gb300 import DenseProduct
    w = torch.zeros(8, 64, dtype=torch.bfloat16, device=dev)
    w[0, 0] = 1.0
    x = torch.zeros(R, 64, dtype=torch.bfloat16, device=dev)
    x[0, 0], x[1, 0] = float("inf"), float("nan")
    for act in ("gelu", "gelu_tanh"):
        got = DenseProduct(w, activation=act)(x, float32=True)[:, 0]
        assert got[0] == float("inf") and got[1].isnan() and got[2:].eq(0).all()
