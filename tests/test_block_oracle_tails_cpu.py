"""Pins of the block oracle where a formula's plain form cancels."""
import numpy as np

from oracle import block as ref


def test_gelu_far_below_zero():
    # Phi(-5.5), Phi(-10), Phi(-20) of the standard normal distribution
    v = np.array([[-5.5, -10.0, -20.0]])
    want = v * np.array([1.8989562465887719e-08, 7.6198530241605261e-24, 2.7536241186062337e-89])
    assert np.allclose(ref.activate(v, "gelu"), want, rtol=1e-13, atol=0)


def test_tanh_gelu_far_below_zero():
    # v / (1 + exp(-y)) with y = sqrt(8 / pi) (v + 0.044715 v^3)
    v = np.array([[-6.0, -10.0]])
    y = np.sqrt(8 / np.pi) * (v + 0.044715 * v ** 3)
    assert np.allclose(ref.activate(v, "gelu_tanh"), v * np.exp(y), rtol=1e-10, atol=0)
    assert (ref.activate(v, "gelu_tanh") < 0).all()
