"""A dense product over a weight that was only just written: its runs read the
weight ahead of earlier work on their stream, so making the handle waits for the
stream that writes it."""
import numpy as np
import pytest
import torch

from test_gpu_prompt import bf16, dev, rng  # noqa: F401

pytestmark = pytest.mark.gpu

N, K, R, L = 512, 1024, 9, 64


def whole(r, *shape):
    return r.integers(-2, 3, shape).astype(float)


@pytest.mark.parametrize("given", [False, True])
def test_the_weights_stream_is_waited_for(dev, given):  # noqa: F811
    # the weight is a product's output, whose launch lets the next one start beside
    # it; whole numbers, so that the sums are exact
    from sparse_expert_gemv_gb300 import DenseProduct
    r = rng(81)
    a, b, x = whole(r, N, L), whole(r, K, L), whole(r, R, K)
    b[:, 2:] = 0                                   # (the weight's values are bf16's)
    first = DenseProduct(bf16(b, dev))
    rows, xs = bf16(a, dev), bf16(x, dev)
    w = torch.full((N, K), 7.0, dtype=torch.bfloat16, device=dev)
    bias = torch.full((N,), 7.0, dtype=torch.bfloat16, device=dev)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)             # a tenth of a second
        bias.fill_(1.0)
        first(rows, out=w)
        if not given:
            product = DenseProduct(w, bias)
            assert side.query()
            got = product(xs, float32=True)
    if given:
        product = DenseProduct(w, bias, stream=side)
        assert side.query()
        with torch.cuda.stream(side):
            got = product(xs, float32=True)
    side.synchronize()
    assert np.array_equal(w.double().cpu().numpy(), a @ b.T)
    assert np.array_equal(got.double().cpu().numpy(), x @ (a @ b.T).T + 1.0)
    assert product.get_error() == 0
