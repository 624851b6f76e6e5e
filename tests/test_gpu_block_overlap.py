"""Calls whose outputs share memory with their inputs: the ones that the
documentation allows give what separate tensors give, all others are refused."""
import pytest
import torch

from test_gpu_block import Dense, Norms
from test_gpu_prompt import bf16, dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(9, 512), (33, 256), (5, 9999), (2100, 1056), (3, 16383), (4, 16384)])
@pytest.mark.parametrize("gate", [None, "full"])
def test_norms_onto_their_inputs(dev, T, H, gate):  # noqa: F811
    from sparse_expert_gemv_gb300 import MoEError, norm_add_norm
    c = Norms(T, H, True, gate, seed=90)
    x, res, post, pre = c.args(dev)
    kw = dict(gate=None if gate is None else bf16(c.gate, dev), mxfp8=H % 32 == 0)
    want = norm_add_norm(x, res, post, pre, **kw)
    for sum_at, y_at in ((None, 0), (None, 1), (0, 1), (1, 0), (0, None)):
        a = [x.clone(), res.clone()]
        bufs = {n: a[i] for n, i in (("sum", sum_at), ("y", y_at)) if i is not None}
        got = norm_add_norm(*a, post, pre, **kw, **bufs)
        for u, v in zip(got, want):
            assert u is None and v is None or torch.equal(u, v)
    flat = torch.empty(T * H + H, dtype=torch.bfloat16, device=dev)
    flat[:T * H] = x.view(-1)
    inside, shifted = flat[:T * H].view(T, H), flat[H:].view(T, H)
    for bufs in (dict(sum=shifted), dict(y=shifted), dict(sum=inside, y=inside)):
        with pytest.raises(MoEError):
            norm_add_norm(inside, res, post, pre, **kw, **bufs)
    assert torch.equal(inside, x)


@pytest.mark.parametrize("R,K,N", [(7, 256, 256), (3000, 256, 256), (2000, 264, 2120)])
def test_dense_outputs_beside_and_over_other_tensors(dev, R, K, N):  # noqa: F811
    from sparse_expert_gemv_gb300 import DenseProduct, MoEError
    c = Dense(R, K, N, True, "relu", True, seed=91)
    w = torch.empty(N * K + R * N, dtype=torch.bfloat16, device=dev)
    w[:N * K] = bf16(c.w, dev).view(-1)
    b = torch.empty(N + R * N, dtype=torch.bfloat16, device=dev)
    b[:N] = bf16(c.b, dev)
    p = DenseProduct(w[:N * K].view(N, K), b[:N], activation="relu")
    res = bf16(c.res, dev)
    flat = torch.empty(R * K + R * N, dtype=torch.bfloat16, device=dev)
    x = flat[:R * K].view(R, K)
    x.copy_(bf16(c.x, dev))
    want = p(x, res)
    c.check(want)
    # right behind x, the weight or the bias: no byte is shared
    for out in (flat[R * K:], w[N * K:], b[N:]):
        assert torch.equal(p(x, res, out=out.view(R, N)), want)
    assert torch.equal(p(x, res.clone(), out=None), want)
    for t, n in ((flat, R * K), (w, N * K), (b, N)):
        out = t[n - 1:][:R * N].view(R, N)
        with pytest.raises(MoEError):
            p(x, res, out=out)
    with pytest.raises(MoEError):
        p(x, flat[R * K:].view(R, N), out=flat[R * K - 8:][:R * N].view(R, N))
    wide = torch.empty(R, N, dtype=torch.float32, device=dev)
    over = wide.view(torch.bfloat16).view(-1)[:R * N].view(R, N)     # its memory's first half
    over.copy_(res)
    with pytest.raises(MoEError):
        p(x, over, out=wide, float32=True)
    assert p.get_error() == 0
    if K == N:
        before = x.clone()
        with pytest.raises(MoEError):
            p(x, res, out=x)
        with pytest.raises(MoEError):
            p(x, out=w[:N * K].view(N, K)[:R] if R <= N else x)
        assert torch.equal(x, before)


def test_routes_over_their_logits(dev):  # noqa: F811
    from sparse_expert_gemv_gb300 import MoEError, route_experts
    flat = torch.randn(20 * 16 + 20 * 4 * 2, device=dev)
    z, k = flat[:320].view(20, 16), 4
    want = route_experts(z, k)
    ids, w = flat[320:400].view(torch.int32).view(20, 4), flat[400:].view(20, 4)
    for got, like in zip(route_experts(z, k, ids=ids, w=w), want):
        assert torch.equal(got, like)
    before = z.clone()
    for bufs in (dict(w=flat[316:396].view(20, 4)), dict(ids=flat[:80].view(torch.int32).view(20, 4)),
                 dict(ids=ids, w=ids.view(torch.float32))):
        with pytest.raises(MoEError):
            route_experts(z, k, **bufs)
    assert torch.equal(z, before)
