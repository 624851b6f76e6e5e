"""Outputs that share memory with other tensors of their call are refused at the C
ABI before any CUDA call: pointers that are never followed."""
import ctypes

import pytest

from test_block_cpu import lib, moe  # noqa: F401  (fixtures)

A = 1 << 20            # tensors 1 MB apart


@pytest.mark.parametrize("kw", [
    dict(ids=A), dict(ids=A + 4 * 16 * 4 - 4), dict(ids=A - 4 * 3 * 4 + 4), dict(w=A + 64), dict(w=2 * A),
    dict(w=3 * A), dict(w=3 * A + 44), dict(ids=2 * A + 60), dict(flags=1, ids=A + 4 * 16 * 2 - 4)])
def test_route(lib, kw):  # noqa: F811
    from sparse_expert_gemv_gb300._lib import MoERouteConfig
    a = dict(flags=0, logits=A, bias=2 * A, ids=3 * A, w=4 * A) | kw
    cfg = MoERouteConfig(16, 3, 1, 1, 1.0, a["flags"])
    assert lib.moe_route_experts(ctypes.byref(cfg), 4, a["logits"], a["bias"], a["ids"], a["w"], 0) == 1


T, H = 3, 64
ROWS = T * H * 2


@pytest.mark.parametrize("kw", [
    dict(y=6 * A), dict(y=6 * A + ROWS - 2), dict(sum=A + 2), dict(sum=A - ROWS + 2), dict(sum=2 * A + 2),
    dict(sum=A, y=A), dict(y=A + 2 * H), dict(sum=3 * A), dict(sum=4 * A + 2 * H - 2), dict(y=5 * A),
    dict(y=5 * A, flags=0x2), dict(y=5 * A + ROWS - 2, flags=0x2), dict(y=5 * A + 2 * T - 2, flags=0x1),
    dict(codes=A), dict(codes=2 * A + ROWS - 1), dict(codes=6 * A), dict(codes=7 * A), dict(scales=A + 5),
    dict(scales=8 * A + ROWS // 2 - 1), dict(scales=7 * A), dict(scales=3 * A + 1)])
def test_norms(lib, kw):  # noqa: F811
    a = dict(x=A, residual=2 * A, post=3 * A, pre=4 * A, gate=5 * A, scale=1.0, rscale=1.0, eps=1e-6,
             flags=0, sum=6 * A, y=7 * A, codes=8 * A, scales=9 * A) | kw
    assert lib.moe_norm_add_norm(T, H, *a.values(), 0) == 1
