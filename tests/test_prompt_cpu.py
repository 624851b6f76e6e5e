"""The prompt operators on a machine without a GPU: the C ABI of
include/moe_prompt.h (symbols, refusals before any CUDA call) and pins of their
float64 oracle."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from oracle import prompt as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 12            # a pointer that is aligned and never followed


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    b = __graft_entry__._build_module()
    if b.stale(b.OUT):
        b.build()
    from sparse_expert_gemv_gb300 import _lib
    return _lib.lib


def declared():
    text = open(os.path.join(ROOT, "include", "moe_prompt.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))


def test_binding_and_library_cover_the_header(lib):
    from sparse_expert_gemv_gb300 import _lib
    assert set(_lib.PROMPT_SIGNATURES) == set(declared())
    for name in declared():
        assert hasattr(lib, name), name


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(x=0), 1),
    (dict(weight=0), 1), (dict(y=0, codes=0, scales=0), 1), (dict(scales=0), 1), (dict(codes=0), 1),
    (dict(H=16385), 2), (dict(H=40), 2), (dict(x=P + 1), 3), (dict(residual=P + 1), 3),
    (dict(y=P + 1), 3), (dict(T=0, x=0), 0)])
def test_norm_refusals(lib, kw, status):
    a = dict(T=2, H=64, x=P, residual=P, weight=P, eps=1e-6, sum=P, y=P, codes=P, scales=P) | kw
    assert lib.moe_add_rms_norm(*a.values(), 0) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(k=0), 1), (dict(E=0), 1), (dict(ids=0), 1), (dict(offsets=0), 1),
    (dict(rows=0), 1), (dict(slots=0), 1), (dict(E=1025), 2), (dict(T=1 << 28, k=8), 2),
    (dict(ids=P + 2), 3), (dict(offsets=P + 2), 3)])
def test_group_refusals(lib, kw, status):
    a = dict(T=2, k=2, E=4, ids=P, offsets=P, rows=P, slots=P) | kw
    assert lib.moe_group(*a.values(), 0) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(k=0), 1), (dict(H=0), 1), (dict(R=-1), 1), (dict(y=0), 1),
    (dict(slots=0), 1), (dict(w=0), 1), (dict(out=0), 1), (dict(y=P + 1), 3), (dict(w=P + 2), 3),
    (dict(T=0, y=0), 0), (dict(T=1 << 30, H=1 << 20), 2)])
def test_combine_refusals(lib, kw, status):
    a = dict(T=2, k=2, H=64, R=4, y=P, slots=P, w=P, residual=P, out=P) | kw
    assert lib.moe_combine(*a.values(), 0) == status


@pytest.mark.parametrize("kw,status", [
    (dict(E=0), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(flags=0x1), 1), (dict(w=0), 1),
    (dict(s=0), 1), (dict(E=1025), 2), (dict(N=12), 2), (dict(K=48), 2), (dict(N=96, flags=0x10), 2),
    (dict(K=64, flags=0x4), 2), (dict(w=P + 16), 3)])
def test_product_create_refusals(lib, kw, status):
    from sparse_expert_gemv_gb300._lib import MoEProductConfig
    a = dict(E=4, N=128, K=128, flags=0, w=P, s=P) | kw
    cfg = MoEProductConfig(a["E"], a["N"], a["K"], a["flags"])
    h = ctypes.c_void_p(77)
    assert lib.moe_product_create(ctypes.byref(cfg), a["w"], a["s"], ctypes.byref(h), 0) == status
    assert h.value is None


def test_product_null_handles(lib):
    assert lib.moe_product_create(None, P, P, None, 0) == 1
    assert lib.moe_product_run(None, 1, 1, P, P, P, 0, P, 0, 0, 0) == 1
    assert lib.moe_product_get_error(None, 0, None) == 1
    assert lib.moe_product_destroy(None) == 0


# ---------------------------------------------------------------------------
# oracle pins
# ---------------------------------------------------------------------------

def test_e4m3_rounding_against_torch_and_midpoints():
    codes = np.array([c for c in range(256) if np.isfinite(oracle.E4M3[c])])
    v = np.unique(oracle.E4M3[codes])
    assert np.array_equal(ref.e4m3_rne(v), v)
    x = np.random.default_rng(3).standard_normal(20000) * np.exp2(
        np.random.default_rng(4).integers(-12, 9, 20000))
    x = np.concatenate([x, (v[1:] + v[:-1]) / 2]).astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3_rne(x.astype(np.float64)), want)


def test_quantisation_against_the_workloads_encoder():
    x = np.random.default_rng(5).standard_normal((7, 160)).astype(np.float32)
    x[2, 32:64], x[3, :32] = 0.0, x[3, :32] * np.float32(2.0 ** -130)
    q, s = ref.quantize_mxfp8(x.astype(np.float64))
    codes, scales = wl.encode_mxfp8(x)
    assert np.array_equal(s, scales) and np.array_equal(q, oracle.E4M3[codes])


def test_norm_against_a_scalar_loop():
    r = np.random.default_rng(6)
    x, res = oracle.bf16_rne(r.standard_normal((2, 5))), oracle.bf16_rne(r.standard_normal((2, 5)))
    w = r.standard_normal(5)
    s, n = ref.add_rms_norm(x, w, res, 0.01)
    for t in range(2):
        row = [float(torch.tensor(x[t, i] + res[t, i]).to(torch.bfloat16)) for i in range(5)]
        rms = math.sqrt(math.fsum(v * v for v in row) / 5 + 0.01)
        for i in range(5):
            assert s[t, i] == row[i] and n[t, i] == pytest.approx(row[i] / rms * w[i], rel=1e-14)


def test_group_against_a_sort():
    ids = np.random.default_rng(7).integers(-2, 9, (50, 3)).astype(np.int32)
    off, rows, slots = ref.group(ids, 7)
    flat = [(e, p) for p, e in enumerate(ids.reshape(-1)) if 0 <= e < 7]
    order = [p for _, p in sorted(flat)]
    assert rows.tolist() == [p // 3 for p in order] + [-1] * (150 - len(order))
    assert [slots.reshape(-1)[p] for p in order] == list(range(len(order)))
    assert off.tolist() == [sum(e < i for e, _ in flat) for i in range(8)]
    assert np.count_nonzero(slots == -1) == 150 - len(order)


def test_products_and_combination_make_the_decode_layer():
    # with rows the oracle's decode layer also takes (MXFP8-exact x), the
    # product, SiLU and combination give its unrounded layer
    w = wl.Workload(89, "pin", 6, 2, 64, 32, 9, 0.1)
    experts = wl.make_experts(w, 3, range(w.E))
    xc, xs = wl.encode_mxfp8(np.random.default_rng(8).standard_normal((9, 64)).astype(np.float32))
    ids, tw = oracle.route(wl.make_logits(w, 3, 9), w.k)
    off, rows, slots = ref.group(ids, w.E)
    stack = [np.stack([experts[e][i] for e in range(w.E)]) for i in range(4)]
    gu, _ = ref.product(stack[0], stack[1], xc, xs, off, rows)
    h = ref.silu_mul(gu)
    y = np.concatenate([h[off[e]:off[e + 1]] @ oracle.dequantize(stack[2][e], stack[3][e]).T
                        for e in range(w.E)])
    got, mag = ref.combine(y, slots, tw)
    want = oracle.layer(oracle.dequantize(xc, xs), ids, tw, experts, w.E, w.H, w.I)["y_pure"]
    assert np.allclose(got, want, rtol=1e-12, atol=1e-14) and np.all(mag >= np.abs(got))
