"""The block operators on a machine without a GPU: the C ABI of
include/moe_block.h (symbols, refusals before any CUDA call), the binding's
checks, and pins of their float64 oracle."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import oracle
from oracle import block as ref
from test_prompt_devices_cpu import fake, moe  # noqa: F401  (moe: the fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 12            # a pointer that is aligned and never followed
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib(moe):  # noqa: F811
    return moe.lib


def declared():
    text = open(os.path.join(ROOT, "include", "moe_block.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text)))


def test_binding_and_library_cover_the_header(lib):
    from sparse_expert_gemv_gb300 import _lib
    assert set(_lib.BLOCK_SIGNATURES) == set(declared())
    for name in declared():
        assert hasattr(lib, name), name


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(groups=0), 1), (dict(top=0), 1),
    (dict(top=5), 1), (dict(groups=3, top=1), 1), (dict(k=9), 1), (dict(k=5, top=1), 1),
    (dict(scale=math.nan), 1), (dict(scale=math.inf), 1), (dict(flags=0x10), 1), (dict(logits=0), 1),
    (dict(ids=0), 1), (dict(w=0), 1), (dict(E=1028), 2), (dict(E=64, k=33), 2),
    (dict(E=66, groups=33, top=4), 2), (dict(logits=P + 2), 3), (dict(logits=P + 1, flags=1), 3),
    (dict(bias=P + 2), 3), (dict(ids=P + 2), 3), (dict(w=P + 2), 3), (dict(T=0, logits=0), 0),
    (dict(T=2 ** 31 - 1), 2)])
def test_route_refusals(lib, kw, status):
    from sparse_expert_gemv_gb300._lib import MoERouteConfig
    a = dict(T=2, E=16, k=4, groups=4, top=2, scale=1.0, flags=0, logits=P, bias=P, ids=P, w=P) | kw
    cfg = MoERouteConfig(a["E"], a["k"], a["groups"], a["top"], a["scale"], a["flags"])
    assert lib.moe_route_experts(ctypes.byref(cfg), a["T"], a["logits"], a["bias"], a["ids"], a["w"],
                                 0) == status


def test_route_without_a_config(lib):
    assert lib.moe_route_experts(None, 1, P, 0, P, P, 0) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(x=0), 1),
    (dict(residual=0), 1), (dict(sum=0), 1), (dict(scale=math.nan), 1), (dict(rscale=math.inf), 1),
    (dict(scales=0), 1), (dict(codes=0), 1), (dict(pre=0), 1), (dict(y=0, codes=0, scales=0), 1),
    (dict(flags=0x3), 1), (dict(flags=0xc), 1), (dict(flags=0x20), 1), (dict(flags=0x1, gate=0), 1),
    (dict(flags=0x4, gate=0), 1), (dict(H=16385), 2), (dict(H=40), 2), (dict(x=P + 1), 3),
    (dict(residual=P + 1), 3), (dict(post=P + 1), 3), (dict(pre=P + 1), 3), (dict(gate=P + 1), 3),
    (dict(sum=P + 1), 3), (dict(y=P + 1), 3), (dict(T=0, x=0), 0), (dict(T=2 ** 31 - 1), 2)])
def test_norm_refusals(lib, kw, status):
    a = dict(T=2, H=64, x=P, residual=P, post=P, pre=P, gate=P, scale=1.0, rscale=1.0, eps=1e-6,
             flags=0, sum=P, y=P, codes=P, scales=P) | kw
    assert lib.moe_norm_add_norm(*a.values(), 0) == status


@pytest.mark.parametrize("kw,status", [
    (dict(N=0), 1), (dict(K=0), 1), (dict(act=-1), 1), (dict(act=6), 1), (dict(w=0), 1),
    (dict(K=12), 2), (dict(N=7, act=5), 2), (dict(w=P + 8), 3), (dict(b=P + 1), 3),
    (dict(N=2 ** 31 - 1), 2), (dict(K=2 ** 31 - 8), 2)])
def test_dense_create_refusals(lib, kw, status):
    from sparse_expert_gemv_gb300._lib import MoEDenseConfig
    a = dict(N=64, K=64, act=0, w=P, b=P) | kw
    h = ctypes.c_void_p(77)
    cfg = MoEDenseConfig(a["N"], a["K"], a["act"])
    assert lib.moe_dense_create(ctypes.byref(cfg), a["w"], a["b"], ctypes.byref(h)) == status
    assert h.value is None


def plan(lib, R, K, N, act=0, sms=152, out_float=0):
    from sparse_expert_gemv_gb300._lib import MoEDenseConfig, MoEDensePlan
    p = MoEDensePlan()
    assert lib.moe_dense_plan(ctypes.byref(MoEDenseConfig(N, K, act)), R, out_float, sms, ctypes.byref(p)) == 0
    return p


def test_dense_plans_keep_the_kernels_limits(lib):
    r = np.random.default_rng(5)
    seen = set()
    for _ in range(3000):
        R, K, N = (int(np.exp(r.uniform(0, np.log(hi)))) for hi in (20000, 1000, 10000))
        K, act, sms = 8 * K, int(r.choice([0, 5])), int(r.choice([1, 2, 76, 148, 152]))
        N += N % 2
        flt, two = int(r.choice([0, 1])), 2 if act == 5 else 1
        p = plan(lib, R, K, N, act, sms, flt)
        M, nk = N // two, -(-K // 64)
        seen.add((p.split, p.parts))
        assert p.stages >= 2
        if p.split:
            assert p.nt % 16 == 0 and 16 <= p.nt <= 128 and p.stages <= 16
            assert p.parts in (1, 2, 4, 8) and p.parts <= nk
            # FP32 sums of up to 1024 K (or an eighth) in the tensor cores
            assert not flt or p.parts == 8 or -(-nk // p.parts) <= 16
            # barriers, ring, sums; at most two CTAs an SM, whose tensor memory it has
            stage, sums = 16384 + p.nt * 128, p.nt * 512
            assert sums <= p.stages * stage
            assert 2048 + p.stages * stage + (sums if p.parts > 1 else 0) <= p.smem <= 226 * 1024
            assert 3 * (p.smem + 1024) > 228 * 1024 and 2 * p.nt <= 512
            assert p.ctas == -(-M // (64 if act else 128)) * -(-R // p.nt) * p.parts
        else:
            assert p.nt % 32 == 0 and 32 <= p.nt <= (128 if flt else 256) and p.smem <= 232448 and p.stages <= 12
            assert 1024 + 4 * 8192 + 1024 + p.stages * (16384 + p.nt * 64) <= p.smem
            assert p.ctas == 2 * min(max(1, sms // 2), -(-M // (256 // two)) * -(-R // p.nt))
    assert seen >= {(0, 1), (1, 1), (1, 2), (1, 4), (1, 8)}


def test_dense_plan_refusals(lib):
    from sparse_expert_gemv_gb300._lib import MoEDenseConfig, MoEDensePlan
    p, ok = MoEDensePlan(), MoEDenseConfig(64, 64, 0)
    assert lib.moe_dense_plan(None, 1, 0, 152, ctypes.byref(p)) == 1
    assert lib.moe_dense_plan(ctypes.byref(ok), 0, 0, 152, ctypes.byref(p)) == 1
    assert lib.moe_dense_plan(ctypes.byref(ok), 1, 0, 0, ctypes.byref(p)) == 1
    assert lib.moe_dense_plan(ctypes.byref(ok), 1, 0, 152, None) == 1
    assert lib.moe_dense_plan(ctypes.byref(MoEDenseConfig(64, 60, 0)), 1, 0, 152, ctypes.byref(p)) == 2
    huge = MoEDenseConfig(2 ** 31 - 2, 8, 0)
    assert lib.moe_dense_plan(ctypes.byref(huge), 2 ** 31 - 1, 0, 152, ctypes.byref(p)) == 2


def test_dense_null_handles(lib):
    assert lib.moe_dense_arm_timeout(None) == 1
    assert lib.moe_dense_create(None, P, P, None) == 1
    assert lib.moe_dense_run(None, 1, P, 0, P, 0, 0) == 1
    flags = ctypes.c_uint32(7)
    assert lib.moe_dense_get_error(None, 0, ctypes.byref(flags)) == 1 and flags.value == 0
    assert lib.moe_dense_destroy(None) == 0


# ---------------------------------------------------------------------------
# the binding's checks
# ---------------------------------------------------------------------------

def test_route_arguments(moe):  # noqa: F811
    z = fake((4, 16), F32)
    for kw, what in ((dict(score="max"), "score must be one of"),
                     (dict(group_score="sum"), "group_score must be one of"),
                     (dict(bias=fake((15,), F32)), "bias: expected shape"),
                     (dict(bias=fake((16,), F32, 1)), "bias: expected a tensor on cuda:0")):
        with pytest.raises(ValueError, match=what):
            moe.route_experts(z, 2, **kw)
    with pytest.raises(TypeError, match="logits: expected torch.float32"):
        moe.route_experts(fake((4, 16), torch.float16), 2)
    with pytest.raises(TypeError, match="bias: expected torch.float32"):
        moe.route_experts(z, 2, bias=fake((16,), BF16))
    with pytest.raises(ValueError, match="k must be positive"):
        moe.route_experts(z, 0)
    with pytest.raises(ValueError, match="contiguous"):
        moe.route_experts(fake((16, 4), F32).T, 2)


def test_norm_arguments(moe):  # noqa: F811
    x, w = fake((4, 64), BF16), fake((64,), BF16)
    for kw, what in ((dict(gate=fake((4, 2), BF16)), "gate: expected a value per"),
                     (dict(gate=fake((4,), BF16)), "gate: expected a value per"),
                     (dict(gate=fake((), BF16)), "gate: expected a value per"),
                     (dict(gate=fake((64,), BF16, 1)), "gate: expected a tensor on cuda:0"),
                     (dict(gate_fn="tanh"), "there is no gate"),
                     (dict(gate=w, gate_fn="relu"), "gate_fn must be one of"),
                     (dict(bf16=False), "ask for bf16 rows"),
                     (dict(pre_weight=None, mxfp8=True), "need a pre_weight"),
                     (dict(post_weight=fake((64,), BF16, 1)), "post_weight: expected a tensor on"),
                     (dict(pre_weight=fake((63,), BF16)), "pre_weight: expected shape"),
                     (dict(residual=fake((4, 64), BF16, 1)), "residual: expected a tensor on")):
        with pytest.raises(ValueError, match=what):
            moe.norm_add_norm(x, **(dict(residual=x, post_weight=w, pre_weight=w) | kw))
    with pytest.raises(TypeError, match="gate: expected torch.bfloat16"):
        moe.norm_add_norm(x, x, w, w, gate=fake((64,), F32))


def test_dense_arguments(moe):  # noqa: F811
    for args, kw, what in (((fake((8, 64), BF16),), dict(activation="swish"), "activation must be"),
                           ((fake((8, 64, 1), BF16),), {}, "two dimensions"),
                           ((fake((8, 64), BF16), fake((7,), BF16)), {}, "bias: expected shape"),
                           ((fake((8, 64), BF16), fake((8,), BF16, 1)), {}, "bias: expected a tensor on")):
        with pytest.raises(ValueError, match=what):
            moe.DenseProduct(*args, **kw)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        moe.DenseProduct([1.0])
    with pytest.raises(TypeError, match="weight: expected torch.bfloat16"):
        moe.DenseProduct(fake((8, 64), F32))

    def run(x, res=None, device=0):
        return moe.block._moe_torch.dense_run(P, device, 64, 8, x, res, None, False, None)
    x = fake((4, 64), BF16)
    for args, what in (((fake((4, 63), BF16),), "x: expected shape"),
                       ((x, fake((4, 64), BF16)), "residual: expected shape"),
                       ((x, fake((4, 8), BF16, 1)), "residual: expected a tensor on cuda:0"),
                       ((x, None, 1), "x: expected a tensor on cuda:1, where the weight is")):
        with pytest.raises(ValueError, match=what):
            run(*args)


# ---------------------------------------------------------------------------
# pins of the oracle
# ---------------------------------------------------------------------------

def test_scores_against_torch():
    z = np.random.default_rng(1).standard_normal((20, 33)) * 4
    t = torch.from_numpy(z)
    assert np.allclose(ref.scores(z, "softmax"), t.softmax(1).numpy(), rtol=1e-14)
    assert np.allclose(ref.scores(z, "sigmoid"), t.sigmoid().numpy(), rtol=1e-14)


def test_choice_without_options_is_the_layers_router():
    z = np.random.default_rng(2).standard_normal((50, 64)).astype(np.float32)
    ids, w = oracle.route(z, 6)
    got, gw = ref.route_experts(z, 6)
    assert np.array_equal(got, ids) and np.allclose(gw, w, rtol=1e-6)


def test_choice_within_groups_by_hand():
    z = np.log(np.array([[1.0, 9.0, 5.0, 6.0, 8.0, 1.0, 3.0, 3.0]]))
    # largest of each pair 9, 6, 8, 3; sums of two 10, 11, 9, 6
    ids, w = ref.route_experts(z, 2, groups=4, top_groups=2)
    assert ids.tolist() == [[1, 4]] and np.allclose(w, [[9 / 17, 8 / 17]])
    ids, w = ref.route_experts(z, 3, groups=4, top_groups=2, group_score="top2", renormalize=False,
                               scale=2.0)
    assert ids.tolist() == [[1, 3, 2]] and np.allclose(w, np.array([[9, 6, 5]]) / 36 * 2)
    # a bias moves the choice and no weight
    ids, w = ref.route_experts(z, 1, bias=np.array([0, 0, 0, 0, 0, 1, 0, 0.0]), renormalize=False)
    assert ids.tolist() == [[5]] and np.allclose(w, 1 / 36)


def test_choice_of_equals_and_of_none():
    z = np.zeros((1, 6))
    assert ref.route_experts(z, 4)[0].tolist() == [[0, 1, 2, 3]]
    assert ref.route_experts(z, 2, groups=3, top_groups=1)[0].tolist() == [[0, 1]]
    z[0, :5] = -np.inf
    ids, w = ref.route_experts(z, 3)
    assert ids.tolist() == [[5, -1, -1]] and w.tolist() == [[1, 0, 0]]
    ids, w = ref.route_experts(np.full((1, 6), np.nan), 2, "sigmoid", np.ones(6))
    assert ids.tolist() == [[-1, -1]] and w.tolist() == [[0, 0]]


def test_norms_against_torch():
    r = np.random.default_rng(3)
    x, res, post = r.standard_normal((4, 24)), r.standard_normal((4, 24)), r.standard_normal(24)
    gate = r.standard_normal((4, 1))
    t, _ = ref.norm_add(x, res, post, gate, "tanh", 0.5, 2.0, 1e-3, unit_offset=True)
    X = torch.from_numpy(x)
    p = torch.nn.functional.rms_norm(X, (24,), torch.from_numpy(1 + post), 1e-3)
    want = 2.0 * torch.from_numpy(res) + 0.5 * p * torch.tanh(torch.from_numpy(gate))
    assert np.allclose(t, want.numpy(), rtol=1e-13)


def test_activations_against_torch():
    y = np.random.default_rng(4).standard_normal((6, 10)) * 3
    t, F = torch.from_numpy(y), torch.nn.functional
    for act, want in (("relu", F.relu(t)), ("silu", F.silu(t)), ("gelu", F.gelu(t)),
                      ("gelu_tanh", F.gelu(t, approximate="tanh")),
                      ("silu_mul", F.silu(t[:, :5]) * t[:, 5:]), (None, t)):
        assert np.allclose(ref.activate(y, act), want.numpy(), rtol=1e-12, atol=1e-15), act
