"""The prompt operators' failure and stream behaviour on a GPU."""
import pytest
import torch

from test_gpu_prompt import Products, dev  # noqa: F401  (dev: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("silu", [False, True])
def test_product_winds_down_when_its_waits_give_up(dev, silu, gather):  # noqa: F811
    # failure detection without a fault: the MMAs' bounded wait runs out (for an
    # arrival that nothing makes), and then every other role's; the launch ends, the
    # handle reports it once, and the next runs are right
    from sparse_expert_gemv_gb300 import MOE_DEVICE_TIMEOUT
    c = Products(dev, "mxfp8", 512, 2048, [200, 0, 31, 400], 31, gather)
    args = c.args()
    p = c.handle(silu)
    want = p(*args)
    assert p.get_error() == 0
    c.check(silu, want)
    for _ in range(3):
        p.arm_timeout()
        p(*args)
        assert p.get_error() == MOE_DEVICE_TIMEOUT
        assert p.get_error() == 0
        got = p(*args)
        for x, y in zip(got if silu else [got], want if silu else [want]):
            assert torch.equal(x, y)
        assert p.get_error() == 0


def test_an_armed_timeout_waits_for_a_run_that_launches(dev):  # noqa: F811
    from sparse_expert_gemv_gb300 import MOE_DEVICE_TIMEOUT
    c = Products(dev, "mxfp8", 128, 1024, [40], 32)
    a, s, off, _ = c.args()
    p = c.handle(False)
    p.arm_timeout()
    p(a[:0], s[:0], off)
    assert p.get_error() == 0
    p(a, s, off)
    assert p.get_error() == MOE_DEVICE_TIMEOUT


def calls(dev):  # noqa: F811
    """Each operator as a call of its keyword arguments, with small inputs."""
    from sparse_expert_gemv_gb300 import add_rms_norm, combine, group_by_expert
    g = torch.Generator(device=dev).manual_seed(33)
    x, res = (torch.randn(64, 512, device=dev, generator=g).bfloat16() for _ in range(2))
    weight = torch.ones(512, dtype=torch.bfloat16, device=dev)
    ids = torch.randint(0, 9, (64, 4), dtype=torch.int32, device=dev, generator=g)
    w = torch.rand(64, 4, device=dev, generator=g)
    y = torch.randn(256, 512, device=dev, generator=g).bfloat16()
    slots = torch.randperm(256, device=dev, generator=g).int().view(64, 4)
    c = Products(dev, "mxfp8", 256, 512, [100, 156], 34)
    plain, gate_up, args = c.handle(False), c.handle(True), c.args()
    return {"norm": lambda **kw: add_rms_norm(x, weight, res, mxfp8=True, **kw),
            "group": lambda **kw: group_by_expert(ids, 9, **kw),
            "combine": lambda **kw: combine(y, slots, w, residual=res, **kw),
            "product": lambda **kw: plain(*args, **kw),
            "gate/up": lambda **kw: gate_up(*args, **kw)} | decode_calls(dev)


def decode_calls(dev):  # noqa: F811
    layer, T = small_layer(dev), 30
    g = torch.Generator(device=dev).manual_seed(37)
    logits = torch.randn(T, layer.E, device=dev, generator=g)
    ids, w = layer.route(logits)
    x = torch.randn(T, layer.H, device=dev, generator=g).bfloat16()
    h = layer.gate_up(x, ids)
    return {"route": lambda **kw: layer.route(logits, **kw),
            "schedule": lambda **kw: layer.dedup_schedule(ids, **kw),
            "decode gate/up": lambda **kw: layer.gate_up(x, ids, **kw),
            "decode down": lambda **kw: layer.down(h, ids, w, **kw),
            "decode layer": lambda **kw: layer.layer(x, ids, w, **kw)}


def small_layer(dev, fmt="mxfp8"):  # noqa: F811
    import numpy as np
    import workloads as wl
    from sparse_expert_gemv_gb300 import MoEDecode
    experts = wl.make_experts(wl.Workload(91, "stream", 8, 2, 256, 128, 30, 0.05), 35, range(8), fmt=fmt)
    stack = [torch.from_numpy(np.stack([experts[e][i] for e in range(8)])).to(dev) for i in range(4)]
    return MoEDecode(*stack, k=2, max_T=30, fmt=fmt)


def listed(out):
    return [out] if isinstance(out, torch.Tensor) else list(out)


@pytest.mark.parametrize("op", ["norm", "group", "combine", "product", "gate/up", "route", "schedule",
                                "decode gate/up", "decode down", "decode layer"])
def test_outputs_on_a_given_stream_are_of_its_memory(dev, op):  # noqa: F811
    call = calls(dev)[op]
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


def prompt_args(dev, layer, T):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(36)
    codes = torch.randint(0, 120, (T, layer.H), dtype=torch.uint8, device=dev, generator=g)
    scales = torch.full((T, layer.H // 32), 120, dtype=torch.uint8, device=dev)
    ids = torch.randint(0, layer.E, (T, layer.k), dtype=torch.int32, device=dev, generator=g)
    return codes, scales, ids, torch.rand(T, layer.k, device=dev, generator=g)


def test_prompt_on_a_given_stream(dev):  # noqa: F811
    layer = small_layer(dev)
    args = prompt_args(dev, layer, 30)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = layer.prompt(*args, stream=side)
    side.synchronize()
    assert torch.equal(got, layer.prompt(*args))


def test_a_stream_is_a_torch_stream(dev):  # noqa: F811
    for name, call in calls(dev).items():
        with pytest.raises((TypeError, AttributeError)):
            call(stream=torch.cuda.Stream().cuda_stream)


def test_get_error_waits_for_a_prompt_on_another_stream(dev):  # noqa: F811
    from sparse_expert_gemv_gb300 import MOE_DEVICE_TIMEOUT
    layer = small_layer(dev)
    args = prompt_args(dev, layer, 30)
    layer.prompt(*args)
    assert layer.get_error() == 0
    side, busy = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for product in layer._products:
        product.arm_timeout()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
        layer.prompt(*args, stream=side)
        over = side.record_event()
        with torch.cuda.stream(busy):
            torch.cuda._sleep(2_000_000_000)
            end = busy.record_event()
        assert layer.get_error() == MOE_DEVICE_TIMEOUT
        # for that call's products, and for no other stream's work
        assert not end.query()
        over.synchronize()
        assert layer.get_error() == 0
        end.synchronize()


def test_product_get_error_waits_for_its_latest_call_and_for_a_replay(dev):  # noqa: F811
    from sparse_expert_gemv_gb300 import MOE_DEVICE_TIMEOUT
    c = Products(dev, "mxfp8", 128, 512, [40, 50], 38)
    args, p = c.args(), c.handle(False)
    out = torch.empty(c.R, 128, dtype=torch.bfloat16, device=dev)
    p(*args, out=out)
    assert p.get_error() == 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    p.arm_timeout()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        p(*args, out=out)
    assert p.get_error() == MOE_DEVICE_TIMEOUT        # from the default stream
    g = torch.cuda.CUDAGraph()
    p.arm_timeout()
    with torch.cuda.graph(g):
        p(*args, out=out)                              # every replay times out
    assert p.get_error() == 0
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        g.replay()
    assert p.get_error(side) == MOE_DEVICE_TIMEOUT


def test_reads_of_the_error_word_lose_no_bit(dev):  # noqa: F811
    # runs that time out and reads of the word from two threads: every timeout is
    # seen by exactly one read, the one that first follows it
    import threading
    from sparse_expert_gemv_gb300 import MOE_DEVICE_TIMEOUT
    c = Products(dev, "mxfp8", 128, 512, [40], 39)
    args, p = c.args(), c.handle(False)
    p(*args)
    assert p.get_error() == 0
    seen = []
    for _ in range(20):
        p.arm_timeout()
        p(*args)
        threads = [threading.Thread(target=lambda: seen.append(p._latest_error())) for _ in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    assert sorted(seen) == [0] * 20 + [MOE_DEVICE_TIMEOUT] * 20


def test_buffers_on_another_device_are_refused(dev):  # noqa: F811
    from test_prompt_devices_cpu import fake
    want = {name: listed(call()) for name, call in calls(dev).items()}
    names = {"norm": ["sum", "y", "codes", "scales"], "group": ["offsets", "rows", "slots"],
             "combine": ["out"], "product": ["out"], "gate/up": ["out", "out_scales"]}
    for op, call in calls(dev).items():
        for name, t in zip(names.get(op, []), want[op]):
            with pytest.raises(ValueError, match=f"{name}: expected a tensor on cuda:0, got one on cuda:1"):
                call(**{name: fake(t.shape, t.dtype, 1)})
