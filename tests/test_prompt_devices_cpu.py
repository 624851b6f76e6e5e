"""Tensors of different devices are refused by the prompt operators before
anything is allocated or launched: fake tensors of two GPUs, on any machine."""
from unittest import mock

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import __graft_entry__

BF16, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32


@pytest.fixture(scope="module")
def moe():
    b = __graft_entry__._build_module()
    if b.stale(b.OUT):
        b.build()
    import sparse_expert_gemv_gb300
    return sparse_expert_gemv_gb300


def fake(shape, dtype, device=0):
    # (where there is a GPU, torch would touch the device of a fake tensor)
    with mock.patch.object(torch.cuda, "is_available", lambda: False), FakeTensorMode():
        return torch.empty(shape, dtype=dtype, device=f"cuda:{device}")


def inputs(other, **spec):
    """Fake tensors on cuda:0, the one named `other` on cuda:1."""
    return {k: fake(*v, device=int(k == other)) for k, v in spec.items()}


@pytest.mark.parametrize("other", ["weight", "residual"])
def test_norm(moe, other):
    a = inputs(other, x=((4, 64), BF16), weight=((64,), BF16), residual=((4, 64), BF16))
    with pytest.raises(ValueError, match=f"{other}: expected a tensor on cuda:0, got one on cuda:1"):
        moe.add_rms_norm(a["x"], a["weight"], a["residual"])


@pytest.mark.parametrize("other", ["slots", "w", "residual"])
def test_combine(moe, other):
    a = inputs(other, y=((4, 64), BF16), slots=((2, 2), I32), w=((2, 2), F32), residual=((2, 64), BF16))
    with pytest.raises(ValueError, match=f"{other}: expected a tensor on cuda:0, got one on cuda:1"):
        moe.combine(a["y"], a["slots"], a["w"], residual=a["residual"])


def run(moe, a, device):
    return moe.prompt._moe_torch.product_run(1 << 12, device, 2, 128, 64, False, a["a"], a["a_scales"],
                                             a["offsets"], a["rows"], None, None, None)


PRODUCT = dict(a=((4, 64), U8), a_scales=((4, 2), U8), offsets=((3,), I32), rows=((6,), I32))


@pytest.mark.parametrize("other", ["a_scales", "offsets", "rows"])
def test_product(moe, other):
    with pytest.raises(ValueError, match=f"{other}: expected a tensor on cuda:0, got one on cuda:1"):
        run(moe, inputs(other, **PRODUCT), 0)


def test_product_on_another_device_than_its_weights(moe):
    with pytest.raises(ValueError, match="a: expected a tensor on cuda:1, where the weights are"):
        run(moe, inputs(None, **PRODUCT), 1)


def test_product_handle_is_made_on_the_weights_device(moe, monkeypatch):
    made, current = [], []

    class Device:
        def __init__(self, device):
            self.device = torch.device(device)

        def __enter__(self):
            current.append(self.device)

        def __exit__(self, *_):
            current.pop()

    class Lib:
        @staticmethod
        def moe_product_create(*_):
            made.append(list(current))
            return 0

    monkeypatch.setattr(moe.prompt.torch.cuda, "device", Device)
    monkeypatch.setattr(moe.prompt, "lib", Lib)
    monkeypatch.setattr(moe.prompt, "_ptr", lambda t: 1 << 12)
    monkeypatch.setattr(moe.prompt, "_stream", lambda s: 0)
    moe.GroupedProduct(fake((2, 128, 64), U8, 1), fake((2, 128, 2), U8, 1))
    assert made == [[torch.device("cuda:1")]]
    with pytest.raises(ValueError, match="w_scales: expected a tensor on cuda:1, got one on cuda:0"):
        moe.GroupedProduct(fake((2, 128, 64), U8, 1), fake((2, 128, 2), U8, 0))
    assert len(made) == 1
