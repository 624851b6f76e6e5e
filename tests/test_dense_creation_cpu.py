"""The stream that a dense product's creation waits for, on a machine without a GPU."""
from types import SimpleNamespace

import pytest
import torch

from test_prompt_devices_cpu import fake, moe  # noqa: F401  (moe: the fixture)


def test_a_stream_of_another_device_is_refused(moe):  # noqa: F811
    other = SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream: expected one of cuda:0, got one of cuda:1"):
        moe.DenseProduct(fake((8, 64), torch.bfloat16), stream=other)


@pytest.mark.parametrize("given", [False, True])
def test_the_stream_is_waited_for_before_the_handle_is_made(moe, given, monkeypatch):  # noqa: F811
    import contextlib
    from sparse_expert_gemv_gb300 import block
    order = []
    stream = SimpleNamespace(device=torch.device("cuda", 0), synchronize=lambda: order.append("waited"))
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: stream)
    monkeypatch.setattr(block, "_ptr", lambda t: 0)
    monkeypatch.setattr(block, "lib", SimpleNamespace(
        moe_dense_create=lambda *a: order.append("made") or 0, moe_dense_destroy=lambda h: 0))
    moe.DenseProduct(fake((8, 64), torch.bfloat16), stream=stream if given else None)
    assert order == ["waited", "made"]
