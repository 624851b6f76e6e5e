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
