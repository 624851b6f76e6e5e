"""The products at the edges of their tiles: groups are cut into the fewest
pieces of at most 192 rows, equal but for rounding to 32, and the weight rows
into pairs of 128 (of 64 neurons with silu_mul). Tolerances as in
test_gpu_prompt.py."""
import pytest
import torch

from test_gpu_prompt import Products, dev  # noqa: F401  (dev: the fixture)

pytestmark = pytest.mark.gpu

COUNTS = [
    [191, 192, 193],                 # one piece up to 192, then two
    [383, 384, 385, 0, 1],           # two, then three
    [1153],                          # six pieces of 192 and a row: seven of 192 and less
    [31, 32, 33, 63, 64, 65, 127, 128, 129, 159, 160, 161],   # the MMA's columns, second scale block
    [576, 577, 768, 769]]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("counts", COUNTS)
def test_groups_at_the_edges_of_a_piece(dev, counts, fmt, silu, gather):  # noqa: F811
    c = Products(dev, fmt, 192, 256, counts, 41, gather)
    a, s, off, rows = c.args()
    p = c.handle(silu)
    shape = (c.R, 96 if silu else 192)
    out = torch.full(shape, 7, dtype=torch.uint8 if silu else torch.bfloat16, device=dev)
    got = p(a, s, off, rows, out=out)
    c.check(silu, got)
    assert p.get_error() == 0


@pytest.mark.parametrize("silu,N", [(False, n) for n in (120, 128, 136, 248, 256, 264, 384, 512)] +
                         [(True, n) for n in (64, 128, 192, 256, 320, 512)])
def test_weight_rows_at_the_edges_of_a_tile(dev, silu, N):  # noqa: F811
    c = Products(dev, "mxfp8", N, 160, [5, 0, 193, 30], 42, gather=silu)
    a, s, off, rows = c.args()
    p = c.handle(silu)
    c.check(silu, p(a, s, off, rows))
    assert p.get_error() == 0


@pytest.mark.parametrize("K", [32, 96, 128, 160, 384, 512, 544, 640, 768, 896, 1024, 7168])
@pytest.mark.parametrize("gather", [False, True])
def test_reduction_lengths_around_stages_and_batches(dev, K, gather):  # noqa: F811
    # 128 elements a stage, four stages a batch of scales, six stages in the ring
    for silu in (False, True):
        c = Products(dev, "mxfp8", 128, K, [70, 193, 1], 43, gather)
        a, s, off, rows = c.args()
        p = c.handle(silu)
        c.check(silu, p(a, s, off, rows))
        assert p.get_error() == 0
