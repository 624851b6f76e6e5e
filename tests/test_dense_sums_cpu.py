"""How long a dense product's sums grow in the tensor cores, which cut them off at
each step: with FP32 outputs no accumulator takes more than 512 K, whatever the
rows and however long K is."""
import numpy as np
import pytest

from test_block_cpu import lib, moe, plan  # noqa: F401  (fixtures)


def stages_an_accumulator(p, K):
    """Of moe_dense_split with FP32 outputs: half of tensor memory, 256 columns, in
    accumulators of 32, 64 or 128."""
    nk = -(-K // 64)
    part = -(-nk // p.parts)
    most = 256 // (32 if p.nt <= 32 else 64 if p.nt <= 64 else 128)
    accumulators = min(-(-part // 8), most)
    return -(-part // accumulators)


@pytest.mark.parametrize("R,K,N", [
    (128, 28672, 1024), (128, 65536, 1024), (128, 131072, 256), (1, 65536, 1024), (1, 8192, 64),
    (16, 32768, 256), (16, 32832, 256), (64, 16384, 384), (3, 1 << 20, 128), (1, 1 << 24, 8)])
@pytest.mark.parametrize("act", [0, 5])
def test_long_k(lib, R, K, N, act):  # noqa: F811
    p = plan(lib, R, K, N, act, out_float=1)
    assert not p.split or stages_an_accumulator(p, K) <= 8


def test_any_k(lib):  # noqa: F811
    r = np.random.default_rng(6)
    for _ in range(4000):
        R, K, N = (int(np.exp(r.uniform(0, np.log(hi)))) for hi in (4000, 40000, 6000))
        K, N, act = 8 * K, 2 * N, int(r.choice([0, 5]))
        sms = int(r.choice([8, 76, 152]))
        p = plan(lib, R, K, N, act, sms, 1)
        assert not p.split or stages_an_accumulator(p, K) <= 8, (R, K, N, act, sms)


def test_k_up_to_8192_is_cut_as_it_was(lib):  # noqa: F811
    # FP32 outputs of few rows, with eight parts
    for R, K, N, nt in ((1, 8192, 64, 16), (8, 7168, 256, 16), (64, 8192, 128, 16), (100, 8192, 256, 16)):
        p = plan(lib, R, K, N, 0, 152, 1)
        assert (p.split, p.parts) == (1, 8) and p.nt == nt, (R, K, N, p.nt, p.parts)
