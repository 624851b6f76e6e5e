"""The block's operators beside the decode layer and the prompt operators: different
kernels side by side on several streams, eager and replayed, give what they give
alone."""
import numpy as np
import pytest
import torch

import workloads as wl
from gpu_util import bf16_tensor, device_weights
from test_gpu_block import Block, Dense
from test_gpu_prompt import bf16, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def calls(dev):  # noqa: F811
    from sparse_expert_gemv_gb300 import MoEDecode
    w = wl.Workload(96, "streams", 16, 4, 512, 256, 64, 0.05)
    experts = wl.make_experts(w, 97, range(w.E))
    layer = MoEDecode(*device_weights(w, experts, dev), k=w.k, max_T=64)
    x = bf16_tensor(wl.make_x(w, 97, 64), dev)
    logits = torch.from_numpy(np.float32(wl.make_logits(w, 97, 64))).to(dev)
    block = Block(dev, 90)
    few, many = Dense(30, 1024, 4096, True, "gelu", True, seed=98), Dense(2500, 512, 2600, True, "silu", True, seed=99)
    handles = few.handle(dev), many.handle(dev)
    args = [(bf16(c.x, dev), bf16(c.res, dev)) for c in (few, many)]

    def decode():
        ids, tw = layer.route(logits, score="sigmoid", groups=4, top_groups=2)
        return [ids, tw, layer.layer(x, ids, tw)]

    def products():
        return [p(*a, float32=f) for p, a in zip(handles, args) for f in (False, True)]
    return [block, decode, products], [layer.get_error, block.router.get_error, handles[0].get_error,
                                       handles[1].get_error]


def test_different_operators_at_once(dev):  # noqa: F811
    work, errors = calls(dev)
    want = [[t.clone() for t in f()] for f in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    graphs = []
    for s, f in zip(streams, work):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = f()
        graphs.append((g, out))
    for replay in (False, True):
        torch.cuda.synchronize()
        got = [[] for _ in work]
        for _ in range(12):
            for i, (s, f) in enumerate(zip(streams, work)):
                with torch.cuda.stream(s):
                    if replay:
                        graphs[i][0].replay()
                        got[i].append([t.clone() for t in graphs[i][1]])
                    else:
                        got[i].append(f())
        torch.cuda.synchronize()
        for outs, like in zip(got, want):
            for out in outs:
                for a, b in zip(out, like):
                    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert [e() for e in errors] == [0] * 4
