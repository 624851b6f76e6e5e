"""The router's choice handed to the decode layer: slots that no expert is left for
add nothing, in every form of the layer, and only they set MOE_DEVICE_BAD_ID."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from gpu_util import Case, assert_within, bf16_tensor, device_weights, tensor_to_f64, tol_y
from test_gpu_prompt import dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("left,padded", [(None, 0), (None, 5), (3, 0), (1, 3)])
@pytest.mark.parametrize("c,path,T", [(0, "warp", 1), (0, "warp", 9), (0, "warp", 40), (1, "warp", 1),
                                      (1, "tensor", 24)])
def test_slots_without_an_expert(dev, c, path, T, left, padded):  # noqa: F811
    # `left`: experts that are not switched off; the last rows are padding
    from sparse_expert_gemv_gb300 import MOE_DEVICE_BAD_ID, MoEDecode, add_rms_norm, route_experts
    case = Case(c, T, tokens=[])
    w = case.w
    z = torch.from_numpy(np.float32(case.logits)).to(dev)
    if left is not None:
        z[:, left:] = -float("inf")
    z[T - min(padded, T):] = -float("inf")
    ids, tw = route_experts(z, w.k, score="sigmoid")
    none = ids.eq(-1)
    assert none.any().item() == (padded > 0 or left is not None and left < w.k) and tw[none].eq(0).all()
    picked = ids.cpu().numpy()
    experts = wl.make_experts(w, case.seed, np.unique(picked[picked >= 0]))
    layer = MoEDecode(*device_weights(w, experts, dev, fill="finite"), k=w.k, max_T=T)
    layer.set_path(path)
    x = bf16_tensor(case.x_bits, dev)
    y = layer.layer(x, ids, tw)
    rows = sorted({0, T // 2, T - 1, max(0, T - 4)})
    want = oracle.layer(case.x64(), picked, tw.cpu().numpy(), experts, w.E, w.H, w.I, tokens=rows)["y_spec"]
    assert_within(tensor_to_f64(y)[rows], want[rows], tol_y(want[rows]), "y")
    assert y[none.all(1)].eq(0).all() and y.isfinite().all()
    assert layer.get_error() == (MOE_DEVICE_BAD_ID if none.any() else 0)
    n = add_rms_norm(x, torch.ones(w.H, dtype=torch.bfloat16, device=dev), bf16=False, mxfp8=True)
    out = layer.prompt(n.codes, n.scales, ids, tw)
    assert out[none.all(1)].eq(0).all() and out.isfinite().all() and layer.get_error() == 0
