"""What a transformer block with routed experts needs between them.

The router's choice, the norms around a block's end and dense products with
their epilogues (include/moe_block.h states each one's arithmetic). With the
operators of prompt.py a block with a shared expert over a prompt is

    n = norm_add_norm(x, residual, post_weight, pre_weight, mxfp8=True)
    logits = router(n.y, float32=True)                     # DenseProduct
    ids, w = route_experts(logits, k, score="sigmoid", bias=bias, groups=8, top_groups=4,
                           group_score="top2", scale=2.5)
    h = shared_gate_up(n.y)                                # DenseProduct, "silu_mul"
    out = layer.prompt(n.codes, n.scales, ids, w, residual=shared_down(h))

and for a decode batch the same with layer.layer (which reports slots without an
expert by MOE_DEVICE_BAD_ID; see route_experts). Like the rest of the package these are forward operators: inputs that require grad are taken as they are,
and the results carry no graph. Every call forwards device pointers and a
stream to libmoe_decode.so through the extension module _moe_torch, which
checks the tensors, allocates the outputs that were not passed in, and takes
the current stream or the torch.cuda.Stream given as `stream`. New outputs
belong to the stream of the call, as if it were current. Outputs that are passed
in share no memory with other tensors of the call, but where it says so; such
calls are refused.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import MoEDenseConfig, check, lib
from ._tensors import _need, _ptr, _stream
from .prompt import RmsNorm, _moe_torch

_SCORES = {"softmax": 0, "sigmoid": 0x2}
_GROUP_SCORES = {"max": 0, "top2": 0x4}
_RENORMALIZE = 0x8
_GATE_FNS = {None: 0, "sigmoid": 0x4, "tanh": 0x8}
_UNIT_OFFSET = 0x10
_ACTIVATIONS = {None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4, "silu_mul": 5}


def _one_of(value, table: dict, name: str) -> int:
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {', '.join(map(repr, table))}, got {value!r}") from None


def route_experts(logits, k: int, *, score: str = "softmax", bias=None, groups: int = 1,
                  top_groups: int | None = None, group_score: str = "max",
                  renormalize: bool = True, scale: float = 1.0, ids=None, w=None, stream=None):
    """(ids int32 [T, k], w float32 [T, k]): the experts every token takes, best
    first, and their weights, from router logits [T, E] in float32 or bf16.

    Experts compare by their scores (`score`, "softmax" or "sigmoid") plus
    `bias` float32 [E], which no weight contains. With `groups` groups of
    neighbouring experts, the choice is made within the `top_groups` groups
    (all of them if not given) of the best group scores: their largest
    compared score ("max"), or the sum of their two largest ("top2"). Of equal
    scores the lower index wins, and close ones are told apart as FP64
    arithmetic does. The weights are the chosen scores, divided by their sum
    (`renormalize`) and times `scale`.

    A logit of NaN or -inf switches its expert off for that token, a bias of
    NaN or -inf for all. Slots that no expert is left for get the id -1 and
    the weight 0. They add nothing to what MoEDecode makes of them; its prompt
    takes them as unused, while to layer, gate_up and down they are ids out of
    range, after which get_error reports MOE_DEVICE_BAD_ID although nothing failed.
    """
    flags = _one_of(score, _SCORES, "score") | _one_of(group_score, _GROUP_SCORES, "group_score")
    if renormalize:
        flags |= _RENORMALIZE
    return _moe_torch.route_experts(logits, bias, k, groups,
                                    groups if top_groups is None else top_groups, scale, flags,
                                    ids, w, stream)


def norm_add_norm(x, residual, post_weight=None, pre_weight=None, *, gate=None, gate_fn=None,
                  scale: float = 1.0, residual_scale: float = 1.0, unit_offset: bool = False,
                  eps: float = 1e-6, bf16: bool = True, mxfp8: bool = False, sum=None, y=None,
                  codes=None, scales=None, stream=None) -> RmsNorm:
    """The end of a block and the start of the next one:

        p = x * rsqrt(mean(x^2) + eps) * post_weight        (x without post_weight)
        s = bf16(residual_scale * residual + scale * gate_fn(gate) * p)
        n = s * rsqrt(mean(s^2) + eps) * pre_weight

    x and residual are bf16 [T, H], the weights bf16 [H]; with unit_offset
    they are stored less one. gate is bf16: [H] (a value per channel), [T, 1]
    (per row) or [T, H]; gate_fn is None, "sigmoid" or "tanh". Returns s as RmsNorm.sum and n in
    bf16 (`bf16`), as MXFP8 codes and scales (`mxfp8`), or both; without
    pre_weight s alone. The buffers sum, y, codes and scales may be passed in;
    sum may be x or residual, which is then updated in place, and y the one of
    them that sum is not.
    """
    flags = _one_of(gate_fn, _GATE_FNS, "gate_fn") | (_UNIT_OFFSET if unit_offset else 0)
    if gate is None and gate_fn is not None:
        raise ValueError("gate_fn: there is no gate")
    return RmsNorm._make(_moe_torch.norm_add_norm(
        x, residual, post_weight, pre_weight, gate, scale, residual_scale, eps, flags, bf16, mxfp8,
        sum, y, codes, scales, stream))


class DenseProduct:
    """Products of bf16 rows with one weight matrix: act(x @ weight.T + bias) + residual.

    weight is bf16 [N, K] with K a multiple of 8, bias bf16 [N] or None; both
    are borrowed (kept alive by this object), are not to be written while it
    lives (a call reads ahead of earlier work on its stream), and lie where the
    rows of every call have to. Making the handle waits for `stream` (the
    current one of the weight's device if not given), on which they may have
    been written. `activation` is None, "relu", "silu", "gelu",
    "gelu_tanh", or "silu_mul": the N = 2I weight rows are then I gate rows and
    I up rows, and the result is the I values SiLU(gate) * up. The handle is
    made outside graph captures; calls may be captured, and calls on several
    streams may overlap.
    """

    def __init__(self, weight, bias=None, *, activation: str | None = None, stream=None):
        act = _one_of(activation, _ACTIVATIONS, "activation")
        if not isinstance(weight, torch.Tensor):
            raise TypeError("weight must be a torch.Tensor")
        if weight.dim() != 2:
            raise ValueError(f"weight: expected two dimensions, got {weight.dim()}")
        N, K = weight.shape
        _need(weight, torch.bfloat16, (N, K), "weight")
        if bias is not None:
            _need(bias, torch.bfloat16, (N,), "bias")
            if bias.device != weight.device:
                raise ValueError(f"bias: expected a tensor on {weight.device}, got one on {bias.device}")
        if stream is not None and stream.device != weight.device:
            raise ValueError(f"stream: expected one of {weight.device}, got one of {stream.device}")
        self.N, self.K, self.activation = N, K, activation
        self.M = N // 2 if activation == "silu_mul" else N
        self._weights, self._device = (weight, bias), weight.device.index
        h = ctypes.c_void_p()
        with torch.cuda.device(weight.device):
            # nothing orders a call's early reads behind what writes the weight
            (torch.cuda.current_stream() if stream is None else stream).synchronize()
            check(lib.moe_dense_create(ctypes.byref(MoEDenseConfig(N, K, act)), _ptr(weight),
                                       _ptr(bias), ctypes.byref(h)), "moe_dense_create")
        self._h = h

    def close(self) -> None:
        if getattr(self, "_h", None):
            lib.moe_dense_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self) -> ctypes.c_void_p:
        return self._h

    def __call__(self, x, residual=None, *, out=None, float32: bool = False, stream=None):
        """bf16 [R, M] (float32 with `float32`) from x bf16 [R, K] and residual
        bf16 [R, M] or None; M is N, or N / 2 with "silu_mul". `out` may be
        passed in, and may be the residual where it is bf16."""
        h = self._h.value if self._h else 0
        return _moe_torch.dense_run(h, self._device, self.K, self.M, x, residual, out, float32,
                                    stream)

    def arm_timeout(self) -> None:
        """Test support: the bounded waits of the next run that launches
        something run out (it sets MOE_DEVICE_TIMEOUT, which get_error
        reports)."""
        check(lib.moe_dense_arm_timeout(self._h), "moe_dense_arm_timeout")

    def get_error(self, stream=None) -> int:
        """Read and clear the handle's device error bits, after waiting for the
        handle's latest call and for the stream (the current one if not given)."""
        flags = ctypes.c_uint32(0)
        with torch.cuda.device(self._device):
            st = lib.moe_dense_get_error(self._h, _stream(stream), ctypes.byref(flags))
        if st not in (0, 5):
            check(st, "moe_dense_get_error")
        return int(flags.value)
