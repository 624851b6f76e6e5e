"""The operators around the routed experts for calls of many tokens.

The mixture-of-experts half of a transformer block over a prompt, with MXFP8
activations between the operators (include/moe_prompt.h states each one's
arithmetic):

    n = add_rms_norm(x, weight, residual)              # n.sum, n.y, n.codes, n.scales
    ids, w = layer.route(router_logits(n.y))
    offsets, rows, slots = group_by_expert(ids, E)
    hc, hs = gate_up(n.codes, n.scales, offsets, rows=rows)   # GroupedProduct, silu_mul=True
    y = down(hc, hs, offsets)                                 # GroupedProduct
    out = combine(y, slots, w, residual=n.sum)

MoEDecode.prompt is the part after the router on a layer's own weights. Like
the rest of the package these are forward operators: inputs that require grad
are taken as they are, and the results carry no graph. As in
the decode layer, every call forwards device pointers and a stream to
libmoe_decode.so; nothing is computed here. The calls a block makes go through
the extension module _moe_torch (csrc/moe_torch.cpp), which checks the tensors,
allocates the outputs that were not passed in, and takes the current stream or
the torch.cuda.Stream given as `stream`. New outputs belong to the stream of
the call, as if it were current.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from ._lib import MOE_FLAG_MXFP4, MOE_PRODUCT_SILU_MUL, MoEError, MoEProductConfig, check, lib
from ._tensors import _need, _ptr, _stream

_BUILD = "build the extension module first (python -c 'import __graft_entry__ as g; g.build()')"
try:
    from . import _moe_torch
except ImportError as e:
    raise ImportError(f"_moe_torch.so is missing or does not load ({e}): {_BUILD}") from e
if _moe_torch.built_for != f"built with torch {torch.__version__}":
    raise ImportError(f"_moe_torch.so was {_moe_torch.built_for}, this is torch {torch.__version__}: "
                      f"{_BUILD}")
_moe_torch.set_error(MoEError)


class RmsNorm(NamedTuple):
    """What add_rms_norm returns; outputs that were not asked for are None."""
    sum: torch.Tensor | None      # bf16 [T, H]: the new residual stream
    y: torch.Tensor | None        # bf16 [T, H]: the normalised rows
    codes: torch.Tensor | None    # uint8 [T, H]: their E4M3 codes
    scales: torch.Tensor | None   # uint8 [T, H/32]: and UE8M0 scale codes


def add_rms_norm(x, weight, residual=None, *, eps: float = 1e-6, bf16: bool = True,
                 mxfp8: bool = False, sum=None, y=None, codes=None, scales=None,
                 stream=None) -> RmsNorm:
    """The residual stream s = bf16(x + residual) and s * rsqrt(mean(s^2) + eps) * weight,
    in bf16 (`bf16`), as MXFP8 codes and scales (`mxfp8`), or both.

    x and residual are bf16 [T, H], weight is bf16 [H]. No result requires grad,
    even where an input (a weight that is a Parameter) does. Without a residual,
    s is x and RmsNorm.sum is None (unless a buffer for it is passed). The
    buffers sum, y, codes and scales may be passed in; sum may be x or
    residual, which is then updated in place.
    """
    return RmsNorm._make(_moe_torch.add_rms_norm(
        x, weight, residual, eps, bf16, mxfp8, sum, y, codes, scales, stream))


def group_by_expert(ids, E: int, *, offsets=None, rows=None, slots=None, stream=None):
    """(offsets, rows, slots) of routed ids int32 [T, k]: group e is the rows
    offsets[e] .. offsets[e + 1] - 1 in the order of the slots t * k + j;
    rows[q] is the token of grouped row q (-1 past the last group) and
    slots[t, j] the grouped row of a slot (-1 for an id outside [0, E), which
    joins no group)."""
    return _moe_torch.group_by_expert(ids, E, offsets, rows, slots, stream)


def combine(y, slots, w, *, residual=None, out=None, stream=None):
    """out[t] = bf16(residual[t] + sum_j w[t, j] * y[slots[t, j]]) over expert
    rows y bf16 [R, H], slots int32 [T, k] (outside [0, R): nothing) and w
    float32 [T, k]; residual bf16 [T, H] is optional and may be `out`. The result
    carries no graph."""
    return _moe_torch.combine(y, slots, w, residual, out, stream)


class GroupedProduct:
    """Ragged products of grouped MXFP8 rows with one stack of expert weights.

    fmt="mxfp8": w uint8 [E, N, K]; fmt="mxfp4": w uint8 [E, N, K/2]; w_scales
    uint8 [E, N, K/32]. With silu_mul the N = 2I rows of an expert are I gate
    rows and I up rows, and the product is finished to MXFP8(SiLU(g) * u).
    The weights are borrowed (kept alive by this object); the scales are
    copied once into the order in which the tensor cores take them, on the
    weights' device, where the rows of every call have to lie.
    """

    def __init__(self, w, w_scales, *, fmt: str = "mxfp8", silu_mul: bool = False, stream=None):
        if fmt not in ("mxfp8", "mxfp4"):
            raise ValueError(f"fmt must be 'mxfp8' or 'mxfp4', got {fmt!r}")
        per = 2 if fmt == "mxfp4" else 1
        if not isinstance(w, torch.Tensor):
            raise TypeError("w must be a torch.Tensor")
        if w.dim() != 3:
            raise ValueError(f"w: expected three dimensions, got {w.dim()}")
        E, N, RB = w.shape
        K = RB * per
        _need(w, torch.uint8, (E, N, RB), "w")
        _need(w_scales, torch.uint8, (E, N, K // 32), "w_scales")
        if w_scales.device != w.device:
            raise ValueError(f"w_scales: expected a tensor on {w.device}, got one on {w_scales.device}")
        if stream is not None and stream.device != w.device:
            raise ValueError(f"stream: expected one of {w.device}, got one of {stream.device}")
        self.E, self.N, self.K, self.fmt, self.silu_mul = E, N, K, fmt, silu_mul
        self._weights, self._device = (w, w_scales), w.device.index
        flags = (MOE_FLAG_MXFP4 if fmt == "mxfp4" else 0) | (MOE_PRODUCT_SILU_MUL if silu_mul else 0)
        h = ctypes.c_void_p()
        with torch.cuda.device(w.device):      # the handle belongs to the weights' device
            check(lib.moe_product_create(ctypes.byref(MoEProductConfig(E, N, K, flags)), _ptr(w),
                                         _ptr(w_scales), ctypes.byref(h), _stream(stream)),
                  "moe_product_create")
        self._h = h

    def close(self) -> None:
        if getattr(self, "_h", None):
            lib.moe_product_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self) -> ctypes.c_void_p:
        return self._h

    def __call__(self, a, a_scales, offsets, rows=None, *, out=None, out_scales=None, stream=None):
        """For every expert e, rows offsets[e] .. offsets[e + 1] - 1 of the
        result from the MXFP8 rows a[rows[q]] (a[q] without `rows`) uint8
        [A, K] with scales uint8 [A, K/32]: bf16 [R, N], or with silu_mul the
        pair codes uint8 [R, I], scales uint8 [R, I/32]. R is the length of
        `rows`, or A. Rows outside every group are left as they are."""
        h = self._h.value if self._h else 0
        return _moe_torch.product_run(h, self._device, self.E, self.N, self.K, self.silu_mul, a,
                                      a_scales, offsets, rows, out, out_scales, stream)

    def arm_timeout(self) -> None:
        """Test support: the bounded waits of the next run that launches
        something run out (it sets MOE_DEVICE_TIMEOUT, which get_error
        reports)."""
        check(lib.moe_product_arm_timeout(self._h), "moe_product_arm_timeout")

    def get_error(self, stream=None) -> int:
        """Read and clear the handle's device error bits, after waiting for the
        handle's latest call and for the stream (the current one if not given)."""
        with torch.cuda.device(self._device):
            return self._error(lib.moe_product_get_error, _stream(stream))

    def _latest_error(self) -> int:
        """The same, after waiting for the handle's latest call alone."""
        return self._error(lib.moe_product_get_error_latest)

    def _error(self, read, *stream) -> int:
        flags = ctypes.c_uint32(0)
        st = read(self._h, *stream, ctypes.byref(flags))
        if st not in (0, 5):
            check(st, "moe_product_get_error")
        return int(flags.value)
