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

MoEDecode.prompt is the part after the router on a layer's own weights. As in
the decode layer, every call forwards device pointers and a stream to
libmoe_decode.so; nothing is computed here.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from ._lib import MOE_FLAG_MXFP4, MOE_PRODUCT_SILU_MUL, MoEProductConfig, check, lib
from ._tensors import _need, _ptr, _stream


_add_rms_norm, _group, _combine = lib.moe_add_rms_norm, lib.moe_group, lib.moe_combine
_product_run = lib.moe_product_run


class RmsNorm(NamedTuple):
    """What add_rms_norm returns; outputs that were not asked for are None."""
    sum: torch.Tensor | None      # bf16 [T, H]: the new residual stream
    y: torch.Tensor | None        # bf16 [T, H]: the normalised rows
    codes: torch.Tensor | None    # uint8 [T, H]: their E4M3 codes
    scales: torch.Tensor | None   # uint8 [T, H/32]: and UE8M0 scale codes


_BF16, _U8, _I32, _F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
_empty = torch.empty


def _matrix(t, dtype, name) -> tuple:
    """The shape of a contiguous CUDA matrix of `dtype`."""
    if isinstance(t, torch.Tensor) and t.dim() != 2:
        raise ValueError(f"{name}: expected two dimensions, got {t.dim()}")
    shape = t.shape if isinstance(t, torch.Tensor) else ()
    _need(t, dtype, shape, name)
    return shape


def add_rms_norm(x, weight, residual=None, *, eps: float = 1e-6, bf16: bool = True,
                 mxfp8: bool = False, sum=None, y=None, codes=None, scales=None,
                 stream=None) -> RmsNorm:
    """The residual stream s = bf16(x + residual) and s * rsqrt(mean(s^2) + eps) * weight,
    in bf16 (`bf16`), as MXFP8 codes and scales (`mxfp8`), or both.

    x and residual are bf16 [T, H], weight is bf16 [H]. Without a residual, s
    is x and RmsNorm.sum is None (unless a buffer for it is passed). The
    buffers sum, y, codes and scales may be passed in; sum may be x or
    residual, which is then updated in place.
    """
    shape = T, H = _matrix(x, _BF16, "x")
    _need(weight, _BF16, (H,), "weight")
    dev = x.device
    ps = py = pc = pz = pr = 0
    if residual is not None:
        _need(residual, _BF16, shape, "residual")
        pr = residual.data_ptr()
        if sum is None:
            sum = _empty(shape, dtype=_BF16, device=dev)
    if sum is not None:
        _need(sum, _BF16, shape, "sum")
        ps = sum.data_ptr()
    if bf16:
        if y is None:
            y = _empty(shape, dtype=_BF16, device=dev)
        else:
            _need(y, _BF16, shape, "y")
        py = y.data_ptr()
    elif mxfp8:
        y = None
    else:
        raise ValueError("add_rms_norm: ask for bf16 rows, mxfp8 rows or both")
    if mxfp8:
        if codes is None:
            codes = _empty(shape, dtype=_U8, device=dev)
        else:
            _need(codes, _U8, shape, "codes")
        if scales is None:
            scales = _empty((T, H // 32), dtype=_U8, device=dev)
        else:
            _need(scales, _U8, (T, H // 32), "scales")
        pc, pz = codes.data_ptr(), scales.data_ptr()
    else:
        codes = scales = None
    st = _add_rms_norm(T, H, x.data_ptr(), pr, weight.data_ptr(), eps, ps, py, pc, pz,
                       _stream(stream))
    if st:
        check(st, "moe_add_rms_norm")
    return RmsNorm(sum, y, codes, scales)


def group_by_expert(ids, E: int, *, offsets=None, rows=None, slots=None, stream=None):
    """(offsets, rows, slots) of routed ids int32 [T, k]: group e is the rows
    offsets[e] .. offsets[e + 1] - 1 in the order of the slots t * k + j;
    rows[q] is the token of grouped row q (-1 past the last group) and
    slots[t, j] the grouped row of a slot (-1 for an id outside [0, E), which
    joins no group)."""
    T, k = _matrix(ids, _I32, "ids")
    dev = ids.device
    if offsets is None:
        offsets = _empty((E + 1,), dtype=_I32, device=dev)
    else:
        _need(offsets, _I32, (E + 1,), "offsets")
    if rows is None:
        rows = _empty((T * k,), dtype=_I32, device=dev)
    else:
        _need(rows, _I32, (T * k,), "rows")
    if slots is None:
        slots = _empty((T, k), dtype=_I32, device=dev)
    else:
        _need(slots, _I32, (T, k), "slots")
    st = _group(T, k, E, ids.data_ptr(), offsets.data_ptr(), rows.data_ptr(), slots.data_ptr(),
                _stream(stream))
    if st:
        check(st, "moe_group")
    return offsets, rows, slots


def combine(y, slots, w, *, residual=None, out=None, stream=None):
    """out[t] = bf16(residual[t] + sum_j w[t, j] * y[slots[t, j]]) over expert
    rows y bf16 [R, H], slots int32 [T, k] (outside [0, R): nothing) and w
    float32 [T, k]; residual bf16 [T, H] is optional and may be `out`."""
    R, H = _matrix(y, _BF16, "y")
    T, k = _matrix(slots, _I32, "slots")
    _need(w, _F32, (T, k), "w")
    if residual is not None:
        _need(residual, _BF16, (T, H), "residual")
    if out is None:
        out = _empty((T, H), dtype=_BF16, device=y.device)
    else:
        _need(out, _BF16, (T, H), "out")
    st = _combine(T, k, H, R, y.data_ptr(), slots.data_ptr(), w.data_ptr(), _ptr(residual),
                  out.data_ptr(), _stream(stream))
    if st:
        check(st, "moe_combine")
    return out


class GroupedProduct:
    """Ragged products of grouped MXFP8 rows with one stack of expert weights.

    fmt="mxfp8": w uint8 [E, N, K]; fmt="mxfp4": w uint8 [E, N, K/2]; w_scales
    uint8 [E, N, K/32]. With silu_mul the N = 2I rows of an expert are I gate
    rows and I up rows, and the product is finished to MXFP8(SiLU(g) * u).
    The weights are borrowed (kept alive by this object); the scales are
    copied once into the order in which the tensor cores take them.
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
        self.E, self.N, self.K, self.fmt, self.silu_mul = E, N, K, fmt, silu_mul
        self._weights = (w, w_scales)
        flags = (MOE_FLAG_MXFP4 if fmt == "mxfp4" else 0) | (MOE_PRODUCT_SILU_MUL if silu_mul else 0)
        h = ctypes.c_void_p()
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
        A = a.shape[0]
        _need(a, _U8, (A, self.K), "a")
        _need(a_scales, _U8, (A, self.K // 32), "a_scales")
        _need(offsets, _I32, (self.E + 1,), "offsets")
        R, pr = A, 0
        if rows is not None:
            R, pr = rows.shape[0], rows.data_ptr()
            _need(rows, _I32, (R,), "rows")
        shape = (R, self.N // 2) if self.silu_mul else (R, self.N)
        dtype = _U8 if self.silu_mul else _BF16
        if out is None:
            out = _empty(shape, dtype=dtype, device=a.device)
        else:
            _need(out, dtype, shape, "out")
        py, pc, pz = out.data_ptr(), 0, 0
        if self.silu_mul:
            if out_scales is None:
                out_scales = _empty((R, self.N // 64), dtype=_U8, device=a.device)
            else:
                _need(out_scales, _U8, (R, self.N // 64), "out_scales")
            py, pc, pz = 0, py, out_scales.data_ptr()
        elif out_scales is not None:
            raise ValueError("out_scales: only a product with silu_mul has scales")
        st = _product_run(self._h, R, A, a.data_ptr(), a_scales.data_ptr(), offsets.data_ptr(), pr,
                          py, pc, pz, _stream(stream))
        if st:
            check(st, "moe_product_run")
        return (out, out_scales) if self.silu_mul else out

    def get_error(self, stream=None) -> int:
        """Read and clear the handle's device error bits, after waiting for the
        stream."""
        flags = ctypes.c_uint32(0)
        st = lib.moe_product_get_error(self._h, _stream(stream), ctypes.byref(flags))
        if st not in (0, 5):
            check(st, "moe_product_get_error")
        return int(flags.value)
