"""Python face of one MoE decode layer: a handle plus the C ABI's calls.

Every method forwards device pointers of torch tensors and the current CUDA
stream to libmoe_decode.so; nothing is computed here.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import (MOE_FLAG_MXFP4, MOE_PATH_AUTO, MOE_PATH_TENSOR, MOE_PATH_WARP, MoEConfig, check,
                   lib)
from ._tensors import _need, _on, _ptr, _stream
from .block import route_experts
from .prompt import GroupedProduct, combine, group_by_expert


class MoEDecode:
    """One MoE decode layer over caller-owned block-scaled weights on the current device.

    fmt="mxfp8": w_gateup uint8 [E, 2I, H] (rows [0, I) gate, [I, 2I) up),
    w_down uint8 [E, H, I], one E4M3 code per byte. fmt="mxfp4": w_gateup
    uint8 [E, 2I, H/2], w_down uint8 [E, H, I/2], two E2M1 codes per byte
    (the even element in the low nibble). Either way s_gateup uint8
    [E, 2I, H/32] and s_down uint8 [E, H, I/32] hold the UE8M0 scales. The
    tensors are borrowed (kept alive by this object, never copied).
    """

    def __init__(self, w_gateup, s_gateup, w_down, s_down, *, k: int, max_T: int = 32,
                 flags: int = 0, fmt: str = "mxfp8"):
        if fmt not in ("mxfp8", "mxfp4"):
            raise ValueError(f"fmt must be 'mxfp8' or 'mxfp4', got {fmt!r}")
        per = 2 if fmt == "mxfp4" else 1          # elements per code byte
        E, twoI, RB = w_gateup.shape
        I, H = twoI // 2, RB * per
        _need(w_gateup, torch.uint8, (E, 2 * I, H // per), "w_gateup")
        _need(s_gateup, torch.uint8, (E, 2 * I, H // 32), "s_gateup")
        _need(w_down, torch.uint8, (E, H, I // per), "w_down")
        _need(s_down, torch.uint8, (E, H, I // 32), "s_down")
        self.E, self.k, self.H, self.I, self.max_T, self.fmt = E, k, H, I, max_T, fmt
        self._weights = (w_gateup, s_gateup, w_down, s_down)
        self._products = None       # prompt()'s two GroupedProducts
        if fmt == "mxfp4":
            flags |= MOE_FLAG_MXFP4
        cfg = MoEConfig(E, k, H, I, max_T, flags)
        h = ctypes.c_void_p()
        check(lib.moe_decode_create(ctypes.byref(cfg), _ptr(w_gateup), _ptr(s_gateup),
                                    _ptr(w_down), _ptr(s_down), ctypes.byref(h)),
              "moe_decode_create")
        self._h = h

    # -- lifetime -------------------------------------------------------------
    def close(self) -> None:
        if getattr(self, "_h", None):
            lib.moe_decode_destroy(self._h)
            self._h = None
        self._products = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self) -> ctypes.c_void_p:
        return self._h

    @property
    def fused_single_token(self) -> bool:
        """True when one-token layer calls run as one persistent launch."""
        return lib.moe_decode_fused_layer(self._h) == 1

    @property
    def tensor_path(self) -> bool:
        """True when this handle can run the expert-centric tensor-core path."""
        return lib.moe_decode_tensor_path(self._h) == 1

    def set_path(self, path: str) -> None:
        """Which form layer calls take: "auto" (the tensor-core path from 16
        tokens when they route 1.5 or more slots per expert on average),
        "warp" or "tensor"."""
        code = {"auto": MOE_PATH_AUTO, "warp": MOE_PATH_WARP, "tensor": MOE_PATH_TENSOR}[path]
        check(lib.moe_decode_set_path(self._h, code), "moe_decode_set_path")

    def path(self, T: int) -> str:
        """The form a layer call with T tokens takes: "warp" or "tensor"."""
        return {MOE_PATH_WARP: "warp", MOE_PATH_TENSOR: "tensor"}[lib.moe_decode_path(self._h, T)]

    def kernel_name(self, T: int, which: str) -> str:
        """The kernel moe_gate_up (which="gate_up") or moe_down ("down")
        launches for T tokens on this handle."""
        w = {"gate_up": 0, "down": 1}[which]
        return lib.moe_decode_kernel_name(self._h, T, w).decode()

    def arm_barrier_timeout(self) -> None:
        """Test support: the next one-launch call's grid barrier times out
        (bounded; it sets MOE_DEVICE_TIMEOUT, which get_error reports)."""
        check(lib.moe_decode_arm_barrier_timeout(self._h), "moe_decode_arm_barrier_timeout")

    def _dev(self, shape, dtype, out, name, stream):
        if out is None:             # of the memory of the stream that writes it
            with _on(stream):
                return torch.empty(shape, dtype=dtype, device=self._weights[0].device)
        _need(out, dtype, shape, name)
        return out

    # -- calls ----------------------------------------------------------------
    def route(self, logits, ids=None, w=None, stream=None, **options):
        """(ids int32 [T, k], w float32 [T, k]) of router logits float32 [T, E]:
        the k most probable experts by a softmax and their probabilities,
        renormalised. With `options`, route_experts' (score, bias, groups,
        top_groups, group_score, renormalize, scale), the choice is that
        operator's, which takes bf16 logits too."""
        if options:
            if logits.shape[-1] != self.E:
                raise ValueError(f"logits: expected {self.E} experts, got {logits.shape[-1]}")
            return route_experts(logits, self.k, ids=ids, w=w, stream=stream, **options)
        T = logits.shape[0]
        _need(logits, torch.float32, (T, self.E), "logits")
        ids = self._dev((T, self.k), torch.int32, ids, "topk_ids", stream)
        w = self._dev((T, self.k), torch.float32, w, "topk_w", stream)
        check(lib.moe_route(self._h, T, _ptr(logits), _ptr(ids), _ptr(w), _stream(stream)),
              "moe_route")
        return ids, w

    def dedup_schedule(self, ids, stream=None):
        T = ids.shape[0]
        _need(ids, torch.int32, (T, self.k), "topk_ids")
        U = min(self.E, T * self.k)
        dev = ids.device
        with _on(stream):           # the fills come before the schedule there
            uniq = torch.full((U,), -1, dtype=torch.int32, device=dev)
            off = torch.full((U + 1,), -1, dtype=torch.int32, device=dev)
            pairs = torch.full((T * self.k,), -1, dtype=torch.int32, device=dev)
            n = torch.zeros((1,), dtype=torch.int32, device=dev)
        check(lib.moe_dedup_schedule(self._h, T, _ptr(ids), _ptr(uniq), _ptr(off), _ptr(pairs),
                                     _ptr(n), _stream(stream)), "moe_dedup_schedule")
        return uniq, off, pairs, n

    def gate_up(self, x, ids, h=None, stream=None):
        T = x.shape[0]
        _need(x, torch.bfloat16, (T, self.H), "x")
        _need(ids, torch.int32, (T, self.k), "topk_ids")
        h = self._dev((T, self.k, self.I), torch.bfloat16, h, "h", stream)
        check(lib.moe_gate_up(self._h, T, _ptr(x), _ptr(ids), _ptr(h), _stream(stream)),
              "moe_gate_up")
        return h

    def down(self, h, ids, w, y=None, stream=None):
        T = h.shape[0]
        _need(h, torch.bfloat16, (T, self.k, self.I), "h")
        _need(ids, torch.int32, (T, self.k), "topk_ids")
        _need(w, torch.float32, (T, self.k), "topk_w")
        y = self._dev((T, self.H), torch.bfloat16, y, "y", stream)
        check(lib.moe_down(self._h, T, _ptr(h), _ptr(ids), _ptr(w), _ptr(y), _stream(stream)),
              "moe_down")
        return y

    def layer(self, x, ids, w, h=None, y=None, stream=None):
        T = x.shape[0]
        _need(x, torch.bfloat16, (T, self.H), "x")
        _need(ids, torch.int32, (T, self.k), "topk_ids")
        _need(w, torch.float32, (T, self.k), "topk_w")
        h = self._dev((T, self.k, self.I), torch.bfloat16, h, "h", stream)
        y = self._dev((T, self.H), torch.bfloat16, y, "y", stream)
        check(lib.moe_decode_layer(self._h, T, _ptr(x), _ptr(ids), _ptr(w), _ptr(h), _ptr(y),
                                   _stream(stream)), "moe_decode_layer")
        return y

    def forward_host(self, x, ids, w, y=None, stream=None):
        """The layer from and to host tensors (pin them for asynchronous copies)."""
        T = x.shape[0]
        _need(x, torch.bfloat16, (T, self.H), "x", cuda=False)
        _need(ids, torch.int32, (T, self.k), "topk_ids", cuda=False)
        _need(w, torch.float32, (T, self.k), "topk_w", cuda=False)
        if y is None:
            y = torch.empty((T, self.H), dtype=torch.bfloat16, pin_memory=True)
        _need(y, torch.bfloat16, (T, self.H), "y", cuda=False)
        check(lib.moe_decode_forward_host(self._h, T, _ptr(x), _ptr(ids), _ptr(w), _ptr(y),
                                          _stream(stream)), "moe_decode_forward_host")
        return y

    def prompt(self, codes, scales, ids, w, residual=None, out=None, stream=None):
        """The routed experts over a prompt's MXFP8 rows (codes uint8 [T, H],
        scales uint8 [T, H/32], e.g. add_rms_norm's): grouping, both products
        on the tensor cores with h in MXFP8, and the weighted sum with
        `residual` (bf16 [T, H], optional) added; bf16 [T, H]. T is not bound
        by max_T; an id outside [0, E) adds nothing. The first call lays out
        the weights' scales for the two products (see GroupedProduct), which
        the layer then keeps: make it before a stream is captured. With MXFP4
        weights H and I must be multiples of 128."""
        if stream is not None:      # the intermediates belong to that stream too
            with torch.cuda.stream(stream):
                return self.prompt(codes, scales, ids, w, residual, out)
        if self._products is None:
            wgu, sgu, wd, sd = self._weights
            self._products = (GroupedProduct(wgu, sgu, fmt=self.fmt, silu_mul=True),
                              GroupedProduct(wd, sd, fmt=self.fmt))
        gate_up, down = self._products
        _need(ids, torch.int32, (codes.shape[0], self.k), "topk_ids")
        offsets, rows, slots = group_by_expert(ids, self.E)
        hc, hs = gate_up(codes, scales, offsets, rows)
        return combine(down(hc, hs, offsets), slots, w, residual=residual, out=out)

    def get_error(self, stream=None) -> int:
        """Read and clear the handle's device error bits. Waits for this
        handle's latest call, or, given a stream, for that stream."""
        flags = ctypes.c_uint32(0)
        if stream is None:
            st = lib.moe_decode_get_error(self._h, ctypes.byref(flags))
        else:
            st = lib.moe_decode_get_error_stream(self._h, _stream(stream), ctypes.byref(flags))
        if st not in (0, 5):
            check(st, "moe_decode_get_error")
        for p in self._products or ():
            flags.value |= p._latest_error() if stream is None else p.get_error(stream)
        return int(flags.value)
