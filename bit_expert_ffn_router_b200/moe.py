"""ctypes binding of libmoe (include/moe.h): argument marshalling, and for the
balance loss and the MX calls a look at their tensors.

Every step of the MoE FFN runs inside libmoe's CUDA kernels; this module turns
torch tensors into device pointers and the current torch stream into a
cudaStream_t. If libmoe.so is missing, loading fails with an error: there is
no fallback.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "lib", "libmoe.so")

OK, EINVAL, EUNSUPPORTED, ECUDA, ETIMEOUT, EDEVICE, ENOSPACE = range(7)
DECODE_MAX_T = 8


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = f"{what}: {status_string(status)} ({status})"
        if status == ECUDA:
            msg += f" [{load_library().moe_last_cuda_error().decode()}]"
        super().__init__(msg)


class _Cfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in
                ("d", "f", "E", "k", "n_shared", "bits", "block", "renorm", "out_fp32", "residual",
                 "skip_from", "hot_slots")]


class _Layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("gu_codes", "dn_codes", "gu_scales", "dn_scales", "bytes")]


class Grouping(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("k", ctypes.c_int), ("E", ctypes.c_int),
                ("n_pairs", ctypes.c_int), ("n_rows", ctypes.c_int)] + [
        (n, ctypes.c_void_p) for n in
        ("expert_count", "expert_offset", "pair_token", "pair_j", "pair_gate", "pair_slot", "pair_pos",
         "uniq_expert", "uniq_slot", "uniq_offset", "n_uniq", "internal")]


class Routing(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("k", ctypes.c_int), ("E", ctypes.c_int),
                ("logits", ctypes.c_void_p), ("idx", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("grouping", Grouping)]


class _WithRef:
    """Room for a configuration's C structure beside its fields, not among them: vars(), copies and pickles hold the
    fields alone."""
    __slots__ = ("_ref",)

    def __getstate__(self):
        return self.__dict__


@dataclasses.dataclass(frozen=True)
class LayerCfg(_WithRef):
    d: int
    f: int
    E: int
    k: int
    n_shared: int = 1
    bits: int = 2
    block: int = 32
    renorm: int = 1
    out_fp32: int = 1
    residual: int = 0
    skip_from: int = 0  # 0: off; else pairs of rank >= skip_from on a slot >= hot_slots are left out (decode)
    hot_slots: int = 0

    def c(self) -> _Cfg:
        """A C structure of these fields, the caller's own."""
        return _Cfg(*(getattr(self, f.name) for f in dataclasses.fields(self)))

    def ref(self):
        """A pointer argument to a structure that is built once (the library only reads it)."""
        try:
            return self._ref
        except AttributeError:
            object.__setattr__(self, "_ref", ctypes.byref(self.c()))
            return self._ref

    def replace(self, **kw) -> "LayerCfg":
        return dataclasses.replace(self, **kw)


# Named shapes: the tiny parity layer and the full Qwen3.8-Flash-Next-shaped layer.
TINY = LayerCfg(d=256, f=128, E=16, k=2)
FULL = LayerCfg(d=2048, f=768, E=512, k=10)

TYPE_BF16, TYPE_FP16, TYPE_FP32 = range(3)  # element types of the MX calls
MX4_GATHER, MX4_SWIGLU, MX4_GATE = 1, 2, 4
MX4_BLOCK = 32  # values per scale


class _Mx4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("code_stride", ctypes.c_size_t),
                ("scale_stride", ctypes.c_size_t), ("n_slots", ctypes.c_int), ("rows", ctypes.c_int),
                ("cols", ctypes.c_int)]


_P, _I, _Z, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
_SIGS = {
    "moe_ctx_create": (_I, [_I, ctypes.POINTER(ctypes.c_void_p)]),
    "moe_ctx_destroy": (None, [_P]),
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_last_cuda_error": (ctypes.c_char_p, []),
    "moe_check_device_status": (_I, [_P, _S]),
    "moe_last_device_error_detail": (_I, [_P]),
    "moe_trace_fetch": (_I, [_P, ctypes.c_void_p, _I, _S]),
    "moe_expert_layout_get": (_I, [ctypes.POINTER(_Cfg), ctypes.POINTER(_Layout)]),
    "moe_workspace_bytes": (_Z, [ctypes.POINTER(_Cfg), _I]),
    "moe_router_topk": (_I, [_P, ctypes.POINTER(_Cfg), _P, _P, _P, _I, _P, _P, _P, _S]),
    "moe_topk": (_I, [_P, ctypes.POINTER(_Cfg), _P, _I, _P, _P, _S]),
    "moe_group_tokens": (_I, [_P, ctypes.POINTER(_Cfg), _P, _P, _I, _P, _I, _P, _Z,
                              ctypes.POINTER(Grouping), _S]),
    "moe_expert_ffn_q2": (_I, [_P, ctypes.POINTER(_Cfg), _P, ctypes.POINTER(Grouping), _P, _Z, _P, _P, _Z,
                               _P, _P, _S]),
    "moe_expert_ffn_q3": (_I, [_P, ctypes.POINTER(_Cfg), _P, ctypes.POINTER(Grouping), _P, _Z, _P, _P, _Z,
                               _P, _P, _S]),
    "moe_combine": (_I, [_P, ctypes.POINTER(_Cfg), ctypes.POINTER(Grouping), _P, _P, _I, _P, _S]),
    "moe_layer_forward": (_I, [_P, ctypes.POINTER(_Cfg), _P, _I, _P, _P, _P, _I, _P, _Z, _P, _P, _Z, _P,
                               _S]),
    "moe_layer_routing": (_I, [ctypes.POINTER(_Cfg), _I, _P, _Z, ctypes.POINTER(Routing)]),
    "moe_stack_workspace_bytes": (_Z, [ctypes.POINTER(_Cfg), _I, _I]),
    "moe_stack_forward": (_I, [_P, ctypes.POINTER(_Cfg), _I, _P, _I, _P, _P, _P, _I, _P, _Z, _P, _P, _Z, _P, _S]),
    "moe_stack_routing": (_I, [ctypes.POINTER(_Cfg), _I, _I, _P, _Z, _I, ctypes.POINTER(Routing)]),
    "moe_layer_forward_static": (_I, [_P, ctypes.POINTER(_Cfg), _P, _I, _P, _P, _P, _I, _P, _Z, _P, _P, _S]),
    "moe_usage_count": (_I, [_P, ctypes.POINTER(_Cfg), _I, _I, _P, _Z, _P, _S]),
    "moe_slot_swap": (_I, [_P, ctypes.POINTER(_Cfg), _P, _Z, _P, _I, _I, _P, _P, _I, _S]),
    "moe_balance_workspace_bytes": (_Z, [ctypes.POINTER(_Cfg)]),
    "moe_balance_loss": (_I, [_P, ctypes.POINTER(_Cfg), _P, _P, _P, _I, _P, _P, _P, _P, _Z, _S]),
    "moe_balance_loss_backward": (_I, [_P, ctypes.POINTER(_Cfg), _P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _S]),
    "moe_mx4_scale_pitch": (_Z, [_I]),
    "moe_mx4_quantize": (_I, [_P, _P, _I, _I, _I, _Z, _P, _P, _S]),
    "moe_mx4_dequantize": (_I, [_P, _P, _P, _I, _I, _P, _I, _Z, _S]),
    "moe_mx4_product": (_I, [_P, _P, _P, _I, ctypes.POINTER(_Mx4), ctypes.POINTER(Grouping), _I, _I, _P, _I, _Z,
                             _S]),
}

_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Opens libmoe.so (built in-tree by bit_expert_ffn_router_b200.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise FileNotFoundError(f"{path} is missing: build it with `python -m bit_expert_ffn_router_b200.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_string(s: int) -> str:
    return load_library().moe_status_string(s).decode()


def _check(status: int, what: str) -> None:
    if status != OK:
        raise MoeError(status, what)


def expert_layout(cfg: LayerCfg) -> dict:
    lay = _Layout()
    _check(load_library().moe_expert_layout_get(cfg.ref(), ctypes.byref(lay)), "moe_expert_layout_get")
    return {n: getattr(lay, n) for n, _ in _Layout._fields_}


def workspace_bytes(cfg: LayerCfg, T: int) -> int:
    return int(load_library().moe_workspace_bytes(cfg.ref(), T))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


class Context:
    """One libmoe context (device status word + SM count) on a CUDA device."""

    def __init__(self, device: int = 0):
        self.lib = load_library()
        h = ctypes.c_void_p()
        _check(self.lib.moe_ctx_create(device, ctypes.byref(h)), "moe_ctx_create")
        self.h = h
        self.device = device
        self._bind_torch()

    def _bind_torch(self):
        import torch
        self._current = torch._C._cuda_getCurrentRawStream  # of a device: its current stream's handle
        self._f32, self._i32 = torch.float32, torch.int32
        self._type_code = {torch.bfloat16: TYPE_BF16, torch.float16: TYPE_FP16, torch.float32: TYPE_FP32}.get

    def close(self):
        if self.h:
            self.lib.moe_ctx_destroy(self.h)
            self.h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- raw entry points (status codes returned, not raised) --------------------
    def router_topk_status(self, cfg, x, w_router, bias, T, logits, idx, gate, stream=None):
        return self.lib.moe_router_topk(self.h, cfg.ref(), _ptr(x), _ptr(w_router), _ptr(bias), T,
                                        _ptr(logits), _ptr(idx), _ptr(gate), _stream(stream))

    def layer_forward_status(self, cfg, x, T, w_router, bias, slot_of, n_slots, pool, stride, shared, ws, y,
                             stream=None):
        return self.lib.moe_layer_forward(self.h, cfg.ref(), _ptr(x), T, _ptr(w_router), _ptr(bias),
                                          _ptr(slot_of), n_slots, _ptr(pool), stride, _ptr(shared), _ptr(ws),
                                          0 if ws is None else ws.numel() * ws.element_size(), _ptr(y),
                                          _stream(stream))

    def stack_forward_status(self, cfg, L, x, T, w_router, bias, slot_of, n_slots, pool, stride, shared, ws, y,
                             stream=None):
        return self.lib.moe_stack_forward(self.h, cfg.ref(), L, _ptr(x), T, _ptr(w_router), _ptr(bias),
                                          _ptr(slot_of), n_slots, _ptr(pool), stride, _ptr(shared), _ptr(ws),
                                          0 if ws is None else ws.numel() * ws.element_size(), _ptr(y),
                                          _stream(stream))

    def stack_forward(self, cfg, L, x, T, w_router, bias, slot_of, n_slots, pool, stride, shared, ws, y,
                      stream=None):
        """moe_stack_forward: L chained decode layers in one launch (layer l + 1 reads y[l])."""
        _check(self.stack_forward_status(cfg, L, x, T, w_router, bias, slot_of, n_slots, pool, stride, shared, ws,
                                         y, stream), "moe_stack_forward")

    def layer_forward_static_status(self, cfg, x, T, w_router, bias, slot_of, n_slots, pool, stride, shared, y,
                                    stream=None):
        """moe_layer_forward with the library's static scratch (no workspace argument)."""
        return self.lib.moe_layer_forward_static(self.h, cfg.ref(), _ptr(x), T, _ptr(w_router),
                                                 _ptr(bias), _ptr(slot_of), n_slots, _ptr(pool), stride,
                                                 _ptr(shared), _ptr(y), _stream(stream))

    # -- checked wrappers ---------------------------------------------------------
    def router_topk(self, cfg, x, w_router, bias, T, logits, idx, gate, stream=None):
        _check(self.router_topk_status(cfg, x, w_router, bias, T, logits, idx, gate, stream), "moe_router_topk")

    def topk(self, cfg, logits, T, idx, gate, stream=None):
        _check(self.lib.moe_topk(self.h, cfg.ref(), _ptr(logits), T, _ptr(idx), _ptr(gate),
                                 _stream(stream)), "moe_topk")

    def group_tokens(self, cfg, idx, gate, T, slot_of, n_slots, ws, stream=None) -> Grouping:
        g = Grouping()
        _check(self.lib.moe_group_tokens(self.h, cfg.ref(), _ptr(idx), _ptr(gate), T, _ptr(slot_of),
                                         n_slots, _ptr(ws), ws.numel() * ws.element_size(), ctypes.byref(g),
                                         _stream(stream)), "moe_group_tokens")
        return g

    def expert_ffn(self, cfg, x, grouping, pool, stride, shared, ws, z_rows=None, y=None, stream=None):
        fn = self.lib.moe_expert_ffn_q2 if cfg.bits == 2 else self.lib.moe_expert_ffn_q3
        _check(fn(self.h, cfg.ref(), _ptr(x), ctypes.byref(grouping), _ptr(pool), stride, _ptr(shared),
                  _ptr(ws), ws.numel() * ws.element_size(), _ptr(z_rows), _ptr(y), _stream(stream)),
               f"moe_expert_ffn_q{cfg.bits}")

    def combine(self, cfg, grouping, z_rows, x, T, y, stream=None):
        _check(self.lib.moe_combine(self.h, cfg.ref(), ctypes.byref(grouping), _ptr(z_rows), _ptr(x),
                                    T, _ptr(y), _stream(stream)), "moe_combine")

    def layer_forward(self, cfg, x, T, w_router, bias, slot_of, n_slots, pool, stride, shared, ws, y,
                      stream=None):
        _check(self.layer_forward_status(cfg, x, T, w_router, bias, slot_of, n_slots, pool, stride, shared, ws, y,
                                         stream), "moe_layer_forward")

    def prepare_layer_forward(self, cfg, T, w_router, bias, slot_of, n_slots, pool, stride, shared, ws,
                              stream=None) -> "PreparedLayer":
        """moe_layer_forward with every argument but x and y marshalled once (for launch loops)."""
        return PreparedLayer(self, cfg, T, w_router, bias, slot_of, n_slots, pool, stride, shared, ws, stream)

    def usage_count_status(self, cfg, L, T, ws, counts, stream=None) -> int:
        return self.lib.moe_usage_count(self.h, cfg.ref(), L, T, _ptr(ws),
                                        ws.numel() * ws.element_size(), _ptr(counts), _stream(stream))

    def usage_count(self, cfg, L, T, ws, counts, stream=None) -> None:
        """moe_usage_count: counts [L*E] int32 (device) += pairs routed to each expert by the call that
        used ws (L = 1 for a single-layer workspace)."""
        _check(self.usage_count_status(cfg, L, T, ws, counts, stream), "moe_usage_count")

    def slot_swap_status(self, cfg, pool, stride, slot_of, n_slots, a, b, stream=None) -> int:
        import numpy as np
        a = np.ascontiguousarray(a, dtype=np.int32)
        b = np.ascontiguousarray(b, dtype=np.int32)
        if a.shape != b.shape or a.ndim != 1:
            return EINVAL
        return self.lib.moe_slot_swap(self.h, cfg.ref(), _ptr(pool), stride, _ptr(slot_of),
                                      slot_of.numel(), n_slots, a.ctypes.data, b.ctypes.data, a.size,
                                      _stream(stream))

    def slot_swap(self, cfg, pool, stride, slot_of, n_slots, a, b, stream=None) -> None:
        """moe_slot_swap: the records at slots slot_of[a[i]] and slot_of[b[i]] trade places, and so
        do the two table entries (a, b: host index arrays into the flat device table slot_of)."""
        _check(self.slot_swap_status(cfg, pool, stride, slot_of, n_slots, a, b, stream), "moe_slot_swap")

    # The calls below take a few microseconds on the GPU at their smallest, so
    # their arguments go to ctypes as plain integers, without objects around them.

    def _raw_stream(self, stream) -> int:
        """The stream's handle; None is the current stream of this context's device."""
        return self._current(self.device) if stream is None else stream.cuda_stream

    # -- the router's balance loss -------------------------------------------------
    # Every tensor has to hold the elements that the call reads or writes, of their type and one after another. Each
    # question costs 0.05 us of a call's 5 us on the host, a function for a tensor's as much again; so they are asked
    # in place, and the device of the first tensor stands for all.

    def balance_loss_status(self, cfg, logits, idx, mask, T, stats, counts, prob, ws, stream=None) -> int:
        f32, i32, E = self._f32, self._i32, cfg.E
        try:
            if (logits.get_device() != self.device
                    or logits.dtype is not f32 or logits.nbytes < 4 * T * E or not logits.is_contiguous()
                    or idx.dtype is not i32 or idx.nbytes < 4 * T * cfg.k or not idx.is_contiguous()
                    or stats.dtype is not f32 or stats.nbytes < 16 or not stats.is_contiguous()
                    or counts.dtype is not i32 or counts.nbytes < 4 * E or not counts.is_contiguous()
                    or prob.dtype is not f32 or prob.nbytes < 4 * E or not prob.is_contiguous()
                    or not ws.is_contiguous()
                    or mask is not None and not _is_mask(mask, T)):
                return EINVAL
            return self.lib.moe_balance_loss(self.h, cfg.ref(), logits.data_ptr(), idx.data_ptr(),
                                             None if mask is None else mask.data_ptr(), T, stats.data_ptr(),
                                             counts.data_ptr(), prob.data_ptr(), ws.data_ptr(), ws.nbytes,
                                             self._raw_stream(stream))
        except AttributeError:  # no tensor
            return EINVAL

    def balance_loss(self, cfg, logits, idx, mask, T, stats, counts, prob, ws, stream=None) -> None:
        """moe_balance_loss: stats [4] fp32 (balance loss, z loss, tokens that count, largest load), counts [E]
        int32 and prob [E] fp32 from logits [T, E] fp32, idx [T, k] int32 and mask [T] of single bytes (uint8,
        bool) or None; ws: balance_workspace. Tensors are contiguous and on the context's device; they may be
        longer than that."""
        status = self.balance_loss_status(cfg, logits, idx, mask, T, stats, counts, prob, ws, stream)
        if status:
            raise MoeError(status, "moe_balance_loss")

    def balance_loss_backward_status(self, cfg, logits, idx, gate, mask, T, stats, counts, d_loss, d_gate, d_logits,
                                     stream=None) -> int:
        f32, i32, E = self._f32, self._i32, cfg.E
        rows, pairs = 4 * T * E, 4 * T * cfg.k
        try:
            if (logits.get_device() != self.device
                    or logits.dtype is not f32 or logits.nbytes < rows or not logits.is_contiguous()
                    or d_logits.dtype is not f32 or d_logits.nbytes < rows or not d_logits.is_contiguous()
                    or idx.dtype is not i32 or idx.nbytes < pairs or not idx.is_contiguous()
                    or stats.dtype is not f32 or stats.nbytes < 16 or not stats.is_contiguous()
                    or counts.dtype is not i32 or counts.nbytes < 4 * E or not counts.is_contiguous()
                    or d_loss.dtype is not f32 or d_loss.nbytes < 8 or not d_loss.is_contiguous()
                    or d_gate is not None and (
                        gate.dtype is not f32 or gate.nbytes < pairs or not gate.is_contiguous()
                        or d_gate.dtype is not f32 or d_gate.nbytes < pairs or not d_gate.is_contiguous())
                    or mask is not None and not _is_mask(mask, T)):
                return EINVAL
            return self.lib.moe_balance_loss_backward(
                self.h, cfg.ref(), logits.data_ptr(), idx.data_ptr(), None if d_gate is None else gate.data_ptr(),
                None if mask is None else mask.data_ptr(), T, stats.data_ptr(), counts.data_ptr(), d_loss.data_ptr(),
                None if d_gate is None else d_gate.data_ptr(), d_logits.data_ptr(), self._raw_stream(stream))
        except AttributeError:  # no tensor
            return EINVAL

    def balance_loss_backward(self, cfg, logits, idx, gate, mask, T, stats, counts, d_loss, d_gate, d_logits,
                              stream=None) -> None:
        """moe_balance_loss_backward: d_logits [T, E] of d_loss[0] * stats[0] + d_loss[1] * stats[1] and, unless
        d_gate is None, of the gates [T, k] (both fp32). Tensors as for balance_loss."""
        status = self.balance_loss_backward_status(cfg, logits, idx, gate, mask, T, stats, counts, d_loss, d_gate,
                                                   d_logits, stream)
        if status:
            raise MoeError(status, "moe_balance_loss_backward")

    # -- 4-bit experts in the MX format ----------------------------------------------
    # As above: the device of the rows (and of the matrices) stands for their codes' and scales'.

    def mx4_quantize_status(self, x, codes, scales, stream=None) -> int:
        rows, cols, ld = _rows(x)
        if x.get_device() != self.device or _bad_mx4(codes, scales, rows, cols):
            return EINVAL
        return self.lib.moe_mx4_quantize(self.h, x.data_ptr(), self._type_code(x.dtype, -1), rows, cols, ld,
                                         codes.data_ptr(), scales.data_ptr(), self._raw_stream(stream))

    def mx4_quantize(self, x, codes, scales, stream=None) -> None:
        """moe_mx4_quantize: x [rows, cols] (bf16, fp16 or fp32, any row stride) to codes and scales as
        mx4_buffers gives them."""
        status = self.mx4_quantize_status(x, codes, scales, stream)
        if status:
            raise MoeError(status, "moe_mx4_quantize")

    def mx4_dequantize_status(self, codes, scales, out, stream=None) -> int:
        rows, cols, ld = _rows(out)
        if out.get_device() != self.device or _bad_mx4(codes, scales, rows, cols):
            return EINVAL
        return self.lib.moe_mx4_dequantize(self.h, codes.data_ptr(), scales.data_ptr(), rows, cols, out.data_ptr(),
                                           self._type_code(out.dtype, -1), ld, self._raw_stream(stream))

    def mx4_dequantize(self, codes, scales, out, stream=None) -> None:
        """moe_mx4_dequantize: the values of codes and scales to out [rows, cols] (bf16, fp16 or fp32)."""
        status = self.mx4_dequantize_status(codes, scales, out, stream)
        if status:
            raise MoeError(status, "moe_mx4_dequantize")

    def mx4_product_status(self, codes, scales, w: "Mx4Matrix", out, grouping=None, shared_slot=-1, gather=False,
                           swiglu=False, gate=False, stream=None) -> int:
        rows, cols, ld = _rows(out)
        x_rows = codes.shape[0]
        if (out.get_device() != self.device or w.device != self.device or _bad_mx4(codes, scales, x_rows, w.cols)
                or cols != (w.rows // 2 if swiglu else w.rows)):
            return EINVAL
        if grouping is None:
            need, g = x_rows, None
        else:
            need, g = grouping.n_pairs + (grouping.T if shared_slot >= 0 else 0), ctypes.byref(grouping)
        if rows < need:
            return EINVAL
        flags = (MX4_GATHER if gather else 0) | (MX4_SWIGLU if swiglu else 0) | (MX4_GATE if gate else 0)
        return self.lib.moe_mx4_product(self.h, codes.data_ptr(), scales.data_ptr(), x_rows, w.ref, g, shared_slot,
                                        flags, out.data_ptr(), self._type_code(out.dtype, -1), ld, self._raw_stream(stream))

    def mx4_product(self, codes, scales, w: "Mx4Matrix", out, grouping=None, shared_slot=-1, gather=False,
                    swiglu=False, gate=False, stream=None) -> None:
        """moe_mx4_product: out = x w^T of 4-bit rows (codes, scales) and the matrices w, one matrix or grouped."""
        status = self.mx4_product_status(codes, scales, w, out, grouping, shared_slot, gather, swiglu, gate, stream)
        if status:
            raise MoeError(status, "moe_mx4_product")

    def expert_ffn_mx4(self, cfg, x, grouping, up: "Mx4Matrix", down: "Mx4Matrix", shared_slot, bufs, z_rows,
                       stream=None) -> None:
        """The expert FFN on 4-bit matrices in the place of expert_ffn (any T): x [T, d] quantised, gate and up
        rows with SwiGLU (up: [slots, 2f, d], row 2c gate and 2c + 1 up of channel c), the hidden rows
        quantised, down rows (down: [slots, d, f]) times the gates, to z_rows [n_rows, d] fp32 for combine.
        shared_slot: the pool slot of the shared expert (-1 where cfg.n_shared is 0); bufs: mx4_ffn_buffers."""
        # combine reads z_rows by its address alone
        if ((shared_slot >= 0) != bool(cfg.n_shared)
                or (up.rows, up.cols, down.rows, down.cols) != (2 * cfg.f, cfg.d, cfg.d, cfg.f)
                or z_rows.dtype is not self._f32 or not z_rows.is_contiguous()
                or z_rows.nbytes < 4 * cfg.d * (grouping.n_pairs + (grouping.T if shared_slot >= 0 else 0))):
            raise MoeError(EINVAL, "expert_ffn_mx4")
        xq, h, hq = bufs
        self.mx4_quantize(x, *xq, stream=stream)
        self.mx4_product(*xq, up, h, grouping=grouping, shared_slot=shared_slot, gather=True, swiglu=True,
                         stream=stream)
        self.mx4_quantize(h, *hq, stream=stream)
        self.mx4_product(*hq, down, z_rows, grouping=grouping, shared_slot=shared_slot, gate=True, stream=stream)

    def layer_routing(self, cfg, T, ws, stack_layers=None, layer=0) -> dict:
        """The routing a whole-step call with workspace `ws` computed (moe_layer_routing; with
        stack_layers=L, layer `layer` of a moe_stack_forward workspace), as torch views into ws:
        logits [T,E], idx [T,k], gate [T,k] and the grouping arrays. Read them after the call has
        completed on its stream."""
        import torch
        r = Routing()
        nbytes = ws.numel() * ws.element_size()
        if stack_layers is None:
            _check(self.lib.moe_layer_routing(cfg.ref(), T, _ptr(ws), nbytes, ctypes.byref(r)),
                   "moe_layer_routing")
        else:
            _check(self.lib.moe_stack_routing(cfg.ref(), stack_layers, T, _ptr(ws), nbytes, layer,
                                              ctypes.byref(r)), "moe_stack_routing")
        raw = ws.view(torch.uint8).view(-1)
        base = ws.data_ptr()

        def view(ptr, n, dtype):
            off = ptr - base
            return raw[off:off + 4 * n].view(dtype)

        g = r.grouping
        n_pairs, nu_max = T * cfg.k, min(T * cfg.k, cfg.E)
        return {
            "logits": view(r.logits, T * cfg.E, torch.float32).view(T, cfg.E),
            "idx": view(r.idx, T * cfg.k, torch.int32).view(T, cfg.k),
            "gate": view(r.gate, T * cfg.k, torch.float32).view(T, cfg.k),
            "expert_count": view(g.expert_count, cfg.E, torch.int32),
            "expert_offset": view(g.expert_offset, cfg.E + 1, torch.int32),
            "pair_token": view(g.pair_token, n_pairs, torch.int32),
            "pair_j": view(g.pair_j, n_pairs, torch.int32),
            "pair_gate": view(g.pair_gate, n_pairs, torch.float32),
            "pair_slot": view(g.pair_slot, n_pairs, torch.int32),
            "pair_pos": view(g.pair_pos, n_pairs, torch.int32),
            "uniq_expert": view(g.uniq_expert, nu_max, torch.int32),
            "uniq_slot": view(g.uniq_slot, nu_max, torch.int32),
            "uniq_offset": view(g.uniq_offset, nu_max + 1, torch.int32),
            "n_uniq": view(g.n_uniq, 1, torch.int32),
        }

    def prepare_stack_forward(self, cfg, L, T, w_router, slot_of, n_slots, pool, stride, shared, ws,
                              stream=None) -> "PreparedStack":
        """moe_stack_forward with every argument but x, the bias and y marshalled once (for launch loops)."""
        return PreparedStack(self, cfg, L, T, w_router, slot_of, n_slots, pool, stride, shared, ws, stream)

    def check_device_status(self, stream=None) -> int:
        return self.lib.moe_check_device_status(self.h, _stream(stream))

    def last_device_error_detail(self) -> int:
        return self.lib.moe_last_device_error_detail(self.h)

    def trace_fetch(self, n_ctas: int, stream=None):
        """Phase timestamps of the last decode-layer launches (MOE_TRACE set at creation)."""
        import numpy as np
        buf = np.zeros((n_ctas, 64), dtype=np.uint64)
        _check(self.lib.moe_trace_fetch(self.h, buf.ctypes.data, buf.size, _stream(stream)), "moe_trace_fetch")
        return buf


class PreparedLayer:
    """A moe_layer_forward call whose layer arguments (configuration, weights,
    slot table, pool, workspace, stream) are converted to ctypes values once;
    each call marshals only x and y. It passes exactly the arguments
    Context.layer_forward_status would, and keeps the tensors it points into
    alive."""

    def __init__(self, ctx, cfg, T, w_router, bias, slot_of, n_slots, pool, stride, shared, ws, stream=None):
        self._fn = ctx.lib.moe_layer_forward
        self._cfg = cfg.c()
        self._keep = (ctx, w_router, bias, slot_of, pool, shared, ws)
        self._head = (ctx.h, ctypes.byref(self._cfg))
        self._mid = (T, _ptr(w_router), _ptr(bias), _ptr(slot_of), n_slots, _ptr(pool), stride, _ptr(shared),
                     _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size())
        self._stream = _stream(stream)

    def status(self, x, y) -> int:
        return self._fn(*self._head, _ptr(x), *self._mid, _ptr(y), self._stream)

    def __call__(self, x, y) -> None:
        _check(self.status(x, y), "moe_layer_forward")


class PreparedStack:
    """A moe_stack_forward call whose fixed arguments (configuration, routers,
    slot table, pool, shared experts, workspace, stream) are converted to
    ctypes values once; each call marshals only x, the bias and y."""

    def __init__(self, ctx, cfg, L, T, w_router, slot_of, n_slots, pool, stride, shared, ws, stream=None):
        self._fn = ctx.lib.moe_stack_forward
        self._cfg = cfg.c()
        self._keep = (ctx, w_router, slot_of, pool, shared, ws)
        self._head = (ctx.h, ctypes.byref(self._cfg), L)
        self._T = T
        self._mid = (_ptr(w_router),)
        self._tail = (_ptr(slot_of), n_slots, _ptr(pool), stride, _ptr(shared), _ptr(ws),
                      ws.numel() * ws.element_size())
        self._stream = _stream(stream)

    def status(self, x, bias, y) -> int:
        return self._fn(*self._head, _ptr(x), self._T, *self._mid, _ptr(bias), *self._tail, _ptr(y), self._stream)

    def __call__(self, x, bias, y) -> None:
        _check(self.status(x, bias, y), "moe_stack_forward")


def _is_mask(t, T) -> bool:
    return t.element_size() == 1 and t.nbytes >= T and t.is_contiguous()


# ------------------------------------------------------------------ 4-bit MX matrices

def _rows(t):
    """(rows, cols, elements from row to row) of a 2-D tensor with contiguous rows."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 2:
        rows, cols = shape
        if rows <= 1 and (cols <= 1 or stride[1] == 1):
            return rows, cols, cols
        if (cols <= 1 or stride[1] == 1) and stride[0] >= cols:
            return rows, cols, stride[0]
    raise MoeError(EINVAL, f"a 2-D tensor with contiguous rows is needed, got {tuple(shape)}, {stride}")


def _bad_mx4(codes, scales, rows, cols) -> bool:
    """Whether codes and scales are not the contiguous bytes of [rows, cols] MX rows (a number of columns
    that no MX row has is left to the library to refuse)."""
    if cols <= 0 or cols % MX4_BLOCK:
        return False
    return (codes.numel() != rows * cols // 2 or scales.numel() != rows * ((cols // MX4_BLOCK + 15) // 16 * 16)
            or codes.element_size() != 1 or scales.element_size() != 1
            or not codes.is_contiguous() or not scales.is_contiguous())


def mx4_scale_pitch(cols: int) -> int:
    """Bytes from one row of scales to the next; 0 where cols is no multiple of 32 or too large."""
    return int(load_library().moe_mx4_scale_pitch(cols))


def mx4_buffers(rows: int, cols: int, device="cuda"):
    """Uninitialised codes [rows, cols/2] and scales [rows, pitch] (uint8) of an MX matrix."""
    import torch
    pitch = mx4_scale_pitch(cols)
    if pitch == 0 or rows < 0:
        raise MoeError(EINVAL if rows < 0 or cols <= 0 else EUNSUPPORTED, "moe_mx4_scale_pitch")
    return (torch.empty(rows, cols // 2, dtype=torch.uint8, device=device),
            torch.empty(rows, pitch, dtype=torch.uint8, device=device))


def mx4_ffn_buffers(cfg: LayerCfg, T: int, device="cuda"):
    """The intermediate rows of expert_ffn_mx4 at T tokens: x's codes and scales, the hidden rows in bf16, and
    their codes and scales."""
    import torch
    n = T * cfg.k + (T if cfg.n_shared else 0)
    return (mx4_buffers(T, cfg.d, device), torch.empty(n, cfg.f, dtype=torch.bfloat16, device=device),
            mx4_buffers(n, cfg.f, device))


class Mx4Matrix:
    """One matrix or a pool of them in MX form: codes [rows, cols/2] or [slots, rows, cols/2] and scales
    [rows, pitch] or [slots, rows, pitch] (uint8; each matrix contiguous, the slots at any 16-byte stride)."""

    def __init__(self, codes, scales, cols: int):
        if codes.dim() == 2:
            codes, scales = codes.unsqueeze(0), scales.unsqueeze(0)
        pitch = mx4_scale_pitch(cols)
        if pitch == 0 or codes.dim() != 3 or scales.dim() != 3 or codes.shape[0] == 0:
            raise MoeError(EINVAL, "Mx4Matrix")
        self.n_slots, self.rows, self.cols = codes.shape[0], codes.shape[1], cols
        for t, n in ((codes, cols // 2), (scales, pitch)):
            if t.element_size() != 1 or tuple(t.shape) != (self.n_slots, self.rows, n) or not t[0].is_contiguous():
                raise MoeError(EINVAL, f"Mx4Matrix: a part of shape {tuple(t.shape)} for {cols} columns")
        if codes.get_device() != scales.get_device():
            raise MoeError(EINVAL, "Mx4Matrix: codes and scales on two devices")
        self.codes, self.scales, self.device = codes, scales, codes.get_device()
        self._c = _Mx4(codes.data_ptr(), scales.data_ptr(), codes.stride(0), scales.stride(0), self.n_slots, self.rows,
                       cols)
        self.ref = ctypes.byref(self._c)

    def c(self) -> _Mx4:
        return self._c


# ------------------------------------------------------------------ buffers

def balance_workspace(cfg: LayerCfg, device="cuda"):
    import torch
    n = int(load_library().moe_balance_workspace_bytes(cfg.ref()))
    if n == 0:
        raise MoeError(EINVAL, "moe_balance_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def workspace(cfg: LayerCfg, T: int, device="cuda"):
    import torch
    n = workspace_bytes(cfg, T)
    if n == 0:
        raise MoeError(EINVAL, "moe_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def stack_workspace(cfg: LayerCfg, L: int, T: int, device="cuda"):
    import torch
    n = int(load_library().moe_stack_workspace_bytes(cfg.ref(), L, T))
    if n == 0:
        raise MoeError(EINVAL, "moe_stack_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def place_records(cfg: LayerCfg, sections: list, device="cuda", stride: int | None = None):
    """Packs per-expert section arrays (gu_codes, dn_codes, gu_scales, dn_scales)
    into one uint8 pool tensor [n, stride] at libmoe's record offsets."""
    import numpy as np
    import torch
    lay = expert_layout(cfg)
    stride = stride or lay["bytes"]
    host = np.zeros((len(sections), stride), dtype=np.uint8)
    for i, sec in enumerate(sections):
        for name in ("gu_codes", "dn_codes", "gu_scales", "dn_scales"):
            raw = np.ascontiguousarray(sec[name]).view(np.uint8).reshape(-1)
            host[i, lay[name]:lay[name] + raw.size] = raw
    return torch.from_numpy(host).to(device), stride
