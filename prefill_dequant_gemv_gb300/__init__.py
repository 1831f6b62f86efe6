"""Python binding of the GB300 quantized GEMV / GEMM library (``libqgemv.so``).

Argument marshalling only: every step of the computation runs in the library's
CUDA kernels.  PyTorch provides device memory and streams.  The functions carry
the C ABI's names (see ``include/qgemv.h``); ``PackedWeight`` and the lower-case
helpers wrap them for torch tensors.

The library must have been built (``prefill_dequant_gemv_gb300.build.build()``);
importing the binding without it raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqgemv.so")

FMT_MLX_AFFINE4_G64, FMT_MXFP4, FMT_NVFP4, FMT_Q6K, FMT_Q5_0, FMT_Q5_1, FMT_Q5_K = 1, 2, 3, 4, 5, 6, 7
OUT_F32, OUT_BF16 = 0, 1
STATUS = {0: "QG_OK", 1: "QG_ERR_INVALID_ARG", 2: "QG_ERR_UNSUPPORTED", 3: "QG_ERR_MISALIGNED",
          4: "QG_ERR_WORKSPACE_TOO_SMALL", 5: "QG_ERR_CUDA", 6: "QG_ERR_TIMEOUT"}


class QGError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


class qg_weight(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("reserved", ctypes.c_int32), ("n", ctypes.c_int64),
                ("k", ctypes.c_int64), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("aux", ctypes.c_void_p), ("tensor_scale", ctypes.c_float), ("reserved2", ctypes.c_float)]


class qg_moe_layer(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("hidden", ctypes.c_int64),
                ("ffn", ctypes.c_int64), ("gu_codes", ctypes.c_void_p), ("gu_scales", ctypes.c_void_p),
                ("gu_aux", ctypes.c_void_p), ("dn_codes", ctypes.c_void_p), ("dn_scales", ctypes.c_void_p),
                ("dn_aux", ctypes.c_void_p), ("tensor_scale", ctypes.c_float), ("has_shared", ctypes.c_int32),
                ("shared_gate_up", qg_weight), ("shared_down", qg_weight)]


class qg_kv_cache(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("page_tokens", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("n_pages", ctypes.c_int64), ("k_codes", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p)]


class qg_kv_batch(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("max_new", ctypes.c_int32), ("max_len", ctypes.c_int64),
                ("q_start", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("pages", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64)]


class qg_norm_rope(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("weight_offset", ctypes.c_float), ("cos_sin", ctypes.c_void_p), ("n_positions", ctypes.c_int64),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


class qg_norm_out(ctypes.Structure):
    _fields_ = [("sum", ctypes.c_void_p), ("ldh", ctypes.c_int64), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("ldc", ctypes.c_int64), ("scales", ctypes.c_void_p), ("lds", ctypes.c_int64),
                ("group", ctypes.c_int64)]


class qg_lora(ctypes.Structure):
    _fields_ = [("n_adapters", ctypes.c_int32), ("max_rank", ctypes.c_int32), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("a", ctypes.c_void_p), ("lda", ctypes.c_int64), ("b", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("ranks", ctypes.c_void_p)]


class qg_route_rule(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("n_groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("group_best", ctypes.c_int32), ("renormalise", ctypes.c_int32), ("scale", ctypes.c_float),
                ("bias", ctypes.c_void_p)]


_lib = None
_P, _I64, _I, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
_SIGNATURES = {
    "qg_status_str": (ctypes.c_char_p, [_I]),
    "qg_packed_sizes": (_I, [_I, _I64, _I64, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)]),
    "qg_pack_host": (_I, [_I, _I64, _I64, _P, _P, _P, _P, _P, _P]),
    "qg_dequant": (_I, [ctypes.POINTER(qg_weight), _I, _P, _I64, _P]),
    "qg_gemv_workspace_size": (_SZ, [_I, _I64, _I64, _I]),
    "qg_workspace_init": (_I, [_P, _SZ, _P]),
    "qg_workspace_status": (_I, [_P, ctypes.POINTER(_I), _P]),
    "qgemv": (_I, [ctypes.POINTER(qg_weight), _P, _I, _I64, _P, _I64, _P, _I64, _P, _SZ, _P]),
    "qgemv_static_ws": (_I, [ctypes.POINTER(qg_weight), _P, _I, _I64, _P, _I64, _P, _I64, _P]),
    "qgemv_static_ws_status": (_I, [ctypes.POINTER(_I), _P]),
    "qg_gemm_workspace_size": (_SZ, [_I, _I64, _I64, _I]),
    "qgemm": (_I, [ctypes.POINTER(qg_weight), _P, _I64, _I64, _P, _I64, _P, _I64, _P, _SZ, _P]),
    "qmoe_route_workspace_size": (_SZ, [_I64, _I, _I]),
    "qmoe_route": (_I, [_P, _I64, _I, _I, _P, _P, _P, _SZ, _P]),
    "qmoe_workspace_size": (_SZ, [ctypes.POINTER(qg_moe_layer), _I64, _I]),
    "qmoe_ffn": (_I, [ctypes.POINTER(qg_moe_layer), _P, _I64, _I64, _I, _P, _P, _P, _P, _I64, _P, _SZ, _P]),
    "qgemm_grouped_workspace_size": (_SZ, [ctypes.POINTER(qg_moe_layer), _I64, _I, _I]),
    "qmoe_forward": (_I, [ctypes.POINTER(qg_moe_layer), _P, _I64, _I64, _P, _I, _P, _P, _P, _P, _SZ, _P, _I64, _P, _SZ,
                          _P]),
    "qgemm_grouped": (_I, [ctypes.POINTER(qg_moe_layer), _I, _P, _I64, _I64, _I, _P, _P, _P, _P, _I64, _P, _SZ, _P]),
    "qg_selftest_wait_timeout": (_I, [_P, _SZ, _P]),
    "qg_quant_act_nvfp4": (_I, [_P, _I64, _I64, _I64, ctypes.c_float, _P, _I64, _P, _I64, _P, _I64, _P]),
    "qgemm_w4a4_workspace_size": (_SZ, [_I, _I64, _I64, _I64]),
    "qgemm_w4a4": (_I, [ctypes.POINTER(qg_weight), _P, _I64, _I64, ctypes.c_float, _P, _I64, _P, _I64, _P, _SZ,
                        _P]),
    "qkv_append_workspace_size": (_SZ, []),
    "qkv_append": (_I, [ctypes.POINTER(qg_kv_cache), ctypes.POINTER(qg_kv_batch), ctypes.POINTER(qg_norm_rope), _I64, _I,
                        _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _SZ, _P]),
    "qattn_workspace_size": (_SZ, [ctypes.POINTER(qg_kv_cache), ctypes.POINTER(qg_kv_batch), _I64, _I]),
    "qattn": (_I, [ctypes.POINTER(qg_kv_cache), ctypes.POINTER(qg_kv_batch), _I64, _I, _P, _I64, _I64, ctypes.c_float,
                   _I64, _P, _I64, _I64, _P, _SZ, _P]),
    "qg_rms_norm": (_I, [_P, _I64, _P, _I64, _I64, _I64, _P, ctypes.c_float, ctypes.c_float, ctypes.POINTER(qg_norm_out), _P]),
    "qlora_workspace_size": (_SZ, [ctypes.POINTER(qg_lora), _I64]),
    "qlora": (_I, [ctypes.POINTER(qg_lora), _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _SZ, _P]),
    "qmoe_route_by": (_I, [ctypes.POINTER(qg_route_rule), _P, _I64, _I, _I, _P, _P, _P, _SZ, _P]),
}

QG_KV_E4M3 = 1
QG_SCORE_SOFTMAX, QG_SCORE_SIGMOID = 1, 2
QG_MOE_GATE_UP_SWIGLU = 1
QG_MOE_DOWN_COMBINE = 2


def lib():
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with prefill_dequant_gemv_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def _check(st: int, what: str):
    if st != 0:
        raise QGError(st, what)


# ------------------------------------------------------------------ C ABI, same names
def qg_status_str(status: int) -> str:
    return lib().qg_status_str(status).decode()


def qg_packed_sizes(fmt: int, n: int, k: int):
    c, s, a = _SZ(), _SZ(), _SZ()
    _check(lib().qg_packed_sizes(fmt, n, k, ctypes.byref(c), ctypes.byref(s), ctypes.byref(a)), "qg_packed_sizes")
    return c.value, s.value, a.value


def qg_pack_host(fmt: int, n: int, k: int, codes: np.ndarray, scales: np.ndarray, aux: Optional[np.ndarray]):
    """Pack logical host arrays; returns (codes, scales, aux) uint8 numpy arrays (aux empty unless Q6_K or
    Q5_K)."""
    cb, sb, ab = qg_packed_sizes(fmt, n, k)
    codes = np.ascontiguousarray(codes, dtype=np.uint8)
    scales = np.ascontiguousarray(scales)
    aux = None if aux is None else np.ascontiguousarray(aux)
    oc, os_, oa = np.empty(cb, np.uint8), np.empty(sb, np.uint8), np.empty(max(ab, 1), np.uint8)
    st = lib().qg_pack_host(fmt, n, k, codes.ctypes.data, scales.ctypes.data,
                            None if aux is None else aux.ctypes.data,
                            oc.ctypes.data, os_.ctypes.data, oa.ctypes.data if ab else None)
    _check(st, "qg_pack_host")
    return oc, os_, oa[:ab]


def qg_dequant(w: qg_weight, out_dtype: int, out_ptr: int, ldo: int, stream: int = 0):
    _check(lib().qg_dequant(ctypes.byref(w), out_dtype, out_ptr, ldo, stream), "qg_dequant")


def qg_gemv_workspace_size(fmt: int, n: int, k: int, m: int) -> int:
    return lib().qg_gemv_workspace_size(fmt, n, k, m)


def qg_workspace_init(ptr: int, nbytes: int, stream: int = 0):
    _check(lib().qg_workspace_init(ptr, nbytes, stream), "qg_workspace_init")


def qg_workspace_status(ptr: int, stream: int = 0) -> int:
    v = _I()
    _check(lib().qg_workspace_status(ptr, ctypes.byref(v), stream), "qg_workspace_status")
    return v.value


def qgemv(w: qg_weight, x_ptr: int, m: int, ldx: int, res_ptr: Optional[int], ldr: int, y_ptr: int, ldy: int,
          ws_ptr: int, ws_bytes: int, stream: int = 0):
    _check(lib().qgemv(ctypes.byref(w), x_ptr, m, ldx, res_ptr, ldr, y_ptr, ldy, ws_ptr, ws_bytes, stream),
           "qgemv")


def qg_gemm_workspace_size(fmt: int, n: int, k: int, m: int) -> int:
    return lib().qg_gemm_workspace_size(fmt, n, k, m)


def qgemm(w: qg_weight, x_ptr: int, m: int, ldx: int, res_ptr: Optional[int], ldr: int, y_ptr: int, ldy: int,
          ws_ptr: int, ws_bytes: int, stream: int = 0):
    _check(lib().qgemm(ctypes.byref(w), x_ptr, m, ldx, res_ptr, ldr, y_ptr, ldy, ws_ptr, ws_bytes, stream), "qgemm")


def qg_quant_act_nvfp4(x_ptr: int, m: int, k: int, ldx: int, act_scale: float, codes_ptr: Optional[int], ldc: int,
                       scales_ptr: Optional[int], lds: int, xe_ptr: Optional[int], lde: int, stream: int = 0):
    _check(lib().qg_quant_act_nvfp4(x_ptr, m, k, ldx, act_scale, codes_ptr, ldc, scales_ptr, lds, xe_ptr, lde, stream),
           "qg_quant_act_nvfp4")


def qgemm_w4a4_workspace_size(fmt: int, n: int, k: int, m: int) -> int:
    return lib().qgemm_w4a4_workspace_size(fmt, n, k, m)


def qgemm_w4a4(w: qg_weight, x_ptr: int, m: int, ldx: int, act_scale: float, res_ptr: Optional[int], ldr: int,
               y_ptr: int, ldy: int, ws_ptr: int, ws_bytes: int, stream: int = 0):
    _check(lib().qgemm_w4a4(ctypes.byref(w), x_ptr, m, ldx, act_scale, res_ptr, ldr, y_ptr, ldy, ws_ptr, ws_bytes,
                            stream), "qgemm_w4a4")


def qmoe_route_workspace_size(t: int, n_experts: int, topk: int) -> int:
    return lib().qmoe_route_workspace_size(t, n_experts, topk)


def qmoe_route(logits_ptr: int, t: int, n_experts: int, topk: int, ids_ptr: int, w_ptr: int, ws_ptr: int,
               ws_bytes: int, stream: int = 0):
    _check(lib().qmoe_route(logits_ptr, t, n_experts, topk, ids_ptr, w_ptr, ws_ptr, ws_bytes, stream), "qmoe_route")


def qmoe_workspace_size(layer: qg_moe_layer, t: int, topk: int) -> int:
    return lib().qmoe_workspace_size(ctypes.byref(layer), t, topk)


def qmoe_ffn(layer: qg_moe_layer, x_ptr: int, t: int, ldx: int, topk: int, w_ptr: int, gate_ptr: Optional[int],
             route_ws_ptr: int, out_ptr: int, ldo: int, ws_ptr: int, ws_bytes: int, stream: int = 0):
    _check(lib().qmoe_ffn(ctypes.byref(layer), x_ptr, t, ldx, topk, w_ptr, gate_ptr, route_ws_ptr, out_ptr, ldo,
                          ws_ptr, ws_bytes, stream), "qmoe_ffn")


def qmoe_forward(layer: qg_moe_layer, x_ptr: int, t: int, ldx: int, logits_ptr: int, topk: int,
                 gate_ptr: Optional[int], ids_ptr: int, w_ptr: int, route_ws_ptr: int, route_ws_bytes: int, out_ptr: int,
                 ldo: int, ws_ptr: int, ws_bytes: int, stream: int = 0):
    _check(lib().qmoe_forward(ctypes.byref(layer), x_ptr, t, ldx, logits_ptr, topk, gate_ptr, ids_ptr, w_ptr,
                              route_ws_ptr, route_ws_bytes, out_ptr, ldo, ws_ptr, ws_bytes, stream), "qmoe_forward")


def qgemm_grouped_workspace_size(layer: qg_moe_layer, t: int, topk: int, stage: int) -> int:
    return lib().qgemm_grouped_workspace_size(ctypes.byref(layer), t, topk, stage)


def qgemm_grouped(layer: qg_moe_layer, stage: int, in_ptr: int, t: int, ldi: int, topk: int, w_ptr: Optional[int],
                  gate_ptr: Optional[int], route_ws_ptr: int, out_ptr: int, ldo: int, ws_ptr: int, ws_bytes: int,
                  stream: int = 0):
    _check(lib().qgemm_grouped(ctypes.byref(layer), stage, in_ptr, t, ldi, topk, w_ptr, gate_ptr, route_ws_ptr,
                               out_ptr, ldo, ws_ptr, ws_bytes, stream), "qgemm_grouped")


def qgemv_static_ws(w: qg_weight, x_ptr: int, m: int, ldx: int, res_ptr: Optional[int], ldr: int, y_ptr: int,
                    ldy: int, stream: int = 0):
    """qgemv without a workspace argument, for callers that cannot allocate device memory
    (its scratch is a fixed array inside the library, shared by all calls)."""
    _check(lib().qgemv_static_ws(ctypes.byref(w), x_ptr, m, ldx, res_ptr, ldr, y_ptr, ldy, stream), "qgemv_static_ws")


def qgemv_static_ws_status(stream: int = 0) -> int:
    """Read and clear the status word of qgemv_static_ws's array on the current device
    (synchronises `stream`): QG_OK, or QG_ERR_TIMEOUT after a bounded wait gave up."""
    v = _I(0)
    _check(lib().qgemv_static_ws_status(ctypes.byref(v), stream), "qgemv_static_ws_status")
    return v.value


def qg_selftest_wait_timeout(ws_ptr: int, ws_bytes: int, stream: int = 0):
    """Launch the bounded-wait self-test (its wait runs out after the library's limit and
    records QG_ERR_TIMEOUT in the workspace status word)."""
    _check(lib().qg_selftest_wait_timeout(ws_ptr, ws_bytes, stream), "qg_selftest_wait_timeout")


def qkv_append_workspace_size() -> int:
    return lib().qkv_append_workspace_size()


def qkv_append(cache: qg_kv_cache, batch: qg_kv_batch, norm_rope: Optional[qg_norm_rope], n_tokens: int, n_q_heads: int,
               q_ptr: Optional[int], ldq: int, hsq: int, k_ptr: int, ldk: int, hsk: int, v_ptr: int, ldv: int, hsv: int,
               q_out_ptr: Optional[int], ldqo: int, hsqo: int, ws_ptr: int, ws_bytes: int, stream: int = 0):
    _check(lib().qkv_append(cache, batch, norm_rope, n_tokens, n_q_heads, q_ptr, ldq, hsq, k_ptr, ldk, hsk, v_ptr, ldv,
                            hsv, q_out_ptr, ldqo, hsqo, ws_ptr, ws_bytes, stream), "qkv_append")


def qattn_workspace_size(cache: qg_kv_cache, batch: qg_kv_batch, n_tokens: int, n_q_heads: int) -> int:
    return lib().qattn_workspace_size(cache, batch, n_tokens, n_q_heads)


def qattn(cache: qg_kv_cache, batch: qg_kv_batch, n_tokens: int, n_q_heads: int, q_ptr: int, ldq: int, hsq: int,
          scale: float, window: int, out_ptr: int, ldo: int, hso: int, ws_ptr: int, ws_bytes: int, stream: int = 0):
    _check(lib().qattn(cache, batch, n_tokens, n_q_heads, q_ptr, ldq, hsq, scale, window, out_ptr, ldo, hso, ws_ptr,
                       ws_bytes, stream), "qattn")


def qg_rms_norm(x_ptr: int, ldx: int, res_ptr: Optional[int], ldr: int, m: int, k: int, w_ptr: int, eps: float,
                weight_offset: float, out: qg_norm_out, stream: int = 0):
    _check(lib().qg_rms_norm(x_ptr, ldx, res_ptr, ldr, m, k, w_ptr, eps, weight_offset, out, stream), "qg_rms_norm")


def qlora_workspace_size(lora: "qg_lora", m: int) -> int:
    return lib().qlora_workspace_size(lora, m)


def qlora(lora: "qg_lora", ids_ptr: int, m: int, x_ptr: int, ldx: int, y_ptr: int, ldy: int, out_ptr: int, ldo: int, ws_ptr: int,
          ws_bytes: int, stream: int = 0):
    _check(lib().qlora(lora, ids_ptr, m, x_ptr, ldx, y_ptr, ldy, out_ptr, ldo, ws_ptr, ws_bytes, stream), "qlora")


def qmoe_route_by(rule: Optional[qg_route_rule], logits_ptr: int, t: int, n_experts: int, topk: int, ids_ptr: int, w_ptr: int,
                  ws_ptr: int, ws_bytes: int, stream: int = 0):
    _check(lib().qmoe_route_by(rule, logits_ptr, t, n_experts, topk, ids_ptr, w_ptr, ws_ptr, ws_bytes, stream), "qmoe_route_by")


# ------------------------------------------------------------------ torch helpers
def _need(ok: bool, what: str):
    if not ok:
        raise QGError(1, what)


def _on(index: int, call, *args):
    """call(*args, the current stream of device `index`), with that device the current one."""
    import torch
    c = torch._C
    if c._cuda_getDevice() == index:
        return call(*args, c._cuda_getCurrentRawStream(index))
    with torch.cuda.device(index):
        return call(*args, _raw_stream(index))


def _stream_ptr(stream=None) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


class PackedWeight:
    """A packed weight resident in device memory plus its ``qg_weight`` descriptor."""

    def __init__(self, fmt: int, n: int, k: int, codes, scales, aux, tensor_scale: float = 1.0):
        self.fmt, self.n, self.k = fmt, n, k
        self.codes, self.scales, self.aux = codes, scales, aux  # torch uint8 device tensors
        self.tensor_scale = float(tensor_scale)
        self.desc = qg_weight(fmt, 0, n, k, codes.data_ptr(), scales.data_ptr(),
                              aux.data_ptr() if aux is not None else None, self.tensor_scale, 0.0)

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel() + (self.aux.numel() if self.aux is not None else 0)

    @staticmethod
    def from_logical(w, device="cuda") -> "PackedWeight":
        """Pack a logical weight (``workloads.QWeight``) on the host and copy it to ``device``."""
        import torch
        c, s, a = qg_pack_host(w.fmt, w.n, w.k, w.codes, w.scales, w.aux)
        tc = torch.from_numpy(c).to(device)
        ts_ = torch.from_numpy(s).to(device)
        ta = torch.from_numpy(a).to(device) if a.size else None
        return PackedWeight(w.fmt, w.n, w.k, tc, ts_, ta, w.tensor_scale if w.fmt == FMT_NVFP4 else 1.0)


class Workspace:
    """A zero-initialised device workspace (caller-owned memory for the kernels' split-K state)."""

    def __init__(self, nbytes: int, device="cuda"):
        import torch
        self.nbytes = max(int(nbytes), 256)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device)
        self.index = self.buf.get_device()

    @property
    def ptr(self) -> int:
        return self.buf.data_ptr()

    def status(self) -> int:
        """The status word, read and cleared; after a wait that gave up the whole workspace is zeroed, as the kernels'
        counters may have been left behind."""
        st = qg_workspace_status(self.ptr, _stream_ptr())
        if st == 6:
            self.buf.zero_()
        return st


def dequant(pw: PackedWeight, out_dtype: int = OUT_F32):
    import torch
    dt = torch.float32 if out_dtype == OUT_F32 else torch.bfloat16
    ldo = (pw.k + 7) // 8 * 8
    out = torch.empty((pw.n, ldo), dtype=dt, device=pw.codes.device)
    qg_dequant(pw.desc, out_dtype, out.data_ptr(), ldo, _stream_ptr())
    return out[:, :pw.k]


def gemv(pw: PackedWeight, x, residual=None, out=None, workspace: Optional[Workspace] = None):
    """y = bf16(W x (+ residual)) for x bf16 [m, k] on the device, m = 1..4."""
    import torch
    m = x.shape[0]
    if out is None:
        out = torch.empty((m, (pw.n + 7) // 8 * 8), dtype=torch.bfloat16, device=x.device)[:, :pw.n]
    if workspace is None:
        workspace = Workspace(qg_gemv_workspace_size(pw.fmt, pw.n, pw.k, m), x.device)
    qgemv(pw.desc, x.data_ptr(), m, x.stride(0), None if residual is None else residual.data_ptr(),
          0 if residual is None else residual.stride(0), out.data_ptr(), out.stride(0), workspace.ptr,
          workspace.nbytes, _stream_ptr())
    return out


def gemm(pw: PackedWeight, x, residual=None, out=None, workspace: Optional[Workspace] = None):
    """y = bf16(W x (+ residual)) for x bf16 [m, k] on the device, any m (tokens)."""
    import torch
    m = x.shape[0]
    if out is None:
        out = torch.empty((m, (pw.n + 7) // 8 * 8), dtype=torch.bfloat16, device=x.device)[:, :pw.n]
    if workspace is None:
        workspace = Workspace(qg_gemm_workspace_size(pw.fmt, pw.n, pw.k, min(m, 2 ** 31 - 1)), x.device)
    qgemm(pw.desc, x.data_ptr(), m, x.stride(0), None if residual is None else residual.data_ptr(),
          0 if residual is None else residual.stride(0), out.data_ptr(), out.stride(0), workspace.ptr,
          workspace.nbytes, _stream_ptr())
    return out


def quant_act_nvfp4(x, act_scale: float):
    """NVFP4-quantise bf16 activations x [m, k] on the device (W4A4).  Returns (codes uint8 [m, k/2], two
    E2M1 codes a byte, the even k in the low nibble; scales uint8 [m, k/16] E4M3; xe bf16 [m, k], the exact
    expansion E4M3(S) * E2M1(code) without act_scale)."""
    import torch
    m, k = x.shape
    dev = x.device
    codes = torch.empty((m, (k // 2 + 7) // 8 * 8), dtype=torch.uint8, device=dev)
    scales = torch.empty((m, k // 16), dtype=torch.uint8, device=dev)
    xe = torch.empty((m, (k + 7) // 8 * 8), dtype=torch.bfloat16, device=dev)
    qg_quant_act_nvfp4(x.data_ptr(), m, k, x.stride(0), act_scale, codes.data_ptr(), codes.stride(0),
                       scales.data_ptr(), scales.stride(0), xe.data_ptr(), xe.stride(0), _stream_ptr())
    return codes[:, :k // 2], scales, xe[:, :k]


def gemm_w4a4(pw: PackedWeight, x, act_scale: float, residual=None, out=None, workspace: Optional[Workspace] = None):
    """y = bf16(W xq (+ residual)) with xq the NVFP4 quantisation of x (bf16 [m, k]) at tensor scale act_scale."""
    import torch
    m = x.shape[0]
    if out is None:
        out = torch.empty((m, (pw.n + 7) // 8 * 8), dtype=torch.bfloat16, device=x.device)[:, :pw.n]
    if workspace is None:
        workspace = Workspace(qgemm_w4a4_workspace_size(pw.fmt, pw.n, pw.k, m), x.device)
    qgemm_w4a4(pw.desc, x.data_ptr(), m, x.stride(0), act_scale, None if residual is None else residual.data_ptr(),
               0 if residual is None else residual.stride(0), out.data_ptr(), out.stride(0), workspace.ptr,
               workspace.nbytes, _stream_ptr())
    return out


class PackedMoE:
    """A mixture-of-experts layer packed on the host and resident in device memory: the
    routed experts' packed matrices back to back, the shared expert separate."""

    def __init__(self, layer, device="cuda"):
        import torch
        self.fmt, self.n_experts, self.hidden, self.ffn = layer.fmt, layer.n_experts, layer.hidden, layer.ffn

        def pack_all(ws):
            parts = [qg_pack_host(w.fmt, w.n, w.k, w.codes, w.scales, w.aux) for w in ws]
            out = []
            for i in range(3):
                cat = np.concatenate([p[i] for p in parts]) if parts[0][i].size else np.zeros(0, np.uint8)
                out.append(torch.from_numpy(cat).to(device) if cat.size else None)
            return out

        self.gu = pack_all(layer.gate_up)
        self.dn = pack_all(layer.down)
        self.shared = None
        if layer.shared_gate_up is not None:
            self.shared = (PackedWeight.from_logical(layer.shared_gate_up, device),
                           PackedWeight.from_logical(layer.shared_down, device))
        ts = layer.gate_up[0].tensor_scale if layer.fmt == FMT_NVFP4 else 1.0
        empty = qg_weight(layer.fmt, 0, 0, 0, None, None, None, 1.0, 0.0)
        self.desc = qg_moe_layer(
            layer.fmt, layer.n_experts, layer.hidden, layer.ffn,
            self.gu[0].data_ptr(), self.gu[1].data_ptr(), self.gu[2].data_ptr() if self.gu[2] is not None else None,
            self.dn[0].data_ptr(), self.dn[1].data_ptr(), self.dn[2].data_ptr() if self.dn[2] is not None else None,
            ts, 1 if self.shared else 0,
            self.shared[0].desc if self.shared else empty, self.shared[1].desc if self.shared else empty)

    @property
    def nbytes_per_expert(self) -> int:
        tot = sum(t.numel() for t in self.gu if t is not None) + sum(t.numel() for t in self.dn if t is not None)
        return tot // self.n_experts


class RouteRule:
    """How experts are chosen and weighed (``qg_route_rule``): ``score`` "softmax" or "sigmoid"; ``bias`` fp32 [experts] added
    for the choice alone; of ``groups`` groups of consecutive experts the ``topk_groups`` best are kept, a group valued by
    the sum of its ``group_best`` (1 or 2) largest; the chosen scores, divided by their sum with ``renormalise``, times ``scale``."""

    def __init__(self, score: str = "softmax", bias=None, groups: int = 1, topk_groups: int = 1, group_best: int = 2,
                 renormalise: bool = True, scale: float = 1.0):
        import torch
        kinds = {"softmax": QG_SCORE_SOFTMAX, "sigmoid": QG_SCORE_SIGMOID}
        _need(score in kinds, "RouteRule: score is softmax or sigmoid")
        _need(bias is None or (bias.dtype == torch.float32 and bias.dim() == 1 and bias.is_contiguous()),
              "RouteRule: bias is contiguous float32 [experts]")
        _need(0 <= min(groups, topk_groups, group_best) and max(groups, topk_groups, group_best) < 1 << 31,
              "RouteRule: groups, topk_groups and group_best are 32-bit counts")
        self.bias = bias
        self.desc = qg_route_rule(kinds[score], groups, topk_groups, group_best, 1 if renormalise else 0, scale,
                                  None if bias is None else bias.data_ptr())


def _route_by(rule: RouteRule, logits, topk: int, workspace: Optional[Workspace]):
    import torch
    t, e = logits.shape
    index = logits.get_device()
    if logits.dtype is not torch.float32 or not logits.is_contiguous() or index < 0:
        raise QGError(1, "route: contiguous float32 logits [tokens, experts] on a CUDA device")
    if rule.bias is not None and (rule.bias.shape[0] != e or rule.bias.get_device() != index):
        raise QGError(1, "route: a bias for every expert, on the logits' device")
    if workspace is None:
        workspace = Workspace(qmoe_route_workspace_size(t, e, topk), logits.device)
    elif workspace.index != index:
        raise QGError(1, "route: the workspace on the logits' device")
    device = logits.device
    ids, w = torch.empty(t, topk, dtype=torch.int32, device=device), torch.empty(t, topk, dtype=torch.float32, device=device)
    st = _on(index, (_lib or lib()).qmoe_route_by, rule.desc, logits.data_ptr(), t, e, topk, ids.data_ptr(), w.data_ptr(),
             workspace.ptr, workspace.nbytes)
    if st:
        raise QGError(st, "qmoe_route_by")
    return ids, w, workspace


def route(logits, topk: int, workspace: Optional[Workspace] = None, rule: Optional[RouteRule] = None):
    """(topk_ids int32 [t, topk], topk_w fp32 [t, topk], route workspace) for fp32 logits [t, E] on the device:
    the largest logits and their softmax, or by a rule (``qmoe_route_by``)."""
    if rule is not None:
        return _route_by(rule, logits, topk, workspace)
    import torch
    t, e = logits.shape
    ids = torch.empty((t, topk), dtype=torch.int32, device=logits.device)
    w = torch.empty((t, topk), dtype=torch.float32, device=logits.device)
    if workspace is None:
        workspace = Workspace(qmoe_route_workspace_size(t, e, topk), logits.device)
    qmoe_route(logits.data_ptr(), t, e, topk, ids.data_ptr(), w.data_ptr(), workspace.ptr, workspace.nbytes,
               _stream_ptr())
    return ids, w, workspace


def moe_ffn(pm: PackedMoE, x, topk_w, route_ws: Workspace, out=None, workspace: Optional[Workspace] = None,
            shared_gate=None):
    """One MoE FFN layer for the routed tokens x bf16 [t, H]: 1..4 tokens take the grouped-GEMV
    decode chain, more tokens the grouped tensor-core prefill chain.  shared_gate: fp32 [t]
    gate logits of the shared expert (its output is weighed by their sigmoid), or None."""
    import torch
    t = x.shape[0]
    topk = topk_w.shape[1]
    if out is None:
        out = torch.empty((t, (pm.hidden + 7) // 8 * 8), dtype=torch.bfloat16, device=x.device)[:, :pm.hidden]
    if workspace is None:
        workspace = Workspace(qmoe_workspace_size(pm.desc, t, topk), x.device)
    qmoe_ffn(pm.desc, x.data_ptr(), t, x.stride(0), topk, topk_w.data_ptr(),
             None if shared_gate is None else shared_gate.data_ptr(), route_ws.ptr, out.data_ptr(),
             out.stride(0), workspace.ptr, workspace.nbytes, _stream_ptr())
    return out


def moe_forward(pm: PackedMoE, x, logits, topk: int, out=None, workspace: Optional[Workspace] = None,
                route_ws: Optional[Workspace] = None, shared_gate=None, rule: Optional[RouteRule] = None):
    """Router and MoE FFN in one call (qmoe_forward; by a rule qmoe_route_by, then qmoe_ffn) for x bf16 [t, H] and fp32
    logits [t, E]: returns (out bf16 [t, H], topk_ids int32 [t, topk], topk_w fp32 [t, topk], route workspace)."""
    import torch
    if rule is not None:
        if logits.get_device() >= 0 and logits.get_device() != torch._C._cuda_getDevice():
            with torch.cuda.device(logits.device):
                return moe_forward(pm, x, logits, topk, out, workspace, route_ws, shared_gate, rule)
        if (x.shape[0], pm.n_experts) != tuple(logits.shape) or x.get_device() != logits.get_device():
            raise QGError(1, f"moe_forward: logits [{x.shape[0]}, {pm.n_experts}] on x's device")
        ids, w, route_ws = _route_by(rule, logits, topk, route_ws)
        return moe_ffn(pm, x, w, route_ws, out, workspace, shared_gate), ids, w, route_ws
    t = x.shape[0]
    e = logits.shape[1]
    ids = torch.empty((t, topk), dtype=torch.int32, device=x.device)
    w = torch.empty((t, topk), dtype=torch.float32, device=x.device)
    if route_ws is None:
        route_ws = Workspace(qmoe_route_workspace_size(t, e, topk), x.device)
    if out is None:
        out = torch.empty((t, (pm.hidden + 7) // 8 * 8), dtype=torch.bfloat16, device=x.device)[:, :pm.hidden]
    if workspace is None:
        workspace = Workspace(qmoe_workspace_size(pm.desc, t, topk), x.device)
    qmoe_forward(pm.desc, x.data_ptr(), t, x.stride(0), logits.data_ptr(), topk,
                 None if shared_gate is None else shared_gate.data_ptr(), ids.data_ptr(), w.data_ptr(), route_ws.ptr,
                 route_ws.nbytes, out.data_ptr(), out.stride(0), workspace.ptr, workspace.nbytes, _stream_ptr())
    return out, ids, w, route_ws


def moe_stage(pm: PackedMoE, stage: int, inp, t: int, topk: int, route_ws: Workspace, topk_w=None, out=None,
              workspace: Optional[Workspace] = None, shared_gate=None):
    """One stage of the MoE FFN (qgemm_grouped): QG_MOE_GATE_UP_SWIGLU takes x bf16 [t, H] and
    returns h bf16 [t*topk + (t if shared), F] in the router's grouped row order;
    QG_MOE_DOWN_COMBINE takes that h, topk_w and optionally the shared expert's gate logits and
    returns out bf16 [t, H]."""
    import torch
    rows = t * topk + (t if pm.desc.has_shared else 0)
    cols = pm.ffn if stage == QG_MOE_GATE_UP_SWIGLU else pm.hidden
    n_out = rows if stage == QG_MOE_GATE_UP_SWIGLU else t
    if out is None:
        out = torch.empty((n_out, (cols + 7) // 8 * 8), dtype=torch.bfloat16, device=inp.device)[:, :cols]
    if workspace is None:
        workspace = Workspace(qgemm_grouped_workspace_size(pm.desc, t, topk, stage), inp.device)
    qgemm_grouped(pm.desc, stage, inp.data_ptr(), t, inp.stride(0), topk,
                  None if topk_w is None else topk_w.data_ptr(),
                  None if shared_gate is None else shared_gate.data_ptr(), route_ws.ptr, out.data_ptr(),
                  out.stride(0), workspace.ptr, workspace.nbytes, _stream_ptr())
    return out


# ------------------------------------------------------------------ RMS norm and low-rank adapters
def _rows(t, shape, dtype, index, what, name):
    """(pointer, row stride) of a matrix of `shape` and `dtype` on device `index`; its rows' elements lie side by side."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index:
        ld, step = t.stride()
        if step == 1 or shape[1] == 1:
            return t.data_ptr(), (ld if shape[0] > 1 else (shape[1] + 7) // 8 * 8)
    raise QGError(1, f"{what}: {name} is {dtype} {[*shape]} with a contiguous last dimension, on the call's CUDA device")


def _new_rows(x, shape, dtype):
    """A new matrix whose rows start at multiples of 16 bytes."""
    import torch
    m, k = shape
    if k % 16 == 0:
        return torch.empty(m, k, dtype=dtype, device=x.device)
    return torch.empty(m, (k + 15) // 16 * 16, dtype=dtype, device=x.device)[:, :k]


def _norm(x, weight, residual, sum_out, bf16, what):
    """The checked inputs of a norm: (x's shape, device, the arguments up to the weight, pointer and stride of the sum, the sum)."""
    index, shape = x.get_device(), x.shape
    if len(shape) != 2 or index < 0:
        raise QGError(1, f"{what}: x is bfloat16 [rows, columns] on a CUDA device")
    m, k = shape
    xp, ldx = _rows(x, shape, bf16, index, what, "x")
    if weight.dtype is not bf16 or weight.shape != (k,) or weight.get_device() != index or (k > 1 and weight.stride(0) != 1):
        raise QGError(1, f"{what}: weight is contiguous bfloat16 [{k}] on x's device")
    if residual is None:
        if sum_out is not None:
            raise QGError(1, f"{what}: a sum needs a residual")
        return shape, index, (xp, ldx, None, 0, m, k, weight.data_ptr()), None, 0, None
    rp, ldr = _rows(residual, shape, bf16, index, what, "residual")
    if sum_out is None:
        sum_out = _new_rows(x, shape, bf16)
    hp, ldh = _rows(sum_out, shape, bf16, index, what, "sum_out")
    return shape, index, (xp, ldx, rp, ldr, m, k, weight.data_ptr()), hp, ldh, sum_out


def rms_norm(x, weight, residual=None, eps: float = 1e-6, weight_offset: float = 0.0, out=None, sum_out=None):
    """RMS norm of x (bf16 [m, k]), after the residual's addition if there is one (``qg_rms_norm``): returns (y bf16 [m, k],
    the sum bf16 [m, k] or None).  out or sum_out may be x or the residual itself."""
    import torch
    bf16 = torch.bfloat16
    shape, index, args, hp, ldh, sum_out = _norm(x, weight, residual, sum_out, bf16, "rms_norm")
    if out is None:
        out = _new_rows(x, shape, bf16)
    yp, ldy = _rows(out, shape, bf16, index, "rms_norm", "out")
    st = _on(index, (_lib or lib()).qg_rms_norm, *args, eps, weight_offset, qg_norm_out(hp, ldh, yp, ldy))
    if st:
        raise QGError(st, "qg_rms_norm")
    return out, sum_out


def rms_norm_fp8(x, weight, residual=None, eps: float = 1e-6, weight_offset: float = 0.0, group: int = 128, out=None, scales=None,
                 sum_out=None, y_out=None):
    """``rms_norm`` with its output in 8 bits: returns (codes float8_e4m3fn [m, k], scales fp32 [m, ceil(k / group)], the
    sum or None); group 32, 64 or 128, or 0 for one scale a row.  y_out (bf16 [m, k]), if given, takes the output in bf16 too."""
    import torch
    bf16 = torch.bfloat16
    shape, index, args, hp, ldh, sum_out = _norm(x, weight, residual, sum_out, bf16, "rms_norm_fp8")
    if group not in (0, 32, 64, 128):
        raise QGError(2, "rms_norm_fp8: group is 32, 64, 128 or 0")
    groups = shape[0], (-(-shape[1] // group) if group else 1)
    if out is None:
        out = _new_rows(x, shape, torch.float8_e4m3fn)
    if scales is None:
        scales = torch.empty(groups, dtype=torch.float32, device=x.device)
    cp, ldc = _rows(out, shape, torch.float8_e4m3fn, index, "rms_norm_fp8", "out")
    if scales.dtype is not torch.float32 or scales.shape != groups or scales.get_device() != index or \
            (groups[1] > 1 and scales.stride(1) != 1):
        raise QGError(1, f"rms_norm_fp8: scales are float32 {[*groups]} with a contiguous last dimension, on x's device")
    lds = scales.stride(0) if groups[0] > 1 else groups[1]
    yp, ldy = (None, 0) if y_out is None else _rows(y_out, shape, bf16, index, "rms_norm_fp8", "y_out")
    st = _on(index, (_lib or lib()).qg_rms_norm, *args, eps, weight_offset,
             qg_norm_out(hp, ldh, yp, ldy, cp, ldc, scales.data_ptr(), lds, group))
    if st:
        raise QGError(st, "qg_rms_norm")
    return out, scales, sum_out


class LoraAdapters:
    """Low-rank adapters of one projection (``qg_lora``): a bf16 [adapters, max_rank, k], b bf16 [adapters, n, max_rank],
    scales fp32 [adapters] and, where they have not all max_rank, ranks int32 [adapters], on one device.  The tensors'
    contents may change between calls."""

    def __init__(self, a, b, scales, ranks=None):
        import torch
        _need(a.dtype == b.dtype == torch.bfloat16 and a.dim() == b.dim() == 3, "LoraAdapters: a and b are bfloat16 of 3 dimensions")
        count, top, k = (int(v) for v in a.shape)
        n = int(b.shape[1])
        _need(b.shape == (count, n, top) and b.is_contiguous(), "LoraAdapters: b is contiguous [adapters, outputs, max_rank]")
        _need(min(count, top, k, n) > 0, "LoraAdapters: no empty dimension")
        lda = int(a.stride(1)) if top > 1 else (k + 7) // 8 * 8
        _need((k == 1 or a.stride(2) == 1) and lda >= k and (count == 1 or a.stride(0) == top * lda),
              "LoraAdapters: a is [adapters, max_rank, inputs] with rows at one distance")
        _need(scales.dtype == torch.float32 and scales.shape == (count,) and scales.is_contiguous(),
              "LoraAdapters: scales are contiguous float32 [adapters]")
        _need(ranks is None or (ranks.dtype == torch.int32 and ranks.shape == (count,) and ranks.is_contiguous()),
              "LoraAdapters: ranks are contiguous int32 [adapters]")
        for t in (b, scales, ranks):
            _need(t is None or t.device == a.device, "LoraAdapters: tensors on one device")
        self.a, self.b, self.scales, self.ranks = a, b, scales, ranks
        self.n, self.k, self.index = n, k, a.get_device()
        self.desc = qg_lora(count, top, n, k, a.data_ptr(), lda, b.data_ptr(), scales.data_ptr(),
                            None if ranks is None else ranks.data_ptr())


def lora_workspace_size(adapters: LoraAdapters, m: int) -> int:
    """Workspace bytes of ``lora`` for m rows."""
    import torch
    with torch.cuda.device(adapters.index):  # -1, not on a GPU: the current one
        return qlora_workspace_size(adapters.desc, m)


def lora(adapters: LoraAdapters, ids, x, y, out=None, workspace: Optional[Workspace] = None):
    """y plus each row's adapter's share (``qlora``): ids int32 [m] (-1: none), x bf16 [m, k] the projection's input, y bf16 [m, n]
    its output.  Without ``out`` y is changed in place."""
    import torch
    bf16 = torch.bfloat16
    index, m = adapters.index, x.shape[0]
    if index < 0 or ids.dtype is not torch.int32 or ids.shape != (m,) or ids.get_device() != index or (m > 1 and ids.stride(0) != 1):
        raise QGError(1, f"lora: contiguous int32 ids [{m}] on the adapters' CUDA device")
    xp, ldx = _rows(x, (m, adapters.k), bf16, index, "lora", "x")
    shape = m, adapters.n
    yp, ldy = _rows(y, shape, bf16, index, "lora", "y")
    if out is None:
        out, op, ldo = y, yp, ldy
    else:
        op, ldo = _rows(out, shape, bf16, index, "lora", "out")
    if workspace is None:
        workspace = Workspace(lora_workspace_size(adapters, m), x.device)
    elif workspace.index != index:
        raise QGError(1, "lora: the workspace on the adapters' device")
    st = _on(index, (_lib or lib()).qlora, adapters.desc, ids.data_ptr(), m, xp, ldx, yp, ldy, op, ldo, workspace.ptr, workspace.nbytes)
    if st:
        raise QGError(st, "qlora")
    return out


# ------------------------------------------------------------------ attention over the 8-bit paged cache
def _raw_stream(index: int) -> int:
    """The current stream of a device, as torch keeps it."""
    import torch
    return torch.cuda.current_stream(index).cuda_stream


def _raw_stream_getter():
    """torch's own accessor of the current stream's handle (0.1 us a call; a Stream object takes 1.2) where it has one."""
    import torch
    return getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


class KVCache:
    """A pool of pages of keys and values in 8 bits (``qg_kv_cache``): codes float8_e4m3fn (or uint8)
    [n_pages, n_kv_heads, page_tokens, head_dim] and scales fp32 [n_pages, n_kv_heads], contiguous on the device."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        import torch
        _need(k_codes.dim() == 4 and k_codes.shape == v_codes.shape, "KVCache: codes are [pages, heads, tokens, dim]")
        _need(k_scales.shape == k_codes.shape[:2] and v_scales.shape == k_codes.shape[:2], "KVCache: scales are [pages, heads]")
        for t in (k_codes, v_codes, k_scales, v_scales):
            _need(t.is_contiguous() and t.device == k_codes.device, "KVCache: contiguous tensors on one device")
        for t in (k_codes, v_codes):
            _need(t.dtype in (torch.float8_e4m3fn, torch.uint8), "KVCache: codes are float8_e4m3fn or uint8")
        for t in (k_scales, v_scales):
            _need(t.dtype == torch.float32, "KVCache: scales are float32")
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.n_pages, self.n_kv_heads, self.page_tokens, self.head_dim = (int(x) for x in k_codes.shape)
        # what each call needs of torch, looked up once: calls of a decode step are short
        self.bf16 = torch.bfloat16
        self.index = k_codes.get_device() if k_codes.is_cuda else -2  # where no tensor is
        self.raw_stream = _raw_stream_getter()
        self.desc = qg_kv_cache(QG_KV_E4M3, self.page_tokens, self.n_kv_heads, self.head_dim, self.n_pages,
                                k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr())

    @staticmethod
    def empty(n_pages: int, n_kv_heads: int, page_tokens: int, head_dim: int, device="cuda") -> "KVCache":
        """A pool with nothing in it yet."""
        import torch
        shape = (n_pages, n_kv_heads, page_tokens, head_dim)
        codes = [torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.ones(shape[:2], dtype=torch.float32, device=device) for _ in range(2)]
        return KVCache(*codes, *scales)


class KVBatch:
    """The sequences of a call (``qg_kv_batch``): q_start int32 [n_seqs + 1], lens int32 [n_seqs] (with the new
    tokens) and pages int32 [n_seqs, m] on the device; max_new and max_len bound every sequence's new tokens
    and length, max_len by m pages at most.  The tensors' contents may change between calls (within the bounds)."""

    def __init__(self, q_start, lens, pages, max_new: int, max_len: int):
        import torch
        for t in (q_start, lens, pages):
            _need(t.dtype == torch.int32 and t.device == lens.device, "KVBatch: int32 tensors on one device")
        n = lens.numel()
        _need(lens.dim() == 1 and lens.is_contiguous(), "KVBatch: lens is contiguous [n_seqs]")
        _need(q_start.shape == (n + 1,) and q_start.is_contiguous(), "KVBatch: q_start is contiguous [n_seqs + 1]")
        _need(pages.dim() == 2 and pages.shape[0] == n and pages.stride(1) == 1, "KVBatch: pages is [n_seqs, m]")
        _need(n == 1 or pages.stride(0) >= pages.shape[1], "KVBatch: pages' rows overlap")
        self.q_start, self.lens, self.pages = q_start, lens, pages
        self.n_seqs, self.max_new, self.max_len = n, int(max_new), int(max_len)
        self.index, self.width = lens.get_device(), int(pages.shape[1])  # (a row's stride may be longer)
        self.desc = qg_kv_batch(n, self.max_new, self.max_len, q_start.data_ptr(), lens.data_ptr(), pages.data_ptr(),
                                pages.stride(0) if n > 1 else pages.shape[1])


class NormRope:
    """Norm weights (bf16 [head_dim], each optional) and rotation table (fp32 [positions, rotary_dim]: the pairs'
    cosines, then their sines) of ``kv_append`` (``qg_norm_rope``)."""

    def __init__(self, q_weight=None, k_weight=None, eps: float = 1e-6, weight_offset: float = 0.0, cos_sin=None,
                 interleaved: bool = False):
        import torch
        for t in (q_weight, k_weight):
            _need(t is None or (t.dtype == torch.bfloat16 and t.dim() == 1 and t.is_contiguous()),
                  "NormRope: weights are contiguous bfloat16 [head_dim]")
        _need(cos_sin is None or (cos_sin.dtype == torch.float32 and cos_sin.dim() == 2 and cos_sin.is_contiguous()),
              "NormRope: cos_sin is contiguous float32 [positions, rotary_dim]")
        self.q_weight, self.k_weight, self.cos_sin = q_weight, k_weight, cos_sin
        places = {t.get_device() for t in (q_weight, k_weight, cos_sin) if t is not None}
        _need(len(places) < 2, "NormRope: tensors on one device")
        self.index = places.pop() if places else None
        dims = {w.numel() for w in (q_weight, k_weight) if w is not None}
        _need(len(dims) < 2, "NormRope: weights of one length")
        self.dim = dims.pop() if dims else None
        self.desc = qg_norm_rope(None if q_weight is None else q_weight.data_ptr(),
                                 None if k_weight is None else k_weight.data_ptr(), eps, weight_offset,
                                 None if cos_sin is None else cos_sin.data_ptr(),
                                 0 if cos_sin is None else cos_sin.shape[0],
                                 0 if cos_sin is None else cos_sin.shape[1], 1 if interleaved else 0)


def _refuse(cache, batch, what):
    """What the descriptors do not tell: the width of the page table, and where the tensors are."""
    if batch.max_len > batch.width * cache.page_tokens:
        raise QGError(1, f"{what}: max_len {batch.max_len} takes more than the {batch.width} pages a sequence of the table")
    raise QGError(1, f"{what}: cache, batch and workspace on one CUDA device")


def _heads(t, n, heads, cache, what):
    """(pointer, token stride, head stride) of bf16 [n, heads, head_dim]; n or heads None: any."""
    s, st = t.shape, t.stride()
    if (t.dtype is not cache.bf16 or len(s) != 3 or s[2] != cache.head_dim or st[2] != 1
            or (n is not None and s[0] != n) or (heads is not None and s[1] != heads) or t.get_device() != cache.index):
        raise QGError(1, f"{what}: bfloat16 [{'tokens' if n is None else n}, {'heads' if heads is None else heads}, "
                         f"{cache.head_dim}] with a contiguous last dimension on the cache's device")
    return t.data_ptr(), st[0], st[1]


def kv_append(cache: KVCache, batch: KVBatch, q, k, v, norm_rope: Optional[NormRope] = None, out=None,
              workspace: Optional[Workspace] = None):
    """Norm and rotate the new tokens' q and k (bf16 [n, heads, head_dim]), write k and v into the cache and
    return the queries (``qkv_append``).  q may be None: only the cache is written."""
    hkv = cache.n_kv_heads
    if (batch.max_len > batch.width * cache.page_tokens or batch.index != cache.index
            or (workspace is not None and workspace.index != cache.index)):
        _refuse(cache, batch, "kv_append")
    kp, ldk, hsk = _heads(k, None, hkv, cache, "kv_append: k")
    n = k.shape[0]
    vp, ldv, hsv = _heads(v, n, hkv, cache, "kv_append: v")
    qp = op = None
    hq = ldq = hsq = ldo = hso = 0
    if q is not None:
        qp, ldq, hsq = _heads(q, n, None, cache, "kv_append: q")
        hq = q.shape[1]
        if out is None:
            out = q.new_empty((n, hq, cache.head_dim))
        op, ldo, hso = _heads(out, n, hq, cache, "kv_append: out")
    nr = None
    if norm_rope is not None:
        nr = norm_rope.desc
        if norm_rope.dim is not None and norm_rope.dim != cache.head_dim:
            raise QGError(1, "kv_append: norm weights of head_dim elements")
        if norm_rope.index is not None and norm_rope.index != cache.index:
            raise QGError(1, "kv_append: norm weights and rotation table on the cache's device")
    if workspace is None:
        workspace = Workspace(qkv_append_workspace_size(), k.device)
    st = (_lib or lib()).qkv_append(cache.desc, batch.desc, nr, n, hq, qp, ldq, hsq, kp, ldk, hsk, vp, ldv, hsv, op, ldo, hso,
                                    workspace.ptr, workspace.nbytes, cache.raw_stream(cache.index))
    if st:
        raise QGError(st, "qkv_append")
    return out


def attention_workspace_size(cache: KVCache, batch: KVBatch, n_tokens: int, n_q_heads: int) -> int:
    """Workspace bytes of ``attention`` for these sizes."""
    return qattn_workspace_size(cache.desc, batch.desc, n_tokens, n_q_heads)


def attention(cache: KVCache, batch: KVBatch, q, scale: Optional[float] = None, window: int = 0, out=None,
              workspace: Optional[Workspace] = None):
    """Causal attention of the new tokens q (bf16 [n, heads, head_dim]) over the cache (``qattn``);
    scale is 1/sqrt(head_dim) unless given, window 0 means none."""
    if (batch.max_len > batch.width * cache.page_tokens or batch.index != cache.index
            or (workspace is not None and workspace.index != cache.index)):
        _refuse(cache, batch, "attention")
    qp, ldq, hsq = _heads(q, None, None, cache, "attention: q")
    n, hq, d = q.shape
    if out is None:
        out = q.new_empty((n, hq, d))
    op, ldo, hso = _heads(out, n, hq, cache, "attention: out")
    if workspace is None:
        workspace = Workspace(attention_workspace_size(cache, batch, n, hq), q.device)
    st = (_lib or lib()).qattn(cache.desc, batch.desc, n, hq, qp, ldq, hsq, d ** -0.5 if scale is None else scale, window,
                               op, ldo, hso, workspace.ptr, workspace.nbytes, cache.raw_stream(cache.index))
    if st:
        raise QGError(st, "qattn")
    return out
