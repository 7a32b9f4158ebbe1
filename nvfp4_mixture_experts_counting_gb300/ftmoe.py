"""ctypes binding of libftmoe.so (argument marshalling only).

The functions carry the C names of ``include/ftmoe.h``.  Torch supplies device
memory and streams; every step of the layer runs in the library's CUDA
kernels.  If the library is missing or fails to load, every call raises:
there is no fallback path.

``Layer`` is a small convenience wrapper that owns one handle.
"""

from __future__ import annotations

import ctypes as C
import os
import struct
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libftmoe.so")

ABI_VERSION = 3
OUT_BF16, OUT_FP32, OUT_ACCUMULATE, ACT_BF16 = 0, 1, 0x100, 0x200

STATUS = {
    0: "OK", -1: "INVALID_ARG", -2: "ALIGNMENT", -3: "NOT_LOADED", -4: "SLICE_OUT_OF_RANGE",
    -5: "OOM", -6: "CUDA", -7: "TIMEOUT", -8: "FAULT_INJECTED", -9: "DEVICE", -10: "DEVICE_CHECK",
    -11: "TOO_LARGE",
}


class FtmoeError(RuntimeError):
    def __init__(self, code: int, where: str, detail: str = ""):
        self.code = code
        self.name = STATUS.get(code, str(code))
        super().__init__(f"{where}: {self.name} ({code}) {detail}".rstrip())


class Config(C.Structure):
    _fields_ = [("abi_version", C.c_int32), ("H", C.c_int32), ("I", C.c_int32), ("E", C.c_int32),
                ("top_k", C.c_int32), ("I_shared", C.c_int32), ("num_layers", C.c_int32),
                ("max_tokens", C.c_int32), ("norm_topk_prob", C.c_int32),
                ("has_router_bias", C.c_int32), ("hbm_slot_bytes", C.c_int64)]


class BankDesc(C.Structure):
    _fields_ = [("router_w", C.c_void_p), ("router_bias", C.c_void_p), ("gu_codes", C.c_void_p),
                ("gu_scales", C.c_void_p), ("gu_global", C.c_void_p), ("dn_codes", C.c_void_p),
                ("dn_scales", C.c_void_p), ("dn_global", C.c_void_p), ("sh_gate_up", C.c_void_p),
                ("sh_down", C.c_void_p), ("sh_gate", C.c_void_p), ("on_device", C.c_int32)]


class Aux(C.Structure):
    _fields_ = [("topk_idx", C.c_void_p), ("topk_w", C.c_void_p), ("offsets", C.c_void_p),
                ("perm", C.c_void_p), ("inv", C.c_void_p), ("logits", C.c_void_p),
                ("h_codes", C.c_void_p), ("h_scales", C.c_void_p)]


class Stats(C.Structure):
    _fields_ = [("touched_experts", C.c_int32), ("resident_slots", C.c_int32),
                ("touched_bytes", C.c_int64), ("hits", C.c_int64), ("misses", C.c_int64),
                ("h2d_bytes", C.c_int64), ("residency", C.c_double), ("device_status", C.c_int32),
                ("reranked_tokens", C.c_int64), ("touched_total", C.c_int64)]


class KernelTime(C.Structure):
    _fields_ = [("name", C.c_char * 48), ("launches", C.c_int64), ("total_ms", C.c_double)]


class PolicyArgs(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("dtype", C.c_int32), ("id_bytes", C.c_int32), ("N", C.c_int64),
                ("V", C.c_int64), ("ld", C.c_int64), ("targets", C.c_void_p), ("old_logp", C.c_void_p),
                ("ref_logp", C.c_void_p), ("advantage", C.c_void_p), ("weight", C.c_void_p),
                ("temperature", C.c_float), ("clip_low", C.c_float), ("clip_high", C.c_float),
                ("kl_coef", C.c_float), ("grad_scale", C.c_float), ("loss", C.c_void_p), ("row_loss", C.c_void_p),
                ("logp", C.c_void_p), ("dlogits", C.c_void_p), ("ld_d", C.c_int64)]


class AdamwTensor(C.Structure):
    _fields_ = [("p", C.c_void_p), ("g", C.c_void_p), ("master", C.c_void_p), ("m", C.c_void_p), ("v", C.c_void_p),
                ("m_scale", C.c_void_p), ("v_scale", C.c_void_p), ("n", C.c_int64), ("weight_decay", C.c_float),
                ("p_dtype", C.c_int32), ("g_dtype", C.c_int32), ("state_bits", C.c_int32)]


class AdamwParams(C.Structure):
    _fields_ = [("lr", C.c_double), ("beta1", C.c_double), ("beta2", C.c_double), ("eps", C.c_double),
                ("step", C.c_int64), ("grad_scale", C.c_void_p)]


class RouteArgs(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("dtype", C.c_int32), ("T", C.c_int32), ("E", C.c_int32), ("ld", C.c_int64),
                ("score", C.c_int32), ("top_k", C.c_int32), ("norm_topk_prob", C.c_int32), ("scale", C.c_float),
                ("bias", C.c_void_p), ("n_groups", C.c_int32), ("top_groups", C.c_int32), ("group_best", C.c_int32),
                ("topk_idx", C.c_void_p), ("topk_w", C.c_void_p)]


class Fp8MatmulArgs(C.Structure):
    _fields_ = [("a", C.c_void_p), ("a_scale", C.c_void_p), ("w", C.c_void_p), ("w_scale", C.c_void_p),
                ("offsets", C.c_void_p), ("M", C.c_int64), ("E", C.c_int32), ("N", C.c_int32), ("K", C.c_int32),
                ("transpose", C.c_int32), ("swiglu", C.c_int32), ("out_dtype", C.c_int32), ("out", C.c_void_p),
                ("out_scale", C.c_void_p)]


_lib = None

#: every symbol the header declares, with its argument and result types
SIGNATURES = {
    "ftmoe_create": ([C.POINTER(Config), C.c_int, C.POINTER(C.c_void_p)], C.c_int),
    "ftmoe_load_bank": ([C.c_void_p, C.c_int, C.POINTER(BankDesc), C.c_int, C.c_int, C.c_void_p], C.c_int),
    "ftmoe_forward": ([C.c_void_p, C.c_int, C.c_void_p, C.c_int, C.c_void_p, C.c_int, C.c_int, C.c_int,
                       C.POINTER(Aux), C.c_void_p], C.c_int),
    "ftmoe_forward_stack": ([C.c_void_p, C.c_void_p, C.c_int, C.c_void_p, C.c_void_p], C.c_int),
    "ftmoe_rms_renorm": ([C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_void_p], C.c_int),
    "ftmoe_destroy": ([C.c_void_p], C.c_int),
    "ftmoe_error_string": ([C.c_int], C.c_char_p),
    "ftmoe_last_cuda_error": ([], C.c_char_p),
    "ftmoe_get_stats": ([C.c_void_p, C.c_int, C.POINTER(Stats)], C.c_int),
    "ftmoe_check_status": ([C.c_void_p, C.c_void_p], C.c_int),
    "ftmoe_profile_enable": ([C.c_void_p, C.c_int], C.c_int),
    "ftmoe_profile_read": ([C.c_void_p, C.POINTER(KernelTime), C.c_int, C.POINTER(C.c_int)], C.c_int),
    "ftmoe_route_static": ([C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int,
                            C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p], C.c_int),
    "ftmoe_route_static_status": ([C.c_void_p], C.c_int),
    "ftmoe_forward_experts": ([C.c_void_p, C.c_int, C.c_void_p, C.c_int, C.c_void_p, C.c_int, C.c_void_p,
                               C.c_int, C.c_int, C.POINTER(Aux), C.c_void_p], C.c_int),
    "ftmoe_reduce_partials": ([C.c_void_p, C.c_int, C.c_int64, C.c_void_p, C.c_int, C.c_void_p], C.c_int),
    "ftmoe_test_withhold_stage": ([C.c_void_p, C.c_int, C.c_int64], C.c_int),
    "ftmoe_slice_format": ([C.c_int, C.c_int, C.c_int, C.c_int, C.c_int, C.c_int, C.c_int,
                            C.POINTER(C.c_void_p), C.POINTER(C.c_void_p), C.c_void_p], C.c_int),
    "ftmoe_quantize_weights": ([C.c_void_p, C.c_int64, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p,
                                C.c_void_p], C.c_int),
    "ftmoe_quantize_activations": ([C.c_void_p, C.c_int64, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p],
                                   C.c_int),
    "ftmoe_dispatch": ([C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_void_p,
                        C.c_void_p, C.c_void_p, C.c_void_p], C.c_int),
    "ftmoe_combine": ([C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p,
                       C.c_void_p], C.c_int),
    "ftmoe_combine_backward": ([C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p,
                                C.c_void_p, C.c_void_p, C.c_void_p], C.c_int),
    "ftmoe_route_backward": ([C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int,
                              C.c_void_p, C.c_void_p], C.c_int),
    "ftmoe_embed": ([C.c_void_p, C.c_int, C.c_int64, C.c_int, C.c_void_p, C.c_int, C.c_int64, C.c_float, C.c_void_p,
                     C.c_void_p], C.c_int),
    "ftmoe_embed_workspace": ([C.c_int64, C.c_int], C.c_int64),
    "ftmoe_embed_backward": ([C.c_void_p, C.c_int, C.c_void_p, C.c_int, C.c_int64, C.c_int64, C.c_int, C.c_float,
                              C.c_int64, C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_int64, C.c_void_p], C.c_int),
    "ftmoe_policy_loss": ([C.POINTER(PolicyArgs), C.c_void_p], C.c_int),
    "ftmoe_test_withhold_policy": ([C.c_int, C.c_int64], C.c_int),
    "ftmoe_adamw": ([C.POINTER(AdamwTensor), C.c_int, C.POINTER(AdamwParams), C.c_void_p], C.c_int),
    "ftmoe_route_topk": ([C.POINTER(RouteArgs), C.c_void_p], C.c_int),
    "ftmoe_route_topk_backward": ([C.POINTER(RouteArgs), C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p], C.c_int),
    "ftmoe_fp8_quantize": ([C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_int, C.c_void_p, C.c_void_p,
                            C.c_void_p, C.c_void_p], C.c_int),
    "ftmoe_fp8_quantize_weights": ([C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p,
                                    C.c_void_p], C.c_int),
    "ftmoe_fp8_matmul": ([C.POINTER(Fp8MatmulArgs), C.c_void_p], C.c_int),
    "ftmoe_test_withhold_matmul": ([C.c_int, C.c_int64], C.c_int),
    "ftmoe_swiglu": ([C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p], C.c_int),
    "ftmoe_swiglu_backward": ([C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p,
                               C.c_void_p], C.c_int),
    "ftmoe_ops_status": ([C.c_void_p], C.c_int),
}


def lib():
    """The loaded libftmoe.so (raises if it is missing: no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libftmoe.so is not built ({LIB_PATH}); run build.build() first")
        L = C.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def _check(rc: int, where: str):
    if rc != 0:
        detail = ""
        if rc == -6:
            detail = lib().ftmoe_last_cuda_error().decode()
        raise FtmoeError(rc, where, detail)


def _ptr(t) -> Optional[int]:
    """Raw address of a torch tensor or numpy array (None stays None)."""
    if t is None:
        return None
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    return t.ctypes.data


_raw_stream = None  # torch's handle of a device's current stream, once torch is there


def _stream(stream) -> Optional[int]:
    if stream is None:
        global _raw_stream
        if _raw_stream is None:
            import torch
            _raw_stream = torch._C._cuda_getCurrentRawStream
        # the handle alone (a Stream object costs some 3 us a call), of the current device (-1)
        return _raw_stream(-1)
    if hasattr(stream, "cuda_stream"):
        return stream.cuda_stream
    return int(stream)


# ----------------------------------------------------------------- C-named calls

def ftmoe_create(config: Config, device: int = 0) -> int:
    h = C.c_void_p()
    _check(lib().ftmoe_create(C.byref(config), device, C.byref(h)), "ftmoe_create")
    return h.value


def ftmoe_load_bank(h: int, layer: int, desc: BankDesc, i0: int, I_loc: int, stream=None):
    _check(lib().ftmoe_load_bank(h, layer, C.byref(desc), i0, I_loc, _stream(stream)), "ftmoe_load_bank")


def ftmoe_forward(h: int, layer: int, x, T: int, out, out_flags: int, i0: int, I_loc: int,
                  aux: Optional[Aux] = None, stream=None):
    _check(lib().ftmoe_forward(h, layer, _ptr(x), T, _ptr(out), out_flags, i0, I_loc,
                               C.byref(aux) if aux is not None else None, _stream(stream)),
           "ftmoe_forward")


def ftmoe_forward_stack(h: int, x, T: int, out, stream=None):
    _check(lib().ftmoe_forward_stack(h, _ptr(x), T, _ptr(out), _stream(stream)), "ftmoe_forward_stack")


def ftmoe_rms_renorm(y, x, T: int, H: int, stream=None):
    _check(lib().ftmoe_rms_renorm(_ptr(y), _ptr(x), T, H, _stream(stream)), "ftmoe_rms_renorm")


def ftmoe_destroy(h: int):
    _check(lib().ftmoe_destroy(h), "ftmoe_destroy")


def ftmoe_error_string(code: int) -> str:
    return lib().ftmoe_error_string(code).decode()


def ftmoe_last_cuda_error() -> str:
    return lib().ftmoe_last_cuda_error().decode()


def ftmoe_get_stats(h: int, layer: int) -> Stats:
    s = Stats()
    _check(lib().ftmoe_get_stats(h, layer, C.byref(s)), "ftmoe_get_stats")
    return s


def ftmoe_check_status(h: int, stream=None) -> int:
    return lib().ftmoe_check_status(h, _stream(stream))


def ftmoe_profile_enable(h: int, enable: bool):
    _check(lib().ftmoe_profile_enable(h, int(enable)), "ftmoe_profile_enable")


def ftmoe_profile_read(h: int, max_entries: int = 64) -> dict:
    """{kernel name: (launches, total ms)} recorded since the last read."""
    arr = (KernelTime * max_entries)()
    n = C.c_int()
    _check(lib().ftmoe_profile_read(h, arr, max_entries, C.byref(n)), "ftmoe_profile_read")
    return {arr[i].name.decode(): (arr[i].launches, arr[i].total_ms) for i in range(n.value)}


def ftmoe_route_static(x, T: int, H: int, router_w, router_bias, E: int, top_k: int, norm_topk_prob: bool,
                       topk_idx, topk_w, offsets, perm, inv, stream=None):
    """Routing with no device allocation (scratch in a fixed device array)."""
    _check(lib().ftmoe_route_static(_ptr(x), T, H, _ptr(router_w), _ptr(router_bias), E, top_k,
                                    int(norm_topk_prob), _ptr(topk_idx), _ptr(topk_w), _ptr(offsets),
                                    _ptr(perm), _ptr(inv), _stream(stream)), "ftmoe_route_static")


def ftmoe_forward_experts(h: int, layer: int, x, T: int, out, out_flags: int, expert_mask,
                          shared_i0: int = 0, shared_I_loc: int = 0, aux: Optional[Aux] = None, stream=None):
    """One expert-parallel rank's share: the routed slots of the experts whose
    mask byte (host numpy uint8 [E]) is set, plus the shared expert's window
    [shared_i0, shared_i0 + shared_I_loc) (none when shared_I_loc is 0)."""
    import numpy as np
    m = np.ascontiguousarray(expert_mask, dtype=np.uint8)
    _check(lib().ftmoe_forward_experts(h, layer, _ptr(x), T, _ptr(out), out_flags, m.ctypes.data, shared_i0,
                                       shared_I_loc, C.byref(aux) if aux is not None else None, _stream(stream)),
           "ftmoe_forward_experts")


def ftmoe_reduce_partials(parts, n_parts: int, n: int, out, out_flags: int = OUT_BF16, stream=None):
    """out <- sum over ranks of fp32 partials [n_parts][n], in rank order."""
    _check(lib().ftmoe_reduce_partials(_ptr(parts), n_parts, n, _ptr(out), out_flags, _stream(stream)),
           "ftmoe_reduce_partials")


def ftmoe_route_static_status(stream=None) -> int:
    """Status of the latest ftmoe_route_static call (0, DEVICE_CHECK or TIMEOUT)."""
    return lib().ftmoe_route_static_status(_stream(stream))


def ftmoe_test_withhold_stage(h: int, enable: bool, wait_limit_ns: int = 0):
    _check(lib().ftmoe_test_withhold_stage(h, int(enable), wait_limit_ns), "ftmoe_test_withhold_stage")


FMT = {"nvfp4": 0, "fp8_block": 1, "q4_0": 2, "mxfp4": 3}
MAT_GATE_UP, MAT_DOWN = 0, 1


def ftmoe_slice_format(fmt: str, matrix: int, E: int, H: int, I: int, i0: int, I_loc: int, src, dst, stream=None):
    """Slice E experts' matrix in bank format `fmt` to a window; src / dst
    are lists of device tensors (the format's arrays, in the header's order)."""
    S = (C.c_void_p * 3)(*[_ptr(t) for t in src] + [None] * (3 - len(src)))
    D = (C.c_void_p * 3)(*[_ptr(t) for t in dst] + [None] * (3 - len(dst)))
    _check(lib().ftmoe_slice_format(FMT[fmt], matrix, E, H, I, i0, I_loc, S, D, _stream(stream)),
           "ftmoe_slice_format")


def ftmoe_quantize_weights(w, rows: int, K: int, codes, scales, globals_, stream=None):
    _check(lib().ftmoe_quantize_weights(_ptr(w), rows, K, _ptr(codes), _ptr(scales), _ptr(globals_),
                                        _stream(stream)), "ftmoe_quantize_weights")


def ftmoe_quantize_activations(a, rows: int, K: int, codes, scales, stream=None):
    _check(lib().ftmoe_quantize_activations(_ptr(a), rows, K, _ptr(codes), _ptr(scales), _stream(stream)),
           "ftmoe_quantize_activations")


# ----------------------------------------------------------------- training operators

BF16, FP32, FP16 = 0, 1, 2
_INT32, _INT64 = 3, 4


class _Codes(dict):
    """torch.dtype -> code, filled once torch is there; -1 for other types."""

    fp32 = int32 = codes = None

    def __missing__(self, dtype):
        import torch
        self.fp32 = torch.float32
        self.int32 = torch.int32
        self.codes = (torch.uint8, torch.float8_e4m3fn)
        self.update({torch.bfloat16: BF16, torch.float32: FP32, torch.float16: FP16, torch.int32: _INT32,
                     torch.int64: _INT64})
        return self.setdefault(dtype, -1)


_CODES = _Codes()


def _dtype(t) -> int:
    code = _CODES[t.dtype]
    if code not in (BF16, FP32, FP16):
        raise TypeError(f"bf16, fp32 or fp16 expected, got {t.dtype}")
    return code


def _array(t, code: int, n: int):
    """Address of a contiguous tensor of n values or more of the type that `code` names (None stays None)."""
    if t is None:
        return None
    if _CODES[t.dtype] != code:
        raise TypeError(f"{('bf16', 'fp32', 'fp16', 'int32', 'int64')[code]} expected, got {t.dtype}")
    if t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{n} or more contiguous values expected, got {t.numel()} with strides {t.stride()}")
    return t.data_ptr()


def _dense(t):
    """Address of a contiguous tensor (None stays None): the C calls take no strides."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("contiguous tensors expected")
    return t.data_ptr()


def _floats(t, n: int, fp32):
    """Address of exactly n contiguous fp32 values (None stays None); `fp32` is torch's name of the type."""
    if t is None:
        return None
    if t.nbytes != 4 * n or t.dtype is not fp32 or not t.is_contiguous():
        raise ValueError(f"{n} contiguous fp32 values expected, got {t.numel()} of {t.dtype}")
    return t.data_ptr()


def ftmoe_dispatch(x, T: int, H: int, topk_idx, top_k: int, E: int, offsets, perm, inv, xs, stream=None):
    """Rows of x sorted by expert into xs, and the sort's tables (x and xs None: the tables alone)."""
    P, dtype = T * top_k, BF16 if x is None else _dtype(x)
    # A decode step's call takes some 5 us on the host: one look at all tensors (6 calls of _array take 0.3 us
    # more), and one by one only where something is absent or wrong.
    if (x is None or xs is None or topk_idx is None or offsets is None or perm is None or inv is None
            or _CODES[inv.dtype] != _INT32 or not topk_idx.dtype is offsets.dtype is perm.dtype is inv.dtype
            or xs.dtype is not x.dtype or x.numel() < T * H or xs.numel() < P * H or topk_idx.numel() < P
            or perm.numel() < P or inv.numel() < P or offsets.numel() <= E
            or not (x.is_contiguous() and xs.is_contiguous() and topk_idx.is_contiguous() and perm.is_contiguous()
                    and inv.is_contiguous() and offsets.is_contiguous())):
        rc = lib().ftmoe_dispatch(_array(x, dtype, T * H), dtype, T, H, _array(topk_idx, _INT32, P), top_k, E,
                                  _array(offsets, _INT32, E + 1), _array(perm, _INT32, P), _array(inv, _INT32, P),
                                  _array(xs, dtype, P * H), _stream(stream))
    else:
        rc = lib().ftmoe_dispatch(x.data_ptr(), dtype, T, H, topk_idx.data_ptr(), top_k, E, offsets.data_ptr(),
                                  perm.data_ptr(), inv.data_ptr(), xs.data_ptr(), _stream(stream))
    _check(rc, "ftmoe_dispatch")


def ftmoe_combine(ys, T: int, H: int, top_k: int, inv, w, out, stream=None):
    """out[t] = sum_j w[t, j] ys[inv[t, j]]; w None: weights of one (the gradient of ftmoe_dispatch)."""
    P, dtype = T * top_k, _dtype(ys)
    _check(lib().ftmoe_combine(_array(ys, dtype, P * H), dtype, T, H, top_k, _array(inv, _INT32, P),
                               _array(w, FP32, P), _array(out, dtype, T * H), _stream(stream)), "ftmoe_combine")


def ftmoe_combine_backward(dout, ys, T: int, H: int, top_k: int, inv, w, dys, dw, stream=None):
    P, dtype = T * top_k, _dtype(dout)
    _check(lib().ftmoe_combine_backward(_array(dout, dtype, T * H), _array(ys, dtype, P * H), dtype, T, H, top_k,
                                        _array(inv, _INT32, P), _array(w, FP32, P), _array(dys, dtype, P * H),
                                        _array(dw, FP32, P), _stream(stream)), "ftmoe_combine_backward")


def ftmoe_route_backward(logits, topk_idx, topk_w, dw, T: int, E: int, top_k: int, norm_topk_prob: bool, dlogits,
                         stream=None):
    P = T * top_k
    _check(lib().ftmoe_route_backward(_array(logits, FP32, T * E), _array(topk_idx, _INT32, P),
                                      _array(topk_w, FP32, P), _array(dw, FP32, P), T, E, top_k, int(norm_topk_prob),
                                      _array(dlogits, FP32, T * E), _stream(stream)), "ftmoe_route_backward")


def _indices(t, n: int):
    """Address and bytes of each of a contiguous tensor's n or more int32 or int64 values."""
    if t is None:
        return None, 8
    code = _CODES[t.dtype]
    if code != _INT32 and code != _INT64:
        raise TypeError(f"int32 or int64 expected, got {t.dtype}")
    if t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{n} or more contiguous values expected, got {t.numel()} with strides {t.stride()}")
    return t.data_ptr(), 4 if code == _INT32 else 8


def ftmoe_embed(table, V: int, H: int, ids, N: int, scale: float, out, stream=None):
    dtype, (at, id_bytes) = _dtype(table), _indices(ids, N)
    _check(lib().ftmoe_embed(_array(table, dtype, V * H), dtype, V, H, at, id_bytes, N, scale,
                             _array(out, dtype, N * H), _stream(stream)), "ftmoe_embed")


def ftmoe_embed_workspace(N: int, H: int) -> int:
    """Bytes of workspace for ftmoe_embed_backward."""
    n = lib().ftmoe_embed_workspace(N, H)
    _check(min(n, 0), "ftmoe_embed_workspace")
    return n


def ftmoe_embed_backward(dout, ids, N: int, V: int, H: int, scale: float, padding_id: int, dtable, accumulate: bool,
                         workspace, stream=None):
    dtype, table_dtype, (at, id_bytes) = _dtype(dout), _dtype(dtable), _indices(ids, N)
    _check(lib().ftmoe_embed_backward(_array(dout, dtype, N * H), dtype, at, id_bytes, N, V, H, scale, padding_id,
                                      _array(dtable, table_dtype, V * H), table_dtype, int(accumulate),
                                      _dense(workspace),
                                      0 if workspace is None else workspace.numel() * workspace.element_size(),
                                      _stream(stream)), "ftmoe_embed_backward")


def policy_args(logits, targets, old_logp, ref_logp, advantage, weight, loss, row_loss, logp=None, dlogits=None,
                temperature: float = 1.0, clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0,
                grad_scale: float = 1.0) -> PolicyArgs:
    """Arguments of ftmoe_policy_loss, kept with references to the tensors; logits and dlogits [N, V] may have any
    row stride (last dimension dense)."""
    shape, dtype = logits.shape, _dtype(logits)
    N, V = shape
    ld, step = logits.stride()
    at, ld_d, step_d = None, 0, 1
    if dlogits is not None:
        if dlogits.dtype is not logits.dtype or dlogits.shape != shape:
            raise TypeError("dlogits has the shape and type of logits")
        at, (ld_d, step_d) = dlogits.data_ptr(), dlogits.stride()
    if V > 1 and (step != 1 or step_d != 1):
        raise ValueError("logits and dlogits need a dense last dimension")
    if N <= 1:  # a single row's stride says nothing
        ld = ld_d = V
    f32, (ids, id_bytes) = _CODES.fp32, _indices(targets, N)
    args = PolicyArgs(logits.data_ptr(), dtype, id_bytes, N, V, ld, ids, _floats(old_logp, N, f32),
                      _floats(ref_logp, N, f32), _floats(advantage, N, f32), _floats(weight, N, f32), temperature,
                      clip_low, clip_high, kl_coef, grad_scale, _floats(loss, 1, f32), _floats(row_loss, N, f32),
                      _floats(logp, N, f32), at, ld_d)
    args.tensors = (logits, targets, old_logp, ref_logp, advantage, weight, loss, row_loss, logp, dlogits)
    return args


def ftmoe_policy_loss(args: PolicyArgs, stream=None):
    _check(lib().ftmoe_policy_loss(C.byref(args), _stream(stream)), "ftmoe_policy_loss")


def ftmoe_test_withhold_policy(enable: bool, wait_limit_ns: int = 0):
    _check(lib().ftmoe_test_withhold_policy(int(enable), wait_limit_ns), "ftmoe_test_withhold_policy")


class AdamwList:
    """The tensors of ftmoe_adamw: made once, kept with references to them."""

    def __init__(self, tensors):
        self.tensors = [dict(t) for t in tensors]  # the entries hold addresses, whatever becomes of the caller's dicts
        entries = []
        for t in self.tensors:
            get = t.get
            p, g, m, v = t["p"], t["g"], t["m"], t["v"]
            n = p.numel()
            if min(g.numel(), m.numel(), v.numel()) < n or m.dtype is not v.dtype:
                raise ValueError("g, m and v have p's values, and m and v one type")
            if m.element_size() != 1 and _CODES[m.dtype] != FP32:
                raise TypeError(f"m and v are fp32 or codes of one byte, got {m.dtype}")
            blocks = (n + 255) // 256
            entries.append((_dense(p), _dense(g), _array(get("master"), FP32, n), _dense(m), _dense(v),
                            _array(get("m_scale"), FP32, blocks), _array(get("v_scale"), FP32, blocks), n,
                            get("weight_decay", 0.0), _dtype(p), _dtype(g), 8 * m.element_size()))
        self.array = (AdamwTensor * len(entries))(*entries)


def adamw_list(tensors) -> AdamwList:
    """A list of dicts: p, g, m, v, and where they apply master, m_scale, v_scale, weight_decay."""
    return AdamwList(list(tensors))


def ftmoe_adamw(tensors: AdamwList, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                step: int = 1, grad_scale=None, stream=None):
    hp = AdamwParams(lr, beta1, beta2, eps, step, _array(grad_scale, FP32, 1))
    _check(lib().ftmoe_adamw(tensors.array, len(tensors.array), C.byref(hp), _stream(stream)), "ftmoe_adamw")


# ----------------------------------------------------------------- the layer on 8-bit codes

SCORES = {"softmax": 0, "sigmoid": 1}
# The fields of RouteArgs and Fp8MatmulArgs, to be filled at once (a third of the time that their constructors take).
_ROUTE, _MATMUL = struct.Struct("@PiiiqiiifPiiiPP"), struct.Struct("@PPPPPqiiiiiiPP")


def _fill():
    """The types of codes, once torch is there."""
    _CODES[None]
    return _CODES.codes


def _codes8(t, n: int):
    """Address of a contiguous tensor of n E4M3 codes or more (float8_e4m3fn, or their bytes)."""
    if t is None:
        return None
    if t.dtype not in (_CODES.codes or _fill()):
        raise TypeError(f"float8_e4m3fn or uint8 expected, got {t.dtype}")
    if t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{n} or more contiguous codes expected, got {t.numel()} with strides {t.stride()}")
    return t.data_ptr()


def _rows(t):
    """(rows, columns, values between rows) of a matrix whose rows are dense."""
    n, width = t.shape
    ld, step = t.stride()
    if width > 1 and step != 1:
        raise ValueError("rows need a dense last dimension")
    return n, width, width if n <= 1 else ld  # a single row's stride says nothing


# The calls below take some 4 us on the host, as long as their smallest kernels: their tensors are looked at together,
# and one by one (_array and the like, which say what is wrong) only where something is absent or wrong.

def route_args(logits, topk_idx, topk_w, score: str = "softmax", norm_topk_prob: bool = True, scale: float = 1.0,
               bias=None, n_groups: int = 1, top_groups: int = 1, group_best: int = 1) -> RouteArgs:
    """Arguments of ftmoe_route_topk and its gradient, kept with references to the tensors; logits [T, E] may have
    any row stride, top_k is the width of topk_idx [T, top_k]."""
    T, E, ld = _rows(logits)
    shape = topk_idx.shape
    if len(shape) != 2 or shape[0] != T or topk_w.shape != shape:
        raise ValueError("topk_idx and topk_w have a row for each of the logits' and one shape")
    k, dtype = shape[1], _dtype(logits)
    if (topk_idx.dtype is _CODES.int32 and topk_w.dtype is _CODES.fp32 and topk_idx.is_contiguous()
            and topk_w.is_contiguous()):
        idx, w = topk_idx.data_ptr(), topk_w.data_ptr()
    else:
        idx, w = _array(topk_idx, _INT32, T * k), _array(topk_w, FP32, T * k)
    args = RouteArgs()
    _ROUTE.pack_into(args, 0, logits.data_ptr(), dtype, T, E, ld, SCORES[score], k, norm_topk_prob, scale,
                     _array(bias, FP32, E) or 0, n_groups, top_groups, group_best, idx, w)
    args.tensors = (logits, topk_idx, topk_w, bias)
    return args


def ftmoe_route_topk(args: RouteArgs, stream=None):
    _check(lib().ftmoe_route_topk(C.byref(args), _stream(stream)), "ftmoe_route_topk")


def ftmoe_route_topk_backward(args: RouteArgs, dw, dlogits, stream=None):
    T, E, ld = _rows(dlogits)
    if T != args.T or E != args.E or _dtype(dlogits) != args.dtype:
        raise TypeError("dlogits has the shape and type of logits")
    _check(lib().ftmoe_route_topk_backward(C.byref(args), _array(dw, FP32, T * args.top_k), dlogits.data_ptr(), ld,
                                           _stream(stream)), "ftmoe_route_topk_backward")


def ftmoe_fp8_quantize(x, T: int, K: int, inv, top_k: int, codes, scales, used=None, stream=None):
    """E4M3 codes of x's rows with a scale for 128 values; with inv, in the rows that ftmoe_dispatch's table names."""
    dtype, rows, blocks = _dtype(x), T * top_k, (K + 127) // 128
    if (inv is not None and used is None and inv.dtype is _CODES.int32 and codes.dtype in _CODES.codes
            and scales.dtype is _CODES.fp32 and x.numel() >= T * K and inv.numel() >= rows
            and codes.numel() >= rows * K and scales.numel() >= blocks * rows and x.is_contiguous()
            and inv.is_contiguous() and codes.is_contiguous() and scales.is_contiguous()):
        rc = lib().ftmoe_fp8_quantize(x.data_ptr(), dtype, T, K, inv.data_ptr(), top_k, None, codes.data_ptr(),
                                      scales.data_ptr(), _stream(stream))
    else:
        rc = lib().ftmoe_fp8_quantize(_array(x, dtype, T * K), dtype, T, K, _array(inv, _INT32, rows), top_k,
                                      _array(used, _INT32, 1), _codes8(codes, rows * K),
                                      _array(scales, FP32, blocks * rows), _stream(stream))
    _check(rc, "ftmoe_fp8_quantize")


def ftmoe_fp8_quantize_weights(w, E: int, N: int, K: int, codes, scales, stream=None):
    dtype, blocks = _dtype(w), (N + 127) // 128 * ((K + 127) // 128)
    _check(lib().ftmoe_fp8_quantize_weights(_array(w, dtype, E * N * K), dtype, E, N, K, _codes8(codes, E * N * K),
                                            _array(scales, FP32, E * blocks), _stream(stream)),
           "ftmoe_fp8_quantize_weights")


def ftmoe_fp8_matmul(a, a_scale, w, w_scale, offsets, M: int, E: int, N: int, K: int, out, out_scale=None,
                     transpose: bool = False, swiglu: bool = False, stream=None):
    """Each expert's rows of codes times its matrix [N, K] (transpose: times its columns; swiglu: h as codes)."""
    width, out_width = (N, K) if transpose else (K, N // 2 if swiglu else N)
    nb, kb = (N + 127) // 128, (K + 127) // 128
    n_scales, n_out = (nb if transpose else kb) * M, M * out_width
    codes, fp32 = _CODES.codes or _fill(), _CODES.fp32
    dtype = 0 if swiglu else _dtype(out)
    if (offsets is not None and a.dtype in codes and w.dtype in codes and a_scale.dtype is fp32
            and w_scale.dtype is fp32 and offsets.dtype is _CODES.int32 and a.numel() >= M * width
            and a_scale.numel() >= n_scales and w.numel() >= E * N * K and w_scale.numel() >= E * nb * kb
            and offsets.numel() > E and out.numel() >= n_out and a.is_contiguous() and a_scale.is_contiguous()
            and w.is_contiguous() and w_scale.is_contiguous() and offsets.is_contiguous() and out.is_contiguous()
            and not swiglu):
        args = Fp8MatmulArgs()
        _MATMUL.pack_into(args, 0, a.data_ptr(), a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(),
                          offsets.data_ptr(), M, E, N, K, transpose, False, dtype, out.data_ptr(), 0)
    else:
        args = Fp8MatmulArgs(_codes8(a, M * width), _array(a_scale, FP32, n_scales), _codes8(w, E * N * K),
                             _array(w_scale, FP32, E * nb * kb), _array(offsets, _INT32, E + 1), M, E, N, K, transpose,
                             swiglu, dtype, _codes8(out, n_out) if swiglu else _array(out, dtype, n_out),
                             _array(out_scale, FP32, out_width // 128 * M) if swiglu else None)
    _check(lib().ftmoe_fp8_matmul(C.byref(args), _stream(stream)), "ftmoe_fp8_matmul")


def ftmoe_test_withhold_matmul(enable: bool, wait_limit_ns: int = 0):
    _check(lib().ftmoe_test_withhold_matmul(int(enable), wait_limit_ns), "ftmoe_test_withhold_matmul")


def _swiglu_out(out, scales, dtype: int, rows: int, width: int):
    if scales is None:
        return _array(out, dtype, rows * width), None
    return _codes8(out, rows * width), _array(scales, FP32, width // 128 * rows)


def ftmoe_swiglu(gu, rows: int, I: int, out, scales=None, used=None, stream=None):
    """out = SiLU(gate) * up, in gu's type or, with scales, as E4M3 codes."""
    dtype = _dtype(gu)
    _check(lib().ftmoe_swiglu(_array(gu, dtype, 2 * rows * I), dtype, rows, I, _array(used, _INT32, 1),
                              *_swiglu_out(out, scales, dtype, rows, I), _stream(stream)), "ftmoe_swiglu")


def ftmoe_swiglu_backward(dh, gu, rows: int, I: int, dgu, scales=None, used=None, stream=None):
    dtype = _dtype(gu)
    _check(lib().ftmoe_swiglu_backward(_array(dh, dtype, rows * I), _array(gu, dtype, 2 * rows * I), dtype, rows, I,
                                       _array(used, _INT32, 1), *_swiglu_out(dgu, scales, dtype, rows, 2 * I),
                                       _stream(stream)), "ftmoe_swiglu_backward")


def ftmoe_ops_status(stream=None) -> int:
    """Status of the training operators' checks and waits since the last call (0, DEVICE_CHECK or TIMEOUT)."""
    return lib().ftmoe_ops_status(_stream(stream))


# ----------------------------------------------------------------- convenience

def make_config(H, I, E, top_k, I_shared, num_layers=1, max_tokens=16, norm_topk_prob=True,
                has_router_bias=False, hbm_slot_bytes=0) -> Config:
    return Config(ABI_VERSION, H, I, E, top_k, I_shared, num_layers, max_tokens, int(norm_topk_prob),
                  int(has_router_bias), hbm_slot_bytes)


def bank_desc(router_w, router_bias, gu_codes, gu_scales, gu_global, dn_codes, dn_scales, dn_global,
              sh_gate_up, sh_down, sh_gate, on_device: bool) -> BankDesc:
    return BankDesc(_ptr(router_w), _ptr(router_bias), _ptr(gu_codes), _ptr(gu_scales), _ptr(gu_global),
                    _ptr(dn_codes), _ptr(dn_scales), _ptr(dn_global), _ptr(sh_gate_up), _ptr(sh_down),
                    _ptr(sh_gate), int(on_device))


class Layer:
    """Owns one ftmoe handle (all layers of one shape)."""

    def __init__(self, config: Config, device: int = 0):
        self.config = config
        self.handle = ftmoe_create(config, device)

    def close(self):
        if self.handle:
            ftmoe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def load_bank(self, layer: int, desc: BankDesc, i0: int = 0, I_loc: Optional[int] = None, stream=None):
        I_loc = self.config.I - i0 if I_loc is None else I_loc
        ftmoe_load_bank(self.handle, layer, desc, i0, I_loc, stream)

    def forward(self, layer: int, x, out, out_flags: int = OUT_BF16, i0: int = 0,
                I_loc: Optional[int] = None, aux: Optional[Aux] = None, stream=None):
        I_loc = self.config.I - i0 if I_loc is None else I_loc
        ftmoe_forward(self.handle, layer, x, x.shape[0], out, out_flags, i0, I_loc, aux, stream)
        return out

    def forward_stack(self, x, out, stream=None):
        ftmoe_forward_stack(self.handle, x, x.shape[0], out, stream)
        return out

    def stats(self, layer: int) -> Stats:
        return ftmoe_get_stats(self.handle, layer)

    def check_status(self, stream=None) -> int:
        return ftmoe_check_status(self.handle, stream)
