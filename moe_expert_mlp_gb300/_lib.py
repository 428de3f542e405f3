"""ctypes binding of libmoe (include/moe.h).

Argument marshalling only: every function here has the name of the C entry
point it calls, turns torch tensors into device pointers and the current
torch stream into a cudaStream_t, and raises on a non-zero status.  All
computation happens in the library's CUDA kernels.  There is no fallback:
if libmoe.so is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os
import sysconfig

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_DTYPE_BF16 = 1
MOE_DTYPE_MXFP8 = 2
MOE_DTYPE_NVFP4 = 3
MOE_DTYPE_FP32 = 4
MOE_MX_SCALES_ROWMAJOR = 0
MOE_MX_SCALES_MMA = 1
ACTS = {"swiglu": 0, "geglu": 1, "srelu": 2, "sreglu": 3}

EXPORTS = (
    "moe_fc1_padded_width", "moe_workspace_size", "moe_repack_fc1", "moe_unpack_fc1",
    "moe_route_permute", "moe_group_offsets", "moe_mlp_fwd", "moe_unpermute_combine",
    "moe_unpermute_combine_bwd", "moe_mlp_bwd", "moe_permute_bwd", "moe_route_bwd",
    "moe_read_device_status", "moe_status_string", "moe_fc1_glu_fwd", "moe_fc2_fwd",
    "moe_fc2_dgrad_dglu", "moe_fc2_wgrad", "moe_fc1_dgrad", "moe_fc1_wgrad", "moe_bias_grads",
    "moe_route_permute_noalloc", "moe_quantize_mx", "moe_selftest_wait_timeout",
    "moe_fc1_glu_fwd_unfused", "moe_fc2_dgrad_dglu_unfused", "moe_fc1_recompute_h",
    "moe_mx_scale_bytes", "moe_quantize_mx_bf16", "moe_quantize_act_mx",
    "moe_quantize_weights_mx", "moe_mlp_fwd_mx", "moe_mlp_bwd_mx", "moe_fc1_glu_fwd_mx",
    "moe_fc2_fwd_mx", "moe_fc2_dgrad_dglu_mx", "moe_fc2_wgrad_mx", "moe_fc1_dgrad_mx",
    "moe_fc1_wgrad_mx", "moe_route_permute_fused", "moe_nvfp4_scale_bytes", "moe_amax_nvfp4",
    "moe_quantize_nvfp4_bf16", "moe_quantize_act_nvfp4", "moe_quantize_weights_nvfp4",
    "moe_fc1_glu_fwd_nv", "moe_fc2_fwd_nv", "moe_fc2_dgrad_dglu_nv", "moe_fc2_wgrad_nv",
    "moe_fc1_dgrad_nv", "moe_fc1_wgrad_nv", "moe_mlp_fwd_nv", "moe_mlp_bwd_nv",
    "moe_fc1_recompute_h_mx", "moe_fc1_recompute_h_nv", "moe_fc1_glu_fwd_mx_unfused",
    "moe_fc2_dgrad_dglu_mx_unfused", "moe_fc2_dgrad_dglu_recompute",
    "moe_fc2_dgrad_dglu_recompute_mx", "moe_route_permute_mx", "moe_unpermute_combine_bwd_mx",
    "moe_transpose_weights_tf32", "moe_transpose_rows_f32", "moe_fc1_glu_fwd_tf32",
    "moe_fc2_fwd_tf32", "moe_fc2_dgrad_dglu_tf32", "moe_fc2_wgrad_tf32", "moe_fc1_dgrad_tf32",
    "moe_fc1_wgrad_tf32", "moe_selftest_grid_wait_timeout", "moe_block_norm_workspace_size",
    "moe_block_pre_norm_fwd", "moe_block_pre_norm_bwd", "moe_block_post_norm_fwd",
    "moe_block_post_norm_bwd", "moe_grad_norm_workspace_size", "moe_grad_norm", "moe_clip_grads",
)

NORMS = {None: 0, "none": 0, "rms": 1, "layer": 2}
GATES = {None: 0, "none": 0, "channel": 1, "token": 2, "full": 3}
GATE_ACTS = {None: 0, "none": 0, "sigmoid": 1, "tanh": 2}
GRAD_NORMS = {"l2": 0, "inf": 1}


class MoeError(RuntimeError):
    pass


class moe_mlp_desc_t(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
        ("d", ctypes.c_int32), ("F", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("act", ctypes.c_int32), ("alpha", ctypes.c_float), ("limit", ctypes.c_float),
        ("linear_offset", ctypes.c_float), ("out_scale", ctypes.c_float),
        ("has_b1", ctypes.c_int32), ("has_b2", ctypes.c_int32), ("align", ctypes.c_int32),
        ("sm_margin", ctypes.c_int32), ("capacity", ctypes.c_int32),
        ("recompute_h", ctypes.c_int32),
    ]


class moe_mx_out_t(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("qt", ctypes.c_void_p),
                ("scale_t", ctypes.c_void_p), ("amax", ctypes.c_void_p),
                ("layout", ctypes.c_int32)]


class moe_mx_weights_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("w1", "w1_s", "w1t", "w1t_s", "w2", "w2_s", "w2t", "w2t_s")]


class moe_nv_weights_t(ctypes.Structure):
    _fields_ = [("q", moe_mx_weights_t), ("amax", ctypes.c_void_p)]


class moe_rows_t(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("ld", ctypes.c_int64)]


class moe_block_norm_desc_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "d", "dtype", "res_dtype", "param_dtype", "pre_norm", "post_norm", "gate",
                 "gate_act")]
    _fields_ += [(n, ctypes.c_float) for n in
                 ("pre_eps", "post_eps", "pre_offset", "post_offset", "res_scale",
                  "branch_scale")]


class moe_block_params_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("pre_w", "pre_b", "post_w", "post_b")]
    _fields_ += [("gate", moe_rows_t)]


class moe_routed_rows_t(ctypes.Structure):
    _fields_ = [("row_of", ctypes.c_void_p), ("topk_w", ctypes.c_void_p), ("k", ctypes.c_int32),
                ("capacity", ctypes.c_int32), ("y_out", moe_rows_t)]


class moe_grad_t(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("ld", ctypes.c_int64), ("ld_out", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


def _nvw(w):
    """dict of the eight NVFP4 weight tensors + "amax" (float[4]) ->
    moe_nv_weights_t pointer."""
    q = moe_mx_weights_t(*[_p(w[k]).value for k in
                           ("w1", "w1_s", "w1t", "w1t_s", "w2", "w2_s", "w2t", "w2t_s")])
    return ctypes.byref(moe_nv_weights_t(q, _p(w["amax"]).value))


def _mx(mx):
    """dict of optional tensors {q, scale, qt, scale_t, amax} (+ "layout":
    "mma" for the MMA scale layout) -> struct pointer."""
    if mx is None:
        return None
    st = moe_mx_out_t(*[(_p(mx[k]).value if mx.get(k) is not None else None)
                        for k in ("q", "scale", "qt", "scale_t", "amax")],
                      MOE_MX_SCALES_MMA if mx.get("layout") == "mma" else MOE_MX_SCALES_ROWMAJOR)
    return ctypes.byref(st)


def _mxw(w):
    """dict of the eight MXFP8 weight tensors -> moe_mx_weights_t pointer."""
    st = moe_mx_weights_t(*[_p(w[k]).value for k in
                            ("w1", "w1_s", "w1t", "w1t_s", "w2", "w2_s", "w2t", "w2t_s")])
    return ctypes.byref(st)


def make_desc(T, E, k, d, F, act="swiglu", alpha=1.0, limit=math.inf, linear_offset=0.0,
              out_scale=1.0, has_b1=False, has_b2=False, sm_margin=0, capacity=None,
              recompute_h=False, dtype="bf16"):
    if capacity is None:
        capacity = T * k + E * 127
        capacity = (capacity + 127) // 128 * 128
    dt = {"bf16": MOE_DTYPE_BF16, "mxfp8": MOE_DTYPE_MXFP8, "nvfp4": MOE_DTYPE_NVFP4,
          "fp32": MOE_DTYPE_FP32}[dtype]
    return moe_mlp_desc_t(T, E, k, d, F, dt, ACTS[act], alpha, limit, linear_offset,
                          out_scale, int(has_b1), int(has_b2), 128, sm_margin, capacity,
                          int(recompute_h))


def make_block_norm_desc(T, d, dtype="bf16", res_dtype=None, param_dtype=None, pre_norm="rms",
                         post_norm=None, pre_eps=1e-6, post_eps=1e-6, pre_offset=0.0,
                         post_offset=0.0, gate=None, gate_act=None, res_scale=1.0,
                         branch_scale=1.0):
    """Descriptor of a residual block's norms (see include/moe.h): norms "rms",
    "layer" or None; gate None, "channel", "token" or "full"; gate_act None,
    "sigmoid" or "tanh"; types "bf16" or "fp32" (res_dtype and param_dtype
    default to dtype)."""
    dt = {"bf16": MOE_DTYPE_BF16, "fp32": MOE_DTYPE_FP32}
    return moe_block_norm_desc_t(
        T, d, dt[dtype], dt[res_dtype or dtype], dt[param_dtype or dtype], NORMS[pre_norm],
        NORMS[post_norm], GATES[gate], GATE_ACTS[gate_act], pre_eps, post_eps, pre_offset,
        post_offset, res_scale, branch_scale)


_lib = None


def lib():
    """Load libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise MoeError(f"{LIB_PATH} is not built; run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        D = ctypes.POINTER(moe_mlp_desc_t)
        R = moe_rows_t
        sig = {
            "moe_fc1_padded_width": (ctypes.c_int32, [ctypes.c_int32]),
            "moe_workspace_size": (ctypes.c_int, [D, ctypes.POINTER(ctypes.c_size_t)]),
            "moe_repack_fc1": (ctypes.c_int, [D, P, P, P, P, P]),
            "moe_unpack_fc1": (ctypes.c_int, [D, P, P, ctypes.c_int32, P]),
            "moe_route_permute": (ctypes.c_int, [D] + [P] * 13 + [ctypes.c_size_t, P]),
            "moe_group_offsets": (ctypes.c_int, [D, P, P, P, P, P]),
            "moe_mlp_fwd": (ctypes.c_int, [D] + [P] * 13 + [ctypes.c_size_t, P]),
            "moe_unpermute_combine": (ctypes.c_int, [D, P, P, P, P, P]),
            "moe_unpermute_combine_bwd": (ctypes.c_int, [D] + [P] * 8 + [P]),
            "moe_mlp_bwd": (ctypes.c_int, [D] + [P] * 17 + [ctypes.c_size_t, P]),
            "moe_permute_bwd": (ctypes.c_int, [D, P, P, P, P]),
            "moe_route_bwd": (ctypes.c_int, [D, P, P, P, P, P]),
            "moe_read_device_status": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int32), ctypes.c_int32]),
            "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "moe_fc1_glu_fwd": (ctypes.c_int, [D] + [P] * 9),
            "moe_fc2_fwd": (ctypes.c_int, [D] + [P] * 8),
            "moe_fc2_dgrad_dglu": (ctypes.c_int, [D] + [P] * 8),
            "moe_fc2_wgrad": (ctypes.c_int, [D] + [P] * 6),
            "moe_fc1_dgrad": (ctypes.c_int, [D] + [P] * 6),
            "moe_fc1_wgrad": (ctypes.c_int, [D] + [P] * 6),
            "moe_bias_grads": (ctypes.c_int, [D] + [P] * 7),
            "moe_route_permute_noalloc": (ctypes.c_int, [D] + [P] * 12 + [P]),
            "moe_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_uint32, P]),
            "moe_selftest_grid_wait_timeout": (ctypes.c_int, [ctypes.c_uint32, P]),
            "moe_fc1_glu_fwd_unfused": (ctypes.c_int, [D] + [P] * 8),
            "moe_fc1_recompute_h": (ctypes.c_int, [D] + [P] * 7),
            "moe_fc2_dgrad_dglu_unfused": (ctypes.c_int, [D] + [P] * 8),
            "moe_quantize_mx": (ctypes.c_int, [P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                               P, P, P]),
            "moe_mx_scale_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
            "moe_quantize_mx_bf16": (ctypes.c_int, [P, ctypes.c_int64, ctypes.c_int64,
                                                    ctypes.c_int64, P, P]),
            "moe_quantize_act_mx": (ctypes.c_int, [D, P, ctypes.c_int32, P, P, P]),
            "moe_quantize_weights_mx": (ctypes.c_int, [D, P, P, P, P]),
            "moe_mlp_fwd_mx": (ctypes.c_int, [D] + [P] * 11),
            "moe_mlp_bwd_mx": (ctypes.c_int, [D] + [P] * 16),
            "moe_fc1_glu_fwd_mx": (ctypes.c_int, [D] + [P] * 9),
            "moe_route_permute_fused": (ctypes.c_int, [D] + [P] * 14 + [ctypes.c_size_t, P]),
            "moe_fc2_fwd_mx": (ctypes.c_int, [D] + [P] * 7),
            "moe_fc2_dgrad_dglu_mx": (ctypes.c_int, [D] + [P] * 8),
            "moe_fc2_wgrad_mx": (ctypes.c_int, [D] + [P] * 6),
            "moe_fc1_dgrad_mx": (ctypes.c_int, [D] + [P] * 6),
            "moe_fc1_wgrad_mx": (ctypes.c_int, [D] + [P] * 6),
            "moe_nvfp4_scale_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
            "moe_amax_nvfp4": (ctypes.c_int, [P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                              P, P, P]),
            "moe_quantize_nvfp4_bf16": (ctypes.c_int, [P, ctypes.c_int64, ctypes.c_int64,
                                                       ctypes.c_int64, P, ctypes.c_int32, P]),
            "moe_quantize_act_nvfp4": (ctypes.c_int, [D, P, ctypes.c_int32, P, P,
                                                      ctypes.c_int32, P]),
            "moe_quantize_weights_nvfp4": (ctypes.c_int, [D, P, P, P, P]),
            "moe_fc1_glu_fwd_nv": (ctypes.c_int, [D] + [P] * 9),
            "moe_fc2_fwd_nv": (ctypes.c_int, [D] + [P] * 7),
            "moe_fc2_dgrad_dglu_nv": (ctypes.c_int, [D] + [P] * 8),
            "moe_fc2_wgrad_nv": (ctypes.c_int, [D] + [P] * 6),
            "moe_fc1_dgrad_nv": (ctypes.c_int, [D] + [P] * 6),
            "moe_fc1_wgrad_nv": (ctypes.c_int, [D] + [P] * 6),
            "moe_mlp_fwd_nv": (ctypes.c_int, [D] + [P] * 12),
            "moe_fc1_recompute_h_mx": (ctypes.c_int, [D] + [P] * 7),
            "moe_fc1_glu_fwd_mx_unfused": (ctypes.c_int, [D] + [P] * 9),
            "moe_fc2_dgrad_dglu_recompute": (ctypes.c_int, [D] + [P] * 10),
            "moe_route_permute_mx": (ctypes.c_int, [D] + [P] * 14 + [ctypes.c_size_t, P]),
            "moe_unpermute_combine_bwd_mx": (ctypes.c_int, [D] + [P] * 9 + [P]),
            "moe_fc2_dgrad_dglu_recompute_mx": (ctypes.c_int, [D] + [P] * 9),
            "moe_fc2_dgrad_dglu_mx_unfused": (ctypes.c_int, [D] + [P] * 9),
            "moe_fc1_recompute_h_nv": (ctypes.c_int, [D] + [P] * 7),
            "moe_mlp_bwd_nv": (ctypes.c_int, [D] + [P] * 16),
            "moe_transpose_weights_tf32": (ctypes.c_int, [D] + [P] * 5),
            "moe_transpose_rows_f32": (ctypes.c_int, [D, P, ctypes.c_int32, P, P, P]),
            "moe_fc1_glu_fwd_tf32": (ctypes.c_int, [D] + [P] * 9),
            "moe_fc2_fwd_tf32": (ctypes.c_int, [D] + [P] * 7),
            "moe_fc2_dgrad_dglu_tf32": (ctypes.c_int, [D] + [P] * 8),
            "moe_fc2_wgrad_tf32": (ctypes.c_int, [D] + [P] * 6),
            "moe_fc1_dgrad_tf32": (ctypes.c_int, [D] + [P] * 6),
            "moe_fc1_wgrad_tf32": (ctypes.c_int, [D] + [P] * 6),
            "moe_block_norm_workspace_size": (ctypes.c_int, [P, ctypes.POINTER(ctypes.c_size_t)]),
            "moe_block_pre_norm_fwd": (ctypes.c_int, [P, R, P, P, R, P]),
            "moe_block_pre_norm_bwd": (ctypes.c_int, [P, R, R, P, R, ctypes.c_float, R, P, P, P,
                                                      ctypes.c_size_t, P]),
            "moe_block_post_norm_fwd": (ctypes.c_int, [P, R, R, P, R, R, P, P]),
            "moe_block_post_norm_bwd": (ctypes.c_int, [P, R, ctypes.c_float, R, R, R, P, R, R, P,
                                                       P, ctypes.c_size_t, P]),
            "moe_grad_norm_workspace_size": (ctypes.c_int, [ctypes.c_int32,
                                                            ctypes.POINTER(ctypes.c_size_t)]),
            "moe_grad_norm": (ctypes.c_int, [P, ctypes.c_int32, ctypes.c_int32, P, P, P,
                                             ctypes.c_size_t, P]),
            "moe_clip_grads": (ctypes.c_int, [P, ctypes.c_int32, P, ctypes.c_float,
                                              ctypes.c_float, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


# the file is named for the Python that it was compiled for
BINDING_PATH = os.path.join(_HERE, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
_binding = None


def binding():
    """The C module that marshals the smallest calls (csrc/moe_binding.c),
    set up with the loaded library's functions."""
    global _binding
    if _binding is None:
        L = lib()
        if not os.path.exists(BINDING_PATH):
            raise MoeError(f"{BINDING_PATH} is not built; run __graft_entry__.build()")
        loader = importlib.machinery.ExtensionFileLoader("_binding", BINDING_PATH)
        spec = importlib.util.spec_from_file_location("_binding", BINDING_PATH, loader=loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        module.setup(torch, *[ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.moe_block_pre_norm_fwd, L.moe_block_pre_norm_bwd, L.moe_block_post_norm_fwd,
            L.moe_block_post_norm_bwd, L.moe_grad_norm, L.moe_clip_grads)])
        _binding = module
    return _binding


def _p(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous CUDA tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    # the current stream's handle without building a torch.cuda.Stream (0.3
    # instead of 3 us a call)
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _check(st):
    if st != 0:
        msg = lib().moe_status_string(st).decode()
        raise MoeError(f"libmoe status {st}: {msg}")


def moe_fc1_padded_width(F):
    return int(lib().moe_fc1_padded_width(F))


def moe_workspace_size(desc):
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_size(ctypes.byref(desc), ctypes.byref(n)))
    return int(n.value)


def moe_repack_fc1(desc, w1, b1, w1p, b1p, stream=None):
    _check(lib().moe_repack_fc1(ctypes.byref(desc), _p(w1), _p(b1), _p(w1p), _p(b1p), _stream(stream)))


def moe_unpack_fc1(desc, w1p, w1, rows_width, stream=None):
    _check(lib().moe_unpack_fc1(ctypes.byref(desc), _p(w1p), _p(w1), rows_width, _stream(stream)))


def moe_route_permute(desc, logits, bias, x, topk_idx, topk_w, counts, offsets, padded_offsets,
                      tile_prefix, row_src, row_of, x_perm, ws, stream=None):
    _check(lib().moe_route_permute(
        ctypes.byref(desc), _p(logits), _p(bias), _p(x), _p(topk_idx), _p(topk_w), _p(counts),
        _p(offsets), _p(padded_offsets), _p(tile_prefix), _p(row_src), _p(row_of), _p(x_perm),
        _p(ws), ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream)))


def moe_route_permute_fused(desc, x, w_router, bias, logits, topk_idx, topk_w, counts, offsets,
                            padded_offsets, tile_prefix, row_src, row_of, x_perm, ws,
                            stream=None):
    _check(lib().moe_route_permute_fused(
        ctypes.byref(desc), _p(x), _p(w_router), _p(bias), _p(logits), _p(topk_idx), _p(topk_w),
        _p(counts), _p(offsets), _p(padded_offsets), _p(tile_prefix), _p(row_src), _p(row_of),
        _p(x_perm), _p(ws), ws.numel() * ws.element_size() if ws is not None else 0,
        _stream(stream)))


def moe_group_offsets(desc, counts, offsets, padded_offsets, tile_prefix, stream=None):
    _check(lib().moe_group_offsets(ctypes.byref(desc), _p(counts), _p(offsets), _p(padded_offsets),
                                   _p(tile_prefix), _stream(stream)))


def moe_mlp_fwd(desc, x_perm, counts, padded_offsets, w1p, b1p, w2, b2, h, a, y, ws=None,
                stream=None, a_mx=None, y_mx=None):
    _check(lib().moe_mlp_fwd(
        ctypes.byref(desc), _p(x_perm), _p(counts), _p(padded_offsets), _p(w1p), _p(b1p), _p(w2),
        _p(b2), _p(h), _p(a), _p(y), _mx(a_mx), _mx(y_mx), _p(ws),
        ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream)))


def moe_unpermute_combine(desc, y, row_of, topk_w, out, stream=None):
    _check(lib().moe_unpermute_combine(ctypes.byref(desc), _p(y), _p(row_of), _p(topk_w), _p(out),
                                       _stream(stream)))


def moe_unpermute_combine_bwd(desc, dout, y, row_of, topk_w, row_src, padded_offsets, dy, dw,
                              stream=None):
    _check(lib().moe_unpermute_combine_bwd(
        ctypes.byref(desc), _p(dout), _p(y), _p(row_of), _p(topk_w), _p(row_src),
        _p(padded_offsets), _p(dy), _p(dw), _stream(stream)))


def moe_mlp_bwd(desc, dy, x_perm, h, a, counts, padded_offsets, w1p, w2, dh, dx_perm, dw1p, db1p,
                dw2, db2, ws=None, stream=None, dh_mx=None, b1p=None):
    _check(lib().moe_mlp_bwd(
        ctypes.byref(desc), _p(dy), _p(x_perm), _p(h), _p(a), _p(counts), _p(padded_offsets),
        _p(w1p), _p(b1p), _p(w2), _p(dh), _p(dx_perm), _p(dw1p), _p(db1p), _p(dw2), _p(db2),
        _mx(dh_mx), _p(ws), ws.numel() * ws.element_size() if ws is not None else 0,
        _stream(stream)))


def moe_permute_bwd(desc, dx_perm, row_of, dx, stream=None):
    _check(lib().moe_permute_bwd(ctypes.byref(desc), _p(dx_perm), _p(row_of), _p(dx), _stream(stream)))


def moe_route_bwd(desc, dw, topk_w, topk_idx, dlogits, stream=None):
    _check(lib().moe_route_bwd(ctypes.byref(desc), _p(dw), _p(topk_w), _p(topk_idx), _p(dlogits),
                               _stream(stream)))


def moe_read_device_status(clear=True):
    v = ctypes.c_int32(0)
    _check(lib().moe_read_device_status(ctypes.byref(v), int(clear)))
    return int(v.value)


def moe_fc1_glu_fwd(desc, x_perm, counts, padded_offsets, w1p, b1p, h, a, stream=None, mx=None):
    _check(lib().moe_fc1_glu_fwd(ctypes.byref(desc), _p(x_perm), _p(counts), _p(padded_offsets),
                                 _p(w1p), _p(b1p), _p(h), _p(a), _mx(mx), _stream(stream)))


def moe_fc2_fwd(desc, a, counts, padded_offsets, w2, b2, y, stream=None, mx=None):
    _check(lib().moe_fc2_fwd(ctypes.byref(desc), _p(a), _p(counts), _p(padded_offsets), _p(w2),
                             _p(b2), _p(y), _mx(mx), _stream(stream)))


def moe_fc2_dgrad_dglu(desc, dy, h, counts, padded_offsets, w2, dh, stream=None, mx=None):
    _check(lib().moe_fc2_dgrad_dglu(ctypes.byref(desc), _p(dy), _p(h), _p(counts),
                                    _p(padded_offsets), _p(w2), _p(dh), _mx(mx), _stream(stream)))


def moe_fc2_wgrad(desc, dy, a, counts, padded_offsets, dw2, stream=None):
    _check(lib().moe_fc2_wgrad(ctypes.byref(desc), _p(dy), _p(a), _p(counts), _p(padded_offsets),
                               _p(dw2), _stream(stream)))


def moe_fc1_dgrad(desc, dh, counts, padded_offsets, w1p, dx_perm, stream=None):
    _check(lib().moe_fc1_dgrad(ctypes.byref(desc), _p(dh), _p(counts), _p(padded_offsets), _p(w1p),
                               _p(dx_perm), _stream(stream)))


def moe_fc1_wgrad(desc, dh, x_perm, counts, padded_offsets, dw1p, stream=None):
    _check(lib().moe_fc1_wgrad(ctypes.byref(desc), _p(dh), _p(x_perm), _p(counts),
                               _p(padded_offsets), _p(dw1p), _stream(stream)))


def moe_bias_grads(desc, dy, dh, counts, padded_offsets, db1p, db2, stream=None):
    _check(lib().moe_bias_grads(ctypes.byref(desc), _p(dy), _p(dh), _p(counts),
                                _p(padded_offsets), _p(db1p), _p(db2), _stream(stream)))


def moe_selftest_wait_timeout(limit_us, stream=None):
    _check(lib().moe_selftest_wait_timeout(int(limit_us), _stream(stream)))


def moe_selftest_grid_wait_timeout(limit_us, stream=None):
    _check(lib().moe_selftest_grid_wait_timeout(int(limit_us), _stream(stream)))


def moe_quantize_mx(x, colwise, q, scales, stream=None):
    """MXFP8-quantize fp32 x [rows, cols] rowwise (colwise=False) or
    columnwise into the transposed q (colwise=True)."""
    rows, cols = x.shape
    _check(lib().moe_quantize_mx(_p(x), rows, cols, int(bool(colwise)), _p(q), _p(scales),
                                 _stream(stream)))


def moe_route_permute_noalloc(desc, logits, bias, x, topk_idx, topk_w, counts, offsets,
                              padded_offsets, tile_prefix, row_src, row_of, x_perm, stream=None):
    """moe_route_permute without a caller-provided workspace (see include/moe.h)."""
    _check(lib().moe_route_permute_noalloc(
        ctypes.byref(desc), _p(logits), _p(bias), _p(x), _p(topk_idx), _p(topk_w), _p(counts),
        _p(offsets), _p(padded_offsets), _p(tile_prefix), _p(row_src), _p(row_of), _p(x_perm),
        _stream(stream)))


def moe_fc1_glu_fwd_unfused(desc, x_perm, counts, padded_offsets, w1p, b1p, h, a, stream=None):
    _check(lib().moe_fc1_glu_fwd_unfused(ctypes.byref(desc), _p(x_perm), _p(counts),
                                         _p(padded_offsets), _p(w1p), _p(b1p), _p(h), _p(a),
                                         _stream(stream)))


def moe_fc2_dgrad_dglu_unfused(desc, dy, h, counts, padded_offsets, w2, da, dh, stream=None):
    _check(lib().moe_fc2_dgrad_dglu_unfused(ctypes.byref(desc), _p(dy), _p(h), _p(counts),
                                            _p(padded_offsets), _p(w2), _p(da), _p(dh),
                                            _stream(stream)))


def moe_fc1_recompute_h(desc, x_perm, counts, padded_offsets, w1p, b1p, h, stream=None):
    _check(lib().moe_fc1_recompute_h(ctypes.byref(desc), _p(x_perm), _p(counts),
                                     _p(padded_offsets), _p(w1p), _p(b1p), _p(h), _stream(stream)))


# ------------------------------------------------------------------ MXFP8
def moe_mx_scale_bytes(rows, cols):
    return int(lib().moe_mx_scale_bytes(rows, cols))


def moe_quantize_mx_bf16(inp, batch, rows, cols, out, stream=None):
    _check(lib().moe_quantize_mx_bf16(_p(inp), batch, rows, cols, _mx(out), _stream(stream)))


def moe_quantize_act_mx(desc, inp, width, padded_offsets, out, stream=None):
    _check(lib().moe_quantize_act_mx(ctypes.byref(desc), _p(inp), width, _p(padded_offsets),
                                     _mx(out), _stream(stream)))


def moe_quantize_weights_mx(desc, w1p, w2, out, stream=None):
    _check(lib().moe_quantize_weights_mx(ctypes.byref(desc), _p(w1p), _p(w2), _mxw(out),
                                         _stream(stream)))


def moe_mlp_fwd_mx(desc, x_mx, counts, padded_offsets, w_mx, b1p, b2, h, a, a_mx, y,
                   stream=None):
    _check(lib().moe_mlp_fwd_mx(ctypes.byref(desc), _mx(x_mx), _p(counts), _p(padded_offsets),
                                _mxw(w_mx), _p(b1p), _p(b2), _p(h), _p(a), _mx(a_mx), _p(y),
                                _stream(stream)))


def moe_mlp_bwd_mx(desc, dy, dy_mx, x_mx, h, a_mx, counts, padded_offsets, w_mx, dh, dh_mx,
                   dx_perm, dw1p, db1p, dw2, db2, stream=None):
    _check(lib().moe_mlp_bwd_mx(ctypes.byref(desc), _p(dy), _mx(dy_mx), _mx(x_mx), _p(h),
                                _mx(a_mx), _p(counts), _p(padded_offsets), _mxw(w_mx), _p(dh),
                                _mx(dh_mx), _p(dx_perm), _p(dw1p), _p(db1p), _p(dw2), _p(db2),
                                _stream(stream)))


def moe_fc1_glu_fwd_mx(desc, x_mx, counts, padded_offsets, w_mx, b1p, h, a, a_mx, stream=None):
    _check(lib().moe_fc1_glu_fwd_mx(ctypes.byref(desc), _mx(x_mx), _p(counts),
                                    _p(padded_offsets), _mxw(w_mx), _p(b1p), _p(h), _p(a),
                                    _mx(a_mx), _stream(stream)))


def moe_fc2_fwd_mx(desc, a_mx, counts, padded_offsets, w_mx, b2, y, stream=None):
    _check(lib().moe_fc2_fwd_mx(ctypes.byref(desc), _mx(a_mx), _p(counts), _p(padded_offsets),
                                _mxw(w_mx), _p(b2), _p(y), _stream(stream)))


def moe_fc2_dgrad_dglu_mx(desc, dy_mx, h, counts, padded_offsets, w_mx, dh, dh_mx,
                          stream=None):
    _check(lib().moe_fc2_dgrad_dglu_mx(ctypes.byref(desc), _mx(dy_mx), _p(h), _p(counts),
                                       _p(padded_offsets), _mxw(w_mx), _p(dh), _mx(dh_mx),
                                       _stream(stream)))


def moe_fc2_wgrad_mx(desc, dy_mx, a_mx, counts, padded_offsets, dw2, stream=None):
    _check(lib().moe_fc2_wgrad_mx(ctypes.byref(desc), _mx(dy_mx), _mx(a_mx), _p(counts),
                                  _p(padded_offsets), _p(dw2), _stream(stream)))


def moe_fc1_dgrad_mx(desc, dh_mx, counts, padded_offsets, w_mx, dx_perm, stream=None):
    _check(lib().moe_fc1_dgrad_mx(ctypes.byref(desc), _mx(dh_mx), _p(counts),
                                  _p(padded_offsets), _mxw(w_mx), _p(dx_perm), _stream(stream)))


def moe_fc1_wgrad_mx(desc, dh_mx, x_mx, counts, padded_offsets, dw1p, stream=None):
    _check(lib().moe_fc1_wgrad_mx(ctypes.byref(desc), _mx(dh_mx), _mx(x_mx), _p(counts),
                                  _p(padded_offsets), _p(dw1p), _stream(stream)))


# ------------------------------------------------------------------ NVFP4
def moe_nvfp4_scale_bytes(rows, cols):
    return int(lib().moe_nvfp4_scale_bytes(rows, cols))


def moe_amax_nvfp4(inp, batch, rows, cols, amax, row_limit=None, stream=None):
    _check(lib().moe_amax_nvfp4(_p(inp), batch, rows, cols, _p(row_limit), _p(amax),
                                _stream(stream)))


def moe_quantize_nvfp4_bf16(inp, batch, rows, cols, out, rotate_t=False, stream=None):
    _check(lib().moe_quantize_nvfp4_bf16(_p(inp), batch, rows, cols, _mx(out),
                                         int(bool(rotate_t)), _stream(stream)))


def moe_quantize_act_nvfp4(desc, inp, width, padded_offsets, out, compute_amax, stream=None):
    _check(lib().moe_quantize_act_nvfp4(ctypes.byref(desc), _p(inp), width, _p(padded_offsets),
                                        _mx(out), int(bool(compute_amax)), _stream(stream)))


def moe_quantize_weights_nvfp4(desc, w1p, w2, out, stream=None):
    _check(lib().moe_quantize_weights_nvfp4(ctypes.byref(desc), _p(w1p), _p(w2), _nvw(out),
                                            _stream(stream)))


def moe_fc1_glu_fwd_nv(desc, x_nv, counts, padded_offsets, w_nv, b1p, h, a, a_amax, stream=None):
    _check(lib().moe_fc1_glu_fwd_nv(ctypes.byref(desc), _mx(x_nv), _p(counts),
                                    _p(padded_offsets), _nvw(w_nv), _p(b1p), _p(h), _p(a),
                                    _p(a_amax), _stream(stream)))


def moe_fc2_fwd_nv(desc, a_nv, counts, padded_offsets, w_nv, b2, y, stream=None):
    _check(lib().moe_fc2_fwd_nv(ctypes.byref(desc), _mx(a_nv), _p(counts), _p(padded_offsets),
                                _nvw(w_nv), _p(b2), _p(y), _stream(stream)))


def moe_fc2_dgrad_dglu_nv(desc, dy_nv, h, counts, padded_offsets, w_nv, dh, dh_amax,
                          stream=None):
    _check(lib().moe_fc2_dgrad_dglu_nv(ctypes.byref(desc), _mx(dy_nv), _p(h), _p(counts),
                                       _p(padded_offsets), _nvw(w_nv), _p(dh), _p(dh_amax),
                                       _stream(stream)))


def moe_fc2_wgrad_nv(desc, dy_nv, a_nv, counts, padded_offsets, dw2, stream=None):
    _check(lib().moe_fc2_wgrad_nv(ctypes.byref(desc), _mx(dy_nv), _mx(a_nv), _p(counts),
                                  _p(padded_offsets), _p(dw2), _stream(stream)))


def moe_fc1_dgrad_nv(desc, dh_nv, counts, padded_offsets, w_nv, dx_perm, stream=None):
    _check(lib().moe_fc1_dgrad_nv(ctypes.byref(desc), _mx(dh_nv), _p(counts),
                                  _p(padded_offsets), _nvw(w_nv), _p(dx_perm), _stream(stream)))


def moe_fc1_wgrad_nv(desc, dh_nv, x_nv, counts, padded_offsets, dw1p, stream=None):
    _check(lib().moe_fc1_wgrad_nv(ctypes.byref(desc), _mx(dh_nv), _mx(x_nv), _p(counts),
                                  _p(padded_offsets), _p(dw1p), _stream(stream)))


def moe_mlp_fwd_nv(desc, x_perm, x_nv, counts, padded_offsets, w_nv, b1p, b2, h, a, a_nv, y,
                   stream=None):
    _check(lib().moe_mlp_fwd_nv(ctypes.byref(desc), _p(x_perm), _mx(x_nv), _p(counts),
                                _p(padded_offsets), _nvw(w_nv), _p(b1p), _p(b2), _p(h), _p(a),
                                _mx(a_nv), _p(y), _stream(stream)))


def moe_mlp_bwd_nv(desc, dy, dy_nv, x_nv, h, a_nv, counts, padded_offsets, w_nv, dh, dh_nv,
                   dx_perm, dw1p, db1p, dw2, db2, stream=None):
    _check(lib().moe_mlp_bwd_nv(ctypes.byref(desc), _p(dy), _mx(dy_nv), _mx(x_nv), _p(h),
                                _mx(a_nv), _p(counts), _p(padded_offsets), _nvw(w_nv), _p(dh),
                                _mx(dh_nv), _p(dx_perm), _p(dw1p), _p(db1p), _p(dw2), _p(db2),
                                _stream(stream)))


def moe_fc1_recompute_h_mx(desc, x_mx, counts, padded_offsets, w_mx, b1p, h, stream=None):
    _check(lib().moe_fc1_recompute_h_mx(ctypes.byref(desc), _mx(x_mx), _p(counts),
                                        _p(padded_offsets), _mxw(w_mx), _p(b1p), _p(h),
                                        _stream(stream)))


def moe_route_permute_mx(desc, logits, bias, x, topk_idx, topk_w, counts, offsets,
                         padded_offsets, tile_prefix, row_src, row_of, x_perm, x_mx, ws,
                         stream=None):
    """moe_route_permute that also writes x_perm's rowwise MXFP8 copy."""
    _check(lib().moe_route_permute_mx(
        ctypes.byref(desc), _p(logits), _p(bias), _p(x), _p(topk_idx), _p(topk_w), _p(counts),
        _p(offsets), _p(padded_offsets), _p(tile_prefix), _p(row_src), _p(row_of), _p(x_perm),
        _mx(x_mx), _p(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_unpermute_combine_bwd_mx(desc, dout, y, row_of, topk_w, row_src, padded_offsets, dy,
                                 dy_mx, dw, stream=None):
    """moe_unpermute_combine_bwd that also writes dy's rowwise MXFP8 copy."""
    _check(lib().moe_unpermute_combine_bwd_mx(
        ctypes.byref(desc), _p(dout), _p(y), _p(row_of), _p(topk_w), _p(row_src),
        _p(padded_offsets), _p(dy), _mx(dy_mx), _p(dw), _stream(stream)))


def moe_fc2_dgrad_dglu_recompute(desc, x_perm, dy, counts, padded_offsets, w1p, b1p, w2, dh,
                                 stream=None, mx=None):
    """FC2 dgrad + dGLU with H recomputed inside the kernel (see include/moe.h)."""
    _check(lib().moe_fc2_dgrad_dglu_recompute(ctypes.byref(desc), _p(x_perm), _p(dy), _p(counts),
                                              _p(padded_offsets), _p(w1p), _p(b1p), _p(w2),
                                              _p(dh), _mx(mx), _stream(stream)))


def moe_fc2_dgrad_dglu_recompute_mx(desc, x_mx, dy_mx, counts, padded_offsets, w_mx, b1p, dh,
                                    dh_mx, stream=None):
    """The same on the MXFP8 operands (see include/moe.h)."""
    _check(lib().moe_fc2_dgrad_dglu_recompute_mx(ctypes.byref(desc), _mx(x_mx), _mx(dy_mx),
                                                 _p(counts), _p(padded_offsets), _mxw(w_mx),
                                                 _p(b1p), _p(dh), _mx(dh_mx), _stream(stream)))


def moe_fc1_glu_fwd_mx_unfused(desc, x_mx, counts, padded_offsets, w_mx, b1p, h, a, a_mx,
                               stream=None):
    """FC1 plain GEMM, GLU pass, MXFP8 quantize pass (see include/moe.h)."""
    _check(lib().moe_fc1_glu_fwd_mx_unfused(ctypes.byref(desc), _mx(x_mx), _p(counts),
                                            _p(padded_offsets), _mxw(w_mx), _p(b1p), _p(h), _p(a),
                                            _mx(a_mx), _stream(stream)))


def moe_fc2_dgrad_dglu_mx_unfused(desc, dy_mx, h, counts, padded_offsets, w_mx, da, dh, dh_mx,
                                  stream=None):
    """FC2 dgrad plain GEMM, dGLU pass, MXFP8 quantize pass (see include/moe.h)."""
    _check(lib().moe_fc2_dgrad_dglu_mx_unfused(ctypes.byref(desc), _mx(dy_mx), _p(h), _p(counts),
                                               _p(padded_offsets), _mxw(w_mx), _p(da), _p(dh),
                                               _mx(dh_mx), _stream(stream)))


def moe_fc1_recompute_h_nv(desc, x_nv, counts, padded_offsets, w_nv, b1p, h, stream=None):
    _check(lib().moe_fc1_recompute_h_nv(ctypes.byref(desc), _mx(x_nv), _p(counts),
                                        _p(padded_offsets), _nvw(w_nv), _p(b1p), _p(h),
                                        _stream(stream)))


# ------------------------------------------------------- fp32 / TF32 path
def moe_transpose_weights_tf32(desc, w1p, w2, w1t, w2t, stream=None):
    _check(lib().moe_transpose_weights_tf32(ctypes.byref(desc), _p(w1p), _p(w2), _p(w1t),
                                            _p(w2t), _stream(stream)))


def moe_transpose_rows_f32(desc, x, width, padded_offsets, out, stream=None):
    _check(lib().moe_transpose_rows_f32(ctypes.byref(desc), _p(x), width, _p(padded_offsets),
                                        _p(out), _stream(stream)))


def moe_fc1_glu_fwd_tf32(desc, x_perm, counts, padded_offsets, w1p, b1p, h, a, a_t=None,
                         stream=None):
    _check(lib().moe_fc1_glu_fwd_tf32(ctypes.byref(desc), _p(x_perm), _p(counts),
                                      _p(padded_offsets), _p(w1p), _p(b1p), _p(h), _p(a),
                                      _p(a_t), _stream(stream)))


def moe_fc2_fwd_tf32(desc, a, counts, padded_offsets, w2, b2, y, stream=None):
    _check(lib().moe_fc2_fwd_tf32(ctypes.byref(desc), _p(a), _p(counts), _p(padded_offsets),
                                  _p(w2), _p(b2), _p(y), _stream(stream)))


def moe_fc2_dgrad_dglu_tf32(desc, dy, h, counts, padded_offsets, w2t, dh, dh_t=None,
                            stream=None):
    _check(lib().moe_fc2_dgrad_dglu_tf32(ctypes.byref(desc), _p(dy), _p(h), _p(counts),
                                         _p(padded_offsets), _p(w2t), _p(dh), _p(dh_t),
                                         _stream(stream)))


def moe_fc2_wgrad_tf32(desc, dy_t, a_t, counts, padded_offsets, dw2, stream=None):
    _check(lib().moe_fc2_wgrad_tf32(ctypes.byref(desc), _p(dy_t), _p(a_t), _p(counts),
                                    _p(padded_offsets), _p(dw2), _stream(stream)))


def moe_fc1_dgrad_tf32(desc, dh, counts, padded_offsets, w1t, dx_perm, stream=None):
    _check(lib().moe_fc1_dgrad_tf32(ctypes.byref(desc), _p(dh), _p(counts), _p(padded_offsets),
                                    _p(w1t), _p(dx_perm), _stream(stream)))


def moe_fc1_wgrad_tf32(desc, dh_t, x_t, counts, padded_offsets, dw1p, stream=None):
    _check(lib().moe_fc1_wgrad_tf32(ctypes.byref(desc), _p(dh_t), _p(x_t), _p(counts),
                                    _p(padded_offsets), _p(dw1p), _stream(stream)))


# ------------------------------------------------- residual block's norms
# Marshalled in C (binding()): tensors are [T,d] with unit stride along the
# channels and any stride between rows, None where absent.
def moe_block_norm_workspace_size(desc):
    n = ctypes.c_size_t(0)
    _check(lib().moe_block_norm_workspace_size(ctypes.byref(desc), ctypes.byref(n)))
    return int(n.value)


def moe_block_pre_norm_fwd(desc, res, w, b, x, stream=None):
    """x = N1(res)."""
    _check((_binding or binding()).pre_norm_fwd(desc, res, w, b, x, stream))


def moe_block_pre_norm_bwd(desc, dx, res, w, dres_in, dres, dw, db, ws, dres_scale=1.0,
                           stream=None):
    """dres = dres_scale*dres_in + N1^T(dx); dw, db or None."""
    _check((_binding or binding()).pre_norm_bwd(desc, dx, res, w, dres_in, dres, dw, db, ws,
                                                dres_scale, stream))


def moe_block_post_norm_fwd(desc, res, y, params, res_out, x=None, routed=None, stream=None):
    """res_out = res_scale*res + branch_scale*G*N2(y), x = N1(res_out) or None.
    params: dict {pre_w, pre_b, post_w, post_b, gate}; routed: dict {row_of,
    topk_w, y_out} with y the expert rows [capacity, d]."""
    _check((_binding or binding()).post_norm_fwd(desc, res, y, params, res_out, x, routed, stream))


def moe_block_post_norm_bwd(desc, dres_in, dx, res_out, y, params, dres, dy, grads, ws,
                            dres_scale=1.0, stream=None):
    """dres = dres_scale*dres_in + N1^T(dx; res_out) (dx None: without the next
    norm), dy = N2^T(branch_scale*G*dres; y) and the parameters' gradients
    (grads: dict like params, each optional)."""
    _check((_binding or binding()).post_norm_bwd(desc, dres_in, dx, res_out, y, params, dres, dy,
                                                 grads, ws, dres_scale, stream))


# ------------------------------------------- gradient norm and clipping
def _runs(t, out):
    """(rows, cols, ld, ld_out) of a tensor whose elements lie in runs of equal
    length and distance, in the memory order of t; out in the same order."""
    if t.numel() == 0:
        return (1, 0, 0, 0)
    dims = sorted((i for i in range(t.dim()) if t.size(i) != 1), key=lambda i: -t.stride(i))
    runs = []                                  # [size, stride, stride of out], outermost first
    for i in dims:
        n, s, so = t.size(i), t.stride(i), out.stride(i)
        if runs and runs[-1][1] == n * s and runs[-1][2] == n * so:
            runs[-1] = [runs[-1][0] * n, s, so]
        else:
            runs.append([n, s, so])
    if not runs or runs[-1][1] != 1 or runs[-1][2] != 1:
        runs.append([1, 1, 1])                 # no unit stride: rows of one element
    cols = runs[-1][0]
    if len(runs) == 1:
        return (1, cols, cols, cols)
    rows, ld, ld_out = runs[0]
    if len(runs) > 2 or ld < cols or ld_out < cols:
        raise ValueError(f"gradient of shape {tuple(t.shape)} and strides {t.stride()} (out: "
                         f"{out.stride()}) is not rows at one distance")
    return (rows, cols, ld, ld_out)


class GradList:
    """Gradient tensors (bf16 or fp32, contiguous or rows at one distance) and
    where their clipped copies go (outs; default: in place), described for
    moe_grad_norm and moe_clip_grads.  The list holds the tensors; one that has
    other memory, strides, size or type since (`tensor.data = ...`) is described
    anew at the next call."""

    def __init__(self, tensors, outs=None):
        self.tensors = list(tensors)
        self.outs = self.tensors if outs is None else list(outs)
        self.describe()

    def __len__(self):
        return len(self.tensors)

    def describe(self):
        if len(self.outs) != len(self.tensors):
            raise ValueError(f"{len(self.tensors)} gradients and {len(self.outs)} outputs")
        kinds = {torch.bfloat16: MOE_DTYPE_BF16, torch.float32: MOE_DTYPE_FP32}
        array = (moe_grad_t * max(len(self.tensors), 1))()
        layouts = []
        for i, (t, o) in enumerate(zip(self.tensors, self.outs)):
            if t.dtype not in kinds or o.dtype not in kinds or not t.is_cuda or not o.is_cuda:
                raise ValueError(f"gradient {i}: expected bf16 or fp32 CUDA tensors, got {t.dtype} "
                                 f"on {t.device} and {o.dtype} on {o.device}")
            if t.shape != o.shape:
                raise ValueError(f"gradient {i}: shapes {tuple(t.shape)} and {tuple(o.shape)}")
            array[i] = moe_grad_t(t.data_ptr(), o.data_ptr(), *_runs(t, o), kinds[t.dtype],
                                  kinds[o.dtype])
            dense = t.is_contiguous() and o.is_contiguous()
            layouts.append((None, None) if dense else tuple((tuple(v.shape), v.stride())
                                                            for v in (t, o)))
        self.array, self.layouts = array, layouts
        # two gradients clipped into the same memory, if there are any: blocks
        # would write it side by side (the norm may read one twice)
        seen, self.shared = {}, None
        for i, o in enumerate(self.outs):
            if o.numel() and seen.setdefault(o.data_ptr(), i) != i:
                self.shared = (seen[o.data_ptr()], i)

    def refresh(self, outs=True):
        """Describes the tensors anew if one (or, if asked, an output) is no
        longer what it was."""
        other = None if self.outs is self.tensors or not outs else self.outs
        if not (_binding or binding()).in_place(self.array, self.tensors, other, self.layouts):
            self.describe()


def _grad_list(grads, outs):
    if not isinstance(grads, GradList):
        return GradList(grads)
    grads.refresh(outs)
    return grads


def moe_grad_norm_workspace_size(n):
    b = ctypes.c_size_t(0)
    _check(lib().moe_grad_norm_workspace_size(n, ctypes.byref(b)))
    return int(b.value)


def moe_grad_norm(grads, norm, norms, norm_type, ws, stream=None):
    """Global norm of a GradList (or a list of tensors) into norm fp32 [1], and
    each tensor's into norms fp32 [n] (or None); norm_type "l2" or "inf"."""
    g = _grad_list(grads, False)
    _check((_binding or binding()).grad_norm(g.array, len(g.tensors), GRAD_NORMS[norm_type], norm,
                                             norms, ws, stream))


def moe_clip_grads(grads, norm, max_norm, eps=1e-6, stream=None):
    """outs = grads * min(1, max_norm / (norm + eps)), norm fp32 [1] on the
    device."""
    g = _grad_list(grads, True)
    if g.shared:
        raise ValueError("gradients {} and {} are clipped into the same memory".format(*g.shared))
    _check((_binding or binding()).clip_grads(g.array, len(g.tensors), norm, max_norm, eps, stream))
