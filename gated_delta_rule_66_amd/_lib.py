"""ctypes view of libgdr.so (include/gdr.h).  Loading fails loudly if the
library has not been built: there is no fallback path."""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgdr.so")

GDR_BF16, GDR_FP16, GDR_FP32 = 0, 1, 2

STATUS = {
    0: "GDR_OK", 1: "GDR_ERR_NULL", 2: "GDR_ERR_SHAPE", 3: "GDR_ERR_HEAD_DIM",
    4: "GDR_ERR_DTYPE", 5: "GDR_ERR_HEADS", 6: "GDR_ERR_VARLEN", 7: "GDR_ERR_WORKSPACE",
    8: "GDR_ERR_DEVICE", 9: "GDR_ERR_HIP", 10: "GDR_ERR_ARG",
}


class Problem(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("Hq", ctypes.c_int32),
        ("Hv", ctypes.c_int32), ("K", ctypes.c_int32), ("V", ctypes.c_int32),
        ("N", ctypes.c_int32),
        ("cu_seqlens_dev", ctypes.c_void_p),
        ("cu_seqlens_host", ctypes.c_void_p),
        ("in_dtype", ctypes.c_int), ("g_dtype", ctypes.c_int),
        ("scale", ctypes.c_float),
        ("state_v_first", ctypes.c_int32),
        ("cp_segments", ctypes.c_int32),
        ("wave_tiles", ctypes.c_int32),
        ("use_qk_l2norm", ctypes.c_int32),
        ("beta_sigmoid", ctypes.c_int32),
        ("neg_eigval", ctypes.c_int32),
        ("use_gate", ctypes.c_int32),
        ("gate_A_log", ctypes.c_void_p),
        ("gate_dt_bias", ctypes.c_void_p),
        ("h_packed", ctypes.c_int32),
    ]


class ConvProblem(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("D", ctypes.c_int32), ("W", ctypes.c_int32),
        ("N", ctypes.c_int32),
        ("cu_seqlens_dev", ctypes.c_void_p),
        ("cu_seqlens_host", ctypes.c_void_p),
        ("dtype", ctypes.c_int), ("w_dtype", ctypes.c_int),
        ("activation", ctypes.c_int32),
        ("x_stride", ctypes.c_int64),
    ]


class SsmProblem(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("G", ctypes.c_int32),
        ("K", ctypes.c_int32), ("V", ctypes.c_int32), ("N", ctypes.c_int32),
        ("cu_seqlens_dev", ctypes.c_void_p),
        ("cu_seqlens_host", ctypes.c_void_p),
        ("in_dtype", ctypes.c_int), ("dt_dtype", ctypes.c_int), ("p_dtype", ctypes.c_int),
        ("dt_softplus", ctypes.c_int32), ("keep_states", ctypes.c_int32),
        ("x_stride", ctypes.c_int64), ("b_stride", ctypes.c_int64), ("c_stride", ctypes.c_int64),
    ]


class NormProblem(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int32), ("D", ctypes.c_int32),
        ("dtype", ctypes.c_int), ("res_dtype", ctypes.c_int), ("w_dtype", ctypes.c_int),
        ("has_residual", ctypes.c_int32), ("quant", ctypes.c_int32),
        ("group_size", ctypes.c_int32), ("eps", ctypes.c_float),
        ("x_stride", ctypes.c_int64),
    ]


class GatedNormProblem(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int32), ("D", ctypes.c_int32), ("norm_size", ctypes.c_int32),
        ("dtype", ctypes.c_int), ("w_dtype", ctypes.c_int),
        ("shared_weight", ctypes.c_int32), ("gate_first", ctypes.c_int32),
        ("activation", ctypes.c_int32), ("quant", ctypes.c_int32),
        ("scale_group", ctypes.c_int32), ("eps", ctypes.c_float),
        ("x_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64),
    ]


class SandwichNormProblem(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int32), ("D", ctypes.c_int32),
        ("dtype", ctypes.c_int), ("res_dtype", ctypes.c_int), ("w_dtype", ctypes.c_int),
        ("activation", ctypes.c_int32), ("quant", ctypes.c_int32),
        ("group_size", ctypes.c_int32), ("eps", ctypes.c_float), ("alpha", ctypes.c_float),
        ("x_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64),
    ]


class QuantizeProblem(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int32), ("D", ctypes.c_int32), ("dtype", ctypes.c_int),
        ("quant", ctypes.c_int32), ("group_size", ctypes.c_int32),
        ("x_stride", ctypes.c_int64),
    ]


class Int8MatmulProblem(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
        ("out_dtype", ctypes.c_int), ("bias_dtype", ctypes.c_int),
        ("x_stride", ctypes.c_int64),
    ]


# every symbol include/gdr.h declares
EXPORTS = [
    "gdr_status_string", "gdr_last_error", "gdr_check_supported", "gdr_check_device",
    "gdr_chunk_fwd_workspace_size", "gdr_chunk_bwd_workspace_size", "gdr_chunk_fwd",
    "gdr_chunk_bwd", "gdr_prepare_lens_i32", "gdr_prepare_lens_i64",
    "gdr_prepare_chunk_indices_i32", "gdr_prepare_chunk_indices_i64",
    "gdr_prepare_chunk_offsets_i32", "gdr_prepare_chunk_offsets_i64",
    "gdr_prepare_chunk_token_starts_i64", "gdr_profile_enable", "gdr_profile_read",
    "gdr_plan_info", "gdr_recurrent_fwd", "gdr_chunk_bwd_gate", "gdr_chunk_fwd_noalloc",
    "gdr_chunk_bwd_states", "gdr_chunk_bwd_states_workspace_size", "gdr_chunk_fwd_states",
    "gdr_chunk_trans_size", "gdr_bwd_pipeline_info",
    "gdr_conv1d_check", "gdr_conv1d_fwd", "gdr_conv1d_bwd_workspace_size", "gdr_conv1d_bwd",
    "gdr_conv1d_update", "gdr_rms_norm_check", "gdr_rms_norm_fwd",
    "gdr_rms_norm_bwd_workspace_size", "gdr_rms_norm_bwd",
    "gdr_ssm_check", "gdr_ssm_fwd_workspace_size", "gdr_ssm_fwd", "gdr_ssm_step",
    "gdr_ssm_bwd_workspace_size", "gdr_ssm_bwd",
    "gdr_gated_norm_check", "gdr_gated_norm_fwd", "gdr_gated_norm_bwd_workspace_size",
    "gdr_gated_norm_bwd", "gdr_sandwich_norm_check", "gdr_sandwich_norm_fwd",
    "gdr_sandwich_norm_bwd_workspace_size", "gdr_sandwich_norm_bwd", "gdr_quantize_check",
    "gdr_quantize_rows", "gdr_int8_matmul_check",
    "gdr_int8_matmul_workspace_size", "gdr_int8_matmul",
]


class GdrError(RuntimeError):
    def __init__(self, status: int, msg: str):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__("%s: %s" % (self.name, msg))


def _declare(lib):
    P = ctypes.c_void_p
    PP = ctypes.POINTER(Problem)
    I64 = ctypes.c_int64
    S = ctypes.c_size_t
    st = ctypes.c_int
    lib.gdr_status_string.argtypes = [st]
    lib.gdr_status_string.restype = ctypes.c_char_p
    lib.gdr_last_error.argtypes = []
    lib.gdr_last_error.restype = ctypes.c_char_p
    lib.gdr_check_supported.argtypes = [PP, ctypes.c_char_p, S]
    lib.gdr_check_supported.restype = st
    lib.gdr_check_device.argtypes = []
    lib.gdr_check_device.restype = st
    lib.gdr_chunk_fwd_workspace_size.argtypes = [PP]
    lib.gdr_chunk_fwd_workspace_size.restype = S
    lib.gdr_chunk_bwd_workspace_size.argtypes = [PP]
    lib.gdr_chunk_bwd_workspace_size.restype = S
    lib.gdr_chunk_fwd.argtypes = [PP, P, P, P, P, P, P, P, P, P, P, P, P, S, P]
    lib.gdr_chunk_fwd.restype = st
    lib.gdr_chunk_bwd_states_workspace_size.argtypes = [PP]
    lib.gdr_chunk_bwd_states_workspace_size.restype = S
    lib.gdr_chunk_bwd_states.argtypes = [PP] + [P] * 12 + [S] + [P] * 9 + [S, P]
    lib.gdr_bwd_pipeline_info.argtypes = [PP, ctypes.POINTER(ctypes.c_int32),
                                          ctypes.POINTER(ctypes.c_int32), ctypes.c_int32]
    lib.gdr_bwd_pipeline_info.restype = st
    lib.gdr_chunk_trans_size.argtypes = [PP]
    lib.gdr_chunk_trans_size.restype = S
    lib.gdr_chunk_fwd_states.argtypes = [PP] + [P] * 11 + [S] + [P] * 2 + [S, P]
    lib.gdr_chunk_fwd_states.restype = st
    lib.gdr_chunk_bwd_states.restype = st
    lib.gdr_chunk_fwd_noalloc.argtypes = [PP, P, P, P, P, P, P, P, P, P, P, P, P]
    lib.gdr_chunk_fwd_noalloc.restype = st
    lib.gdr_chunk_bwd.argtypes = [PP, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, S, P]
    lib.gdr_chunk_bwd.restype = st
    lib.gdr_chunk_bwd_gate.argtypes = [PP, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P,
                                       P, S, P]
    lib.gdr_chunk_bwd_gate.restype = st
    lib.gdr_recurrent_fwd.argtypes = [PP, P, P, P, P, P, P, P, P, P]
    lib.gdr_recurrent_fwd.restype = st
    for name in ("gdr_prepare_lens_i32", "gdr_prepare_lens_i64"):
        getattr(lib, name).argtypes = [P, I64, P]
        getattr(lib, name).restype = st
    for name in ("gdr_prepare_chunk_indices_i32", "gdr_prepare_chunk_indices_i64",
                 "gdr_prepare_chunk_offsets_i32", "gdr_prepare_chunk_offsets_i64",
                 "gdr_prepare_chunk_token_starts_i64"):
        getattr(lib, name).argtypes = [P, I64, I64, P, ctypes.POINTER(I64)]
        getattr(lib, name).restype = st


def _declare_profile(lib):
    lib.gdr_profile_enable.argtypes = [ctypes.c_int]
    lib.gdr_profile_enable.restype = ctypes.c_int
    lib.gdr_profile_read.argtypes = [ctypes.c_char_p, ctypes.c_size_t, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_int]
    lib.gdr_profile_read.restype = ctypes.c_int
    lib.gdr_plan_info.argtypes = [ctypes.POINTER(Problem), ctypes.c_int,
                                  ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]
    lib.gdr_plan_info.restype = ctypes.c_int


def _declare_ops(lib):
    P, S, st = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int

    def fn(name, args, res=st):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res

    CP = ctypes.POINTER(ConvProblem)
    fn("gdr_conv1d_check", [CP, ctypes.c_char_p, S])
    fn("gdr_conv1d_fwd", [CP] + [P] * 7)
    fn("gdr_conv1d_bwd_workspace_size", [CP], S)
    fn("gdr_conv1d_bwd", [CP] + [P] * 11 + [S, P])
    fn("gdr_conv1d_update", [CP] + [P] * 6)
    SP = ctypes.POINTER(SsmProblem)
    fn("gdr_ssm_check", [SP, ctypes.c_char_p, S])
    fn("gdr_ssm_fwd_workspace_size", [SP], S)
    fn("gdr_ssm_fwd", [SP] + [P] * 11 + [S, P])
    fn("gdr_ssm_step", [SP] + [P] * 11)
    fn("gdr_ssm_bwd_workspace_size", [SP], S)
    fn("gdr_ssm_bwd", [SP] + [P] * 20 + [S, P])
    NP = ctypes.POINTER(NormProblem)
    fn("gdr_rms_norm_check", [NP, ctypes.c_char_p, S])
    fn("gdr_rms_norm_fwd", [NP] + [P] * 8)
    fn("gdr_rms_norm_bwd_workspace_size", [NP], S)
    fn("gdr_rms_norm_bwd", [NP] + [P] * 9 + [S, P])
    GP = ctypes.POINTER(GatedNormProblem)
    fn("gdr_gated_norm_check", [GP, ctypes.c_char_p, S])
    fn("gdr_gated_norm_fwd", [GP] + [P] * 7)
    fn("gdr_gated_norm_bwd_workspace_size", [GP], S)
    fn("gdr_gated_norm_bwd", [GP] + [P] * 9 + [S, P])
    WP = ctypes.POINTER(SandwichNormProblem)
    fn("gdr_sandwich_norm_check", [WP, ctypes.c_char_p, S])
    fn("gdr_sandwich_norm_fwd", [WP] + [P] * 12)
    fn("gdr_sandwich_norm_bwd_workspace_size", [WP], S)
    fn("gdr_sandwich_norm_bwd", [WP] + [P] * 17 + [S, P])
    QP = ctypes.POINTER(QuantizeProblem)
    fn("gdr_quantize_check", [QP, ctypes.c_char_p, S])
    fn("gdr_quantize_rows", [QP] + [P] * 4)
    MP = ctypes.POINTER(Int8MatmulProblem)
    fn("gdr_int8_matmul_check", [MP, ctypes.c_char_p, S])
    fn("gdr_int8_matmul_workspace_size", [MP], S)
    fn("gdr_int8_matmul", [MP] + [P] * 7 + [S, P])


def load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            "libgdr.so is not built (expected at %s); run gated_delta_rule_66_amd/build.py"
            % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    _declare(lib)
    _declare_profile(lib)
    _declare_ops(lib)
    return lib


lib = load()


def check(status: int):
    if status != 0:
        raise GdrError(status, lib.gdr_last_error().decode(errors="replace"))
