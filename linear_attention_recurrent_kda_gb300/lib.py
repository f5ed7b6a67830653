"""ctypes view of the C ABI in include/kda.h (``libkda_gb300.so``).

Argument marshalling only: every step of the KDA decode/verify path runs in
the CUDA library.  Loading fails loudly when the library is missing; there is
no CPU fallback.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import warnings

from . import build as _build

_P = ctypes.c_void_p

# Return codes and device error flags (include/kda.h).
KDA_SUCCESS = 0
KDA_ERR_NULL_ARGS = 1
KDA_ERR_TOKENS = 2
KDA_ERR_GATE_MODE = 3
KDA_ERR_RECORD = 4
KDA_ERR_NULL_POINTER = 5
KDA_ERR_CONV_WIDTH = 6
KDA_ERR_ALIGNMENT = 7
KDA_ERR_SHAPE = 8
KDA_ERR_DEVICE = 9
KDA_ERR_LAUNCH = 10
KDA_ERR_PATH = 11
KDA_ERR_WORKSPACE = 12
KDA_ERR_ACTIVATION = 13
KDA_PATH_AUTO, KDA_PATH_PERSISTENT, KDA_PATH_SPLIT = 0, 1, 2
KDA_DEVERR_SLOT = 1
KDA_DEVERR_ACCEPTED = 2
KDA_DEVERR_TIMEOUT = 4
KDA_DEVERR_SEQ = 8

EXPORTED = ("kda_decode", "kda_verify", "kda_step_noalloc", "kda_recover", "kda_oproj",
            "kda_lin_prompt_workspace", "kda_lin_prompt", "kda_lin_step",
            "kda_snapshot_save", "kda_snapshot_load",
            "kda_conv_prompt", "kda_conv_step", "kda_ssm_prompt_workspace", "kda_ssm_prompt",
            "kda_ssm_step", "kda_linear", "kda_linear_path",
            "kda_selftest_wait_timeout", "kda_selftest_lin_wait_timeout",
            "kda_strerror", "kda_abi_version")


class KdaArgs(ctypes.Structure):
    """Mirror of ``struct kda_args``."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("heads", ctypes.c_int32),
        ("tokens", ctypes.c_int32), ("num_slots", ctypes.c_int32),
        ("conv_width", ctypes.c_int32), ("slot_cols", ctypes.c_int32),
        ("gate_mode", ctypes.c_int32), ("has_bias", ctypes.c_int32),
        ("record", ctypes.c_int32), ("use_pdl", ctypes.c_int32),
        ("x", _P), ("conv_weight", _P), ("conv_bias", _P), ("f_a", _P),
        ("f_b", _P), ("beta", _P), ("gate", _P), ("norm_weight", _P),
        ("a_log", _P), ("dt_bias", _P), ("slots", _P), ("accepted", _P),
        ("conv_state", _P), ("state", _P), ("output", _P),
        ("rec_u", _P), ("rec_kg", _P),
        ("lower_bound", ctypes.c_float), ("scale", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("err", _P), ("dbg", _P), ("path", ctypes.c_int32),
        ("conv_f32", ctypes.c_int32), ("sched", _P),
    ]


class KdaRecoverArgs(ctypes.Structure):
    """Mirror of ``struct kda_recover_args``."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("heads", ctypes.c_int32),
        ("tokens", ctypes.c_int32), ("num_slots", ctypes.c_int32),
        ("src_slots", _P), ("dst_slots", _P), ("accepted", _P),
        ("rec_u", _P), ("rec_kg", _P), ("a_log", _P), ("dt_bias", _P),
        ("lower_bound", ctypes.c_float), ("state", _P), ("err", _P), ("sched", _P),
    ]


class KdaOprojArgs(ctypes.Structure):
    """Mirror of ``struct kda_oproj_args``."""
    _fields_ = [
        ("tp", ctypes.c_int32), ("tokens", ctypes.c_int32),
        ("hidden", ctypes.c_int32), ("nb", ctypes.c_int32),
        ("has_delta", ctypes.c_int32),
        ("partials", _P), ("blocks", _P), ("norm", _P), ("query", _P),
        ("out_norm", _P), ("prefix", _P), ("output", _P),
        ("eps", ctypes.c_float), ("out_eps", ctypes.c_float),
    ]


class KdaLinPromptArgs(ctypes.Structure):
    """Mirror of ``struct kda_lin_prompt_args``."""
    _fields_ = [
        ("seqs", ctypes.c_int32), ("heads", ctypes.c_int32),
        ("qk_heads", ctypes.c_int32), ("tokens", ctypes.c_int32),
        ("max_seq", ctypes.c_int32), ("num_slots", ctypes.c_int32),
        ("decay_rows", ctypes.c_int32), ("path", ctypes.c_int32),
        ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64), ("o_stride", ctypes.c_int64),
        ("q", _P), ("k", _P), ("v", _P), ("decay", _P), ("seq_starts", _P),
        ("src_slots", _P), ("dst_slots", _P), ("state", _P), ("output", _P),
        ("scale", ctypes.c_float), ("err", _P), ("workspace", _P),
        ("workspace_bytes", ctypes.c_int64),
    ]


class KdaLinStepArgs(ctypes.Structure):
    """Mirror of ``struct kda_lin_step_args``."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("heads", ctypes.c_int32),
        ("qk_heads", ctypes.c_int32), ("num_slots", ctypes.c_int32),
        ("decay_rows", ctypes.c_int32),
        ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64), ("o_stride", ctypes.c_int64),
        ("q", _P), ("k", _P), ("v", _P), ("decay", _P), ("slots", _P),
        ("state", _P), ("output", _P), ("scale", ctypes.c_float), ("err", _P),
    ]


class KdaSnapshotArgs(ctypes.Structure):
    """Mirror of ``struct kda_snapshot_args``."""
    _fields_ = [
        ("count", ctypes.c_int32), ("heads", ctypes.c_int32),
        ("num_slots", ctypes.c_int32), ("num_snaps", ctypes.c_int32),
        ("bits", ctypes.c_int32),
        ("slots", _P), ("snaps", _P), ("state", _P), ("codes", _P), ("scales", _P),
        ("err", _P),
    ]


class KdaConvPromptArgs(ctypes.Structure):
    """Mirror of ``struct kda_conv_prompt_args``."""
    _fields_ = [
        ("seqs", ctypes.c_int32), ("channels", ctypes.c_int32), ("parts", ctypes.c_int32),
        ("taps", ctypes.c_int32), ("tokens", ctypes.c_int32), ("num_slots", ctypes.c_int32),
        ("width", ctypes.c_int32), ("window_f32", ctypes.c_int32), ("silu", ctypes.c_int32),
        ("x_stride", ctypes.c_int64), ("o_stride", ctypes.c_int64),
        ("x", _P), ("weight", _P), ("bias", _P), ("seq_starts", _P), ("src_slots", _P),
        ("dst_slots", _P), ("window", _P), ("output", _P), ("err", _P),
    ]


class KdaConvStepArgs(ctypes.Structure):
    """Mirror of ``struct kda_conv_step_args``."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("channels", ctypes.c_int32), ("parts", ctypes.c_int32),
        ("taps", ctypes.c_int32), ("num_slots", ctypes.c_int32), ("width", ctypes.c_int32),
        ("window_f32", ctypes.c_int32), ("silu", ctypes.c_int32),
        ("x_stride", ctypes.c_int64), ("o_stride", ctypes.c_int64),
        ("x", _P), ("weight", _P), ("bias", _P), ("slots", _P), ("window", _P), ("output", _P),
        ("err", _P),
    ]


class KdaSsmPromptArgs(ctypes.Structure):
    """Mirror of ``struct kda_ssm_prompt_args``."""
    _fields_ = [
        ("seqs", ctypes.c_int32), ("channels", ctypes.c_int32), ("states", ctypes.c_int32),
        ("groups", ctypes.c_int32), ("tokens", ctypes.c_int32), ("max_seq", ctypes.c_int32),
        ("num_slots", ctypes.c_int32), ("softplus", ctypes.c_int32), ("path", ctypes.c_int32),
        ("x_stride", ctypes.c_int64), ("dt_stride", ctypes.c_int64),
        ("b_stride", ctypes.c_int64), ("c_stride", ctypes.c_int64),
        ("z_stride", ctypes.c_int64), ("o_stride", ctypes.c_int64),
        ("x", _P), ("dt", _P), ("a", _P), ("b", _P), ("c", _P), ("d", _P), ("z", _P),
        ("dt_bias", _P), ("seq_starts", _P), ("src_slots", _P), ("dst_slots", _P),
        ("state", _P), ("output", _P), ("err", _P), ("workspace", _P),
        ("workspace_bytes", ctypes.c_int64),
    ]


class KdaSsmStepArgs(ctypes.Structure):
    """Mirror of ``struct kda_ssm_step_args``."""
    _fields_ = [
        ("batch", ctypes.c_int32), ("channels", ctypes.c_int32), ("states", ctypes.c_int32),
        ("groups", ctypes.c_int32), ("num_slots", ctypes.c_int32), ("softplus", ctypes.c_int32),
        ("x_stride", ctypes.c_int64), ("dt_stride", ctypes.c_int64),
        ("b_stride", ctypes.c_int64), ("c_stride", ctypes.c_int64),
        ("z_stride", ctypes.c_int64), ("o_stride", ctypes.c_int64),
        ("x", _P), ("dt", _P), ("a", _P), ("b", _P), ("c", _P), ("d", _P), ("z", _P),
        ("dt_bias", _P), ("slots", _P), ("state", _P), ("output", _P), ("err", _P),
    ]


class KdaLinearArgs(ctypes.Structure):
    """Mirror of ``struct kda_linear_args``."""
    _fields_ = [
        ("rows", ctypes.c_int32), ("inner", ctypes.c_int32), ("outer", ctypes.c_int32),
        ("activation", ctypes.c_int32),
        ("x_stride", ctypes.c_int64), ("w_stride", ctypes.c_int64),
        ("r_stride", ctypes.c_int64), ("o_stride", ctypes.c_int64),
        ("x", _P), ("weight", _P), ("bias", _P), ("residual", _P), ("output", _P), ("err", _P),
    ]


class KdaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"KDA error {code}: {msg}")
        self.code = code


_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load (building first if needed) the CUDA library."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _build.LIB_PATH
    if path is None and not os.path.exists(p):
        _build.build()
    if not os.path.exists(p):
        raise ImportError(f"KDA CUDA library not found at {p}")
    lib = ctypes.CDLL(p)
    for name in ("kda_decode", "kda_verify", "kda_step_noalloc"):
        fn = getattr(lib, name)
        fn.argtypes = [ctypes.POINTER(KdaArgs), ctypes.c_void_p]
        fn.restype = ctypes.c_int
    lib.kda_recover.argtypes = [ctypes.POINTER(KdaRecoverArgs), ctypes.c_void_p]
    lib.kda_recover.restype = ctypes.c_int
    lib.kda_oproj.argtypes = [ctypes.POINTER(KdaOprojArgs), ctypes.c_void_p]
    lib.kda_oproj.restype = ctypes.c_int
    for name, args, res in (("kda_lin_prompt_workspace", [ctypes.POINTER(KdaLinPromptArgs)],
                             ctypes.c_int64),
                            ("kda_lin_prompt", [ctypes.POINTER(KdaLinPromptArgs), _P],
                             ctypes.c_int),
                            ("kda_lin_step", [ctypes.POINTER(KdaLinStepArgs), _P], ctypes.c_int),
                            ("kda_snapshot_save", [ctypes.POINTER(KdaSnapshotArgs), _P],
                             ctypes.c_int),
                            ("kda_snapshot_load", [ctypes.POINTER(KdaSnapshotArgs), _P],
                             ctypes.c_int),
                            ("kda_conv_prompt", [ctypes.POINTER(KdaConvPromptArgs), _P],
                             ctypes.c_int),
                            ("kda_conv_step", [ctypes.POINTER(KdaConvStepArgs), _P],
                             ctypes.c_int),
                            ("kda_ssm_prompt_workspace", [ctypes.POINTER(KdaSsmPromptArgs)],
                             ctypes.c_int64),
                            ("kda_ssm_prompt", [ctypes.POINTER(KdaSsmPromptArgs), _P],
                             ctypes.c_int),
                            ("kda_ssm_step", [ctypes.POINTER(KdaSsmStepArgs), _P], ctypes.c_int),
                            ("kda_linear", [ctypes.POINTER(KdaLinearArgs), _P], ctypes.c_int),
                            ("kda_linear_path", [ctypes.POINTER(KdaLinearArgs), ctypes.c_int32, _P],
                             ctypes.c_int)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res
    for fn in (lib.kda_selftest_wait_timeout, lib.kda_selftest_lin_wait_timeout):
        fn.argtypes, fn.restype = [ctypes.c_void_p, ctypes.c_void_p], ctypes.c_int
    lib.kda_strerror.argtypes = [ctypes.c_int]
    lib.kda_strerror.restype = ctypes.c_char_p
    lib.kda_abi_version.argtypes = []
    lib.kda_abi_version.restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


def strerror(code: int) -> str:
    return load().kda_strerror(int(code)).decode()


def call(entry: str, args, stream_handle: int, *more) -> int:
    """Raw call: returns the library's code without raising (``more``: what an entry takes
    between its struct and its stream)."""
    return getattr(_lib or load(), entry)(args, *more, stream_handle or None)


_bind = None


class _General:
    """In the binding's place where there is none: leaves every call to the general checks."""

    @staticmethod
    def _leave(*args):
        return None

    conv_prompt = ssm_prompt = linear = _leave


def _load_bind():
    path = _build.BIND_PATH
    if path is None:
        raise ImportError("PyTorch's version is not known")
    if not os.path.exists(path):
        _build.build()
    loader = importlib.machinery.ExtensionFileLoader("kda_bind", path)
    module = importlib.util.module_from_spec(
        importlib.util.spec_from_file_location("kda_bind", path, loader=loader))
    loader.exec_module(module)
    return module


def bind():
    """The short way to kda_conv_prompt, kda_ssm_prompt and kda_linear (building first if
    needed): functions that launch and return the library's code, or return None for
    what they leave to the general checks.  Where the binding cannot be built or loaded
    they leave everything, after a warning."""
    global _bind
    if _bind is None:
        lib = load()
        try:
            module = _load_bind()
        except (ImportError, OSError) as e:
            warnings.warn(f"no short way from Python, calls take the general one: {e}", RuntimeWarning,
                          stacklevel=3)
            module = _General()
        else:
            module.setup(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in (
                "kda_conv_prompt", "kda_ssm_prompt_workspace", "kda_ssm_prompt", "kda_linear")))
        _bind = module
    return _bind


def prompt_workspace(args) -> int:
    """Bytes of workspace that ``kda_lin_prompt`` needs for these sizes."""
    return (_lib or load()).kda_lin_prompt_workspace(args)


def ssm_workspace(args) -> int:
    """Bytes of workspace that ``kda_ssm_prompt`` needs for these sizes."""
    return (_lib or load()).kda_ssm_prompt_workspace(args)
