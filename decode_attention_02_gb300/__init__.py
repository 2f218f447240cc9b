"""MFA decode attention for GB300 (sm_103a).

Thin ctypes binding over ``libmfa.so`` (CUDA kernels + C ABI, see include/mfa.h).
Every step of the decode runs in the library's kernels; this module only
marshals arguments.  PyTorch supplies device memory and the current stream.

The operation is Step-3's MFA decode step (paperlayer.ai/abs/2507.19427v1,
section 2 "Step-3 Model Card" and section 5 "Model-System Co-design"): 64 query
heads of width 256 over one shared K head and one shared V head held in a paged
KV cache of 64-token pages, out = softmax(q K^T * scale) V and its log-sum-exp.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmfa.so")

MFA_OK = 0
MFA_ERR_INVALID_ARG = 1
MFA_ERR_UNSUPPORTED = 2
MFA_ERR_WORKSPACE = 3
MFA_ERR_CUDA = 4
MFA_ERR_DEVICE_CHECK = 5

MFA_KV_BF16 = 0
MFA_KV_FP8_E4M3 = 1
MFA_KV_MXFP4 = 2
# the cache formats by the names the input generator uses
KV_DTYPES = {"bf16": MFA_KV_BF16, "fp8_e4m3": MFA_KV_FP8_E4M3, "mxfp4": MFA_KV_MXFP4}

MFA_OUT_BF16 = 0
MFA_OUT_FP32 = 1

MFA_DEV_TIMEOUT = 0x1
MFA_DEV_BAD_BLOCK = 0x2
MFA_DEV_BAD_LENGTH = 0x4
MFA_DEV_SCHEDULE = 0x8
MFA_DEV_RANGE = 0x10

MFA_PLAN_CHECK = 0x1
MFA_PLAN_NO_COMBINE = 0x2
MFA_PLAN_EARLY_METADATA = 0x4
MFA_PLAN_EVEN_SPLIT = 0x100      # set by mfa_block_decode_plan alone
MFA_PLAN_UNIT_CLUSTERS = 0x200   # likewise
MFA_PLAN_WINDOW = 0x400          # set by mfa_window_decode_plan alone
MFA_PLAN_TREE = 0x800            # set by mfa_tree_decode_plan alone

MFA_ROPE_HALF = 0
MFA_ROPE_ADJACENT = 1
MFA_ROPE_MAX_AXES = 4
MFA_ROPE_INTERLEAVED = 0x1
MFA_ROPE_OWN_SPECTRUM = 0x2
MFA_NORM_ROPE_GRAD_PARTS = 512

MFA_TREE_MAX_NODES = 64

NUM_Q_HEADS = 64
HEAD_DIM = 256
PAGE_SIZE = 64

# Every symbol include/mfa.h declares.
EXPORTED_SYMBOLS = ("mfa_decode_plan", "mfa_decode_run", "mfa_combine", "mfa_read_device_status",
                    "mfa_status_string", "mfa_abi_version", "mfa_last_cuda_error",
                    "mfa_decode_run_static_workspace", "mfa_kv_append", "mfa_decode_run_host",
                    "mfa_decode_append_run", "mfa_block_decode_plan", "mfa_block_decode_run", "mfa_block_kv_append",
                    "mfa_window_decode_plan", "mfa_window_decode_run", "mfa_tree_decode_plan", "mfa_tree_decode_run",
                    "mfa_rope_table", "mfa_rope_run", "mfa_norm_rope_run", "mfa_norm_rope_grad_run")

# Size of the library's own scratch array used by mfa_decode_run_static_workspace.
MFA_STATIC_WORKSPACE_BYTES = 24 * 1024 * 1024


class MfaProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
                ("out_dtype", ctypes.c_int32), ("tokens_per_seq", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("kv_shared", ctypes.c_int32)]


class MfaPlan(ctypes.Structure):
    _fields_ = [("num_ctas", ctypes.c_int32), ("tile_tokens", ctypes.c_int32),
                ("max_tiles_per_cta", ctypes.c_int32), ("num_partials", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("num_sms", ctypes.c_int32),
                ("total_tiles", ctypes.c_uint64), ("workspace_bytes", ctypes.c_uint64),
                ("tokens_per_seq", ctypes.c_int32)]


class MfaWindow(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("sinks", ctypes.c_int32)]


class MfaRopeConfig(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("sections", ctypes.c_int32 * MFA_ROPE_MAX_AXES), ("pairing", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("theta", ctypes.c_double), ("position_scale", ctypes.c_double)]


class MfaRopePair(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_uint64), ("axis", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MfaRopeRows(ctypes.Structure):
    _fields_ = [("data_in", ctypes.c_void_p), ("data_out", ctypes.c_void_p), ("in_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64), ("heads", ctypes.c_int32)]


class MfaNorm(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("weight_dtype", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class MfaNormGradRows(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("dy", ctypes.c_void_p), ("dx", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
                ("dy_stride", ctypes.c_int64), ("dx_stride", ctypes.c_int64), ("heads", ctypes.c_int32)]


class MfaError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = f"{where}: {status_string(status)} (status {status})"
        if status == MFA_ERR_CUDA and _lib is not None:
            msg += ": " + _lib.mfa_last_cuda_error().decode()
        super().__init__(msg)
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libmfa.so; raises if it has not been built (no fallback path exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with decode_attention_02_gb300.build.build_library()")
    lib = ctypes.CDLL(path)
    P = ctypes.c_void_p
    lib.mfa_decode_plan.argtypes = [ctypes.POINTER(MfaProblem), P, ctypes.c_int32, ctypes.c_int32,
                                    ctypes.c_int32, ctypes.c_uint32, ctypes.POINTER(MfaPlan)]
    lib.mfa_decode_plan.restype = ctypes.c_int
    lib.mfa_decode_run.argtypes = [ctypes.POINTER(MfaPlan), ctypes.POINTER(MfaProblem), P, P, P, P, P, P, P,
                                   P, P, P, ctypes.c_uint64, P]
    lib.mfa_decode_run.restype = ctypes.c_int
    lib.mfa_combine.argtypes = [ctypes.POINTER(MfaPlan), ctypes.POINTER(MfaProblem), P, ctypes.c_uint64, P, P,
                                P, P]
    lib.mfa_combine.restype = ctypes.c_int
    lib.mfa_read_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_uint32), ctypes.c_int32, P]
    lib.mfa_read_device_status.restype = ctypes.c_int
    lib.mfa_status_string.argtypes = [ctypes.c_int]
    lib.mfa_status_string.restype = ctypes.c_char_p
    lib.mfa_abi_version.argtypes = []
    lib.mfa_abi_version.restype = ctypes.c_int32
    lib.mfa_last_cuda_error.argtypes = []
    lib.mfa_last_cuda_error.restype = ctypes.c_char_p
    lib.mfa_decode_run_static_workspace.argtypes = [ctypes.POINTER(MfaPlan), ctypes.POINTER(MfaProblem), P, P, P,
                                                    P, P, P, P, P, P, P]
    lib.mfa_decode_run_static_workspace.restype = ctypes.c_int
    lib.mfa_kv_append.argtypes = [ctypes.POINTER(MfaProblem), P, P, P, P, P, P, P, P, P, P]
    lib.mfa_kv_append.restype = ctypes.c_int
    lib.mfa_decode_run_host.argtypes = [ctypes.POINTER(MfaPlan), ctypes.POINTER(MfaProblem), P, P, P, P, P,
                                        P, P, P, P, P, P, P, P, P, P, ctypes.c_uint64, P]
    lib.mfa_decode_run_host.restype = ctypes.c_int
    lib.mfa_decode_append_run.argtypes = [ctypes.POINTER(MfaPlan), ctypes.POINTER(MfaProblem), P, P, P, P, P, P, P,
                                          P, P, P, P, P, P, ctypes.c_uint64, P]
    lib.mfa_decode_append_run.restype = ctypes.c_int
    lib.mfa_block_decode_plan.argtypes = [ctypes.POINTER(MfaProblem), ctypes.c_int32, P, ctypes.c_int32,
                                          ctypes.c_int32, ctypes.c_int32, ctypes.c_uint32, ctypes.POINTER(MfaPlan)]
    lib.mfa_block_decode_plan.restype = ctypes.c_int
    lib.mfa_block_decode_run.argtypes = [ctypes.POINTER(MfaPlan), ctypes.POINTER(MfaProblem), ctypes.c_int32, P, P, P,
                                         P, P, P, P, P, P, P, ctypes.c_uint64, P]
    lib.mfa_block_decode_run.restype = ctypes.c_int
    lib.mfa_window_decode_plan.argtypes = [ctypes.POINTER(MfaProblem), ctypes.c_int32, ctypes.POINTER(MfaWindow), P,
                                           ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_uint32,
                                           ctypes.POINTER(MfaPlan)]
    lib.mfa_window_decode_plan.restype = ctypes.c_int
    lib.mfa_window_decode_run.argtypes = [ctypes.POINTER(MfaPlan), ctypes.POINTER(MfaProblem), ctypes.c_int32,
                                          ctypes.POINTER(MfaWindow), P, P, P, P, P, P, P, P, P, P, ctypes.c_uint64, P]
    lib.mfa_window_decode_run.restype = ctypes.c_int
    lib.mfa_tree_decode_plan.argtypes = lib.mfa_block_decode_plan.argtypes
    lib.mfa_tree_decode_plan.restype = ctypes.c_int
    lib.mfa_tree_decode_run.argtypes = [ctypes.POINTER(MfaPlan), ctypes.POINTER(MfaProblem), ctypes.c_int32, P, P, P, P, P,
                                        P, P, P, P, P, P, ctypes.c_uint64, P]
    lib.mfa_tree_decode_run.restype = ctypes.c_int
    lib.mfa_block_kv_append.argtypes = [ctypes.POINTER(MfaProblem), ctypes.c_int32, P, P, ctypes.c_int32, P,
                                        ctypes.c_int32, P, P, P, P, P, P, P, P]
    lib.mfa_block_kv_append.restype = ctypes.c_int
    lib.mfa_rope_table.argtypes = [ctypes.POINTER(MfaRopeConfig), P]
    lib.mfa_rope_table.restype = ctypes.c_int
    lib.mfa_rope_run.argtypes = [ctypes.POINTER(MfaRopeConfig), P, P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                 ctypes.POINTER(MfaRopeRows), ctypes.POINTER(MfaRopeRows), P]
    lib.mfa_rope_run.restype = ctypes.c_int
    lib.mfa_norm_rope_run.argtypes = [ctypes.POINTER(MfaRopeConfig), P, P, ctypes.c_int32, ctypes.c_int32,
                                      ctypes.POINTER(MfaNorm), ctypes.POINTER(MfaRopeRows), ctypes.POINTER(MfaRopeRows), P]
    lib.mfa_norm_rope_run.restype = ctypes.c_int
    lib.mfa_norm_rope_grad_run.argtypes = [ctypes.POINTER(MfaRopeConfig), P, P, ctypes.c_int32, ctypes.c_int32,
                                           ctypes.POINTER(MfaNorm), ctypes.POINTER(MfaNormGradRows),
                                           ctypes.POINTER(MfaNormGradRows), P, P, P, ctypes.c_uint64, P]
    lib.mfa_norm_rope_grad_run.restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load_library().mfa_status_string(int(status)).decode()
    except ImportError:
        return "library not loaded"


def _check(status: int, where: str):
    if status != MFA_OK:
        raise MfaError(status, where)


def _ptr(x) -> Optional[int]:
    """Device pointer of a torch tensor (must be CUDA and contiguous), an int, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not x.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return x.data_ptr()


def _nbytes(x) -> int:
    return x.numel() * x.element_size()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# The attention shapes the library runs: (num_q_heads, head_dim, num_kv_heads, kv_shared).
SHAPE_MFA = (64, 256, 1, False)     # Step-3's MFA: one shared K head and one shared V head
SHAPE_GQA = (64, 128, 4, False)     # grouped-query attention: 4 key/value heads of 128
SHAPE_MLA = (128, 512, 1, True)     # one 512-wide latent that is both key and value


def make_problem(batch: int, max_pages_per_seq: int, num_blocks: int, kv_dtype: int = MFA_KV_BF16,
                 softmax_scale: Optional[float] = None, num_q_heads: int = NUM_Q_HEADS,
                 head_dim: int = HEAD_DIM, page_size: int = PAGE_SIZE, out_dtype: int = MFA_OUT_BF16,
                 tokens_per_seq: int = 1, num_kv_heads: int = 1, kv_shared: bool = False) -> MfaProblem:
    if softmax_scale is None:
        softmax_scale = head_dim ** -0.5
    return MfaProblem(batch, num_q_heads, head_dim, page_size, max_pages_per_seq, num_blocks, kv_dtype,
                      softmax_scale, out_dtype, tokens_per_seq, num_kv_heads, 1 if kv_shared else 0)


def mfa_decode_plan(problem: MfaProblem, host_seq_lens: Optional[Sequence[int]] = None, max_seq_len: int = 0,
                    num_sms: int = 0, force_ctas: int = 0, flags: int = 0) -> MfaPlan:
    lib = load_library()
    plan = MfaPlan()
    lens_arr = None
    if host_seq_lens is not None:
        vals = [int(v) for v in host_seq_lens]
        lens_arr = (ctypes.c_int32 * max(1, len(vals)))(*vals)
    st = lib.mfa_decode_plan(ctypes.byref(problem), lens_arr, int(max_seq_len), int(num_sms), int(force_ctas),
                             int(flags), ctypes.byref(plan))
    _check(st, "mfa_decode_plan")
    return plan


def mfa_decode_run(plan: MfaPlan, problem: MfaProblem, q, k_cache, v_cache, k_scale, v_scale, block_table,
                   seq_lens, out, lse, workspace, stream=None, workspace_bytes: Optional[int] = None) -> None:
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    st = lib.mfa_decode_run(ctypes.byref(plan), ctypes.byref(problem), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                            _ptr(k_scale), _ptr(v_scale), _ptr(block_table), _ptr(seq_lens), _ptr(out),
                            _ptr(lse), _ptr(workspace), int(workspace_bytes), _stream(stream))
    _check(st, "mfa_decode_run")


def mfa_decode_append_run(plan: MfaPlan, problem: MfaProblem, q, k_cache, v_cache, k_scale, v_scale, block_table,
                          seq_lens, k_new, v_new, positions, out, lse, workspace, stream=None,
                          workspace_bytes: Optional[int] = None) -> None:
    """mfa_kv_append then mfa_decode_run in one call (one kernel for one new token per sequence)."""
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    st = lib.mfa_decode_append_run(ctypes.byref(plan), ctypes.byref(problem), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                   _ptr(k_scale), _ptr(v_scale), _ptr(block_table), _ptr(seq_lens), _ptr(k_new),
                                   _ptr(v_new), _ptr(positions), _ptr(out), _ptr(lse), _ptr(workspace),
                                   int(workspace_bytes), _stream(stream))
    _check(st, "mfa_decode_append_run")


def mfa_decode_run_static_workspace(plan: MfaPlan, problem: MfaProblem, q, k_cache, v_cache, k_scale, v_scale,
                                    block_table, seq_lens, out, lse, stream=None) -> None:
    """mfa_decode_run with the library's own fixed scratch array instead of a workspace.

    For callers that must not allocate device memory; see include/mfa.h for the
    size limit and the rule that calls sharing a device must not overlap.
    """
    lib = load_library()
    st = lib.mfa_decode_run_static_workspace(ctypes.byref(plan), ctypes.byref(problem), _ptr(q), _ptr(k_cache),
                                             _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(block_table),
                                             _ptr(seq_lens), _ptr(out), _ptr(lse), _stream(stream))
    _check(st, "mfa_decode_run_static_workspace")


def _host_ptr(x) -> Optional[int]:
    """Address of a CPU torch tensor (contiguous), an int, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if x.is_cuda:
        raise ValueError("expected a CPU (pinned) tensor")
    if not x.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return x.data_ptr()


def mfa_decode_run_host(plan: MfaPlan, problem: MfaProblem, q_host, block_table_host, seq_lens_host, out_host,
                        lse_host, q_dev, block_table_dev, seq_lens_dev, out_dev, lse_dev, k_cache, v_cache, k_scale,
                        v_scale, workspace, stream=None, workspace_bytes: Optional[int] = None) -> None:
    """One decode step from host buffers (copies in, decode, copies out on one stream)."""
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    st = lib.mfa_decode_run_host(ctypes.byref(plan), ctypes.byref(problem), _host_ptr(q_host),
                                 _host_ptr(block_table_host), _host_ptr(seq_lens_host), _host_ptr(out_host),
                                 _host_ptr(lse_host), _ptr(q_dev), _ptr(block_table_dev), _ptr(seq_lens_dev),
                                 _ptr(out_dev), _ptr(lse_dev), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                                 _ptr(v_scale), _ptr(workspace), int(workspace_bytes), _stream(stream))
    _check(st, "mfa_decode_run_host")


def mfa_combine(plan: MfaPlan, problem: MfaProblem, workspace, seq_lens, out, lse, stream=None,
                workspace_bytes: Optional[int] = None) -> None:
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    st = lib.mfa_combine(ctypes.byref(plan), ctypes.byref(problem), _ptr(workspace), int(workspace_bytes),
                         _ptr(seq_lens), _ptr(out), _ptr(lse), _stream(stream))
    _check(st, "mfa_combine")


def mfa_kv_append(problem: MfaProblem, k_new, v_new, positions, block_table, k_cache, v_cache, k_scale=None,
                  v_scale=None, device_status=None, stream=None) -> None:
    """Write each sequence's new key/value row into the paged cache (FP8: quantised).

    k_new/v_new: bf16 [B*T, 256] (T = problem.tokens_per_seq new rows per sequence);
    positions: int32 [B] (index of each sequence's first new row, < 0 = none);
    device_status: a uint32 device tensor (or a decode workspace, whose first word is
    the status word) that collects bad-position / bad-page bits, or None.
    """
    lib = load_library()
    st = lib.mfa_kv_append(ctypes.byref(problem), _ptr(k_new), _ptr(v_new), _ptr(positions), _ptr(block_table),
                           _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(device_status),
                           _stream(stream))
    _check(st, "mfa_kv_append")


def _host_lengths(problem: MfaProblem, host_seq_lens: Optional[Sequence[int]]):
    """The lengths as the library takes them, one for each sequence (None: none)."""
    if host_seq_lens is None:
        return None
    vals = [int(v) for v in host_seq_lens]
    if len(vals) != problem.batch:
        raise ValueError(f"host_seq_lens holds {len(vals)} lengths, the batch is {problem.batch}")
    return (ctypes.c_int32 * max(1, len(vals)))(*vals)


def mfa_block_decode_plan(problem: MfaProblem, scale_tokens: int, host_seq_lens: Optional[Sequence[int]] = None,
                          max_seq_len: int = 0, num_sms: int = 0, force_ctas: int = 0, flags: int = 0) -> MfaPlan:
    """Split the work of mfa_block_decode_run (host only); see include/mfa.h."""
    lib = load_library()
    plan = MfaPlan()
    lens_arr = _host_lengths(problem, host_seq_lens)
    st = lib.mfa_block_decode_plan(ctypes.byref(problem), int(scale_tokens), lens_arr, int(max_seq_len), int(num_sms),
                                   int(force_ctas), int(flags), ctypes.byref(plan))
    _check(st, "mfa_block_decode_plan")
    return plan


def mfa_block_decode_run(plan: MfaPlan, problem: MfaProblem, scale_tokens: int, q, k_cache, v_cache, k_scale, v_scale,
                         block_table, seq_lens, out, lse, workspace, stream=None,
                         workspace_bytes: Optional[int] = None) -> None:
    """One decode step over a block-scaled 8-bit cache (see include/mfa.h)."""
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    st = lib.mfa_block_decode_run(ctypes.byref(plan), ctypes.byref(problem), scale_tokens, _ptr(q), _ptr(k_cache),
                                  _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(block_table), _ptr(seq_lens),
                                  _ptr(out), _ptr(lse), _ptr(workspace), int(workspace_bytes), _stream(stream))
    _check(st, "mfa_block_decode_run")


def mfa_window_decode_plan(problem: MfaProblem, scale_tokens: int, window: MfaWindow,
                           host_seq_lens: Optional[Sequence[int]] = None, max_seq_len: int = 0, num_sms: int = 0,
                           force_ctas: int = 0, flags: int = 0) -> MfaPlan:
    """Split the work of mfa_window_decode_run (host only); see include/mfa.h."""
    lib = load_library()
    plan = MfaPlan()
    lens_arr = _host_lengths(problem, host_seq_lens)
    st = lib.mfa_window_decode_plan(ctypes.byref(problem), int(scale_tokens), ctypes.byref(window), lens_arr,
                                    int(max_seq_len), int(num_sms), int(force_ctas), int(flags), ctypes.byref(plan))
    _check(st, "mfa_window_decode_plan")
    return plan


def mfa_window_decode_run(plan: MfaPlan, problem: MfaProblem, scale_tokens: int, window: MfaWindow, q, k_cache, v_cache,
                          k_scale, v_scale, block_table, seq_lens, out, lse, workspace, stream=None,
                          workspace_bytes: Optional[int] = None) -> None:
    """One decode step over the window and the first tokens of a block-scaled 8-bit cache (see include/mfa.h)."""
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    st = lib.mfa_window_decode_run(ctypes.byref(plan), ctypes.byref(problem), scale_tokens, ctypes.byref(window), _ptr(q),
                                   _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(block_table),
                                   _ptr(seq_lens), _ptr(out), _ptr(lse), _ptr(workspace), int(workspace_bytes),
                                   _stream(stream))
    _check(st, "mfa_window_decode_run")


def mfa_tree_decode_plan(problem: MfaProblem, scale_tokens: int, host_seq_lens: Optional[Sequence[int]] = None,
                         max_seq_len: int = 0, num_sms: int = 0, force_ctas: int = 0, flags: int = 0) -> MfaPlan:
    """Split the work of mfa_tree_decode_run (host only); see include/mfa.h."""
    lib = load_library()
    plan = MfaPlan()
    lens_arr = _host_lengths(problem, host_seq_lens)
    st = lib.mfa_tree_decode_plan(ctypes.byref(problem), int(scale_tokens), lens_arr, int(max_seq_len), int(num_sms),
                                  int(force_ctas), int(flags), ctypes.byref(plan))
    _check(st, "mfa_tree_decode_plan")
    return plan


def mfa_tree_decode_run(plan: MfaPlan, problem: MfaProblem, scale_tokens: int, q, k_cache, v_cache, k_scale, v_scale,
                        block_table, seq_lens, tree, out, lse, workspace, stream=None,
                        workspace_bytes: Optional[int] = None) -> None:
    """Attention of a tree of drafted tokens over a block-scaled 8-bit cache (see include/mfa.h)."""
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = _nbytes(workspace)
    st = lib.mfa_tree_decode_run(ctypes.byref(plan), ctypes.byref(problem), scale_tokens, _ptr(q), _ptr(k_cache),
                                 _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(block_table), _ptr(seq_lens), _ptr(tree),
                                 _ptr(out), _ptr(lse), _ptr(workspace), int(workspace_bytes), _stream(stream))
    _check(st, "mfa_tree_decode_run")


def mfa_block_kv_append(problem: MfaProblem, scale_tokens: int, k_new, v_new, num_new: int, new_offsets, max_new: int,
                        positions, block_table, k_cache, v_cache, k_scale, v_scale, device_status=None,
                        stream=None) -> None:
    """Quantise new key/value rows into a block-scaled 8-bit cache (see include/mfa.h)."""
    lib = load_library()
    st = lib.mfa_block_kv_append(ctypes.byref(problem), scale_tokens, _ptr(k_new), _ptr(v_new), num_new,
                                 _ptr(new_offsets), max_new, _ptr(positions), _ptr(block_table), _ptr(k_cache),
                                 _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(device_status), _stream(stream))
    _check(st, "mfa_block_kv_append")


def mfa_rope_table(config: MfaRopeConfig):
    """The table of ``config``'s rotary pairs as a host array (rotary_dim / 2 entries)."""
    lib = load_library()
    table = (MfaRopePair * max(1, config.rotary_dim // 2))()
    _check(lib.mfa_rope_table(ctypes.byref(config), ctypes.cast(table, ctypes.c_void_p)), "mfa_rope_table")
    return table


def mfa_rope_run(config: MfaRopeConfig, table, positions, num_rows: int, dtype: int, inverse: int,
                 q: Optional[MfaRopeRows], k: Optional[MfaRopeRows], stream=None) -> None:
    """Turn query and key rows by their positions (see include/mfa.h)."""
    lib = load_library()
    st = lib.mfa_rope_run(ctypes.byref(config), _ptr(table), _ptr(positions), num_rows, dtype, inverse,
                          None if q is None else ctypes.byref(q), None if k is None else ctypes.byref(k),
                          _stream(stream))
    _check(st, "mfa_rope_run")


def mfa_norm_rope_run(config: MfaRopeConfig, table, positions, num_rows: int, dtype: int, norm: MfaNorm,
                      q: Optional[MfaRopeRows], k: Optional[MfaRopeRows], stream=None) -> None:
    """Norm each head's rows, weigh and turn them (see include/mfa.h)."""
    lib = load_library()
    st = lib.mfa_norm_rope_run(ctypes.byref(config), _ptr(table), _ptr(positions), num_rows, dtype, ctypes.byref(norm),
                               None if q is None else ctypes.byref(q), None if k is None else ctypes.byref(k),
                               _stream(stream))
    _check(st, "mfa_norm_rope_run")


def mfa_norm_rope_grad_run(config: MfaRopeConfig, table, positions, num_rows: int, dtype: int, norm: MfaNorm,
                           q: Optional[MfaNormGradRows], k: Optional[MfaNormGradRows], q_weight_grad, k_weight_grad,
                           workspace, stream=None, workspace_bytes: Optional[int] = None) -> None:
    """The gradient of mfa_norm_rope_run (see include/mfa.h)."""
    lib = load_library()
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else _nbytes(workspace)
    st = lib.mfa_norm_rope_grad_run(ctypes.byref(config), _ptr(table), _ptr(positions), num_rows, dtype, ctypes.byref(norm),
                                    None if q is None else ctypes.byref(q), None if k is None else ctypes.byref(k),
                                    _ptr(q_weight_grad), _ptr(k_weight_grad), _ptr(workspace), int(workspace_bytes),
                                    _stream(stream))
    _check(st, "mfa_norm_rope_grad_run")


def mfa_read_device_status(workspace, clear: bool = True, stream=None) -> int:
    lib = load_library()
    word = ctypes.c_uint32(0)
    st = lib.mfa_read_device_status(_ptr(workspace), ctypes.byref(word), 1 if clear else 0, _stream(stream))
    _check(st, "mfa_read_device_status")
    return int(word.value)


def workspace_layout(plan: MfaPlan, head_dim: int = HEAD_DIM):
    """Byte offsets of (partial O, partial lse) inside the workspace (see include/mfa.h)."""
    o_off = 256
    lse_off = (o_off + plan.num_partials * NUM_Q_HEADS * head_dim * 4 + 255) // 256 * 256
    return o_off, lse_off


class Decoder:
    """Plan + workspace for one batch shape; ``__call__`` enqueues a decode step.

    Device buffers come from PyTorch's allocator; the step itself is
    ``mfa_decode_run`` (decode kernel + combine kernel).
    """

    def __init__(self, batch: int, max_pages_per_seq: int, num_blocks: int, kv_dtype: int = MFA_KV_BF16,
                 softmax_scale: Optional[float] = None, host_seq_lens=None, max_seq_len: int = 0,
                 force_ctas: int = 0, flags: int = 0, device=None, out_dtype: int = MFA_OUT_BF16,
                 tokens_per_seq: int = 1, shape=SHAPE_MFA):
        import torch
        H, d, G, shared = shape
        self.problem = make_problem(batch, max_pages_per_seq, num_blocks, kv_dtype, softmax_scale,
                                    num_q_heads=H, head_dim=d, out_dtype=out_dtype, tokens_per_seq=tokens_per_seq,
                                    num_kv_heads=G, kv_shared=shared)
        if host_seq_lens is None and max_seq_len == 0:
            max_seq_len = max_pages_per_seq * PAGE_SIZE
        self.plan = mfa_decode_plan(self.problem, host_seq_lens, max_seq_len, 0, force_ctas, flags)
        self.device = torch.device("cuda") if device is None else torch.device(device)
        self.workspace = torch.zeros(int(self.plan.workspace_bytes), dtype=torch.uint8, device=self.device)

    def __call__(self, q, k_cache, v_cache, block_table, seq_lens, k_scale=None, v_scale=None, out=None,
                 lse=None, stream=None):
        import torch
        pr = self.problem
        rows = pr.batch * pr.tokens_per_seq   # (sequence, new token) pairs
        if out is None:
            dt = torch.float32 if pr.out_dtype == MFA_OUT_FP32 else torch.bfloat16
            out = torch.empty((rows, pr.num_q_heads, pr.head_dim), dtype=dt, device=q.device)
        if lse is None:
            lse = torch.empty((rows, pr.num_q_heads), dtype=torch.float32, device=q.device)
        mfa_decode_run(self.plan, self.problem, q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
                       out, lse, self.workspace, stream)
        return out, lse

    def run_host(self, q_host, block_table_host, seq_lens_host, out_host, lse_host, k_cache, v_cache, k_scale=None,
                 v_scale=None, stream=None):
        """One step from pinned host buffers into pinned host outputs (mfa_decode_run_host),
        on device staging buffers this decoder owns.  Asynchronous on ``stream``."""
        import torch
        if not hasattr(self, "_staging"):
            dev = self.device
            pr = self.problem
            B = pr.batch
            rows = B * pr.tokens_per_seq
            odt = torch.float32 if pr.out_dtype == MFA_OUT_FP32 else torch.bfloat16
            self._staging = dict(
                q=torch.empty((rows, pr.num_q_heads, pr.head_dim), dtype=torch.bfloat16, device=dev),
                table=torch.empty((B, pr.max_pages_per_seq), dtype=torch.int32, device=dev),
                lens=torch.empty((B,), dtype=torch.int32, device=dev),
                out=torch.empty((rows, pr.num_q_heads, pr.head_dim), dtype=odt, device=dev),
                lse=torch.empty((rows, pr.num_q_heads), dtype=torch.float32, device=dev))
        st = self._staging
        mfa_decode_run_host(self.plan, self.problem, q_host, block_table_host, seq_lens_host, out_host, lse_host,
                            st["q"], st["table"], st["lens"], st["out"], None if lse_host is None else st["lse"],
                            k_cache, v_cache, k_scale, v_scale, self.workspace, stream)


def _fits(x, dtype, shape, index: int) -> bool:
    """x is a contiguous tensor of this dtype and shape on CUDA device ``index``."""
    return x.dtype is dtype and x.shape == shape and x.get_device() == index and x.is_contiguous()


def _refuse(index: int, *wanted) -> None:
    """Raise for the first (name, tensor, dtype, shape) that _fits does not hold for."""
    for name, x, dtype, shape in wanted:
        if not _fits(x, dtype, shape, index):
            raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}, got "
                             f"{x.dtype} {tuple(x.shape)} strides {x.stride()} on {x.device}")


class _OnDevice:
    """The device that a handle's buffers live on; a call makes it current where another one is."""

    def __init__(self, device):
        import torch
        self.device = torch.device("cuda") if device is None else torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("expected a CUDA device")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._torch, self._index, self._lib = torch, self.device.index, load_library()
        # the current stream's handle without a Stream object around it, where torch has that
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self._current = raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)
        self._home = self._current(self._index)   # the stream that the handle's own buffers are allocated on

    def _stream(self, stream):
        """A torch stream of a stream or its handle."""
        cuda = self._torch.cuda
        if isinstance(stream, int):   # (0 and 1 both name the default stream)
            return cuda.ExternalStream(stream, device=self.device) if stream > 1 else cuda.default_stream(self.device)
        return stream

    def _new(self, shape, dtype, stream):
        """Memory that a call on ``stream`` writes.  (Of that stream's: what the current stream has freed may still be
        written by its work.  The caller may use and drop it on the current stream.)"""
        torch = self._torch
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self._stream(stream)):
            x = torch.empty(shape, dtype=dtype, device=self.device)
        x.record_stream(torch.cuda.current_stream(self._index))
        return x

    def _keep(self, stream, tensors) -> None:
        """Memory that a call on ``stream`` uses: not given out again before that is done."""
        stream = self._stream(stream)
        for x in tensors:
            if x is not None:
                x.record_stream(stream)

    def _call(self, function, where: str, args, stream, own=(), used=()) -> None:
        """One library call on ``stream`` (None: the device's current stream), with the handle's ``own`` tensors
        and the call's: those stay until it is done, on whichever stream they were allocated.  (On the current
        stream the call's tensors do without that, as for any call of torch's.)"""
        index = self._index
        if stream is None:
            handle = self._current(index)
        else:
            handle = stream if isinstance(stream, int) else stream.cuda_stream
        if self._torch.cuda.current_device() == index:
            status = function(*args, handle)
        else:
            with self._torch.cuda.device(index):
                status = function(*args, handle)
        if stream is not None:
            self._keep(stream, (*own, *used))
        elif handle != self._home:
            self._keep(self._torch.cuda.current_stream(index), own)
        if status != MFA_OK:
            raise MfaError(status, where)


class BlockDecoder(_OnDevice):
    """Decode and append over a block-scaled 8-bit cache: plan and workspace for one batch shape.

    The cache: ``k_cache``, ``v_cache`` uint8 [num_blocks, num_kv_heads, 64, head_dim] (e4m3
    codes), ``k_scale``, ``v_scale`` fp32 [num_blocks, num_kv_heads, 64 // scale_tokens];
    ``block_table`` int32 [batch, max_pages_per_seq].  Device buffers come from PyTorch's
    allocator.  Calls that may overlap on the GPU need a decoder (a workspace) each.  A call runs on
    ``stream`` (a torch stream or its handle; None: the current one), and so must what made its
    inputs, or be waited for by it.  What it uses stays allocated until it is done: the decoder's
    workspace always, the tensors of a call with ``stream`` too.  A captured call's decoder and
    tensors have to outlive the graph.

    ``window``: a new token sees only itself, the ``window - 1`` tokens before it and the sequence's first
    ``sinks`` tokens; the pages between are not read.  (None: all tokens before it.)
    """

    def __init__(self, batch: int, max_pages_per_seq: int, num_blocks: int, num_q_heads: int = NUM_Q_HEADS,
                 num_kv_heads: int = 1, head_dim: int = HEAD_DIM, scale_tokens: int = 64,
                 softmax_scale: Optional[float] = None, host_seq_lens=None, max_seq_len: int = 0, force_ctas: int = 0,
                 flags: int = 0, device=None, out_dtype: int = MFA_OUT_BF16, tokens_per_seq: int = 1,
                 window: Optional[int] = None, sinks: int = 0):
        super().__init__(device)
        torch = self._torch
        self.scale_tokens = int(scale_tokens)
        if window is None and sinks:
            raise ValueError("sinks: first tokens stay visible beside a window, and there is none")
        # (the library takes 32 bits, and cuts both to the table's tokens)
        self.window = None if window is None else MfaWindow(*(max(-1, min(int(x), 2 ** 31 - 1)) for x in (window, sinks)))
        self.problem = make_problem(batch, max_pages_per_seq, num_blocks, MFA_KV_FP8_E4M3, softmax_scale,
                                    num_q_heads=num_q_heads, head_dim=head_dim, out_dtype=out_dtype,
                                    tokens_per_seq=tokens_per_seq, num_kv_heads=num_kv_heads)
        if host_seq_lens is None and max_seq_len == 0:
            max_seq_len = max_pages_per_seq * PAGE_SIZE
        with torch.cuda.device(self.device):
            self.plan = self._split(host_seq_lens, max_seq_len, 0, force_ctas, flags)
            self.workspace = torch.zeros(int(self.plan.workspace_bytes), dtype=torch.uint8, device=self.device)
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()   # (the first call may be on another stream)
        self._refs = (ctypes.byref(self.plan), ctypes.byref(self.problem))
        self._own = (self.workspace,)   # buffers that calls use
        self._run = self._decode_call()
        self._append_ref = self._refs[1]
        rows = batch * tokens_per_seq
        self._q_shape = torch.Size((rows, num_q_heads, head_dim))
        self._lse_shape = self._q_shape[:2]
        self._cache_shape = torch.Size((num_blocks, num_kv_heads, PAGE_SIZE, head_dim))
        self._scale_shape = torch.Size((num_blocks, num_kv_heads, PAGE_SIZE // self.scale_tokens))
        self._table_shape = torch.Size((batch, max_pages_per_seq))
        self._batch_shape = self._table_shape[:1]
        self._row_shape = (num_kv_heads, head_dim)
        self._types = (torch.bfloat16, torch.uint8, torch.float32, torch.int32)
        self._out_dtype = torch.float32 if out_dtype == MFA_OUT_FP32 else torch.bfloat16
        # appends whose status a checked decode has yet to report (it clears the word for its own)
        self._checked, self._unreported = bool(flags & MFA_PLAN_CHECK), False

    def _split(self, *args) -> MfaPlan:
        """The plan of this decoder's calls."""
        if self.window is None:
            return mfa_block_decode_plan(self.problem, self.scale_tokens, *args)
        return mfa_window_decode_plan(self.problem, self.scale_tokens, self.window, *args)

    def _decode_call(self):
        """The library's decode, its name, and its arguments up to q."""
        if self.window is None:
            return self._lib.mfa_block_decode_run, "mfa_block_decode_run", (*self._refs, self.scale_tokens)
        return (self._lib.mfa_window_decode_run, "mfa_window_decode_run",
                (*self._refs, self.scale_tokens, ctypes.byref(self.window)))

    def _cache_fits(self, k_cache, v_cache, k_scale, v_scale, block_table) -> bool:
        _, u8, f32, i32 = self._types
        i, codes, scales = self._index, self._cache_shape, self._scale_shape
        return (_fits(k_cache, u8, codes, i) and _fits(v_cache, u8, codes, i) and _fits(k_scale, f32, scales, i) and
                _fits(v_scale, f32, scales, i) and _fits(block_table, i32, self._table_shape, i))

    def _cache_wants(self, k_cache, v_cache, k_scale, v_scale, block_table):
        _, u8, f32, i32 = self._types
        return (("k_cache", k_cache, u8, self._cache_shape), ("v_cache", v_cache, u8, self._cache_shape),
                ("k_scale", k_scale, f32, self._scale_shape), ("v_scale", v_scale, f32, self._scale_shape),
                ("block_table", block_table, i32, self._table_shape))

    def __call__(self, q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, out=None, lse=None, stream=None):
        """One decode step: (out [batch * tokens, num_q_heads, head_dim], lse [.., num_q_heads]).  With
        MFA_PLAN_CHECK it reports what appends since the last one could not place, too."""
        return self._step(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, (), out, lse, stream)

    def _step(self, q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, more, out, lse, stream):
        """A decode step; ``more``: the (checked) tensors of the library's call between seq_lens and out."""
        bf16, _, f32, i32 = self._types
        i = self._index
        if not (_fits(q, bf16, self._q_shape, i) and _fits(seq_lens, i32, self._batch_shape, i) and
                self._cache_fits(k_cache, v_cache, k_scale, v_scale, block_table)):
            _refuse(i, ("q", q, bf16, self._q_shape), ("seq_lens", seq_lens, i32, self._batch_shape),
                    *self._cache_wants(k_cache, v_cache, k_scale, v_scale, block_table))
        if out is None:
            out = self._new(self._q_shape, self._out_dtype, stream)
        elif not _fits(out, self._out_dtype, self._q_shape, i):
            _refuse(i, ("out", out, self._out_dtype, self._q_shape))
        if lse is None:
            lse = self._new(self._lse_shape, f32, stream)
        elif not _fits(lse, f32, self._lse_shape, i):
            _refuse(i, ("lse", lse, f32, self._lse_shape))
        before = self._take_status(stream) if self._unreported else 0
        try:
            self._decode(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, more, out, lse, stream)
        finally:
            if before:
                self._leave_status(before, stream)
        if before:
            raise MfaError(MFA_ERR_DEVICE_CHECK, "mfa_block_kv_append")
        return out, lse

    def _take_status(self, stream) -> int:
        """The status word's bits, which the checked decode about to run clears."""
        self._unreported = False
        word = ctypes.c_uint32(0)
        self._call(self._lib.mfa_read_device_status, "mfa_read_device_status",
                   (self.workspace.data_ptr(), ctypes.byref(word), 0), stream)
        return word.value

    def _leave_status(self, bits: int, stream) -> None:
        """Put bits back beside the checked decode's own (which has synchronised), for mfa_read_device_status."""
        self.workspace[:4].bitwise_or_(self._torch.tensor(list(bits.to_bytes(4, "little")), dtype=self._torch.uint8,
                                                          device=self.device))
        self._torch.cuda.current_stream(self._index).synchronize()

    def _decode(self, q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, more, out, lse, stream) -> None:
        function, where, head = self._run
        self._call(function, where,
                   (*head, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                    block_table.data_ptr(), seq_lens.data_ptr(), *[x.data_ptr() for x in more], out.data_ptr(),
                    lse.data_ptr(), self.workspace.data_ptr(), self.plan.workspace_bytes), stream, self._own,
                   (q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, *more, out, lse))

    def append(self, k_new, v_new, positions, block_table, k_cache, v_cache, k_scale, v_scale, offsets=None,
               max_new: int = 0, device_status=None, stream=None):
        """Quantise new rows into the cache: bf16 ``k_new``, ``v_new`` [rows, num_kv_heads, head_dim], sequence b's
        being rows offsets[b] .. offsets[b + 1] - 1 (``offsets`` int32 [batch + 1], ``max_new`` their largest
        count), or ``tokens_per_seq`` each.  ``device_status``: a tensor of 4 bytes or more, or an address; the
        decoder's workspace by default, so that mfa_read_device_status(decoder.workspace) reports both steps."""
        bf16, _, _, i32 = self._types
        i = self._index
        rows = k_new.shape[0]
        shape = (rows, *self._row_shape)
        counts = (self._batch_shape[0] + 1,)
        if not (_fits(k_new, bf16, shape, i) and _fits(v_new, bf16, shape, i) and
                _fits(positions, i32, self._batch_shape, i) and (offsets is None or _fits(offsets, i32, counts, i)) and
                self._cache_fits(k_cache, v_cache, k_scale, v_scale, block_table)):
            _refuse(i, ("k_new", k_new, bf16, shape), ("v_new", v_new, bf16, shape),
                    ("positions", positions, i32, self._batch_shape),
                    *(() if offsets is None else (("offsets", offsets, i32, counts),)),
                    *self._cache_wants(k_cache, v_cache, k_scale, v_scale, block_table))
        if device_status is None:
            status = self.workspace.data_ptr()
        elif isinstance(device_status, int):
            status, device_status = device_status, None
        else:
            status = device_status.data_ptr()
            if device_status.get_device() != i or _nbytes(device_status) < 4 or not device_status.is_contiguous():
                raise ValueError(f"device_status: expected at least 4 contiguous bytes on {self.device}, got "
                                 f"{device_status.dtype} {tuple(device_status.shape)} on {device_status.device}")
        if self._checked and status == self.workspace.data_ptr():
            self._unreported = True
        self._call(self._lib.mfa_block_kv_append, "mfa_block_kv_append",
                   (self._append_ref, self.scale_tokens, k_new.data_ptr(), v_new.data_ptr(), rows,
                    None if offsets is None else offsets.data_ptr(), max_new, positions.data_ptr(),
                    block_table.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                    v_scale.data_ptr(), status), stream, self._own,
                   (k_new, v_new, offsets, positions, block_table, k_cache, v_cache, k_scale, v_scale, device_status))


class TreeDecoder(BlockDecoder):
    """Attention of trees of drafted tokens over a block-scaled 8-bit cache, and the append of their rows.

    Each sequence's last ``tree_tokens`` cached tokens (1 to 64) are the nodes of a tree: node i sees the tokens
    before the tree, and node j where bit j of its mask is set.  The other arguments, the cache and the rules of
    streams and workspaces are those of BlockDecoder.  A shorter tree takes its nodes first and masks that leave
    out the rest.  Once some nodes are accepted, ``append`` their rows again from the tree's first position, and
    the cache goes on behind them.  (Blocks whose scale a rejected node's row has raised keep that scale.)
    """

    def __init__(self, batch: int, max_pages_per_seq: int, num_blocks: int, tree_tokens: int, num_q_heads: int = NUM_Q_HEADS,
                 num_kv_heads: int = 1, head_dim: int = HEAD_DIM, scale_tokens: int = 64,
                 softmax_scale: Optional[float] = None, host_seq_lens=None, max_seq_len: int = 0, force_ctas: int = 0,
                 flags: int = 0, device=None, out_dtype: int = MFA_OUT_BF16):
        super().__init__(batch, max_pages_per_seq, num_blocks, num_q_heads, num_kv_heads, head_dim, scale_tokens,
                         softmax_scale, host_seq_lens, max_seq_len, force_ctas, flags, device, out_dtype, tree_tokens)
        torch = self._torch
        # appends: rows of any number a sequence (offsets), by default the tree's
        self._append_problem = make_problem(batch, max_pages_per_seq, num_blocks, MFA_KV_FP8_E4M3, softmax_scale,
                                            num_q_heads=num_q_heads, head_dim=head_dim, num_kv_heads=num_kv_heads)
        self._append_ref = ctypes.byref(self._append_problem)
        self._tree_type, self._tree_shape = torch.int64, torch.Size((batch, tree_tokens))
        with torch.cuda.device(self.device):
            self._offsets = torch.arange(0, (batch + 1) * tree_tokens, tree_tokens, dtype=torch.int32, device=self.device)
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()   # (the first call may be on another stream)
        self._own = (self.workspace, self._offsets)

    def _split(self, *args) -> MfaPlan:
        return mfa_tree_decode_plan(self.problem, self.scale_tokens, *args)

    def _decode_call(self):
        return self._lib.mfa_tree_decode_run, "mfa_tree_decode_run", (*self._refs, self.scale_tokens)

    def __call__(self, q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, tree, out=None, lse=None, stream=None):
        """One step: (out [batch * tree_tokens, num_q_heads, head_dim], lse [.., num_q_heads]); ``tree`` int64
        [batch, tree_tokens], the masks (bit 63 is the sign).  seq_lens count the trees' tokens."""
        if not _fits(tree, self._tree_type, self._tree_shape, self._index):
            _refuse(self._index, ("tree", tree, self._tree_type, self._tree_shape))
        return self._step(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, (tree,), out, lse, stream)

    def append(self, k_new, v_new, positions, block_table, k_cache, v_cache, k_scale, v_scale, offsets=None,
               max_new: int = 0, device_status=None, stream=None):
        """As BlockDecoder.append; without ``offsets`` each sequence's rows are its tree's."""
        if offsets is None:
            offsets, max_new = self._offsets, self._tree_shape[1]
            if k_new.shape[0] != self._tree_shape.numel():
                raise ValueError(f"k_new: expected {self._tree_shape.numel()} rows, {max_new} a sequence, got {k_new.shape[0]}")
        super().append(k_new, v_new, positions, block_table, k_cache, v_cache, k_scale, v_scale, offsets, max_new,
                       device_status, stream)


class Rope(_OnDevice):
    """Rotary positions with one to four axes for query heads and new key rows.

    ``sections``: rotary pairs of each axis (their sum is half the rotated width, at most
    head_dim / 2).  ``pairing``: "half" (elements i and i + rotated / 2) or "adjacent" (2 i and
    2 i + 1).  ``interleaved``: the axes are dealt to the pairs in turn instead of one run each;
    ``own_spectrum``: each axis has frequencies of its own.  See include/mfa.h.
    """

    def __init__(self, head_dim: int, sections: Sequence[int], theta: float = 1e4, pairing: str = "half",
                 interleaved: bool = False, own_spectrum: bool = False, position_scale: float = 1.0, device=None):
        super().__init__(device)
        torch = self._torch
        if pairing not in ("half", "adjacent"):
            raise ValueError(f"pairing: expected 'half' or 'adjacent', got {pairing!r}")
        if not 1 <= len(sections) <= MFA_ROPE_MAX_AXES:
            raise ValueError(f"sections: expected 1 to {MFA_ROPE_MAX_AXES} axes, got {len(sections)}")
        self.head_dim, self.axes = int(head_dim), len(sections)
        self.config = MfaRopeConfig(self.head_dim, 2 * int(sum(sections)), self.axes,
                                    (ctypes.c_int32 * MFA_ROPE_MAX_AXES)(*[int(n) for n in sections]),
                                    MFA_ROPE_HALF if pairing == "half" else MFA_ROPE_ADJACENT,
                                    (MFA_ROPE_INTERLEAVED if interleaved else 0) |
                                    (MFA_ROPE_OWN_SPECTRUM if own_spectrum else 0), float(theta), float(position_scale))
        table = mfa_rope_table(self.config)
        self.table = torch.frombuffer(bytearray(bytes(table)), dtype=torch.uint8).to(self.device)
        self._config_ref = ctypes.byref(self.config)
        self._dtypes = {torch.bfloat16: MFA_OUT_BF16, torch.float32: MFA_OUT_FP32}

    def _row_stride(self, t, name: str, line: int) -> int:
        """Elements from one row of t to the next; a row's heads lie side by side, `line` elements of them."""
        if t.is_contiguous():
            return line
        a, b, c = t.stride()
        if c != 1 or (t.shape[1] > 1 and b != self.head_dim):
            raise ValueError(f"{name}: each row's heads must lie side by side, got strides {t.stride()}")
        return a if t.shape[0] > 1 else line   # (a single row has no stride of its own)

    def _rows(self, x, out, name: str, rows: int, dtype, stream):
        """x and its output (x's shape; None: a new tensor) as the library takes them, and the output."""
        shape, d = x.shape, self.head_dim
        if len(shape) != 3 or shape[0] != rows or shape[2] != d or x.dtype is not dtype or x.get_device() != self._index:
            raise ValueError(f"{name}: expected {dtype} [{rows}, heads, {d}] on {self.device}, got {x.dtype} "
                             f"{tuple(shape)} on {x.device}")
        line = shape[1] * d
        if out is None:
            out = self._new(shape, dtype, stream)
        elif out is not x and (out.shape != shape or out.dtype is not dtype or out.get_device() != self._index):
            raise ValueError(f"{name}_out: expected {dtype} {tuple(shape)} on {self.device}, got {out.dtype} "
                             f"{tuple(out.shape)} on {out.device}")
        return MfaRopeRows(x.data_ptr(), out.data_ptr(), self._row_stride(x, name, line), self._row_stride(out, name, line),
                           shape[1]), out

    def __call__(self, q, k, positions, inverse: bool = False, q_out=None, k_out=None, stream=None):
        """Turned rows (q_out, k_out) of q and k, [rows, heads, head_dim] in bf16 or fp32 (either may be None; rows
        may be strided, as columns of one projection); positions int32 [axes, rows].  Pass q_out = q and k_out = k
        to turn in place.  ``inverse``: by the negative angles, which is the gradient of the forward call."""
        some = k if q is None else q
        if some is None:
            raise ValueError("expected q or k")
        rows, dtype = some.shape[0], some.dtype
        kind = self._dtypes.get(dtype)
        if kind is None:
            raise ValueError(f"expected bf16 or fp32 rows, got {dtype}")
        if not _fits(positions, self._torch.int32, (self.axes, rows), self._index):
            _refuse(self._index, ("positions", positions, self._torch.int32, (self.axes, rows)))
        rq = rk = None
        if q is not None:
            rq, q_out = self._rows(q, q_out, "q", rows, dtype, stream)
        if k is not None:
            rk, k_out = self._rows(k, k_out, "k", rows, dtype, stream)
        self._call(self._lib.mfa_rope_run, "mfa_rope_run",
                   (self._config_ref, self.table.data_ptr(), positions.data_ptr(), rows, kind, 1 if inverse else 0,
                    rq, rk), stream, (self.table,), (q, k, positions, q_out, k_out))
        return q_out, k_out


class NormRope(Rope):
    """Norms of query and key heads with their rotary positions in one pass, and the gradient.

    y = turn(x (mean x^2 + eps)^(-1/2) w) for each head x, with one weight for each element of a query
    head and one for each of a key head.  The other arguments are those of Rope.
    """

    def __init__(self, head_dim: int, sections: Sequence[int], eps: float = 1e-6, theta: float = 1e4, pairing: str = "half",
                 interleaved: bool = False, own_spectrum: bool = False, position_scale: float = 1.0, device=None):
        super().__init__(head_dim, sections, theta, pairing, interleaved, own_spectrum, position_scale, device)
        self.eps = float(eps)
        self._weight_shape = self._torch.Size((self.head_dim,))

    def _start(self, q, k, q_weight, k_weight, positions):
        """(rows, row type, its code, MfaNorm) of a call's arguments."""
        some = k if q is None else q
        if some is None:
            raise ValueError("expected q or k")
        rows, dtype = some.shape[0], some.dtype
        kind = self._dtypes.get(dtype)
        if kind is None:
            raise ValueError(f"expected bf16 or fp32 rows, got {dtype}")
        if not _fits(positions, self._torch.int32, (self.axes, rows), self._index):
            _refuse(self._index, ("positions", positions, self._torch.int32, (self.axes, rows)))
        weight_type = None
        for name, x, w in (("q_weight", q, q_weight), ("k_weight", k, k_weight)):
            if x is None:
                continue
            if w is None:
                raise ValueError(f"{name}: expected a weight for each element of a head")
            weight_type = weight_type or w.dtype
            if weight_type not in self._dtypes or not _fits(w, weight_type, self._weight_shape, self._index):
                raise ValueError(f"{name}: expected contiguous bf16 or fp32 weights (of one type) of shape "
                                 f"({self.head_dim},) on {self.device}, got {w.dtype} {tuple(w.shape)} on {w.device}")
        norm = MfaNorm(None if q is None else q_weight.data_ptr(), None if k is None else k_weight.data_ptr(),
                       self._dtypes[weight_type], self.eps)
        return rows, dtype, kind, norm

    def __call__(self, q, k, q_weight, k_weight, positions, q_out=None, k_out=None, stream=None):
        """Normed, weighed and turned rows (q_out, k_out) of q and k, [rows, heads, head_dim] in bf16 or fp32 (either
        may be None; rows may be strided, as columns of one projection); weights [head_dim] in bf16 or fp32;
        positions int32 [axes, rows].  Pass q_out = q and k_out = k to do it in place."""
        rows, dtype, kind, norm = self._start(q, k, q_weight, k_weight, positions)
        rq = rk = None
        if q is not None:
            rq, q_out = self._rows(q, q_out, "q", rows, dtype, stream)
        if k is not None:
            rk, k_out = self._rows(k, k_out, "k", rows, dtype, stream)
        self._call(self._lib.mfa_norm_rope_run, "mfa_norm_rope_run",
                   (self._config_ref, self.table.data_ptr(), positions.data_ptr(), rows, kind, norm, rq, rk), stream,
                   (self.table,), (q, k, q_weight, k_weight, positions, q_out, k_out))
        return q_out, k_out

    def _grad_rows(self, x, dy, dx, name: str, rows: int, dtype, stream):
        """x, dy and dx (x's shape; None: a new tensor) as the library takes them, and dx."""
        if dy is None:
            raise ValueError(f"d{name}: expected the gradient of {name}'s output")
        if dy.shape != x.shape or dy.dtype is not dtype or dy.get_device() != self._index:
            raise ValueError(f"d{name}: expected {dtype} {tuple(x.shape)} on {self.device}, got {dy.dtype} {tuple(dy.shape)} "
                             f"on {dy.device}")
        r, dx = self._rows(x, dx, name, rows, dtype, stream)
        line = x.shape[1] * self.head_dim
        return MfaNormGradRows(r.data_in, dy.data_ptr(), r.data_out, r.in_stride, self._row_stride(dy, "d" + name, line),
                               r.out_stride, r.heads), dx

    def grad(self, dq, dk, q, k, q_weight, k_weight, positions, q_grad=None, k_grad=None, stream=None):
        """The gradient of a call: (q_grad, k_grad, q_weight_grad, k_weight_grad) from dq and dk, the gradients of
        its q_out and k_out, and the call's own arguments.  The weights' gradients are fp32; q_grad and k_grad may be
        given (dq and dk, or q and k, themselves too)."""
        torch = self._torch
        rows, dtype, kind, norm = self._start(q, k, q_weight, k_weight, positions)
        rq = rk = wq = wk = None
        if q is not None:
            rq, q_grad = self._grad_rows(q, dq, q_grad, "q", rows, dtype, stream)
            wq = self._new(self._weight_shape, torch.float32, stream)
        if k is not None:
            rk, k_grad = self._grad_rows(k, dk, k_grad, "k", rows, dtype, stream)
            wk = self._new(self._weight_shape, torch.float32, stream)
        size = 8 * self.head_dim * MFA_NORM_ROPE_GRAD_PARTS
        scratch = self._new(size, torch.uint8, stream)
        self._call(self._lib.mfa_norm_rope_grad_run, "mfa_norm_rope_grad_run",
                   (self._config_ref, self.table.data_ptr(), positions.data_ptr(), rows, kind, norm, rq, rk,
                    None if wq is None else wq.data_ptr(), None if wk is None else wk.data_ptr(), scratch.data_ptr(), size),
                   stream, (self.table,), (dq, dk, q, k, q_weight, k_weight, positions, q_grad, k_grad, wq, wk, scratch))
        return q_grad, k_grad, wq, wk
