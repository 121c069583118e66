"""ctypes binding of the C ABI in ``include/sv.h`` (same names, same
arguments).  Tensors are passed by device pointer; the stream defaults to
PyTorch's current stream on the tensors' device."""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

SV_F32, SV_BF16 = 0, 1
SV_ROW_BAD_TOKEN, SV_ROW_BAD_LENGTH, SV_ROW_BAD_TEMPERATURE = 1, 2, 4
SV_NOTE_ZERO_RESIDUAL, SV_NOTE_CDF_FALLBACK, SV_NOTE_TIMEOUT = 8, 16, 32
SV_ROW_BAD_SLOT, SV_ROW_BAD_PENALTY, SV_ROW_BAD_BIAS = 64, 128, 256
SV_ROW_BAD_MASK, SV_ROW_EMPTY_MASK = 512, 1024
SV_HISTORY_PROMPT, SV_HISTORY_OUTPUT = 0, 1
_STATUS = {0: "SV_OK", 1: "SV_ERR_ARG", 2: "SV_ERR_SHAPE", 3: "SV_ERR_DTYPE",
           4: "SV_ERR_WORKSPACE", 5: "SV_ERR_CUDA"}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libsv.so")
_lib = None


class SVError(RuntimeError):
    def __init__(self, fn: str, code: int):
        extra = ""
        if code == 5 and _lib is not None:
            extra = f" (cuda error {_lib.sv_last_cuda_error()})"
        super().__init__(f"{fn} failed: {_STATUS.get(code, code)}{extra}")
        self.code = code


def library_path() -> str:
    return _LIB_PATH


def lib():
    """Load ``libsv.so``; raises if it is missing (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is missing: build it with "
                          "`python -m speculative_decoding_verification_93_b200.build`")
    L = ctypes.CDLL(_LIB_PATH)
    vp, i32, i64, u64, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64,
                             ctypes.c_size_t)
    L.sv_schedule.argtypes = [vp, i32, i32, ctypes.c_float, vp, vp]
    L.sv_schedule_admit.argtypes = [vp, i32, i32, vp, i32, vp, vp, vp]
    L.sv_sts_workspace_bytes.argtypes = [i32, i32]
    L.sv_sts_workspace_bytes.restype = sz
    L.sv_sts_fit.argtypes = [vp, vp, i32, i32, ctypes.c_float, ctypes.c_float, vp, vp, vp, sz,
                             vp]
    L.sv_sts_apply.argtypes = [vp, vp, i32, i32, vp, vp]
    L.sv_debug_sts_wait_limit.argtypes = [u64]
    L.sv_debug_sts_wait_limit.restype = i32
    L.sv_debug_sts_timeouts.argtypes = []
    L.sv_debug_sts_timeouts.restype = i32
    L.sv_verify_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.sv_verify_workspace_bytes.restype = sz
    L.sv_verify.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, u64, i64, vp, vp, vp, sz, vp,
                            vp]
    L.sv_schedule_verify.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, ctypes.c_float, vp, vp,
                                     u64, i64, vp, vp, vp, sz, vp, vp]
    L.sv_verify_debug.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, u64, i64, vp, vp, vp,
                                  sz, vp, vp, vp]
    L.sv_verify_noalloc.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, u64, i64, vp, vp, vp,
                                    vp]
    sp = ctypes.POINTER(sv_vp_slice)
    L.sv_vp_stats_bytes.argtypes = [sp]
    L.sv_vp_stats_bytes.restype = sz
    L.sv_vp_workspace_bytes.argtypes = [sp]
    L.sv_vp_workspace_bytes.restype = sz
    L.sv_vp_stats.argtypes = [sp, vp, vp, vp, vp, vp]
    L.sv_vp_decide.argtypes = [sp, vp, vp, vp, vp, u64, i64, vp, vp, vp, vp, vp, sz, vp, vp]
    L.sv_vp_draw.argtypes = [sp, vp, vp, vp, sz, vp, vp]
    L.sv_verify_host_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.sv_verify_host_workspace_bytes.restype = sz
    L.sv_verify_host.argtypes = [vp, vp, i32, i32, i32, i32, vp, ctypes.c_float, vp, vp, u64, i64,
                                 vp, vp, vp, vp, i32, vp, sz, vp, vp]
    hp, rp, wp = (ctypes.POINTER(t) for t in (_History, _Rules, _W4))
    L.sv_history_reset.argtypes = [hp, vp, i32, vp, vp]
    L.sv_history_add.argtypes = [hp, vp, i32, vp, i32, vp, i32, i32, vp, vp]
    L.sv_logits_process.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, vp, i32, i32, vp, i32,
                                    rp, vp, vp]
    L.sv_head_w4_workspace_bytes.argtypes = [wp, i32, i32]
    L.sv_head_w4_workspace_bytes.restype = sz
    L.sv_head_w4.argtypes = [wp, vp, i32, i32, vp, i32, vp, i32, vp, sz, vp, vp]
    L.sv_philox_uniforms.argtypes = [u64, vp, vp, vp, i32, vp, vp]
    L.sv_philox4x32_10.argtypes = [vp, vp, i32, vp, vp]
    L.sv_profile_begin.argtypes = [i32]
    L.sv_profile_read.argtypes = [vp, i32]
    L.sv_profile_read.restype = i32
    L.sv_status_string.argtypes = [i32]
    L.sv_status_string.restype = ctypes.c_char_p
    for name in ("sv_schedule", "sv_schedule_admit", "sv_sts_fit", "sv_sts_apply", "sv_verify",
                 "sv_verify_debug", "sv_verify_noalloc", "sv_verify_host", "sv_vp_stats",
                 "sv_vp_decide",
                 "sv_vp_draw",
                 "sv_philox_uniforms",
                 "sv_philox4x32_10", "sv_profile_begin", "sv_history_reset", "sv_history_add",
                 "sv_logits_process", "sv_head_w4"):
        getattr(L, name).restype = i32
    L.sv_last_cuda_error.restype = i32
    L.sv_version.restype = i32
    L.sv_verify_launches.restype = i32
    _lib = L
    return L


class sv_vp_slice(ctypes.Structure):
    """This rank's slice of the vocabulary (``sv_vp_slice`` in include/sv.h)."""
    _fields_ = [("target_logits", ctypes.c_void_p), ("draft_logits", ctypes.c_void_p),
                ("dtype", ctypes.c_int), ("B", ctypes.c_int), ("K", ctypes.c_int),
                ("V", ctypes.c_int), ("v0", ctypes.c_int), ("Vs", ctypes.c_int),
                ("nshards", ctypes.c_int), ("shard", ctypes.c_int)]


def vp_slice(target_logits, draft_logits, V: int, v0: int, nshards: int,
             shard: int) -> sv_vp_slice:
    """Describe a slice from its logits: target [B, K+1, Vs], draft [B, K, Vs]
    or None, holding tokens v0 .. v0+Vs-1 of a vocabulary of V."""
    B, K1, Vs = target_logits.shape
    dt = _dtype(target_logits)
    if not target_logits.is_contiguous():
        raise TypeError("target_logits must be contiguous")
    if draft_logits is not None and (draft_logits.dtype != target_logits.dtype
                                     or not draft_logits.is_contiguous()
                                     or tuple(draft_logits.shape) != (B, K1 - 1, Vs)):
        raise TypeError("draft_logits must be a contiguous [B, K, Vs] tensor of the target dtype")
    return sv_vp_slice(target_logits.data_ptr(),
                       None if draft_logits is None else draft_logits.data_ptr(),
                       dt, B, K1 - 1, int(V), int(v0), Vs, int(nshards), int(shard))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, like: torch.Tensor):
    if stream is None:
        stream = torch.cuda.current_stream(like.device)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(fn: str, code: int):
    if code != 0:
        raise SVError(fn, code)


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SV_F32
    if t.dtype == torch.bfloat16:
        return SV_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _need(t: torch.Tensor, dtype, name: str):
    if t.dtype != dtype or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} tensor")


def sv_schedule(conf: torch.Tensor, load: float, lengths: torch.Tensor, stream=None) -> None:
    _need(conf, torch.float32, "conf")
    _need(lengths, torch.int32, "lengths")
    B, K = conf.shape
    _check("sv_schedule", lib().sv_schedule(_ptr(conf), B, K, float(load), _ptr(lengths),
                                            _stream(stream, conf)))


def sv_schedule_admit(conf: torch.Tensor, speed: torch.Tensor, lengths: torch.Tensor,
                      tau_out: Optional[torch.Tensor] = None, stream=None) -> None:
    _need(conf, torch.float32, "conf")
    _need(speed, torch.float32, "speed")
    _need(lengths, torch.int32, "lengths")
    B, K = conf.shape
    _check("sv_schedule_admit", lib().sv_schedule_admit(
        _ptr(conf), B, K, _ptr(speed), speed.numel(), _ptr(lengths), _ptr(tau_out),
        _stream(stream, conf)))


def sv_sts_workspace_bytes(N: int, K: int) -> int:
    return int(lib().sv_sts_workspace_bytes(N, K))


def sv_sts_fit(logits: torch.Tensor, accept_len: torch.Tensor, temperature: torch.Tensor,
               ece: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               tmin: float = 1e-2, tmax: float = 1e2, stream=None) -> None:
    _need(logits, torch.float32, "logits")
    _need(accept_len, torch.int32, "accept_len")
    _need(temperature, torch.float32, "temperature")
    N, K = logits.shape
    if workspace is None:
        workspace = torch.empty(sv_sts_workspace_bytes(N, K), dtype=torch.uint8,
                                device=logits.device)
    _check("sv_sts_fit", lib().sv_sts_fit(
        _ptr(logits), _ptr(accept_len), N, K, float(tmin), float(tmax), _ptr(temperature),
        _ptr(ece), _ptr(workspace), workspace.numel(), _stream(stream, logits)))


def sv_sts_apply(logits: torch.Tensor, temperature: torch.Tensor, conf_out: torch.Tensor,
                 stream=None) -> None:
    _need(logits, torch.float32, "logits")
    _need(temperature, torch.float32, "temperature")
    _need(conf_out, torch.float32, "conf_out")
    N, K = logits.shape
    _check("sv_sts_apply", lib().sv_sts_apply(_ptr(logits), _ptr(temperature), N, K,
                                              _ptr(conf_out), _stream(stream, logits)))


def sv_debug_sts_wait_limit(limit_ns: int) -> None:
    """Test export: wall-time limit of the calibration barrier's wait on the
    current device (0 restores the 1 s default)."""
    _check("sv_debug_sts_wait_limit", lib().sv_debug_sts_wait_limit(int(limit_ns)))


def sv_debug_sts_timeouts() -> int:
    """Test export: barrier waits that ran out since the previous call."""
    n = lib().sv_debug_sts_timeouts()
    if n < 0:
        raise SVError("sv_debug_sts_timeouts", 5)
    return n


def sv_verify_workspace_bytes(B: int, K: int, V: int, dtype: int) -> int:
    return int(lib().sv_verify_workspace_bytes(B, K, V, dtype))


def _verify_args(target_logits, draft_logits, draft_tokens, lengths, temperature):
    B, K1, V = target_logits.shape
    K = K1 - 1
    dt = _dtype(target_logits)
    if not target_logits.is_contiguous():
        raise TypeError("target_logits must be contiguous")
    if draft_logits is not None and (draft_logits.dtype != target_logits.dtype
                                     or not draft_logits.is_contiguous()
                                     or tuple(draft_logits.shape) != (B, K, V)):
        raise TypeError("draft_logits must be a contiguous [B, K, V] tensor of the target dtype")
    _need(draft_tokens, torch.int32, "draft_tokens")
    _need(lengths, torch.int32, "lengths")
    _need(temperature, torch.float32, "temperature")
    return B, K, V, dt


def sv_verify(target_logits, draft_logits, draft_tokens, lengths, temperature, seed: int,
              out_tokens, out_accept_len, workspace, status=None, row_base: int = 0,
              stream=None) -> None:
    B, K, V, dt = _verify_args(target_logits, draft_logits, draft_tokens, lengths, temperature)
    _check("sv_verify", lib().sv_verify(
        _ptr(target_logits), _ptr(draft_logits), dt, B, K, V, _ptr(draft_tokens), _ptr(lengths),
        _ptr(temperature), ctypes.c_uint64(seed & (2**64 - 1)), int(row_base), _ptr(out_tokens),
        _ptr(out_accept_len), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(status), _stream(stream, target_logits)))


def sv_schedule_verify(target_logits, draft_logits, draft_tokens, conf, load: float, lengths,
                       temperature, seed: int, out_tokens, out_accept_len, workspace, status=None,
                       row_base: int = 0, stream=None) -> None:
    """sv_schedule then sv_verify in one call: `lengths` receives the
    scheduled lengths (see include/sv.h)."""
    B, K, V, dt = _verify_args(target_logits, draft_logits, draft_tokens, lengths, temperature)
    _need(conf, torch.float32, "conf")
    if tuple(conf.shape) != (B, K):
        raise TypeError("conf must be a [B, K] float32 tensor")
    _check("sv_schedule_verify", lib().sv_schedule_verify(
        _ptr(target_logits), _ptr(draft_logits), dt, B, K, V, _ptr(draft_tokens), _ptr(conf),
        float(load), _ptr(lengths), _ptr(temperature), ctypes.c_uint64(seed & (2**64 - 1)),
        int(row_base), _ptr(out_tokens), _ptr(out_accept_len), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream, target_logits)))


def sv_verify_debug(target_logits, draft_logits, draft_tokens, lengths, temperature, seed: int,
                    out_tokens, out_accept_len, workspace, stats_out, status=None,
                    row_base: int = 0, stream=None) -> None:
    B, K, V, dt = _verify_args(target_logits, draft_logits, draft_tokens, lengths, temperature)
    _check("sv_verify_debug", lib().sv_verify_debug(
        _ptr(target_logits), _ptr(draft_logits), dt, B, K, V, _ptr(draft_tokens), _ptr(lengths),
        _ptr(temperature), ctypes.c_uint64(seed & (2**64 - 1)), int(row_base), _ptr(out_tokens),
        _ptr(out_accept_len), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _ptr(status), _ptr(stats_out), _stream(stream, target_logits)))


def sv_verify_noalloc(target_logits, draft_logits, draft_tokens, lengths, temperature, seed: int,
                      out_tokens, out_accept_len, status=None, row_base: int = 0,
                      stream=None) -> None:
    """sv_verify with the library's own fixed scratch instead of a workspace,
    for callers that must not allocate device memory (see include/sv.h)."""
    B, K, V, dt = _verify_args(target_logits, draft_logits, draft_tokens, lengths, temperature)
    _check("sv_verify_noalloc", lib().sv_verify_noalloc(
        _ptr(target_logits), _ptr(draft_logits), dt, B, K, V, _ptr(draft_tokens), _ptr(lengths),
        _ptr(temperature), ctypes.c_uint64(seed & (2**64 - 1)), int(row_base), _ptr(out_tokens),
        _ptr(out_accept_len), _ptr(status), _stream(stream, target_logits)))


def sv_vp_stats_bytes(slice_: sv_vp_slice) -> int:
    return int(lib().sv_vp_stats_bytes(ctypes.byref(slice_)))


def sv_vp_workspace_bytes(slice_: sv_vp_slice) -> int:
    return int(lib().sv_vp_workspace_bytes(ctypes.byref(slice_)))


def sv_vp_stats(slice_: sv_vp_slice, draft_tokens, lengths, temperature, stats_local,
                stream=None) -> None:
    _need(draft_tokens, torch.int32, "draft_tokens")
    _need(lengths, torch.int32, "lengths")
    _need(temperature, torch.float32, "temperature")
    _check("sv_vp_stats", lib().sv_vp_stats(
        ctypes.byref(slice_), _ptr(draft_tokens), _ptr(lengths), _ptr(temperature),
        _ptr(stats_local), _stream(stream, lengths)))


def sv_vp_decide(slice_: sv_vp_slice, stats_all, draft_tokens, lengths, temperature, seed: int,
                 out_tokens, out_accept_len, mass_local, workspace, status=None, norm_out=None,
                 row_base: int = 0, stream=None) -> None:
    _need(draft_tokens, torch.int32, "draft_tokens")
    _need(lengths, torch.int32, "lengths")
    _need(temperature, torch.float32, "temperature")
    _check("sv_vp_decide", lib().sv_vp_decide(
        ctypes.byref(slice_), _ptr(stats_all), _ptr(draft_tokens), _ptr(lengths),
        _ptr(temperature), ctypes.c_uint64(seed & (2**64 - 1)), int(row_base), _ptr(out_tokens),
        _ptr(out_accept_len), _ptr(mass_local), _ptr(norm_out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream, lengths)))


def sv_vp_draw(slice_: sv_vp_slice, mass_all, out_tokens, workspace, status=None,
               stream=None) -> None:
    _check("sv_vp_draw", lib().sv_vp_draw(
        ctypes.byref(slice_), _ptr(mass_all), _ptr(out_tokens), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(status), _stream(stream, out_tokens)))


def sv_verify_host_workspace_bytes(B: int, K: int, V: int, dtype: int) -> int:
    return int(lib().sv_verify_host_workspace_bytes(B, K, V, dtype))


def _need_host(t: torch.Tensor, dtype, name: str):
    if t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} host tensor")


def sv_verify_host(target_logits, draft_logits, conf, load: float, draft_tokens, temperature,
                   seed: int, out_tokens, out_accept_len, lengths, workspace, status=None,
                   row_base: int = 0, levelwise: bool = False, stream=None) -> int:
    """Host-resident inputs and outputs (pinned CPU tensors), device
    workspace; returns the bytes copied host-to-device.  With conf None,
    `lengths` is an input and no schedule runs.  levelwise copies only the
    logits the outcome depends on, one position level at a time.  The
    outputs are valid once `stream` has drained."""
    B, K1, V = target_logits.shape
    K = K1 - 1
    if target_logits.is_cuda or not target_logits.is_contiguous():
        raise TypeError("target_logits must be a contiguous host tensor")
    dt = _dtype(target_logits)
    if draft_logits is not None:
        _need_host(draft_logits, target_logits.dtype, "draft_logits")
        if tuple(draft_logits.shape) != (B, K, V):
            raise TypeError("draft_logits must be [B, K, V]")
    if conf is not None:
        _need_host(conf, torch.float32, "conf")
    _need_host(draft_tokens, torch.int32, "draft_tokens")
    _need_host(temperature, torch.float32, "temperature")
    _need_host(out_tokens, torch.int32, "out_tokens")
    _need_host(out_accept_len, torch.int32, "out_accept_len")
    _need_host(lengths, torch.int32, "lengths")
    if status is not None:
        _need_host(status, torch.int32, "status")
    if not workspace.is_cuda:
        raise TypeError("workspace must be device memory")
    h2d = ctypes.c_size_t(0)
    _check("sv_verify_host", lib().sv_verify_host(
        _ptr(target_logits), _ptr(draft_logits), dt, B, K, V, _ptr(conf), float(load),
        _ptr(draft_tokens), _ptr(temperature), ctypes.c_uint64(seed & (2**64 - 1)), int(row_base),
        _ptr(out_tokens), _ptr(out_accept_len), _ptr(lengths), _ptr(status),
        1 if levelwise else 0, _ptr(workspace),
        workspace.numel() * workspace.element_size(), ctypes.byref(h2d),
        _stream(stream, workspace)))
    return int(h2d.value)


# ---------------------------------------------------------------------------
# Token history, logit rules, 4-bit head.
# ---------------------------------------------------------------------------
class _History(ctypes.Structure):
    _fields_ = [("prompt_bits", ctypes.c_void_p), ("output_bits", ctypes.c_void_p),
                ("output_counts", ctypes.c_void_p), ("R", ctypes.c_int), ("V", ctypes.c_int)]


class _Rules(ctypes.Structure):
    _fields_ = [("history", ctypes.POINTER(_History)), ("slots", ctypes.c_void_p),
                ("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("presence", ctypes.c_void_p), ("bias_begin", ctypes.c_void_p),
                ("bias_tokens", ctypes.c_void_p), ("bias_values", ctypes.c_void_p),
                ("n_bias", ctypes.c_int), ("mask", ctypes.c_void_p), ("n_masks", ctypes.c_int),
                ("mask_index", ctypes.c_void_p)]


class _W4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("zero", ctypes.c_void_p),
                ("scale_dtype", ctypes.c_int), ("V", ctypes.c_int), ("H", ctypes.c_int),
                ("group", ctypes.c_int)]


# The raw handle of the current stream, without a Stream object around it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _given(t, dtype, name: str, dev: int, shape=None):
    """An optional tensor argument on device `dev` (-1: the host): its address, or
    None."""
    if t is None:
        return None
    if t.dtype != dtype or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} tensor")
    if t.get_device() != dev:
        raise TypeError(f"{name} must be on {f'cuda:{dev}' if dev >= 0 else 'cpu'}, "
                        f"is on {t.device}")
    if shape is not None and t.shape != shape:
        raise TypeError(f"{name} must have the shape {shape}, has {tuple(t.shape)}")
    return t.data_ptr()


def _call(fn: str, dev: int, stream, *args) -> None:
    """Call `fn` on device `dev`, with the stream (default: the current one of
    that device) as the last argument."""
    if dev < 0:
        raise TypeError(f"{fn}: the tensors must be on a GPU")
    if stream is None:
        stream = _raw_stream(dev)
    elif isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    if torch.cuda.current_device() == dev:
        code = getattr(lib(), fn)(*args, int(stream))
    else:
        with torch.cuda.device(dev):
            code = getattr(lib(), fn)(*args, int(stream))
    if code != 0:
        raise SVError(fn, code)


class TokenHistory:
    """``sv_history``: the bit planes [R, ceil(V / 32)] (int32 words) and counts
    [R, V] (int32) of R slots.  Holds its tensors; zero-filled ones are empty."""

    def __init__(self, V: int, prompt_bits, output_bits, output_counts):
        R, W = output_counts.shape[0], (V + 31) // 32
        dev = output_counts.get_device()
        at = [_given(t, torch.int32, name, dev, shape) for name, t, shape in (
            ("prompt_bits", prompt_bits, (R, W)), ("output_bits", output_bits, (R, W)),
            ("output_counts", output_counts, (R, V)))]
        self.prompt_bits, self.output_bits = prompt_bits, output_bits
        self.output_counts = output_counts
        self.R, self.V, self.dev = R, V, dev
        self.desc = _History(*at, R, V)

    @classmethod
    def empty(cls, R: int, V: int, device) -> "TokenHistory":
        planes = torch.zeros(2, R, (V + 31) // 32, dtype=torch.int32, device=device)
        return cls(V, planes[0], planes[1],
                   torch.zeros(R, V, dtype=torch.int32, device=device))


class LogitRules:
    """``sv_logit_rules``: every part may be None.  Per-row tensors have B
    entries; biases are B lists, row b the entries bias_begin[b] ..
    bias_begin[b + 1] - 1; mask is [n, ceil(V / 32)] int32 words, bit 1 =
    allowed, and mask_index [B, P] names each position's mask (-1: none)."""

    def __init__(self, history: Optional[TokenHistory] = None, slots=None, repetition=None,
                 frequency=None, presence=None, bias_begin=None, bias_tokens=None,
                 bias_values=None, mask=None, mask_index=None):
        f32, i32 = torch.float32, torch.int32
        rows = (("slots", slots, i32), ("repetition", repetition, f32),
                ("frequency", frequency, f32), ("presence", presence, f32))
        given = [t for _, t, _ in rows] + [bias_begin, mask, mask_index]
        given += [] if history is None else [history.output_counts]
        dev = next((t.get_device() for t in given if t is not None), None)
        n = None
        at = []
        for name, t, dtype in rows:
            at.append(_given(t, dtype, name, dev))
            if t is not None:
                if t.dim() != 1 or n not in (None, t.numel()):
                    raise TypeError("the per-row tensors must be vectors of the same length")
                n = t.numel()
        if history is not None:
            _given(history.output_counts, i32, "history", dev)
        if (bias_begin is None) != (bias_tokens is None) or \
                (bias_begin is None) != (bias_values is None):
            raise TypeError("bias_begin, bias_tokens and bias_values go together")
        n_bias = 0
        if bias_begin is not None:
            n_bias = bias_tokens.numel()
            if n not in (None, bias_begin.numel() - 1):
                raise TypeError("bias_begin must have one entry more than there are rows")
            n = bias_begin.numel() - 1
        at += [_given(bias_begin, i32, "bias_begin", dev),
               _given(bias_tokens, i32, "bias_tokens", dev, (n_bias,)),
               _given(bias_values, f32, "bias_values", dev, (n_bias,))]
        n_masks = 0
        if mask is not None:
            if mask.dim() != 2:
                raise TypeError("mask must be [n, ceil(V / 32)]")
            n_masks = mask.shape[0]
        elif mask_index is not None:
            raise TypeError("mask_index needs a mask")
        self.rows, self.n_masks = n, n_masks
        self.words = None if mask is None else mask.shape[1]
        self.index_shape = None if mask_index is None else tuple(mask_index.shape)
        self.history, self.dev = history, dev
        self._keep = (slots, repetition, frequency, presence, bias_begin, bias_tokens,
                      bias_values, mask, mask_index)
        self.desc = _Rules(None if history is None else ctypes.pointer(history.desc), *at, n_bias,
                           _given(mask, i32, "mask", dev), n_masks,
                           _given(mask_index, i32, "mask_index", dev))


class W4Weight:
    """``sv_w4``: codes [V, H / 2] uint8 (even k in the low half of a byte),
    scale [V, H / group] float32 or bfloat16, zero [V, H / group] uint8 or
    None (8).  Holds its tensors."""

    def __init__(self, codes, scale, zero=None):
        V, H, G = codes.shape[0], 2 * codes.shape[1], scale.shape[1]
        if G < 1 or H % G:
            raise TypeError("scale must be [V, H / group] for codes [V, H / 2]")
        dev = codes.get_device()
        at = (_given(codes, torch.uint8, "codes", dev),
              _given(scale, torch.float32 if scale.dtype == torch.float32 else torch.bfloat16,
                     "scale", dev, (V, G)),
              _given(zero, torch.uint8, "zero", dev, (V, G)))
        self.codes, self.scale, self.zero = codes, scale, zero
        self.V, self.H, self.group, self.dev = V, H, H // G, dev
        self.desc = _W4(*at, SV_F32 if scale.dtype == torch.float32 else SV_BF16, V, H, H // G)


def sv_history_reset(history: TokenHistory, slots=None, n: Optional[int] = None, status=None,
                     stream=None) -> None:
    """Empty the listed slots, or the first n (default: all)."""
    dev = history.dev
    if slots is not None:
        n = slots.numel()
    elif n is None:
        n = history.R
    _call("sv_history_reset", dev, stream, history.desc,
          _given(slots, torch.int32, "slots", dev), int(n),
          _given(status, torch.int32, "status", dev))


def sv_history_add(history: TokenHistory, tokens, lens=None, kind: int = SV_HISTORY_OUTPUT,
                   slots=None, extra: int = 0, status=None, stream=None) -> None:
    """Append the first lens[b] + extra (default: all) tokens of each row of
    tokens [B, S]; sv_verify's results go in as tokens = out_tokens,
    lens = out_accept_len, extra = 1."""
    dev, (B, S) = history.dev, tokens.shape
    _call("sv_history_add", dev, stream, history.desc,
          _given(slots, torch.int32, "slots", dev, (B,)), B,
          _given(tokens, torch.int32, "tokens", dev), S,
          _given(lens, torch.int32, "lens", dev, (B,)), extra, kind,
          _given(status, torch.int32, "status", dev))


def sv_logits_process(logits, out, rules: LogitRules, draft_tokens=None, lengths=None,
                      extra: int = 0, pos0: int = 0, V: Optional[int] = None, v0: int = 0,
                      status=None, stream=None) -> None:
    """Apply `rules` to logits [B, P, Vs] into `out` (which may be `logits`);
    V and v0 place a vocabulary slice (default: the whole vocabulary)."""
    dev, (B, P, Vs) = logits.get_device(), logits.shape
    dt = _dtype(logits)
    V = Vs if V is None else int(V)
    if rules.dev is not None and rules.dev != dev:
        raise TypeError(f"the rules must be on {logits.device}")
    if rules.rows is not None and rules.rows != B:
        raise TypeError(f"the rules are for {rules.rows} rows, the logits have {B}")
    if rules.words is not None and rules.words != (V + 31) // 32:
        raise TypeError(f"mask must have {(V + 31) // 32} words a row, has {rules.words}")
    if rules.index_shape is not None and rules.index_shape != (B, P):
        raise TypeError(f"mask_index must be [{B}, {P}], is {list(rules.index_shape)}")
    K = 0
    if draft_tokens is not None:
        if draft_tokens.dim() != 2 or draft_tokens.shape[0] != B:
            raise TypeError("draft_tokens must be [B, K]")
        K = draft_tokens.shape[1]
    at = _given(logits, logits.dtype, "logits", dev)
    _call("sv_logits_process", dev, stream, at,
          at if out is logits else _given(out, logits.dtype, "out", dev, (B, P, Vs)),
          dt, B, P, V, v0, Vs,
          _given(draft_tokens, torch.int32, "draft_tokens", dev), K, pos0,
          _given(lengths, torch.int32, "lengths", dev, (B,)), extra, rules.desc,
          _given(status, torch.int32, "status", dev))


def sv_head_w4_workspace_bytes(weight: W4Weight, B: int, P: int) -> int:
    return int(lib().sv_head_w4_workspace_bytes(weight.desc, B, P))


def sv_head_w4(weight: W4Weight, x, out, workspace=None, lengths=None, extra: int = 0, status=None,
               stream=None) -> None:
    """out [B, P, V] (float32 or bfloat16) = x [B, P, H] (bfloat16) times the
    4-bit weights; positions p >= lengths[b] + extra are left as they were."""
    dev, (B, P, H) = x.get_device(), x.shape
    if H != weight.H:
        raise TypeError(f"x must be [B, P, {weight.H}]")
    if weight.dev != dev:
        raise TypeError(f"the weights must be on {x.device}")
    _call("sv_head_w4", dev, stream, weight.desc, _given(x, torch.bfloat16, "x", dev), B, P,
          _given(lengths, torch.int32, "lengths", dev, (B,)), extra,
          _given(out, out.dtype, "out", dev, (B, P, weight.V)), _dtype(out),
          None if workspace is None else _given(workspace, workspace.dtype, "workspace", dev),
          0 if workspace is None else workspace.numel() * workspace.element_size(),
          _given(status, torch.int32, "status", dev))


def sv_philox_uniforms(seed: int, row, pos, draw, out, stream=None) -> None:
    n = out.numel()
    _check("sv_philox_uniforms", lib().sv_philox_uniforms(
        ctypes.c_uint64(seed & (2**64 - 1)), _ptr(row), _ptr(pos), _ptr(draw), n, _ptr(out),
        _stream(stream, out)))


def sv_philox4x32_10(ctr, key, out, stream=None) -> None:
    n = out.numel() // 4
    _check("sv_philox4x32_10", lib().sv_philox4x32_10(_ptr(ctr), _ptr(key), n, _ptr(out),
                                                      _stream(stream, out)))


def sv_profile_begin(capacity: int) -> None:
    _check("sv_profile_begin", lib().sv_profile_begin(int(capacity)))


def sv_profile_read(max_n: int = 4096):
    buf = (ctypes.c_float * max_n)()
    n = lib().sv_profile_read(ctypes.cast(buf, ctypes.c_void_p), max_n)
    return [buf[i] for i in range(n)]


def sv_verify_launches() -> int:
    return int(lib().sv_verify_launches())


def sv_status_string(code: int) -> str:
    return lib().sv_status_string(int(code)).decode()


def verify(target_logits, draft_logits, draft_tokens, lengths, temperature, seed: int,
           row_base: int = 0, workspace=None, status=None, stream=None):
    """Allocate the outputs (and workspace, if not given) with PyTorch and call
    :func:`sv_verify`.  Returns (out_tokens [B, K+1], out_accept_len [B])."""
    B, K1, V = target_logits.shape
    dev = target_logits.device
    out_tokens = torch.empty(B, K1, dtype=torch.int32, device=dev)
    out_acc = torch.empty(B, dtype=torch.int32, device=dev)
    if workspace is None:
        n = sv_verify_workspace_bytes(B, K1 - 1, V, _dtype(target_logits))
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    sv_verify(target_logits, draft_logits, draft_tokens, lengths, temperature, seed, out_tokens,
              out_acc, workspace, status=status, row_base=row_base, stream=stream)
    return out_tokens, out_acc
