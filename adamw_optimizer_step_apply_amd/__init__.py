"""Python binding of the MI355X fused AdamW step (``libadamw_amd.so``).

Argument marshalling only: every step of the optimizer runs in the library's
HIP kernels.  The functions carry the names of the C ABI in ``include/adamw.h``
and accept torch tensors (their ``data_ptr()`` is passed) or raw integer device
addresses.  PyTorch supplies device memory and streams; with ``stream=None`` the
work goes on ``torch.cuda.current_stream()``.

There is no fallback: if the shared library has not been built the import
fails, and every non-OK status raises :class:`AdamWError`.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field
from typing import Sequence

import torch  # loads the HIP runtime the library then binds to

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libadamw_amd.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python adamw_optimizer_step_apply_amd/build.py` "
                      "(or __graft_entry__.build())")

_lib = None

# enums of adamw.h
OK, E_INVALID, E_UNSUPPORTED, E_NOMEM, E_HIP = 0, 1, 2, 3, 4
F32, BF16, F16 = 0, 1, 2
MIXED, PURE_KAHAN, MIXED_SPLIT = 0, 1, 2
KAHAN_NONE, KAHAN_BF16, KAHAN_F32 = 0, 1, 2   # compensation buffer of a pure-bf16 step (PurePrecision.kahan)
STREAM_PARAM, STREAM_GRAD, STREAM_EXP_AVG, STREAM_EXP_AVG_SQ, STREAM_AUX = range(5)
BLOCKED_STATE = 1 << 8        # flat_mask bit: exp_avg / exp_avg_sq / aux in one blocked buffer
FLAT_PAD8 = 1 << 9            # flat_mask bit: every tensor starts at a multiple of 8 in the flat index
STATE_BLOCK_ELEMS = 16384     # elements per block of a blocked state buffer (ADAMW_STATE_BLOCK_ELEMS)
NOALLOC_SCRATCH_BYTES = 16 << 20   # the allocation-free step's per-GPU workspace (ADAMW_NOALLOC_SCRATCH_BYTES)
MUON_SCALE_NONE, MUON_SCALE_SPECTRAL, MUON_SCALE_RMS = 0, 1, 2   # factor of a Muon step's update (MuonHParams.scaling)
NS_MAX_STEPS = 16             # most Newton-Schulz steps (ADAMW_NS_MAX_STEPS)
NUM_STREAMS = 5
_STATUS = {0: "ADAMW_OK", 1: "ADAMW_E_INVALID", 2: "ADAMW_E_UNSUPPORTED", 3: "ADAMW_E_NOMEM", 4: "ADAMW_E_HIP"}


EXPORTED = ("adamw_step", "adamw_multi_tensor_step", "adamw_multi_tensor_step_noalloc", "adamw_multi_tensor_step_amp",
            "adamw_pure_multi_tensor_step",
            "adamw_check_finite", "adamw_grad_norm", "adamw_tensor_norms", "adamw_clip_grads",
            "adamw_multi_tensor_step_clipped",
           "adamw_orthogonalize_workspace_bytes", "adamw_orthogonalize", "adamw_muon_multi_tensor_step",
            "adamw_last_error", "adamw_release_workspace", "adamw_abi_version", "adamw_plan_inspect",
            "adamw_plan_inspect_bytes", "adamw_set_chunk_elems", "adamw_set_single_launch_max_workgroups",
            "adamw_blocked_state_bytes", "adamw_blocked_state_copy")


class adamw_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float), ("inv_loss_scale", ctypes.c_float)]


class adamw_pure_precision(ctypes.Structure):
    _fields_ = [("exp_avg", ctypes.c_int), ("exp_avg_sq", ctypes.c_int), ("kahan", ctypes.c_int32)]


class adamw_loss_scaler(ctypes.Structure):
    _fields_ = [("growth_factor", ctypes.c_float), ("backoff_factor", ctypes.c_float),
                ("growth_interval", ctypes.c_int32)]


class adamw_grad_clip(ctypes.Structure):
    _fields_ = [("d_sumsq", ctypes.c_void_p), ("max_norm", ctypes.c_float), ("eps", ctypes.c_float)]


class adamw_newton_schulz(ctypes.Structure):
    _fields_ = [("a", ctypes.c_float), ("b", ctypes.c_float), ("c", ctypes.c_float), ("eps", ctypes.c_float),
                ("steps", ctypes.c_int32)]


class adamw_muon_hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("inv_loss_scale", ctypes.c_float), ("nesterov", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("ns", adamw_newton_schulz)]


class adamw_tensor_list(ctypes.Structure):
    _fields_ = [("n_tensors", ctypes.c_int64), ("numel", ctypes.POINTER(ctypes.c_int64)),
                ("ptr", ctypes.POINTER(ctypes.c_void_p) * NUM_STREAMS),
                ("shard_begin", ctypes.c_int64), ("shard_end", ctypes.c_int64), ("flat_mask", ctypes.c_uint32)]


_vp = ctypes.c_void_p


def _load(path: str) -> None:
    """Loads the library at ``path`` and declares its C signatures."""
    global _lib
    lib = ctypes.CDLL(path)
    _declare(lib)
    _lib = lib


def _declare(_lib):
    _lib.adamw_step.restype = ctypes.c_int
    _lib.adamw_step.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int64, _vp, _vp, _vp, _vp, _vp,
                                ctypes.POINTER(adamw_hparams), _vp, _vp, _vp]
    _lib.adamw_multi_tensor_step.restype = ctypes.c_int
    _lib.adamw_multi_tensor_step.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(adamw_tensor_list),
                                             ctypes.POINTER(adamw_hparams), _vp, _vp, _vp]
    _lib.adamw_multi_tensor_step_noalloc.restype = ctypes.c_int
    _lib.adamw_multi_tensor_step_noalloc.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(adamw_tensor_list),
                                                     ctypes.POINTER(adamw_hparams), _vp, _vp, _vp]
    _lib.adamw_multi_tensor_step_amp.restype = ctypes.c_int
    _lib.adamw_multi_tensor_step_amp.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(adamw_tensor_list),
                                                 ctypes.POINTER(adamw_hparams), _vp, _vp, _vp,
                                                 ctypes.POINTER(adamw_loss_scaler), _vp]
    _lib.adamw_pure_multi_tensor_step.restype = ctypes.c_int
    _lib.adamw_pure_multi_tensor_step.argtypes = [ctypes.POINTER(adamw_pure_precision),
                                                  ctypes.POINTER(adamw_tensor_list), ctypes.POINTER(adamw_hparams),
                                                  _vp, _vp, _vp]
    _lib.adamw_check_finite.restype = ctypes.c_int
    _lib.adamw_check_finite.argtypes = [ctypes.c_int, ctypes.POINTER(adamw_tensor_list), _vp, _vp]
    _lib.adamw_grad_norm.restype = ctypes.c_int
    _lib.adamw_grad_norm.argtypes = [ctypes.c_int, ctypes.POINTER(adamw_tensor_list), ctypes.c_int, _vp, _vp, _vp, _vp]
    _lib.adamw_tensor_norms.restype = ctypes.c_int
    _lib.adamw_tensor_norms.argtypes = [ctypes.c_int, ctypes.POINTER(adamw_tensor_list), _vp, _vp, _vp, _vp]
    _lib.adamw_clip_grads.restype = ctypes.c_int
    _lib.adamw_clip_grads.argtypes = [ctypes.c_int, ctypes.POINTER(adamw_tensor_list), ctypes.POINTER(adamw_grad_clip),
                                      ctypes.c_float, _vp, _vp]
    _lib.adamw_multi_tensor_step_clipped.restype = ctypes.c_int
    _lib.adamw_multi_tensor_step_clipped.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(adamw_pure_precision),
                                                     ctypes.POINTER(adamw_tensor_list), ctypes.POINTER(adamw_hparams),
                                                     ctypes.POINTER(adamw_grad_clip), _vp, _vp, _vp,
                                                     ctypes.POINTER(adamw_loss_scaler), _vp]
    _lib.adamw_orthogonalize_workspace_bytes.restype = ctypes.c_int64
    _lib.adamw_orthogonalize_workspace_bytes.argtypes = [ctypes.POINTER(adamw_tensor_list),
                                                         ctypes.POINTER(ctypes.c_int64), ctypes.c_int]
    _lib.adamw_orthogonalize.restype = ctypes.c_int
    _lib.adamw_orthogonalize.argtypes = [ctypes.c_int, ctypes.POINTER(adamw_tensor_list),
                                         ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(adamw_newton_schulz), _vp,
                                         ctypes.c_int64, _vp]
    _lib.adamw_muon_multi_tensor_step.restype = ctypes.c_int
    _lib.adamw_muon_multi_tensor_step.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(adamw_pure_precision),
                                                  ctypes.POINTER(adamw_tensor_list), ctypes.POINTER(ctypes.c_int64),
                                                  ctypes.POINTER(adamw_muon_hparams), ctypes.POINTER(adamw_grad_clip),
                                                  _vp, _vp, _vp, _vp, ctypes.c_int64, _vp]
    _lib.adamw_last_error.restype = ctypes.c_char_p
    _lib.adamw_last_error.argtypes = []
    _lib.adamw_release_workspace.restype = None
    _lib.adamw_release_workspace.argtypes = []
    _lib.adamw_abi_version.restype = ctypes.c_int
    _lib.adamw_abi_version.argtypes = []
    _lib.adamw_plan_inspect.restype = ctypes.c_int64
    _lib.adamw_plan_inspect.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(adamw_tensor_list), ctypes.c_int,
                                        ctypes.POINTER(ctypes.c_int64), ctypes.c_int64]
    _lib.adamw_plan_inspect_bytes.restype = ctypes.c_int64
    _lib.adamw_plan_inspect_bytes.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(adamw_pure_precision),
                                              ctypes.POINTER(adamw_tensor_list), ctypes.c_int,
                                              ctypes.POINTER(ctypes.c_uint64), ctypes.c_int64]
    _lib.adamw_blocked_state_bytes.restype = ctypes.c_int64
    _lib.adamw_blocked_state_bytes.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(adamw_pure_precision),
                                               ctypes.POINTER(adamw_tensor_list)]
    _lib.adamw_blocked_state_copy.restype = ctypes.c_int
    _lib.adamw_blocked_state_copy.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(adamw_pure_precision),
                                              ctypes.POINTER(adamw_tensor_list), _vp, ctypes.c_int, _vp]
    _lib.adamw_set_chunk_elems.restype = ctypes.c_int64
    _lib.adamw_set_chunk_elems.argtypes = [ctypes.c_int64]
    _lib.adamw_set_single_launch_max_workgroups.restype = ctypes.c_int64
    _lib.adamw_set_single_launch_max_workgroups.argtypes = [ctypes.c_int64]


_load(LIB_PATH)
ABI_VERSION = 10              # ADAMW_ABI_VERSION of the header this binding follows
if _lib.adamw_abi_version() != ABI_VERSION:
    raise ImportError(f"{LIB_PATH} has ABI version {_lib.adamw_abi_version()}, this binding expects {ABI_VERSION}: "
                      "rebuild the library")


class AdamWError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


@dataclass
class HParams:
    """AdamW hyper-parameters (fp32 in the library).  Defaults: the opt-1.3b
    recipe of "[pure bf16 training] w/ AnyPrecisionAdamW and Kahan summation"
    (lr 0.0002, betas 0.9/0.95, weight decay 0.1) and eps 1e-8."""
    lr: float = 2e-4
    beta1: float = 0.9
    beta2: float = 0.95
    eps: float = 1e-8
    weight_decay: float = 0.1
    inv_loss_scale: float = 1.0

    def c(self) -> adamw_hparams:
        return adamw_hparams(self.lr, self.beta1, self.beta2, self.eps, self.weight_decay, self.inv_loss_scale)


def _addr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, torch.Tensor):
        return x.data_ptr()
    return int(x)


def _result(x, dtype: torch.dtype, numel: int, name: str) -> int:
    """The address of a device result or input of the gradient norms; a tensor given has
    to be of the type and length that the library reads or writes there."""
    if isinstance(x, torch.Tensor) and not (x.is_cuda and x.dtype == dtype and x.numel() >= numel and x.is_contiguous()):
        raise ValueError(f"{name}: a contiguous {dtype} tensor of at least {numel} on the GPU is needed, got "
                         f"{tuple(x.shape)} {x.dtype} on {x.device}")
    return _addr(x)


def _scale(x) -> int:
    """The address of a device loss-scale state (8 bytes)."""
    if isinstance(x, torch.Tensor) and not (x.is_cuda and x.numel() * x.element_size() >= 8 and x.is_contiguous()):
        raise ValueError(f"d_scale: a contiguous tensor of 8 bytes on the GPU is needed (loss_scale_state), got "
                         f"{tuple(x.shape)} {x.dtype} on {x.device}")
    return _addr(x)


# The current stream's address without a torch.cuda.Stream object around it, whose making takes
# 2.7 us of host time per call (a small list's kernel takes 3.6); None on a torch without it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is None:
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int):
    if status != OK:
        raise AdamWError(status, (_lib.adamw_last_error() or b"").decode())


def _hp(hp) -> adamw_hparams:
    if isinstance(hp, adamw_hparams):
        return hp
    if hp is None:
        hp = HParams()
    return hp.c()


class TensorList:
    """Marshals a tensor list into an ``adamw_tensor_list`` and keeps the ctypes
    arrays, and every tensor given, alive as long as it lives (addresses given
    as integers are the caller's to keep valid).  ``streams`` is a sequence of
    5 sequences (param, grad, exp_avg, exp_avg_sq, aux) of tensors or
    addresses; a stream flagged in ``flat_mask`` holds one flat shard buffer;
    ``None`` leaves a stream unset."""

    def __init__(self, numels: Sequence[int], streams, shard_begin: int = 0, shard_end: int = -1,
                 flat_mask: int = 0):
        n = len(numels)
        self._numel = (ctypes.c_int64 * max(n, 1))(*[int(x) for x in numels])
        self._arrays = []
        self._tensors = [x for items in streams if items is not None for x in items if isinstance(x, torch.Tensor)]
        s = adamw_tensor_list()
        s.n_tensors = n
        s.numel = ctypes.cast(self._numel, ctypes.POINTER(ctypes.c_int64))
        for k in range(NUM_STREAMS):
            items = streams[k] if k < len(streams) else None
            if items is None:
                s.ptr[k] = ctypes.POINTER(ctypes.c_void_p)()
                continue
            # a stream with too few entries has null in the others' place, which a call that uses it refuses
            arr = (ctypes.c_void_p * max(len(items), n, 1))(*[_addr(x) for x in items])
            self._arrays.append(arr)
            s.ptr[k] = ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p))
        s.shard_begin = int(shard_begin)
        s.shard_end = int(shard_end)
        s.flat_mask = int(flat_mask)
        self.c = s
        self.numels = [int(x) for x in numels]


def adamw_step(mode: int, p_dtype: int, n: int, param, grad, exp_avg, exp_avg_sq, aux, hp, d_step,
               d_found_inf=None, stream=None) -> None:
    """One AdamW step over one contiguous range of ``n`` elements (C ABI adamw_step)."""
    h = _hp(hp)
    _check(_lib.adamw_step(mode, p_dtype, int(n), _addr(param), _addr(grad), _addr(exp_avg), _addr(exp_avg_sq),
                           _addr(aux), ctypes.byref(h), _addr(d_step), _addr(d_found_inf), _stream(stream)))


def adamw_multi_tensor_step(mode: int, p_dtype: int, tensors: TensorList, hp, d_step, d_found_inf=None,
                            stream=None) -> None:
    """One AdamW step over a tensor list or its ZeRO shard (C ABI adamw_multi_tensor_step)."""
    h = _hp(hp)
    _check(_lib.adamw_multi_tensor_step(mode, p_dtype, ctypes.byref(tensors.c), ctypes.byref(h), _addr(d_step),
                                        _addr(d_found_inf), _stream(stream)))


def adamw_multi_tensor_step_noalloc(mode: int, p_dtype: int, tensors: TensorList, hp, d_step, d_found_inf=None,
                                    stream=None) -> None:
    """adamw_multi_tensor_step without any device allocation: the workspace is
    the library's static per-GPU array (C ABI adamw_multi_tensor_step_noalloc)."""
    h = _hp(hp)
    _check(_lib.adamw_multi_tensor_step_noalloc(mode, p_dtype, ctypes.byref(tensors.c), ctypes.byref(h),
                                                _addr(d_step), _addr(d_found_inf), _stream(stream)))


@dataclass
class LossScaler:
    """Dynamic loss-scaling rule (growth after growth_interval clean steps,
    back-off on an inf/NaN gradient)."""
    growth_factor: float = 2.0
    backoff_factor: float = 0.5
    growth_interval: int = 2000

    def c(self) -> adamw_loss_scaler:
        return adamw_loss_scaler(self.growth_factor, self.backoff_factor, int(self.growth_interval))


def loss_scale_state(scale: float = 65536.0, device="cuda") -> torch.Tensor:
    """A device adamw_loss_scale_state {float scale; int32 growth_tracker} as an
    8-byte tensor (view it as float32 for the scale, int32 for the tracker)."""
    t = torch.zeros(2, dtype=torch.float32, device=device)
    t[0] = scale
    return t


def adamw_multi_tensor_step_amp(mode: int, p_dtype: int, tensors: TensorList, hp, d_step, d_found_inf,
                                d_scale, scaler: LossScaler = None, stream=None) -> None:
    """AdamW step that unscales by a device-resident dynamic loss scale and then
    advances it from the overflow flag (C ABI adamw_multi_tensor_step_amp)."""
    h = _hp(hp)
    sc = (scaler or LossScaler()).c()
    _check(_lib.adamw_multi_tensor_step_amp(mode, p_dtype, ctypes.byref(tensors.c), ctypes.byref(h), _addr(d_step),
                                            _addr(d_found_inf), _scale(d_scale), ctypes.byref(sc),
                                            _stream(stream)))


@dataclass
class PurePrecision:
    """State precisions of a pure-bf16 step: exp_avg / exp_avg_sq dtype (F32 or
    BF16) and the aux stream's compensation buffer: KAHAN_NONE (False),
    KAHAN_BF16 (True) or KAHAN_F32."""
    exp_avg: int = BF16
    exp_avg_sq: int = BF16
    kahan: int = KAHAN_BF16

    def c(self) -> adamw_pure_precision:
        return adamw_pure_precision(int(self.exp_avg), int(self.exp_avg_sq), int(self.kahan))

    @classmethod
    def from_optim_args(cls, text: str) -> "PurePrecision":
        """The precisions named by an AnyPrecisionAdamW option string of the
        form used with ``--optim_args`` ("key=value, ..."): momentum_dtype and
        variance_dtype (bfloat16 or float32, default bfloat16),
        use_kahan_summation (true/false, default false) and
        compensation_buffer_dtype (bfloat16 or float32, default bfloat16).
        Other keys, or other values, raise ValueError."""
        dtypes = {"bfloat16": BF16, "torch.bfloat16": BF16, "float32": F32, "torch.float32": F32}
        opts = {"momentum_dtype": "bfloat16", "variance_dtype": "bfloat16", "use_kahan_summation": "false",
                "compensation_buffer_dtype": "bfloat16"}
        for item in filter(None, (x.strip() for x in text.split(","))):
            key, sep, value = (x.strip() for x in item.partition("="))
            if not sep or key not in opts:
                raise ValueError(f"optim_args: unknown or malformed entry {item!r}")
            opts[key] = value.lower()
        for key in ("momentum_dtype", "variance_dtype", "compensation_buffer_dtype"):
            if opts[key] not in dtypes:
                raise ValueError(f"optim_args: {key}={opts[key]} (bfloat16 or float32)")
        if opts["use_kahan_summation"] not in ("true", "false", "1", "0"):
            raise ValueError(f"optim_args: use_kahan_summation={opts['use_kahan_summation']} (true or false)")
        kahan = KAHAN_NONE
        if opts["use_kahan_summation"] in ("true", "1"):
            kahan = KAHAN_F32 if dtypes[opts["compensation_buffer_dtype"]] == F32 else KAHAN_BF16
        return cls(dtypes[opts["momentum_dtype"]], dtypes[opts["variance_dtype"]], kahan)


def adamw_pure_multi_tensor_step(prec: PurePrecision, tensors: TensorList, hp, d_step, d_found_inf=None,
                                 stream=None) -> None:
    """Pure-bf16 step with chosen state precisions (C ABI adamw_pure_multi_tensor_step)."""
    h = _hp(hp)
    pc = prec.c()
    _check(_lib.adamw_pure_multi_tensor_step(ctypes.byref(pc), ctypes.byref(tensors.c), ctypes.byref(h),
                                             _addr(d_step), _addr(d_found_inf), _stream(stream)))


def adamw_check_finite(g_dtype: int, grads: TensorList, d_found_inf, stream=None) -> None:
    """Zero ``d_found_inf``, then set it to 1 if any gradient is inf/NaN (C ABI adamw_check_finite)."""
    _check(_lib.adamw_check_finite(g_dtype, ctypes.byref(grads.c), _addr(d_found_inf), _stream(stream)))


def adamw_grad_norm(g_dtype: int, grads: TensorList, d_sumsq, d_norm=None, d_found_inf=None,
                    accumulate: bool = False, stream=None) -> None:
    """The global gradient norm: the list's sum of squares into ``d_sumsq`` (one
    float64; added to it with ``accumulate``), its square root into ``d_norm``
    (one float32) and whether it is inf or NaN into ``d_found_inf`` (one int32)
    (C ABI adamw_grad_norm)."""
    _check(_lib.adamw_grad_norm(g_dtype, ctypes.byref(grads.c), int(bool(accumulate)),
                                _result(d_sumsq, torch.float64, 1, "d_sumsq"), _result(d_norm, torch.float32, 1, "d_norm"),
                                _result(d_found_inf, torch.int32, 1, "d_found_inf"), _stream(stream)))


def adamw_tensor_norms(g_dtype: int, grads: TensorList, d_tensor_norms=None, d_tensor_sumsq=None, d_sumsq=None,
                       stream=None) -> None:
    """Every tensor's norm into ``d_tensor_norms`` (float32, one per tensor) and sum
    of squares into ``d_tensor_sumsq`` (float64), and the list's sum of squares into
    ``d_sumsq`` (C ABI adamw_tensor_norms)."""
    n = len(grads.numels)
    _check(_lib.adamw_tensor_norms(g_dtype, ctypes.byref(grads.c),
                                   _result(d_tensor_norms, torch.float32, n, "d_tensor_norms"),
                                   _result(d_tensor_sumsq, torch.float64, n, "d_tensor_sumsq"),
                                   _result(d_sumsq, torch.float64, 1, "d_sumsq"), _stream(stream)))


@dataclass
class GradClip:
    """Clipping by the global norm: ``d_sumsq`` is adamw_grad_norm's sum of squares
    (a float64 tensor of one element, or its device address), read when the call
    that clips runs."""
    d_sumsq: object
    max_norm: float = 1.0
    eps: float = 1e-6

    def c(self) -> adamw_grad_clip:
        return adamw_grad_clip(_result(self.d_sumsq, torch.float64, 1, "d_sumsq"), self.max_norm, self.eps)


def adamw_clip_grads(g_dtype: int, grads: TensorList, clip: GradClip, inv_loss_scale: float = 1.0, d_scale=None,
                     stream=None) -> None:
    """Multiplies the list's gradients by min(1, max_norm / (norm + eps)) in place; the
    norm is the unscaled gradients', by ``d_scale`` (a device loss-scale state) or
    ``inv_loss_scale`` (C ABI adamw_clip_grads)."""
    c = clip.c()
    _check(_lib.adamw_clip_grads(g_dtype, ctypes.byref(grads.c), ctypes.byref(c), inv_loss_scale, _scale(d_scale),
                                 _stream(stream)))


def adamw_multi_tensor_step_clipped(mode: int, p_dtype: int, tensors: TensorList, hp, clip: GradClip, d_step,
                                    d_found_inf=None, d_scale=None, scaler: LossScaler = None,
                                    prec: "PurePrecision" = None, stream=None, advance_scale: bool = True) -> None:
    """One AdamW step that multiplies the gradients by the clipping factor as it reads
    them, and is skipped if ``clip.d_sumsq`` is not finite; ``d_scale`` and ``scaler``
    as adamw_multi_tensor_step_amp (``advance_scale`` false: the scale is only read, as
    for every parameter group but the last), ``prec`` selects
    adamw_pure_multi_tensor_step's step (C ABI adamw_multi_tensor_step_clipped)."""
    h, c, sc = _hp(hp), clip.c(), (scaler or LossScaler()).c()
    pc = ctypes.byref(prec.c()) if prec is not None else None
    _check(_lib.adamw_multi_tensor_step_clipped(mode, p_dtype, pc, ctypes.byref(tensors.c), ctypes.byref(h),
                                                ctypes.byref(c), _addr(d_step), _addr(d_found_inf), _scale(d_scale),
                                                ctypes.byref(sc) if advance_scale else None, _stream(stream)))


class MatrixList(TensorList):
    """A list of row-major matrices: a TensorList with each tensor's (rows, columns).
    Tensors given have to be contiguous and of rows * columns elements (a flat
    shard buffer: of the shard's at least), since only their addresses go to the library."""

    def __init__(self, shapes: Sequence[Sequence[int]], streams, shard_begin: int = 0, shard_end: int = -1,
                 flat_mask: int = 0):
        self.shapes = [(int(r), int(c)) for r, c in shapes]
        numels = [r * c for r, c in self.shapes]
        length = shard_end - shard_begin if shard_end >= 0 else sum(
            -(-n // 8) * 8 if flat_mask & FLAT_PAD8 else n for n in numels) - shard_begin
        for k, items in enumerate(streams):
            for i, x in enumerate(items or ()):
                if not isinstance(x, torch.Tensor):
                    continue
                if not x.is_contiguous():
                    raise ValueError(f"stream {k}, tensor {i}: a contiguous tensor is needed, got strides {x.stride()}")
                if (flat_mask >> k) & 1:
                    if x.numel() < length:
                        raise ValueError(f"stream {k}: a flat buffer of {x.numel()} elements for a shard of {length}")
                elif i >= len(numels) or x.numel() != numels[i]:
                    raise ValueError(f"stream {k}, tensor {i}: {x.numel()} elements are no matrix of "
                                     f"{self.shapes[i] if i < len(numels) else 'the list'}")
        super().__init__(numels, streams, shard_begin, shard_end, flat_mask)
        self.cols = (ctypes.c_int64 * max(len(numels), 1))(*[max(c, 1) for _, c in self.shapes])
        # of each stream's tensors, for _check_streams and _check_types
        self._types = [{x.dtype for x in items or () if isinstance(x, torch.Tensor)} for items in streams]
        # for _check_devices
        self._devices = frozenset(x.device.index for items in streams for x in items or ()
                                  if isinstance(x, torch.Tensor) and x.is_cuda)
        self._kinds = [{(x.element_size(), x.is_cuda) for x in items or () if isinstance(x, torch.Tensor)}
                       for items in streams]


@dataclass
class NewtonSchulz:
    """Newton-Schulz products: ``steps`` times X <- a X + b (X X^T) X + c (X X^T)^2 X
    from X = U / (|U| + eps)."""
    a: float = 3.4445
    b: float = -4.7750
    c: float = 2.0315
    steps: int = 5
    eps: float = 1e-7

    def struct(self) -> adamw_newton_schulz:
        return adamw_newton_schulz(self.a, self.b, self.c, self.eps, int(self.steps))


@dataclass
class MuonHParams:
    """Hyper-parameters of a Muon step; lr and weight decay as in the AdamW step's
    recipe, which MUON_SCALE_RMS makes fit."""
    lr: float = 2e-4
    momentum: float = 0.95
    weight_decay: float = 0.1
    inv_loss_scale: float = 1.0
    nesterov: bool = True
    scaling: int = MUON_SCALE_RMS
    ns: NewtonSchulz = field(default_factory=NewtonSchulz)

    def c(self) -> adamw_muon_hparams:
        return adamw_muon_hparams(self.lr, self.momentum, self.weight_decay, self.inv_loss_scale,
                                  int(self.nesterov), int(self.scaling), self.ns.struct())


def adamw_orthogonalize_workspace_bytes(matrices: MatrixList, least: bool = False) -> int:
    """Bytes of device workspace for the two calls below: for full speed, or with
    ``least`` the smallest that they take."""
    n = _lib.adamw_orthogonalize_workspace_bytes(ctypes.byref(matrices.c), matrices.cols, int(bool(least)))
    if n < 0:
        raise AdamWError(E_INVALID, adamw_last_error())
    return n


def make_orthogonalize_workspace(matrices: MatrixList, device=None) -> torch.Tensor:
    """A workspace of adamw_orthogonalize_workspace_bytes on ``device`` (default: the
    list's tensors')."""
    if device is None:
        if not matrices._tensors:
            raise ValueError("make_orthogonalize_workspace: pass device= when the matrices are given as addresses")
        device = matrices._tensors[0].device
    return torch.empty(adamw_orthogonalize_workspace_bytes(matrices), dtype=torch.uint8, device=device)


def _workspace(x):
    """Address and bytes of a workspace: a contiguous tensor on the GPU, or (address, bytes)."""
    if isinstance(x, torch.Tensor):
        if not x.is_contiguous():
            raise ValueError("workspace: a contiguous tensor is needed")
        if not x.is_cuda:
            raise ValueError(f"workspace: a tensor on the GPU is needed, got {x.device}")
        return x.data_ptr(), x.numel() * x.element_size()
    address, nbytes = x
    return int(address), int(nbytes)


_ELEMENT_BYTES = {F32: 4, BF16: 2, F16: 2}


def _check_streams(matrices: MatrixList, sizes) -> None:
    """The tensors of a list of matrices are on the GPU and of the element sizes that a call reads and writes (0 or
    None: not looked at)."""
    for k, (kinds, size) in enumerate(zip(matrices._kinds, sizes)):
        for got, on_gpu in kinds if size else ():
            if not on_gpu or got != size:
                raise ValueError(f"stream {k}: tensors of {size} bytes an element on the GPU are needed, got "
                                 f"{got} bytes{'' if on_gpu else ' on the host'}")


_TYPES = {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16}


def _check_types(matrices: MatrixList, types) -> None:
    """Floating-point tensors of a list of matrices are of the types that a call reads and writes (None: not looked at);
    others, such as int16 words, stand for whatever the call takes them for."""
    for k, (got, want) in enumerate(zip(matrices._types, types)):
        for t in got if want else ():
            if t.is_floating_point and t != want:
                raise ValueError(f"stream {k}: {want} tensors are needed, got {t}")


def _check_devices(matrices: MatrixList, workspace, stream) -> None:
    """A list's tensors and the workspace are on the GPU that the call's stream is on."""
    devices = matrices._devices
    if isinstance(workspace, torch.Tensor):
        devices = devices | {workspace.device.index}
    if devices and stream is None:
        devices = devices | {torch.cuda.current_device()}
    elif isinstance(stream, torch.cuda.Stream):
        devices = devices | {stream.device.index}
    if len(devices) > 1:
        raise ValueError(f"matrices, workspace and stream (the current device's by default) are on the GPUs {sorted(devices)}: "
                         "one is needed")


def adamw_orthogonalize(u_dtype: int, matrices: MatrixList, workspace, ns: NewtonSchulz = None, stream=None) -> None:
    """Orthogonalises every matrix of a list: the Newton-Schulz products of stream 1
    (``u_dtype``) into stream 0 (bf16), which may be the same bf16 tensors; ``workspace``
    from make_orthogonalize_workspace (C ABI adamw_orthogonalize)."""
    c = (ns or NewtonSchulz()).struct()
    ws = _workspace(workspace)
    _check_streams(matrices, (2, _ELEMENT_BYTES.get(u_dtype)))
    _check_types(matrices, (torch.bfloat16, _TYPES.get(u_dtype)))
    _check_devices(matrices, workspace, stream)
    _check(_lib.adamw_orthogonalize(u_dtype, ctypes.byref(matrices.c), matrices.cols, ctypes.byref(c), *ws,
                                    _stream(stream)))


def adamw_muon_multi_tensor_step(mode: int, p_dtype: int, matrices: MatrixList, hp, d_step, workspace,
                                 d_found_inf=None, clip: GradClip = None, d_scale=None, prec: "PurePrecision" = None,
                                 stream=None) -> None:
    """One Muon step over a list of matrices: momentum, Newton-Schulz products of it,
    decoupled weight decay and the update of the weights.  ``clip`` and ``d_scale`` as
    adamw_multi_tensor_step_clipped with ``advance_scale`` false, ``prec`` selects the pure-bf16
    precisions (C ABI adamw_muon_multi_tensor_step)."""
    h = (hp or MuonHParams()).c()
    pc = ctypes.byref(prec.c()) if prec is not None else None
    cc = ctypes.byref(clip.c()) if clip is not None else None
    ws = _workspace(workspace)
    f32, bf16, p16 = torch.float32, torch.bfloat16, _TYPES.get(p_dtype)
    if prec is not None:
        sizes = (2, 2, _ELEMENT_BYTES.get(prec.exp_avg), None, {KAHAN_BF16: 2, KAHAN_F32: 4}.get(prec.kahan))
        types = (bf16, bf16, _TYPES.get(prec.exp_avg), None, {KAHAN_BF16: bf16, KAHAN_F32: f32}.get(prec.kahan))
    else:
        sizes = {MIXED: (2, 2, 4, None, 4), MIXED_SPLIT: (2, 2, 4, None, 2), PURE_KAHAN: (2, 2, 2, None, 2)}.get(mode, ())
        types = {MIXED: (p16, p16, f32, None, f32), MIXED_SPLIT: (bf16, bf16, f32, None, torch.int16),
                 PURE_KAHAN: (bf16, bf16, bf16, None, bf16)}.get(mode, ())
    _check_streams(matrices, sizes)
    _check_types(matrices, types)
    _check_devices(matrices, workspace, stream)
    _check(_lib.adamw_muon_multi_tensor_step(mode, p_dtype, pc, ctypes.byref(matrices.c), matrices.cols, ctypes.byref(h),
                                             cc, _result(d_step, torch.int32, 1, "d_step"),
                                             _result(d_found_inf, torch.int32, 1, "d_found_inf"), _scale(d_scale),
                                             *ws, _stream(stream)))


def adamw_last_error() -> str:
    return (_lib.adamw_last_error() or b"").decode()


def adamw_release_workspace() -> None:
    _lib.adamw_release_workspace()


def adamw_abi_version() -> int:
    return _lib.adamw_abi_version()


def adamw_plan_inspect(mode: int, p_dtype: int, tensors: TensorList, for_check: int = False):
    """The chunk plan as a list of (tensor, offset_in_tensor, count, kind, flat_pos, segment);
    ``for_check`` 1 for the overflow check's, 2 for the gradient norms', 3 for the clipping's."""
    n = _lib.adamw_plan_inspect(mode, p_dtype, ctypes.byref(tensors.c), int(for_check), None, 0)
    if n < 0:
        raise AdamWError(E_INVALID, adamw_last_error())
    buf = (ctypes.c_int64 * (6 * max(n, 1)))()
    n2 = _lib.adamw_plan_inspect(mode, p_dtype, ctypes.byref(tensors.c), int(for_check), buf, n)
    assert n2 == n
    return [tuple(buf[6 * i:6 * i + 6]) for i in range(n)]


def adamw_plan_inspect_bytes(mode: int, p_dtype: int, tensors: TensorList, for_check: int = False,
                             prec: "PurePrecision" = None):
    """The chunk plan with the device bytes of every chunk: (rows, ranges), rows
    an int64 array (chunks, 6) of adamw_plan_inspect's fields, ranges a uint64
    array (chunks, 5, 2) of [lo, hi) per stream, (0, 0) for an untouched stream;
    ``for_check`` 4: the items of the step's launch table instead of its plan's chunks."""
    import numpy as np
    pc = ctypes.byref(prec.c()) if prec is not None else None
    n = _lib.adamw_plan_inspect_bytes(mode, p_dtype, pc, ctypes.byref(tensors.c), int(for_check), None, 0)
    if n < 0:
        raise AdamWError(E_INVALID, adamw_last_error())
    out = np.zeros((max(n, 1), 16), dtype=np.uint64)
    n2 = _lib.adamw_plan_inspect_bytes(mode, p_dtype, pc, ctypes.byref(tensors.c), int(for_check),
                                       out.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)), n)
    assert n2 == n
    out = out[:n]
    return out[:, :6].view(np.int64), out[:, 6:].reshape(n, NUM_STREAMS, 2)


def adamw_blocked_state_bytes(mode: int, p_dtype: int, tensors: TensorList, prec: "PurePrecision" = None) -> int:
    """Bytes of the blocked state buffer for the per-tensor state that ``tensors``
    describes (C ABI adamw_blocked_state_bytes)."""
    pc = ctypes.byref(prec.c()) if prec is not None else None
    n = _lib.adamw_blocked_state_bytes(mode, p_dtype, pc, ctypes.byref(tensors.c))
    if n < 0:
        raise AdamWError(E_INVALID, adamw_last_error())
    return n


def adamw_blocked_state_copy(mode: int, p_dtype: int, tensors: TensorList, blocked, to_blocked: bool = True,
                             prec: "PurePrecision" = None, stream=None) -> None:
    """Copies the state between per-tensor buffers and a blocked buffer, either way
    (C ABI adamw_blocked_state_copy); returns when the copy is done."""
    pc = ctypes.byref(prec.c()) if prec is not None else None
    _check(_lib.adamw_blocked_state_copy(mode, p_dtype, pc, ctypes.byref(tensors.c), _addr(blocked),
                                         int(bool(to_blocked)), _stream(stream)))


def make_blocked_state(mode: int, p_dtype: int, numels: Sequence[int], exp_avg, exp_avg_sq, aux=None,
                       shard_begin: int = 0, shard_end: int = -1, pad8: bool = True, flat_mask: int = 0,
                       prec: "PurePrecision" = None, stream=None, device=None):
    """Optimizer-owned state in the blocked layout, filled from per-tensor state.

    ``exp_avg``, ``exp_avg_sq`` and ``aux`` are sequences of per-tensor tensors
    (one per entry of ``numels``; with flat_mask bits 2-4, one flat shard tensor)
    holding the state to start from -- e.g. zero moments and the fp32 master
    weights (tensors, or device addresses with ``device`` given).  Allocates one
    zero-filled uint8 tensor on their device, copies the state in with the
    library's copy kernel, and returns ``(blocked, step_mask)``:
    a step then takes ``TensorList(numels, [params, grads, [blocked], None, None],
    shard_begin, shard_end, step_mask)``.  ``pad8`` lays the buffer out in the
    padded flat index (ADAMW_FLAT_PAD8), which keeps every tensor of any length on
    the 16-byte vector path when params and grads are 16-byte aligned."""
    streams = [None, None, list(exp_avg), list(exp_avg_sq), None if aux is None else list(aux)]
    mask = (flat_mask & 0x1c) | (FLAT_PAD8 if pad8 else 0)
    tl = TensorList(numels, streams, shard_begin, shard_end, mask)
    nbytes = adamw_blocked_state_bytes(mode, p_dtype, tl, prec)
    if device is None:
        tensors = [t for t in streams[2] if isinstance(t, torch.Tensor)]
        if not tensors:
            raise ValueError("make_blocked_state: pass device= when the state is given as addresses")
        device = tensors[0].device
    blocked = torch.zeros(max(nbytes, 16), dtype=torch.uint8, device=device)
    adamw_blocked_state_copy(mode, p_dtype, tl, blocked, True, prec, stream)
    return blocked, mask | BLOCKED_STATE


def adamw_set_chunk_elems(elems: int) -> int:
    r = _lib.adamw_set_chunk_elems(int(elems))
    if r < 0:
        raise AdamWError(E_INVALID, f"chunk size {elems} rejected")
    return r


def adamw_set_single_launch_max_workgroups(max_workgroups: int) -> int:
    """Largest grid (in workgroups: 8 per chunk of a step, 1 per short one and per check chunk)
    that runs as one launch; 0 = always two launches, < 0 = the default.
    Returns the value now in force."""
    return _lib.adamw_set_single_launch_max_workgroups(int(max_workgroups))


def library_path() -> str:
    return LIB_PATH
