"""Python binding of the gfx950 Muon step library (``libmuon.so``).

Argument marshalling only: every step of the optimizer runs in the HIP
kernels behind the C ABI declared in ``include/muon.h``.  PyTorch provides
device memory and streams.  There is no CPU fallback: if the library is not
built, or the device is not gfx950, the calls raise.

The names mirror the C entry points:
``muon_step``, ``muon_step_noalloc``, ``muon_ns``, ``muon_workspace_bytes``,
``muon_ns_workspace_bytes``, ``muon_adamw_step``,
``muon_adamw_workspace_bytes``, ``muon_cayley_step``,
``muon_cayley_workspace_bytes``, ``muon_block_norm``,
``muon_block_norm_backward``, ``muon_block_norm_backward_workspace_bytes``,
``muon_token_logp``, ``muon_token_logp_backward``,
``muon_token_logp_saved_bytes``, ``muon_token_logp_workspace_bytes``,
``muon_token_logp_backward_workspace_bytes``, ``muon_preference_loss``,
``muon_preference_loss_workspace_bytes``, ``muon_policy_loss``,
``muon_policy_loss_workspace_bytes``, ``muon_status_string``,
``muon_last_error_message``, ``muon_profile_enable``, ``muon_profile_read``
(C: ``muon_profile_read`` and ``muon_profile_read_classes``),
``muon_version``.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Iterable, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmuon.so")

MUON_OK = 0
MUON_ERR_INVALID_ARG = -1
MUON_ERR_UNSUPPORTED = -2
MUON_ERR_WORKSPACE = -3
MUON_ERR_HIP = -4

MUON_F32 = 0
MUON_BF16 = 1

SCALE_RULES = {"naive": 0, "kellerjordan": 1, "mup": 2, "moonlight": 3}
MUON_FLAG_NESTEROV = 1
GATE_NONE, GATE_CHANNEL, GATE_FULL = 0, 1, 2
PREFERENCE_KINDS = {"sigmoid": 0, "hinge": 1, "squared": 2}
KL_KINDS = {"none": 0, "k1": 1, "k2": 2, "k3": 3}
LOSS_REDUCTIONS = {"token": 0, "sequence": 1}
MUON_KCLASS_COUNT = 9
KERNEL_CLASSES = ("momentum_norm", "norm_finalize", "gram", "poly", "update", "apply", "adamw", "cayley",
                  "update_apply", "block_norm", "token_logp", "preference_loss", "policy_loss")


class MuonMatrix(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("momentum", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class MuonNsCoeffs(ctypes.Structure):
    _fields_ = [("a", ctypes.c_float), ("b", ctypes.c_float), ("c", ctypes.c_float)]


class MuonHparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("eps", ctypes.c_float), ("scale_rule", ctypes.c_int32), ("ns_steps", ctypes.c_int32),
                ("schedule", ctypes.POINTER(MuonNsCoeffs)), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class MuonNsMatrix(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64)]


class MuonAdamwTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("numel", ctypes.c_int64)]


class MuonAdamwHparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float), ("step", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class MuonCayleyMatrix(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("momentum", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class MuonCayleyHparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta", ctypes.c_float)]


def _fields(spec):
    kinds = {"p": ctypes.c_void_p, "q": ctypes.c_int64, "f": ctypes.c_float, "i": ctypes.c_int32}
    return [(name, kinds[kind]) for kind, names in spec for name in names.split()]


class MuonBlockNormArgs(ctypes.Structure):
    _fields_ = _fields([("p", "x residual post_weight gate pre_weight out_residual out_norm rstd"),
                        ("q", "rows cols ld_x ld_residual ld_gate ld_out_residual ld_out_norm"),
                        ("f", "residual_scale eps"), ("i", "dtype weight_dtype gate_kind")])


class MuonBlockNormBackwardArgs(ctypes.Structure):
    _fields_ = _fields([("p", "x out_residual rstd grad_norm grad_out_residual post_weight gate pre_weight grad_x "
                              "grad_residual grad_post_weight grad_gate grad_pre_weight"),
                        ("q", "rows cols ld_x ld_out_residual ld_grad_norm ld_grad_out_residual ld_gate ld_grad_x "
                              "ld_grad_residual ld_grad_gate"),
                        ("f", "residual_scale"), ("i", "dtype weight_dtype gate_kind")])


class MuonTokenLogpArgs(ctypes.Structure):
    _fields_ = _fields([("p", "hidden head targets logp lse saved"), ("q", "tokens cols vocab ld_hidden ld_head"),
                        ("f", "scale"), ("i", "dtype")])


class MuonTokenLogpBackwardArgs(ctypes.Structure):
    _fields_ = _fields([("p", "hidden head targets lse grad_logp saved grad_hidden grad_head"),
                        ("q", "tokens cols vocab ld_hidden ld_head ld_grad_hidden ld_grad_head"),
                        ("f", "scale"), ("i", "dtype")])


class MuonPreferenceArgs(ctypes.Structure):
    _fields_ = _fields([("p", "logp ref_logp mask offsets loss rewards grad_logp"), ("q", "tokens sequences"),
                        ("f", "beta margin label_smoothing grad_scale"), ("i", "kind average dtype")])


class MuonPolicyArgs(ctypes.Structure):
    _fields_ = _fields([("p", "logp old_logp ref_logp advantages mask offsets loss stats grad_logp"),
                        ("q", "tokens sequences"), ("f", "clip_low clip_high dual_clip kl_coef grad_scale"),
                        ("i", "kl reduction advantage_per_sequence dtype")])


class MuonProfile(ctypes.Structure):
    _fields_ = [("ms", ctypes.c_double * MUON_KCLASS_COUNT), ("launches", ctypes.c_int64 * MUON_KCLASS_COUNT)]


_WORKSPACE_OPS = ("block_norm_backward", "token_logp", "token_logp_backward", "preference_loss", "policy_loss")

# Every symbol include/muon.h declares, with its ctypes signature.
SIGNATURES = {
    "muon_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(MuonMatrix), ctypes.c_int32, ctypes.POINTER(MuonHparams)]),
    "muon_step": (ctypes.c_int32, [ctypes.POINTER(MuonMatrix), ctypes.c_int32, ctypes.POINTER(MuonHparams),
                                   ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "muon_step_noalloc": (ctypes.c_int32, [ctypes.POINTER(MuonMatrix), ctypes.c_int32, ctypes.POINTER(MuonHparams),
                                           ctypes.c_void_p]),
    "muon_ns_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(MuonNsMatrix), ctypes.c_int32,
                                                  ctypes.POINTER(MuonHparams)]),
    "muon_ns": (ctypes.c_int32, [ctypes.POINTER(MuonNsMatrix), ctypes.c_int32, ctypes.POINTER(MuonHparams),
                                 ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "muon_adamw_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(MuonAdamwTensor), ctypes.c_int32,
                                                     ctypes.POINTER(MuonAdamwHparams)]),
    "muon_adamw_step": (ctypes.c_int32, [ctypes.POINTER(MuonAdamwTensor), ctypes.c_int32,
                                         ctypes.POINTER(MuonAdamwHparams), ctypes.c_void_p, ctypes.c_size_t,
                                         ctypes.c_void_p]),
    "muon_cayley_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(MuonCayleyMatrix), ctypes.c_int32,
                                                      ctypes.POINTER(MuonCayleyHparams)]),
    "muon_cayley_step": (ctypes.c_int32, [ctypes.POINTER(MuonCayleyMatrix), ctypes.c_int32,
                                          ctypes.POINTER(MuonCayleyHparams), ctypes.c_void_p, ctypes.c_size_t,
                                          ctypes.c_void_p]),
    # the operators' arguments are one struct, by address (a ctypes instance or packed bytes)
    "muon_block_norm": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_void_p]),
    **{f"muon_{op}_workspace_bytes": (ctypes.c_size_t, [ctypes.c_void_p]) for op in _WORKSPACE_OPS},
    **{f"muon_{op}": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p])
       for op in _WORKSPACE_OPS},
    "muon_token_logp_saved_bytes": (ctypes.c_size_t, [ctypes.c_void_p]),
    "muon_status_string": (ctypes.c_char_p, [ctypes.c_int32]),
    "muon_last_error_message": (ctypes.c_char_p, []),
    "muon_profile_enable": (ctypes.c_int32, [ctypes.c_int32]),
    "muon_profile_read": (ctypes.c_int32, [ctypes.POINTER(MuonProfile)]),
    "muon_profile_read_classes": (ctypes.c_int32, [ctypes.c_int32, ctypes.POINTER(ctypes.c_double),
                                                   ctypes.POINTER(ctypes.c_int64)]),
    "muon_version": (ctypes.c_int32, []),
}

_lib = None


class MuonError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{_status_string(status)} ({detail})")


def load(path: str = LIB_PATH):
    """Load the HIP library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`"
                           " or `python matrix_aware_optimizer_amd/build.py`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _status_string(status: int) -> str:
    return load().muon_status_string(int(status)).decode()


def muon_status_string(status: int) -> str:
    return _status_string(status)


def muon_last_error_message() -> str:
    return load().muon_last_error_message().decode()


def muon_version() -> int:
    return int(load().muon_version())


def _check(status: int):
    if status != MUON_OK:
        raise MuonError(status, muon_last_error_message())


# --------------------------------------------------------------------------
# Marshalling helpers
# --------------------------------------------------------------------------

def _dtype_code(t) -> int:
    import torch
    dtype = t if isinstance(t, torch.dtype) else t.dtype
    if dtype == torch.bfloat16:
        return MUON_BF16
    if dtype == torch.float32:
        return MUON_F32
    raise ValueError(f"unsupported dtype {dtype}; use bfloat16 or float32")


def _check_matrix(t, what):
    if t.dim() != 2:
        raise ValueError(f"{what} must be 2-D, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous (row-major)")


def make_hparams(*, lr=0.02, beta=0.95, weight_decay=0.0, eps=1e-7, scale_rule="naive",
                 schedule: Sequence[Sequence[float]] = (), dtype=MUON_BF16, nesterov=False):
    """Build a muon_hparams struct.  Returns (struct, keepalive)."""
    sched = (MuonNsCoeffs * max(1, len(schedule)))()
    for k, (a, b, c) in enumerate(schedule):
        sched[k] = MuonNsCoeffs(a, b, c)
    rule = SCALE_RULES[scale_rule] if isinstance(scale_rule, str) else int(scale_rule)
    hp = MuonHparams(lr, beta, weight_decay, eps, rule, len(schedule),
                     ctypes.cast(sched, ctypes.POINTER(MuonNsCoeffs)), int(dtype),
                     MUON_FLAG_NESTEROV if nesterov else 0)
    return hp, sched


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(int(stream.cuda_stream))


def _workspace_for(need: int, workspace, device, stream):
    """The workspace a call runs with, safe for torch's caching allocator.

    The kernels use the workspace on ``stream``.  A workspace allocated here
    is allocated on that stream, so the allocator orders its reuse after the
    work enqueued there; a caller's workspace used on a stream other than the
    current one is recorded on it (``record_stream``), so dropping it does not
    hand its memory to other work while the call's kernels still read it.
    """
    import torch
    if workspace is None:
        if stream is None:
            return allocate_workspace(need, device)
        with torch.cuda.stream(stream):
            return allocate_workspace(need, device)
    if workspace.numel() * workspace.element_size() < need:
        raise MuonError(MUON_ERR_WORKSPACE, f"workspace has {workspace.numel()} bytes, {need} needed")
    if stream is not None and stream != torch.cuda.current_stream(workspace.device):
        workspace.record_stream(stream)
    return workspace


def _matrices(weights, grads, moms):
    weights, grads, moms = list(weights), list(grads), list(moms)
    if not (len(weights) == len(grads) == len(moms)):
        raise ValueError("weights, grads and momenta must have equal lengths")
    arr = (MuonMatrix * max(1, len(weights)))()
    dtype = None
    for i, (w, g, m) in enumerate(zip(weights, grads, moms)):
        _check_matrix(w, f"weight[{i}]")
        _check_matrix(m, f"momentum[{i}]")
        if g is not None:
            _check_matrix(g, f"grad[{i}]")
            if g.shape != w.shape or g.dtype != w.dtype:
                raise ValueError(f"grad[{i}] must match weight[{i}] in shape and dtype")
        if m.shape != w.shape or m.dtype != w.dtype:
            raise ValueError(f"momentum[{i}] must match weight[{i}] in shape and dtype")
        code = _dtype_code(w)
        if dtype is None:
            dtype = code
        elif code != dtype:
            raise ValueError("all matrices of one call must share a dtype")
        arr[i] = MuonMatrix(w.data_ptr(), g.data_ptr() if g is not None else None, m.data_ptr(),
                            w.shape[0], w.shape[1])
    return arr, len(weights), (MUON_BF16 if dtype is None else dtype)


# --------------------------------------------------------------------------
# Entry points
# --------------------------------------------------------------------------

def muon_workspace_bytes(weights, grads, moms, **hp_kwargs) -> int:
    arr, n, dtype = _matrices(weights, grads, moms)
    hp, keep = make_hparams(dtype=dtype, **hp_kwargs)
    size = load().muon_workspace_bytes(arr, n, ctypes.byref(hp))
    if size == 0:
        raise MuonError(MUON_ERR_INVALID_ARG, muon_last_error_message())
    return int(size)


def allocate_workspace(nbytes: int, device=None):
    """Device workspace through torch (256-byte aligned by torch's allocator)."""
    import torch
    ws = torch.empty(max(1, nbytes), dtype=torch.uint8, device=device or "cuda")
    if ws.data_ptr() % 256:
        raise RuntimeError("torch returned a workspace that is not 256-byte aligned")
    return ws


def muon_step(weights: Iterable, grads: Iterable, moms: Iterable, *, lr, beta=0.95, weight_decay=0.0,
              schedule=(), scale_rule="naive", eps=1e-7, nesterov=False, workspace=None, stream=None):
    """One grouped Muon step, in place on ``weights`` and ``moms`` (torch tensors on the GPU).

    A ``None`` gradient skips its matrix.  ``workspace`` is an optional uint8
    device tensor of at least :func:`muon_workspace_bytes` bytes; one is
    allocated through torch otherwise.  Asynchronous on ``stream`` (default:
    torch's current stream).
    """
    weights, grads, moms = list(weights), list(grads), list(moms)
    arr, n, dtype = _matrices(weights, grads, moms)
    hp, keep = make_hparams(lr=lr, beta=beta, weight_decay=weight_decay, eps=eps, scale_rule=scale_rule,
                            schedule=schedule, dtype=dtype, nesterov=nesterov)
    lib = load()
    need = lib.muon_workspace_bytes(arr, n, ctypes.byref(hp))
    if need == 0:
        raise MuonError(MUON_ERR_INVALID_ARG, muon_last_error_message())
    workspace = _workspace_for(need, workspace, weights[0].device if weights else None, stream)
    _check(lib.muon_step(arr, n, ctypes.byref(hp), ctypes.c_void_p(workspace.data_ptr()),
                         workspace.numel() * workspace.element_size(), _stream_handle(stream)))
    return workspace


NOALLOC_SCRATCH_BYTES = 128 << 20   # MUON_NOALLOC_SCRATCH_BYTES


def muon_step_noalloc(weights: Iterable, grads: Iterable, moms: Iterable, *, lr, beta=0.95, weight_decay=0.0,
                      schedule=(), scale_rule="naive", eps=1e-7, nesterov=False, stream=None):
    """:func:`muon_step` without a workspace and without any allocation: the library
    uses its own per-GPU device array of ``NOALLOC_SCRATCH_BYTES``.  Calls that
    overlap on one GPU race; lists that need more workspace raise MuonError."""
    weights, grads, moms = list(weights), list(grads), list(moms)
    arr, n, dtype = _matrices(weights, grads, moms)
    hp, keep = make_hparams(lr=lr, beta=beta, weight_decay=weight_decay, eps=eps, scale_rule=scale_rule,
                            schedule=schedule, dtype=dtype, nesterov=nesterov)
    _check(load().muon_step_noalloc(arr, n, ctypes.byref(hp), _stream_handle(stream)))


def _ns_matrices(inputs, outputs):
    inputs, outputs = list(inputs), list(outputs)
    if len(inputs) != len(outputs):
        raise ValueError("inputs and outputs must have equal lengths")
    import torch
    arr = (MuonNsMatrix * max(1, len(inputs)))()
    dtype = None
    for i, (x, o) in enumerate(zip(inputs, outputs)):
        _check_matrix(x, f"in[{i}]")
        _check_matrix(o, f"out[{i}]")
        if o.dtype != torch.float32 or o.shape != x.shape:
            raise ValueError(f"out[{i}] must be float32 with the input's shape")
        code = _dtype_code(x)
        if dtype is None:
            dtype = code
        elif code != dtype:
            raise ValueError("all inputs of one call must share a dtype")
        arr[i] = MuonNsMatrix(x.data_ptr(), o.data_ptr(), x.shape[0], x.shape[1])
    return arr, len(inputs), (MUON_BF16 if dtype is None else dtype)


def muon_ns_workspace_bytes(inputs, outputs, *, schedule=(), eps=1e-7) -> int:
    arr, n, dtype = _ns_matrices(inputs, outputs)
    hp, keep = make_hparams(schedule=schedule, eps=eps, dtype=dtype)
    size = load().muon_ns_workspace_bytes(arr, n, ctypes.byref(hp))
    if size == 0:
        raise MuonError(MUON_ERR_INVALID_ARG, muon_last_error_message())
    return int(size)


def muon_ns(inputs, outputs, *, schedule, eps=1e-7, workspace=None, stream=None):
    """outputs[i] = NS(inputs[i] / (||inputs[i]||_F + eps)), fp32 outputs."""
    inputs, outputs = list(inputs), list(outputs)
    arr, n, dtype = _ns_matrices(inputs, outputs)
    hp, keep = make_hparams(schedule=schedule, eps=eps, dtype=dtype)
    lib = load()
    need = lib.muon_ns_workspace_bytes(arr, n, ctypes.byref(hp))
    if need == 0:
        raise MuonError(MUON_ERR_INVALID_ARG, muon_last_error_message())
    workspace = _workspace_for(need, workspace, inputs[0].device if inputs else None, stream)
    _check(lib.muon_ns(arr, n, ctypes.byref(hp), ctypes.c_void_p(workspace.data_ptr()),
                       workspace.numel() * workspace.element_size(), _stream_handle(stream)))
    return workspace


def _adamw_tensors(params, grads, exp_avgs, exp_avg_sqs):
    import torch
    params, grads, exp_avgs, exp_avg_sqs = list(params), list(grads), list(exp_avgs), list(exp_avg_sqs)
    if not (len(params) == len(grads) == len(exp_avgs) == len(exp_avg_sqs)):
        raise ValueError("params, grads, exp_avgs and exp_avg_sqs must have equal lengths")
    arr = (MuonAdamwTensor * max(1, len(params)))()
    dtype = None
    for i, (p, g, m, v) in enumerate(zip(params, grads, exp_avgs, exp_avg_sqs)):
        for t, what in ((p, "param"), (m, "exp_avg"), (v, "exp_avg_sq")):
            if not t.is_contiguous():
                raise ValueError(f"{what}[{i}] must be contiguous")
        if g is not None and (not g.is_contiguous() or g.shape != p.shape or g.dtype != p.dtype):
            raise ValueError(f"grad[{i}] must be contiguous and match param[{i}] in shape and dtype")
        for t, what in ((m, "exp_avg"), (v, "exp_avg_sq")):
            if t.dtype != torch.float32 or t.numel() != p.numel():
                raise ValueError(f"{what}[{i}] must be float32 with param[{i}]'s number of elements")
        code = _dtype_code(p)
        if dtype is None:
            dtype = code
        elif code != dtype:
            raise ValueError("all params of one call must share a dtype")
        arr[i] = MuonAdamwTensor(p.data_ptr(), g.data_ptr() if g is not None else None, m.data_ptr(),
                                 v.data_ptr(), p.numel())
    return arr, len(params), (MUON_BF16 if dtype is None else dtype)


def muon_adamw_workspace_bytes(params, grads, exp_avgs, exp_avg_sqs, *, lr=1e-3, betas=(0.9, 0.999),
                               eps=1e-8, weight_decay=0.0, step=1) -> int:
    arr, n, dtype = _adamw_tensors(params, grads, exp_avgs, exp_avg_sqs)
    hp = MuonAdamwHparams(lr, betas[0], betas[1], eps, weight_decay, int(step), dtype)
    size = load().muon_adamw_workspace_bytes(arr, n, ctypes.byref(hp))
    if size == 0:
        raise MuonError(MUON_ERR_INVALID_ARG, muon_last_error_message())
    return int(size)


def muon_adamw_step(params, grads, exp_avgs, exp_avg_sqs, *, lr, betas=(0.9, 0.999), eps=1e-8,
                    weight_decay=0.0, step, workspace=None, stream=None):
    """One grouped AdamW step, in place on params and the fp32 moments.

    ``step`` counts calls and starts at 1 (it sets the bias corrections).  A
    ``None`` gradient skips its tensor.  Asynchronous on ``stream``.
    """
    params = list(params)
    arr, n, dtype = _adamw_tensors(params, grads, exp_avgs, exp_avg_sqs)
    hp = MuonAdamwHparams(lr, betas[0], betas[1], eps, weight_decay, int(step), dtype)
    lib = load()
    need = lib.muon_adamw_workspace_bytes(arr, n, ctypes.byref(hp))
    if need == 0:
        raise MuonError(MUON_ERR_INVALID_ARG, muon_last_error_message())
    workspace = _workspace_for(need, workspace, params[0].device if params else None, stream)
    _check(lib.muon_adamw_step(arr, n, ctypes.byref(hp), ctypes.c_void_p(workspace.data_ptr()),
                               workspace.numel() * workspace.element_size(), _stream_handle(stream)))
    return workspace


def _cayley_matrices(weights, grads, moms):
    import torch
    weights, grads, moms = list(weights), list(grads), list(moms)
    if not (len(weights) == len(grads) == len(moms)):
        raise ValueError("weights, grads and momenta must have equal lengths")
    arr = (MuonCayleyMatrix * max(1, len(weights)))()
    for i, (w, g, m) in enumerate(zip(weights, grads, moms)):
        for t, what in ((w, "weight"), (m, "momentum")) + (((g, "grad"),) if g is not None else ()):
            _check_matrix(t, f"{what}[{i}]")
            if t.dtype != torch.float32 or t.shape != w.shape:
                raise ValueError(f"{what}[{i}] must be float32 with weight[{i}]'s shape")
        arr[i] = MuonCayleyMatrix(w.data_ptr(), g.data_ptr() if g is not None else None, m.data_ptr(),
                                  w.shape[0], w.shape[1])
    return arr, len(weights)


def muon_cayley_workspace_bytes(weights, grads, moms, *, lr=1e-3, beta=0.9) -> int:
    arr, n = _cayley_matrices(weights, grads, moms)
    hp = MuonCayleyHparams(lr, beta)
    size = load().muon_cayley_workspace_bytes(arr, n, ctypes.byref(hp))
    if size == 0:
        raise MuonError(MUON_ERR_INVALID_ARG, muon_last_error_message())
    return int(size)


def muon_cayley_step(weights, grads, moms, *, lr, beta=0.9, workspace=None, stream=None):
    """One grouped Muon-Cayley step (fp32), in place on ``weights`` and ``moms``.

    Each weight must have orthonormal columns (orthonormal rows when it is wide);
    the update keeps it so.  A ``None`` gradient skips its matrix.
    """
    weights = list(weights)
    arr, n = _cayley_matrices(weights, grads, moms)
    hp = MuonCayleyHparams(lr, beta)
    lib = load()
    need = lib.muon_cayley_workspace_bytes(arr, n, ctypes.byref(hp))
    if need == 0:
        raise MuonError(MUON_ERR_INVALID_ARG, muon_last_error_message())
    workspace = _workspace_for(need, workspace, weights[0].device if weights else None, stream)
    _check(lib.muon_cayley_step(arr, n, ctypes.byref(hp), ctypes.c_void_p(workspace.data_ptr()),
                                workspace.numel() * workspace.element_size(), _stream_handle(stream)))
    return workspace


# --------------------------------------------------------------------------
# Training operators (norms around a block, token log-probabilities, losses)
# --------------------------------------------------------------------------
# These calls come once or more per step, some on a few kilobytes, so the binding keeps its own cost to a few
# microseconds: arguments go to the library as one packed struct (the layout of the ctypes class of the same name)
# and the current stream and device come from torch's raw accessors.

def _packer(cls):
    kinds = {ctypes.c_void_p: "P", ctypes.c_int64: "q", ctypes.c_float: "f", ctypes.c_int32: "i"}
    return struct.Struct("".join(kinds[t] for _, t in cls._fields_)).pack


_pack_norm, _pack_norm_backward = _packer(MuonBlockNormArgs), _packer(MuonBlockNormBackwardArgs)
_pack_logp, _pack_logp_backward = _packer(MuonTokenLogpArgs), _packer(MuonTokenLogpBackwardArgs)
_pack_preference, _pack_policy = _packer(MuonPreferenceArgs), _packer(MuonPolicyArgs)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _raw_stream(stream, first, *others):
    """The stream to launch on; every tensor has to be on ``first``'s device, the current GPU."""
    import torch
    dev = first.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensors must be on the current GPU, got {first.device}")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors must share one device, got {first.device} and {t.device}")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _pitch(t, what, shape, dtype):
    """Row pitch in elements of a matrix that has to have this shape and dtype and unit column stride."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype} of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    pitch, step = t.stride()
    rows, cols = shape
    if step != 1 and cols > 1:
        raise ValueError(f"{what} must have unit column stride")
    if rows <= 1:
        return cols
    if pitch < cols:
        raise ValueError(f"{what} has overlapping rows")
    return pitch


def _check_vector(t, what, n, *dtypes):
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous vector of {n}, got {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{what} must be one of {dtypes}, got {t.dtype}")


def _size(size_fn, packed) -> int:
    need = size_fn(packed)
    if need == 0:
        raise MuonError(MUON_ERR_INVALID_ARG, muon_last_error_message())
    return int(need)


def _call(fn, size_fn, packed, workspace, device, stream, raw):
    """Runs one operator with the caller's workspace or one of its own; returns the workspace."""
    if workspace is None:
        workspace = _workspace_for(_size(size_fn, packed), None, device, stream)
    elif stream is not None:
        workspace = _workspace_for(0, workspace, device, stream)
    _check(fn(packed, workspace.data_ptr(), workspace.numel() * workspace.element_size(), raw))
    return workspace


def _norm_weights(x, post_weight, gate, pre_weight):
    """(weight dtype code, gate kind, gate pitch) of the norm's weights, checked against x."""
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D, got shape {tuple(x.shape)}")
    cols = x.shape[1]
    kind, ld_gate, dtype = GATE_NONE, cols, None
    if post_weight is not None:
        dtype = post_weight.dtype
        _check_vector(post_weight, "post_weight", cols, dtype)
    if gate is not None:
        if gate.dim() == 1:
            kind = GATE_CHANNEL
            dtype = dtype or gate.dtype
            _check_vector(gate, "gate", cols, dtype)
        else:
            kind = GATE_FULL
            ld_gate = _pitch(gate, "gate", x.shape, x.dtype)
    if pre_weight is not None:
        dtype = dtype or pre_weight.dtype
        _check_vector(pre_weight, "pre_weight", cols, dtype)
    return _dtype_code(x if dtype is None else dtype), kind, ld_gate


def _check_rstd(rstd, rows):
    import torch
    if rstd.dtype != torch.float32 or rstd.shape != (2, rows) or not rstd.is_contiguous():
        raise ValueError(f"rstd must be contiguous float32 of shape (2, {rows})")


def muon_block_norm(x, residual, out_residual, out_norm=None, *, post_weight=None, gate=None, pre_weight=None,
                    rstd=None, residual_scale=1.0, eps=1e-6, stream=None):
    """Post-norm of a block's output, its gated and scaled residual add, and the next block's pre-norm.

    ``out_residual = residual_scale * residual + gate * (x / rms(x) * post_weight)`` and
    ``out_norm = out_residual / rms(out_residual) * pre_weight``, ``rms(v) = sqrt(mean(v^2) + eps)`` per row.
    Without ``post_weight`` x is taken as it is; ``gate`` is a vector over the columns, a matrix like x, or None;
    ``out_norm`` and ``pre_weight`` go together.  ``out_residual`` may be ``residual`` itself.  ``rstd`` (float32,
    2 x rows) keeps the two inverse rms for :func:`muon_block_norm_backward`.
    """
    wdt, kind, ld_gate = _norm_weights(x, post_weight, gate, pre_weight)
    shape, dtype = x.shape, x.dtype
    rows, cols = shape
    if rstd is not None:
        _check_rstd(rstd, rows)
    packed = _pack_norm(
        x.data_ptr(), residual.data_ptr(), _ptr(post_weight), _ptr(gate), _ptr(pre_weight), out_residual.data_ptr(),
        _ptr(out_norm), _ptr(rstd), rows, cols, _pitch(x, "x", shape, dtype),
        _pitch(residual, "residual", shape, dtype), ld_gate, _pitch(out_residual, "out_residual", shape, dtype),
        cols if out_norm is None else _pitch(out_norm, "out_norm", shape, dtype), residual_scale, eps, _dtype_code(x),
        wdt, kind)
    raw = _raw_stream(stream, x, residual, post_weight, gate, pre_weight, out_residual, out_norm, rstd)
    _check(load().muon_block_norm(packed, raw))


def muon_block_norm_backward_workspace_bytes(x, *, post_weight=None, gate=None, pre_weight=None) -> int:
    """Workspace of :func:`muon_block_norm_backward` for these shapes (gradients shaped like what they are of)."""
    wdt, kind, ld_gate = _norm_weights(x, post_weight, gate, pre_weight)
    rows, cols = x.shape
    # sizes only: distinct stand-in addresses, never dereferenced
    at = iter(range(1 << 44, 1 << 62, 1 << 44))

    def some(t=x):
        return 0 if t is None else next(at)
    packed = _pack_norm_backward(
        some(), some(), some(), some() if pre_weight is not None else 0, some(), some(post_weight), some(gate),
        some(pre_weight), some(), some(), some(post_weight), some(gate), some(pre_weight), rows, cols,
        cols, cols, cols, cols, cols, cols, cols, cols, 1.0, _dtype_code(x), wdt, kind)
    return _size(load().muon_block_norm_backward_workspace_bytes, packed)


def muon_block_norm_backward(x, out_residual, rstd, grad_norm, grad_x, grad_residual, *, grad_out_residual=None,
                             post_weight=None, gate=None, pre_weight=None, grad_post_weight=None, grad_gate=None,
                             grad_pre_weight=None, residual_scale=1.0, workspace=None, stream=None):
    """Gradients of :func:`muon_block_norm`.

    ``grad_norm`` and ``grad_out_residual`` are the gradients of its two outputs (either may be None);
    ``out_residual`` and ``rstd`` are what it wrote.  ``grad_residual`` may be ``grad_out_residual`` itself.
    Weight gradients are summed over the rows.
    """
    wdt, kind, ld_gate = _norm_weights(x, post_weight, gate, pre_weight)
    shape, dtype = x.shape, x.dtype
    rows, cols = shape
    _check_rstd(rstd, rows)
    for w, g, what in ((post_weight, grad_post_weight, "post_weight"), (pre_weight, grad_pre_weight, "pre_weight"),
                       (gate, grad_gate, "gate")):
        if (w is None) != (g is None):
            raise ValueError(f"{what} and its gradient go together")
        if g is not None and w.dim() == 1:
            _check_vector(g, f"gradient of {what}", cols, w.dtype)

    def pitch(t, what):
        return cols if t is None else _pitch(t, what, shape, dtype)
    packed = _pack_norm_backward(
        x.data_ptr(), out_residual.data_ptr(), rstd.data_ptr(), _ptr(grad_norm), _ptr(grad_out_residual),
        _ptr(post_weight), _ptr(gate), _ptr(pre_weight), grad_x.data_ptr(), grad_residual.data_ptr(),
        _ptr(grad_post_weight), _ptr(grad_gate), _ptr(grad_pre_weight), rows, cols, pitch(x, "x"),
        pitch(out_residual, "out_residual"), pitch(grad_norm, "grad_norm"),
        pitch(grad_out_residual, "grad_out_residual"), ld_gate, pitch(grad_x, "grad_x"),
        pitch(grad_residual, "grad_residual"), pitch(grad_gate, "grad_gate") if kind == GATE_FULL else cols,
        residual_scale, _dtype_code(x), wdt, kind)
    raw = _raw_stream(stream, x, out_residual, rstd, grad_norm, grad_out_residual, post_weight, gate, pre_weight,
                      grad_x, grad_residual, grad_post_weight, grad_gate, grad_pre_weight, workspace)
    lib = load()
    return _call(lib.muon_block_norm_backward, lib.muon_block_norm_backward_workspace_bytes, packed, workspace,
                 x.device, stream, raw)


def _logp_shape(hidden, head):
    """(tokens, cols, vocab, pitch of hidden, pitch of head, dtype code)."""
    dtype = hidden.dtype
    if hidden.dim() != 2 or head.dim() != 2 or hidden.shape[1] != head.shape[1] or head.dtype != dtype:
        raise ValueError(f"hidden {tuple(hidden.shape)} {dtype} and head {tuple(head.shape)} {head.dtype} "
                         "must be matrices of one dtype and width")
    tokens, cols = hidden.shape
    return (tokens, cols, head.shape[0], _pitch(hidden, "hidden", hidden.shape, dtype),
            _pitch(head, "head", head.shape, dtype), _dtype_code(dtype))


def _logp_stand_ins(hidden, head):
    """Stand-in addresses for calls that ask for sizes, never dereferenced; aligned like the operands."""
    at = [k << 44 for k in range(1, 9)]
    return [at[0] + hidden.data_ptr() % 256, at[1] + head.data_ptr() % 256] + at[2:]


def muon_token_logp_saved_bytes(hidden, head) -> int:
    """Bytes of the ``saved`` buffer that :func:`muon_token_logp` can keep for the backward pass."""
    tokens, cols, vocab, ldh, ldw, code = _logp_shape(hidden, head)
    return _size(load().muon_token_logp_saved_bytes,
                 _pack_logp(*_logp_stand_ins(hidden, head)[:5], 0, tokens, cols, vocab, ldh, ldw, 1.0, code))


def muon_token_logp_workspace_bytes(hidden, head) -> int:
    """Workspace of :func:`muon_token_logp` for these operands, with ``saved`` or without."""
    tokens, cols, vocab, ldh, ldw, code = _logp_shape(hidden, head)
    at = _logp_stand_ins(hidden, head)
    size = load().muon_token_logp_workspace_bytes
    return max(_size(size, _pack_logp(*at[:5], saved, tokens, cols, vocab, ldh, ldw, 1.0, code)) for saved in (0, at[5]))


def _check_saved(lib, saved, packed):
    if saved is not None:
        need, have = lib.muon_token_logp_saved_bytes(packed), saved.numel() * saved.element_size()
        if have < need:
            raise MuonError(MUON_ERR_WORKSPACE, f"saved has {have} bytes, {need} needed")


def muon_token_logp(hidden, head, targets, logp, lse, *, scale=1.0, saved=None, workspace=None, stream=None):
    """``logp[i] = z[i, targets[i]] - lse[i]`` with ``z = scale * hidden @ head.T`` and ``lse`` its log-sum-exp.

    The tokens x vocab logits never exist as an output.  ``targets`` is int64; a negative one marks a token that is
    not scored (logp = lse = 0).  ``logp`` and ``lse`` are float32.  ``saved`` (uint8, at least
    :func:`muon_token_logp_saved_bytes`) keeps what spares the backward pass the logits' product.
    """
    import torch
    tokens, cols, vocab, ldh, ldw, code = _logp_shape(hidden, head)
    _check_vector(targets, "targets", tokens, torch.int64)
    _check_vector(logp, "logp", tokens, torch.float32)
    _check_vector(lse, "lse", tokens, torch.float32)
    packed = _pack_logp(hidden.data_ptr(), head.data_ptr(), targets.data_ptr(), logp.data_ptr(), lse.data_ptr(),
                        _ptr(saved), tokens, cols, vocab, ldh, ldw, scale, code)
    raw = _raw_stream(stream, head, hidden, targets, logp, lse, saved, workspace)
    lib = load()
    _check_saved(lib, saved, packed)
    return _call(lib.muon_token_logp, lib.muon_token_logp_workspace_bytes, packed, workspace, head.device, stream, raw)


def muon_token_logp_backward_workspace_bytes(hidden, head, *, use_saved=False) -> int:
    tokens, cols, vocab, ldh, ldw, code = _logp_shape(hidden, head)
    at = _logp_stand_ins(hidden, head)
    return _size(load().muon_token_logp_backward_workspace_bytes,
                 _pack_logp_backward(*at[:5], at[5] if use_saved else 0, at[6], at[7], tokens, cols, vocab, ldh, ldw,
                                     cols, cols, 1.0, code))


def muon_token_logp_backward(hidden, head, targets, lse, grad_logp, grad_hidden=None, grad_head=None, *, scale=1.0,
                             saved=None, workspace=None, stream=None):
    """Gradients of :func:`muon_token_logp` for the gradient ``grad_logp`` (float32) of its ``logp``.

    ``grad_hidden`` and ``grad_head`` have their operands' dtype and shape; one of them may be None.  ``saved`` is the
    buffer that the forward call filled for the same inputs, or None: then the logits are formed again.
    """
    import torch
    tokens, cols, vocab, ldh, ldw, code = _logp_shape(hidden, head)
    _check_vector(targets, "targets", tokens, torch.int64)
    _check_vector(lse, "lse", tokens, torch.float32)
    _check_vector(grad_logp, "grad_logp", tokens, torch.float32)
    packed = _pack_logp_backward(
        hidden.data_ptr(), head.data_ptr(), targets.data_ptr(), lse.data_ptr(), grad_logp.data_ptr(), _ptr(saved),
        _ptr(grad_hidden), _ptr(grad_head), tokens, cols, vocab, ldh, ldw,
        cols if grad_hidden is None else _pitch(grad_hidden, "grad_hidden", hidden.shape, hidden.dtype),
        cols if grad_head is None else _pitch(grad_head, "grad_head", head.shape, head.dtype), scale, code)
    raw = _raw_stream(stream, head, hidden, targets, lse, grad_logp, saved, grad_hidden, grad_head, workspace)
    lib = load()
    if saved is not None:
        _check_saved(lib, saved, _pack_logp(0, 0, 0, 0, 0, 0, tokens, cols, vocab, cols, cols, scale, code))
    return _call(lib.muon_token_logp_backward, lib.muon_token_logp_backward_workspace_bytes, packed, workspace,
                 head.device, stream, raw)


def _loss_inputs(logp, offsets, mask, loss, grad_logp, *same):
    """Checks shared by the losses; returns (tokens, sequences, dtype code)."""
    import torch
    n, dt = logp.shape[0] if logp.dim() == 1 else -1, logp.dtype
    _check_vector(logp, "logp", n, torch.float32, torch.bfloat16)
    for t, what in same:
        if t is not None:
            _check_vector(t, what, n, dt)
    if grad_logp is not None:
        _check_vector(grad_logp, "grad_logp", n, dt)
    if mask is not None:
        _check_vector(mask, "mask", n, torch.uint8, torch.bool)
    if offsets.dim() != 1 or offsets.shape[0] < 1 or offsets.dtype != torch.int64 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous int64 vector of sequences + 1")
    if loss is not None and (loss.numel() != 1 or loss.dtype != torch.float32):
        raise ValueError("loss must be one float32")
    return n, offsets.shape[0] - 1, _dtype_code(dt)


def _choice(table, value, what):
    if value not in table:
        raise ValueError(f"unknown {what} {value!r}; one of {sorted(table)}")
    return table[value]


def muon_preference_loss_workspace_bytes(logp, offsets) -> int:
    n, sequences, code = _loss_inputs(logp, offsets, None, None, None)
    return _size(load().muon_preference_loss_workspace_bytes,
                 _pack_preference(1 << 44, 0, 0, 2 << 44, 3 << 44, 0, 4 << 44, n, sequences, 1.0, 0.0, 0.0, 1.0, 0, 0, code))


def muon_preference_loss(logp, offsets, loss, grad_logp=None, *, ref_logp=None, mask=None, beta=0.1, kind="sigmoid",
                         label_smoothing=0.0, margin=0.0, average=False, rewards=None, grad_scale=1.0, workspace=None,
                         stream=None):
    """Mean preference loss over pairs of sequences, and its gradient with respect to ``logp``.

    Sequence s is ``logp[offsets[s]:offsets[s + 1]]`` (offsets: int64 on the GPU); sequence 2p is preferred to
    2p + 1.  Tokens with ``mask`` 0 count for nothing.  ``kind`` is "sigmoid", "hinge" or "squared"; ``average``
    divides each sequence's log ratio by its counted tokens.  ``rewards`` (float32, one per sequence) receives
    ``beta`` times the log ratios.  ``grad_logp`` is scaled by ``grad_scale``.
    """
    import torch
    n, sequences, code = _loss_inputs(logp, offsets, mask, loss, grad_logp, (ref_logp, "ref_logp"))
    if rewards is not None:
        _check_vector(rewards, "rewards", sequences, torch.float32)
    packed = _pack_preference(logp.data_ptr(), _ptr(ref_logp), _ptr(mask), offsets.data_ptr(), loss.data_ptr(),
                              _ptr(rewards), _ptr(grad_logp), n, sequences, beta, margin, label_smoothing, grad_scale,
                              _choice(PREFERENCE_KINDS, kind, "kind"), 1 if average else 0, code)
    raw = _raw_stream(stream, offsets, logp, ref_logp, mask, loss, rewards, grad_logp, workspace)
    lib = load()
    return _call(lib.muon_preference_loss, lib.muon_preference_loss_workspace_bytes, packed, workspace, offsets.device,
                 stream, raw)


def muon_policy_loss_workspace_bytes(logp, offsets) -> int:
    n, sequences, code = _loss_inputs(logp, offsets, None, None, None)
    return _size(load().muon_policy_loss_workspace_bytes,
                 _pack_policy(1 << 44, 2 << 44, 0, 3 << 44, 0, 4 << 44, 5 << 44, 0, 6 << 44, n, sequences, 0.2, 0.2, 0.0,
                              0.0, 1.0, 0, 0, 0, code))


def muon_policy_loss(logp, old_logp, advantages, offsets, loss, grad_logp=None, *, ref_logp=None, mask=None,
                     clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0, kl="none", reduction="token",
                     per_sequence=False, stats=None, grad_scale=1.0, workspace=None, stream=None):
    """Clipped policy loss with a KL term, and its gradient with respect to ``logp``.

    ``advantages`` (float32) is one per token, or one per sequence with ``per_sequence``.  ``kl`` is "none", "k1",
    "k2" or "k3" (then with ``ref_logp``), ``reduction`` "token" or "sequence".  ``stats`` (float32, 4) receives the
    mean KL, the share of tokens held at a bound, the mean ratio and the number of counted tokens.  Sequences,
    ``mask`` and ``grad_scale`` are as in :func:`muon_preference_loss`.
    """
    import torch
    n, sequences, code = _loss_inputs(logp, offsets, mask, loss, grad_logp, (old_logp, "old_logp"),
                                      (ref_logp, "ref_logp"))
    _check_vector(advantages, "advantages", sequences if per_sequence else n, torch.float32)
    if stats is not None:
        _check_vector(stats, "stats", 4, torch.float32)
    packed = _pack_policy(logp.data_ptr(), old_logp.data_ptr(), _ptr(ref_logp), advantages.data_ptr(), _ptr(mask),
                          offsets.data_ptr(), loss.data_ptr(), _ptr(stats), _ptr(grad_logp), n, sequences, clip_low,
                          clip_high, dual_clip, kl_coef, grad_scale, _choice(KL_KINDS, kl, "kl"),
                          _choice(LOSS_REDUCTIONS, reduction, "reduction"), 1 if per_sequence else 0, code)
    raw = _raw_stream(stream, offsets, logp, old_logp, ref_logp, advantages, mask, loss, stats, grad_logp, workspace)
    lib = load()
    return _call(lib.muon_policy_loss, lib.muon_policy_loss_workspace_bytes, packed, workspace, offsets.device, stream,
                 raw)


def muon_profile_enable(on: bool = True):
    _check(load().muon_profile_enable(1 if on else 0))


def muon_profile_read() -> dict:
    n = len(KERNEL_CLASSES)
    ms, launches = (ctypes.c_double * n)(), (ctypes.c_int64 * n)()
    _check(load().muon_profile_read_classes(n, ms, launches))
    return {name: {"ms": ms[i], "launches": int(launches[i])} for i, name in enumerate(KERNEL_CLASSES)}
