"""MI355X (gfx950) selective scan of Mamba-1 (S6): Python binding of ``libssm.so``.

Argument marshalling only.  Every step of the computation runs in the HIP
kernels behind the C ABI declared in ``include/ssm.h``; this module checks
shapes, dtypes and devices, allocates outputs with PyTorch (device memory
and streams are PyTorch's job here), and calls the library on the current
PyTorch stream of the tensors' device.  There is no CPU fallback: if the
library is missing or the tensors are not on a GPU, the call raises.

Functions (same names as the C entry points):

* ``ssm_scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None,
  softplus=False, y=None, last_state=None, return_last_state=True,
  initial_state=None, saved_states=None, tuning=None)`` -> ``(y, last_state)``;
  ``tuning`` (a dict with keys ``path`` in "auto" / "chunked" /
  "single_pass", ``min_chunk``, ``target_waves``) selects the C entry point
  ``ssm_scan_fwd_tuned``
* ``ssm_scan_fwd_noalloc(u, delta, A, B, C, D=None, z=None, delta_bias=None,
  softplus=False, initial_state=None, y=None, last_state=None)`` ->
  ``(y, last_state)``: the same scan with the library's fixed workspace buffer
  (no device allocation in the library)
* ``ssm_scan_plan(b, L, E, N, dtype="bf16", tuning=None)`` ->
  ``(path, chunk_len, n_chunks)``: how the forward runs at that size
* ``ssm_state_update(state, x, delta, A, B, C, D=None, z=None,
  delta_bias=None, softplus=False, y=None)`` -> ``y`` (``state`` is updated
  in place)
* ``ssm_scan_bwd(u, delta, A, B, C, dy, D=None, z=None, delta_bias=None,
  softplus=False, initial_state=None, d_last_state=None)`` -> dict of
  gradients (du, ddelta, dA, dB, dC, dD, dz, d_delta_bias, d_initial_state)
* ``ssm_ssd_fwd(x, delta, A, B, C, D=None, z=None, delta_bias=None,
  softplus=False, initial_state=None, y=None, last_state=None,
  return_last_state=True)`` -> ``(y, last_state)``: the scan with a scalar
  transition per head (x [b, L, H*64], delta [b, L, H], A, D, delta_bias [H]),
  bf16 only
* ``ssm_linattn_fwd(q, k, v, g=None, A=None, scale=None, lengths=None,
  initial_state=None, y=None, last_state=None, return_last_state=True)`` ->
  ``(y, last_state)``: linear attention with a decay for each head over whole
  sequences; ``ssm_linattn_bwd`` its gradients, ``ssm_linattn_update`` its step
  for one token
* ``ssm_deltarule_fwd(q, k, v, beta=None, g=None, A=None, scale=None,
  lengths=None, initial_state=None, y=None, last_state=None,
  return_last_state=True)`` -> ``(y, last_state)``: the gated delta rule over
  whole sequences; ``ssm_deltarule_bwd`` its gradients,
  ``ssm_deltarule_update`` its step for one token
* ``ssm_layernorm_fwd(x, weight=None, bias=None, eps=1e-5, y=None)`` ->
  ``(y, mean, rstd)``: layer norm over the last axis; ``ssm_layernorm_bwd`` its
  gradients
* ``ssm_blocknorm_fwd(x, post_weight=None, z=None, scale=None, residual=None,
  pre_weight=None, norms="both", eps=1e-5, return_h=True, h=None, n=None)`` ->
  ``(h, n, rstd_post, rstd_pre)``: what stands between two blocks, RMS norm
  after one, gate, scale, residual, RMS norm before the next;
  ``ssm_blocknorm_bwd`` its gradients
* ``ssm_conv_fwd(v, weight, conv_bias=None, state_in=None, x=None,
  state_out=None, return_state=True)`` -> ``(x, state_out)``: causal depthwise
  convolution + SiLU over the sequence
* ``ssm_conv_update(conv_state, v, weight, conv_bias=None, x=None)`` -> ``x``
  (``conv_state`` is shifted and appended to in place)

Shapes: u, delta, z, y [b, L, E]; A [E, N] (float32); B, C [b, L, N];
D, delta_bias [E] (float32); state / last_state [b, E, N] (float32).
Linear attention and the delta rule: q, k [b, L, G, Dk]; v, y [b, L, H, Dv];
beta, g [b, L, H]; A [H] float32; lengths [b] int32; states [b, H, Dk, Dv] float32 (G divides H;
Dk, Dv <= 128).
Convolution: v, x [b, L, E]; weight [E, K] float32 (1 <= K <= 8); conv_bias
[E] float32; convolution state [b, E, K] in the streamed dtype, oldest sample
first.  Streamed tensors are all float32 or all bfloat16.
"""
import contextlib
import ctypes
import os

__all__ = [
    "ssm_scan_fwd", "ssm_scan_fwd_from", "ssm_scan_fwd_noalloc", "ssm_scan_bwd", "ssm_ssd_fwd", "ssm_state_update", "ssm_conv_fwd", "ssm_conv_update",
    "ssm_linattn_fwd", "ssm_linattn_bwd", "ssm_linattn_update", "ssm_linattn_workspace",
    "ssm_deltarule_fwd", "ssm_deltarule_bwd", "ssm_deltarule_update", "ssm_deltarule_workspace",
    "ssm_layernorm_fwd", "ssm_layernorm_bwd", "ssm_layernorm_workspace",
    "ssm_blocknorm_fwd", "ssm_blocknorm_bwd", "ssm_blocknorm_workspace", "ssm_scan_plan", "ssm_profile_enable", "ssm_profile_read",
    "ssm_status_string", "library_path", "SSMError", "ScanTuning", "SCAN_PATHS",
    "SSM_F32", "SSM_BF16", "load_library",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libssm.so")
_lib = None

SSM_F32 = 0
SSM_BF16 = 1

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_f32 = ctypes.c_float


# ssm_scan_path values
SCAN_PATHS = {"auto": 0, "chunked": 1, "single_pass": 2}
_PATH_NAMES = {v: k for k, v in SCAN_PATHS.items()}


class ScanTuning(ctypes.Structure):
    """``ssm_scan_tuning``: path (ssm_scan_path), min_chunk, target_waves; zero fields mean the library's choice."""
    _fields_ = [("path", ctypes.c_int32), ("min_chunk", ctypes.c_int32), ("target_waves", ctypes.c_int32)]


def _tuning(tuning):
    """A ScanTuning from None, a ScanTuning or a dict {path, min_chunk, target_waves}."""
    if tuning is None or isinstance(tuning, ScanTuning):
        return tuning
    unknown = set(tuning) - {"path", "min_chunk", "target_waves"}
    if unknown:
        raise ValueError(f"unknown tuning keys {sorted(unknown)}")
    path = tuning.get("path", "auto")
    return ScanTuning(SCAN_PATHS[path] if isinstance(path, str) else int(path), int(tuning.get("min_chunk", 0)),
                      int(tuning.get("target_waves", 0)))


class SSMError(RuntimeError):
    """A call into libssm.so returned a non-zero ssm_status."""

    def __init__(self, fn, status, detail=""):
        self.status = status
        msg = f"{fn} failed: {ssm_status_string(status)} (status {status})"
        if detail:
            msg += f": {detail}"
        super().__init__(msg)


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libssm.so (built in-tree by ``python -m selective_state_space_35_amd.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is missing: build the HIP library first "
            "(python -m selective_state_space_35_amd.build)")
    lib = ctypes.CDLL(_LIB_PATH)
    lib.ssm_scan_fwd.restype = _int
    lib.ssm_scan_fwd.argtypes = [_vp] * 8 + [_int, _vp, _vp] + [_i64] * 4 + [_int, _vp]
    lib.ssm_scan_fwd_from.restype = _int
    lib.ssm_scan_fwd_from.argtypes = [_vp] * 8 + [_int, _vp, _vp, _vp] + [_i64] * 4 + [_int, _vp]
    lib.ssm_scan_fwd_save.restype = _int
    lib.ssm_scan_fwd_save.argtypes = [_vp] * 8 + [_int, _vp, _vp, _vp, _vp] + [_i64] * 4 + [_int, _vp]
    lib.ssm_scan_fwd_noalloc.restype = _int
    lib.ssm_scan_fwd_noalloc.argtypes = [_vp] * 8 + [_int, _vp, _vp, _vp] + [_i64] * 4 + [_int, _vp]
    lib.ssm_scan_fwd_tuned.restype = _int
    lib.ssm_scan_fwd_tuned.argtypes = ([_vp] * 8 + [_int, _vp, _vp, _vp, _vp, ctypes.POINTER(ScanTuning)] +
                                       [_i64] * 4 + [_int, _vp])
    lib.ssm_state_update.restype = _int
    lib.ssm_state_update.argtypes = [_vp] * 9 + [_int, _vp] + [_i64] * 3 + [_int, _vp]
    lib.ssm_scan_bwd.restype = _int
    lib.ssm_scan_bwd.argtypes = [_vp] * 8 + [_int] + [_vp] * 12 + [_i64] * 4 + [_int, _vp]
    lib.ssm_scan_bwd_saved.restype = _int
    lib.ssm_scan_bwd_saved.argtypes = [_vp] * 8 + [_int] + [_vp] * 13 + [_i64] * 4 + [_int, _vp]
    lib.ssm_ssd_fwd.restype = _int
    lib.ssm_ssd_fwd.argtypes = [_vp] * 8 + [_int] + [_vp] * 3 + [_i64] * 5 + [_int, _vp]
    lib.ssm_conv_fwd.restype = _int
    lib.ssm_conv_fwd.argtypes = [_vp] * 6 + [_i64] * 4 + [_int, _vp]
    lib.ssm_conv_update.restype = _int
    lib.ssm_conv_update.argtypes = [_vp] * 5 + [_i64] * 3 + [_int, _vp]
    lib.ssm_linattn_fwd.restype = _int
    lib.ssm_linattn_fwd.argtypes = [_vp] * 6 + [_f32] + [_vp] * 3 + [_i64] * 6 + [_int, _vp, _i64, _vp]
    lib.ssm_linattn_bwd.restype = _int
    lib.ssm_linattn_bwd.argtypes = [_vp] * 6 + [_f32] + [_vp] * 8 + [_i64] * 6 + [_int, _vp, _i64, _vp]
    lib.ssm_linattn_update.restype = _int
    lib.ssm_linattn_update.argtypes = [_vp] * 7 + [_f32, _vp] + [_i64] * 5 + [_int, _vp]
    lib.ssm_linattn_workspace.restype = _i64
    lib.ssm_linattn_workspace.argtypes = [_i64] * 6 + [_int, _int]
    lib.ssm_deltarule_fwd.restype = _int
    lib.ssm_deltarule_fwd.argtypes = [_vp] * 7 + [_f32] + [_vp] * 3 + [_i64] * 6 + [_int, _vp, _i64, _vp]
    lib.ssm_deltarule_bwd.restype = _int
    lib.ssm_deltarule_bwd.argtypes = [_vp] * 7 + [_f32] + [_vp] * 9 + [_i64] * 6 + [_int, _vp, _i64, _vp]
    lib.ssm_deltarule_update.restype = _int
    lib.ssm_deltarule_update.argtypes = [_vp] * 8 + [_f32, _vp] + [_i64] * 5 + [_int, _vp]
    lib.ssm_deltarule_workspace.restype = _i64
    lib.ssm_deltarule_workspace.argtypes = [_i64] * 6 + [_int, _int]
    lib.ssm_layernorm_fwd.restype = _int
    lib.ssm_layernorm_fwd.argtypes = [_vp] * 3 + [_f32] + [_vp] * 3 + [_i64] * 3 + [_int, _vp]
    lib.ssm_layernorm_bwd.restype = _int
    lib.ssm_layernorm_bwd.argtypes = [_vp] * 8 + [_i64] * 3 + [_int, _vp, _i64, _vp]
    lib.ssm_layernorm_workspace.restype = _i64
    lib.ssm_layernorm_workspace.argtypes = [_i64] * 3 + [_int]
    lib.ssm_blocknorm_fwd.restype = _int
    lib.ssm_blocknorm_fwd.argtypes = [_vp] * 6 + [_f32, _int] + [_vp] * 4 + [_i64] * 3 + [_int, _int, _vp]
    lib.ssm_blocknorm_bwd.restype = _int
    lib.ssm_blocknorm_bwd.argtypes = [_vp] * 6 + [_int] + [_vp] * 10 + [_i64] * 3 + [_int, _int, _vp, _i64, _vp]
    lib.ssm_blocknorm_workspace.restype = _i64
    lib.ssm_blocknorm_workspace.argtypes = [_i64] * 3 + [_int, _int]
    lib.ssm_status_string.restype = ctypes.c_char_p
    lib.ssm_status_string.argtypes = [_int]
    lib.ssm_last_hip_error.restype = ctypes.c_char_p
    lib.ssm_last_hip_error.argtypes = []
    lib.ssm_version.restype = _int
    lib.ssm_version.argtypes = []
    lib.ssm_profile_enable.restype = _int
    lib.ssm_profile_enable.argtypes = [_int]
    lib.ssm_profile_read.restype = _int
    lib.ssm_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_i64), _int]
    lib.ssm_profile_kind_name.restype = ctypes.c_char_p
    lib.ssm_profile_kind_name.argtypes = [_int]
    lib.ssm_scan_plan.restype = _int
    lib.ssm_scan_plan.argtypes = [_i64, _i64, _i64, _i64, _int, ctypes.POINTER(ScanTuning), ctypes.POINTER(_int),
                                  ctypes.POINTER(_i64), ctypes.POINTER(_i64)]
    _lib = lib
    return lib


def ssm_status_string(status: int) -> str:
    return load_library().ssm_status_string(int(status)).decode()


def ssm_scan_plan(b, L, E, N, dtype="bf16", tuning=None):
    """(path, chunk_len, n_chunks) of a forward scan of this size (host-only query).

    path is "chunked" or "single_pass"; see ssm_scan_plan in include/ssm.h.
    """
    code = {"f32": SSM_F32, "bf16": SSM_BF16}.get(dtype, dtype)
    t = _tuning(tuning)
    path, cl, nc = _int(0), _i64(0), _i64(0)
    status = load_library().ssm_scan_plan(int(b), int(L), int(E), int(N), int(code),
                                          ctypes.byref(t) if t is not None else None, ctypes.byref(path),
                                          ctypes.byref(cl), ctypes.byref(nc))
    _raise_on("ssm_scan_plan", status)
    return _PATH_NAMES[path.value], cl.value, nc.value


PROFILE_KINDS = 35
_SCAN_KINDS = 17  # the kinds of the scans and the convolution, always in the answer


def ssm_profile_enable(on=True):
    """Bracket every library kernel with HIP events on its stream (benchmark timing)."""
    load_library().ssm_profile_enable(int(bool(on)))


def ssm_profile_read():
    """Wait for the recorded events; return {kind name: (total ms, launches)} and clear the record.

    The kinds of linear attention, the delta rule and the norms are there where they ran.
    """
    lib = load_library()
    ms = (ctypes.c_double * PROFILE_KINDS)()
    cnt = (_i64 * PROFILE_KINDS)()
    _raise_on("ssm_profile_read", lib.ssm_profile_read(ms, cnt, PROFILE_KINDS))
    return {lib.ssm_profile_kind_name(k).decode(): (ms[k], cnt[k]) for k in range(PROFILE_KINDS)
            if k < _SCAN_KINDS or cnt[k]}


def _ptr(t):
    return None if t is None else t.data_ptr()  # an int: ctypes passes it as the void* argument


def _dtype_code(torch, dt):
    if dt == torch.float32:
        return SSM_F32
    if dt == torch.bfloat16:
        return SSM_BF16
    raise TypeError(f"streamed tensors must be float32 or bfloat16, got {dt}")


def _check(torch, name, t, shape, dtype, device, optional=False):
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    try:  # the common case in one pass; anything off falls through to the checks that name it
        if t.dtype is dtype and t.shape == shape and t.get_device() == device.index and t.is_contiguous():
            return
    except (AttributeError, TypeError):
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream_of(torch, device):
    """The current PyTorch stream of ``device`` as a raw handle."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(device.index)
    return torch.cuda.current_stream(device).cuda_stream


_NULL_CTX = contextlib.nullcontext()


def _on(torch, device):
    """A context with ``device`` current: a no-op when it already is (switching costs microseconds)."""
    get = getattr(torch._C, "_cuda_getDevice", None)
    current = get() if get is not None else torch.cuda.current_device()
    return _NULL_CTX if current == device.index else torch.cuda.device(device)


def _raise_on(fn, status):
    if status != 0:
        detail = load_library().ssm_last_hip_error().decode() if status == -6 else ""
        raise SSMError(fn, status, detail)


SAVE_INTERVAL = 64  # SSM_SAVE_INTERVAL of include/ssm.h


def saved_states_shape(b, L, E, N):
    """Shape of the states ``ssm_scan_fwd_save`` keeps: one [E, N] slice per 64 steps but the last."""
    return (b, max((L + SAVE_INTERVAL - 1) // SAVE_INTERVAL - 1, 0), E, N)


def _scan_outputs(torch, u, delta, A, B, C, D, z, delta_bias, y, last_state, return_last_state, initial_state,
                  saved_states):
    """Checks the forward's tensors; returns (b, L, E, N, dtype code, device, y, last_state)."""
    if not isinstance(u, torch.Tensor) or u.dim() != 3:
        raise ValueError("u must be a [b, L, E] tensor")
    device = u.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU device, got {device}")
    b, L, E = u.shape
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be an [E, N] tensor")
    N = A.shape[1]
    io = u.dtype
    code = _dtype_code(torch, io)
    _check(torch, "delta", delta, (b, L, E), io, device)
    _check(torch, "A", A, (E, N), torch.float32, device)
    _check(torch, "B", B, (b, L, N), io, device)
    _check(torch, "C", C, (b, L, N), io, device)
    _check(torch, "D", D, (E,), torch.float32, device, optional=True)
    _check(torch, "z", z, (b, L, E), io, device, optional=True)
    _check(torch, "delta_bias", delta_bias, (E,), torch.float32, device, optional=True)
    _check(torch, "u", u, (b, L, E), io, device)
    if y is None:
        y = torch.empty((b, L, E), dtype=io, device=device)
    else:
        _check(torch, "y", y, (b, L, E), io, device)
    if last_state is None and return_last_state:
        last_state = torch.empty((b, E, N), dtype=torch.float32, device=device)
    elif last_state is not None:
        _check(torch, "last_state", last_state, (b, E, N), torch.float32, device)
    _check(torch, "initial_state", initial_state, (b, E, N), torch.float32, device, optional=True)
    if initial_state is not None and last_state is not None and initial_state.data_ptr() == last_state.data_ptr():
        raise ValueError("initial_state must not be the last_state buffer")
    if saved_states is not None:
        _check(torch, "saved_states", saved_states, saved_states_shape(b, L, E, N), torch.float32, device)
    return b, L, E, N, code, device, y, last_state


def ssm_scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=False, y=None,
                 last_state=None, return_last_state=True, initial_state=None, saved_states=None, tuning=None):
    """Selective scan forward on the GPU.  Returns ``(y, last_state)`` (last_state None if not requested).

    ``initial_state`` [b, E, N] float32 continues the recurrence from that state
    (the C entry point ``ssm_scan_fwd_from``); None starts from zero.  A given
    ``saved_states`` buffer (``saved_states_shape``, float32) receives the state
    every 64 steps (the C entry point ``ssm_scan_fwd_save``).  ``tuning`` (dict
    or ScanTuning) fixes the form and split (the C entry point ``ssm_scan_fwd_tuned``).
    """
    import torch

    lib = load_library()
    b, L, E, N, code, device, y, last_state = _scan_outputs(torch, u, delta, A, B, C, D, z, delta_bias, y, last_state,
                                                            return_last_state, initial_state, saved_states)
    t = _tuning(tuning)
    if t is not None:
        with _on(torch, device):
            status = lib.ssm_scan_fwd_tuned(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                                            _ptr(delta_bias), int(bool(softplus)), _ptr(initial_state), _ptr(y),
                                            _ptr(last_state), _ptr(saved_states), ctypes.byref(t), b, L, E, N, code,
                                            _stream_of(torch, device))
        _raise_on("ssm_scan_fwd_tuned", status)
        return y, last_state
    if saved_states is not None:
        with _on(torch, device):
            status = lib.ssm_scan_fwd_save(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                                           _ptr(delta_bias), int(bool(softplus)), _ptr(initial_state), _ptr(y),
                                           _ptr(last_state), _ptr(saved_states), b, L, E, N, code,
                                           _stream_of(torch, device))
        _raise_on("ssm_scan_fwd_save", status)
        return y, last_state
    with _on(torch, device):
        if initial_state is None:
            status = lib.ssm_scan_fwd(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                                      _ptr(delta_bias), int(bool(softplus)), _ptr(y), _ptr(last_state),
                                      b, L, E, N, code, _stream_of(torch, device))
        else:
            status = lib.ssm_scan_fwd_from(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                                           _ptr(delta_bias), int(bool(softplus)), _ptr(initial_state), _ptr(y),
                                           _ptr(last_state), b, L, E, N, code, _stream_of(torch, device))
    _raise_on("ssm_scan_fwd" if initial_state is None else "ssm_scan_fwd_from", status)
    return y, last_state


def ssm_scan_fwd_noalloc(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=False, initial_state=None,
                         y=None, last_state=None, return_last_state=True):
    """``ssm_scan_fwd_from`` whose library side allocates no device memory (the C entry point
    ``ssm_scan_fwd_noalloc``): a workspace comes from the library's fixed buffer.  The outputs y and
    last_state are the caller's; pass them to keep this call free of allocations on the PyTorch side too."""
    import torch

    lib = load_library()
    b, L, E, N, code, device, y, last_state = _scan_outputs(torch, u, delta, A, B, C, D, z, delta_bias, y, last_state,
                                                            return_last_state, initial_state, None)
    with _on(torch, device):
        status = lib.ssm_scan_fwd_noalloc(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                                          _ptr(delta_bias), int(bool(softplus)), _ptr(initial_state), _ptr(y),
                                          _ptr(last_state), b, L, E, N, code, _stream_of(torch, device))
    _raise_on("ssm_scan_fwd_noalloc", status)
    return y, last_state


def ssm_scan_fwd_from(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=False, initial_state=None,
                      y=None, last_state=None, return_last_state=True):
    """``ssm_scan_fwd`` continuing from ``initial_state`` (same name as the C entry point)."""
    return ssm_scan_fwd(u, delta, A, B, C, D, z, delta_bias, softplus, y=y, last_state=last_state,
                        return_last_state=return_last_state, initial_state=initial_state)


def ssm_scan_fwd_save(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=False, initial_state=None,
                      y=None, last_state=None, saved_states=None, tuning=None):
    """``ssm_scan_fwd_from`` that also keeps the state every 64 steps for ``ssm_scan_bwd_saved``.

    Returns ``(y, last_state, saved_states)``; saved_states [b, ceil(L / 64) - 1, E, N] float32 holds
    the state entering steps 64, 128, ...
    """
    import torch

    b, L, E = u.shape
    N = A.shape[1]
    if saved_states is None:
        saved_states = torch.empty(saved_states_shape(b, L, E, N), dtype=torch.float32, device=u.device)
    y, last_state = ssm_scan_fwd(u, delta, A, B, C, D, z, delta_bias, softplus, y=y, last_state=last_state,
                                 initial_state=initial_state, saved_states=saved_states, tuning=tuning)
    return y, last_state, saved_states


def ssm_scan_bwd_saved(u, delta, A, B, C, dy, saved_states, D=None, z=None, delta_bias=None, softplus=False,
                       initial_state=None, d_last_state=None):
    """``ssm_scan_bwd`` with the states entering its chunks from ``ssm_scan_fwd_save``."""
    return ssm_scan_bwd(u, delta, A, B, C, dy, D, z, delta_bias, softplus, initial_state=initial_state,
                        d_last_state=d_last_state, saved_states=saved_states)


def ssm_scan_bwd(u, delta, A, B, C, dy, D=None, z=None, delta_bias=None, softplus=False, initial_state=None,
                 d_last_state=None, saved_states=None):
    """Gradients of sum(dy * y) + sum(d_last_state * last_state) for ``ssm_scan_fwd_from``'s arguments.

    Returns a dict: du, ddelta (and dz when z is given) [b, L, E] in the streamed dtype;
    dA [E, N], dB and dC [b, L, N], d_initial_state [b, E, N], dD and d_delta_bias [E]
    (None when D / delta_bias are None), all float32.  ``saved_states`` from
    ``ssm_scan_fwd_save`` on the same inputs replaces the recomputed chunk states
    (the C entry point ``ssm_scan_bwd_saved``).
    """
    import torch

    lib = load_library()
    if not isinstance(u, torch.Tensor) or u.dim() != 3:
        raise ValueError("u must be a [b, L, E] tensor")
    device = u.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU device, got {device}")
    b, L, E = u.shape
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be an [E, N] tensor")
    N = A.shape[1]
    io = u.dtype
    code = _dtype_code(torch, io)
    f32 = torch.float32
    _check(torch, "u", u, (b, L, E), io, device)
    _check(torch, "delta", delta, (b, L, E), io, device)
    _check(torch, "A", A, (E, N), f32, device)
    _check(torch, "B", B, (b, L, N), io, device)
    _check(torch, "C", C, (b, L, N), io, device)
    _check(torch, "dy", dy, (b, L, E), io, device)
    _check(torch, "D", D, (E,), f32, device, optional=True)
    _check(torch, "z", z, (b, L, E), io, device, optional=True)
    _check(torch, "delta_bias", delta_bias, (E,), f32, device, optional=True)
    _check(torch, "initial_state", initial_state, (b, E, N), f32, device, optional=True)
    _check(torch, "d_last_state", d_last_state, (b, E, N), f32, device, optional=True)
    g = {
        "du": torch.empty((b, L, E), dtype=io, device=device),
        "ddelta": torch.empty((b, L, E), dtype=io, device=device),
        "dz": torch.empty((b, L, E), dtype=io, device=device) if z is not None else None,
        "dA": torch.empty((E, N), dtype=f32, device=device),
        "dB": torch.empty((b, L, N), dtype=f32, device=device),
        "dC": torch.empty((b, L, N), dtype=f32, device=device),
        "dD": torch.empty((E,), dtype=f32, device=device) if D is not None else None,
        "d_delta_bias": torch.empty((E,), dtype=f32, device=device) if delta_bias is not None else None,
        "d_initial_state": torch.empty((b, E, N), dtype=f32, device=device),
    }
    if saved_states is not None:
        _check(torch, "saved_states", saved_states, saved_states_shape(b, L, E, N), f32, device)
        with _on(torch, device):
            status = lib.ssm_scan_bwd_saved(
                _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
                int(bool(softplus)), _ptr(initial_state), _ptr(saved_states), _ptr(dy), _ptr(d_last_state),
                _ptr(g["du"]), _ptr(g["ddelta"]), _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]),
                _ptr(g["dz"]), _ptr(g["d_delta_bias"]), _ptr(g["d_initial_state"]), b, L, E, N, code,
                _stream_of(torch, device))
        _raise_on("ssm_scan_bwd_saved", status)
        return g
    with _on(torch, device):
        status = lib.ssm_scan_bwd(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
                                  int(bool(softplus)), _ptr(initial_state), _ptr(dy), _ptr(d_last_state), _ptr(g["du"]),
                                  _ptr(g["ddelta"]), _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]),
                                  _ptr(g["dz"]), _ptr(g["d_delta_bias"]), _ptr(g["d_initial_state"]), b, L, E, N, code,
                                  _stream_of(torch, device))
    _raise_on("ssm_scan_bwd", status)
    return g


def ssm_ssd_fwd(x, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=False, initial_state=None, y=None,
                last_state=None, return_last_state=True):
    """The scan with a scalar transition per head on the GPU (bf16).  Returns ``(y, last_state)``."""
    import torch

    lib = load_library()
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [b, L, H*P] tensor")
    device = x.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU device, got {device}")
    if not isinstance(delta, torch.Tensor) or delta.dim() != 3:
        raise ValueError("delta must be a [b, L, H] tensor")
    b, L, E = x.shape
    H = delta.shape[2]
    if H == 0 or E % H:
        raise ValueError("the channels of x must split evenly into the heads of delta")
    P = E // H
    N = B.shape[2] if isinstance(B, torch.Tensor) and B.dim() == 3 else -1
    io = x.dtype
    code = _dtype_code(torch, io)
    f32 = torch.float32
    _check(torch, "x", x, (b, L, E), io, device)
    _check(torch, "delta", delta, (b, L, H), io, device)
    _check(torch, "A", A, (H,), f32, device)
    _check(torch, "B", B, (b, L, N), io, device)
    _check(torch, "C", C, (b, L, N), io, device)
    _check(torch, "D", D, (H,), f32, device, optional=True)
    _check(torch, "z", z, (b, L, E), io, device, optional=True)
    _check(torch, "delta_bias", delta_bias, (H,), f32, device, optional=True)
    _check(torch, "initial_state", initial_state, (b, E, N), f32, device, optional=True)
    if y is None:
        y = torch.empty((b, L, E), dtype=io, device=device)
    else:
        _check(torch, "y", y, (b, L, E), io, device)
    if last_state is None and return_last_state:
        last_state = torch.empty((b, E, N), dtype=f32, device=device)
    elif last_state is not None:
        _check(torch, "last_state", last_state, (b, E, N), f32, device)
    with _on(torch, device):
        status = lib.ssm_ssd_fwd(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
                                 int(bool(softplus)), _ptr(initial_state), _ptr(y), _ptr(last_state), b, L, H, P, N,
                                 code, _stream_of(torch, device))
    _raise_on("ssm_ssd_fwd", status)
    return y, last_state


def ssm_state_update(state, x, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=False, y=None):
    """One recurrent step on the GPU; ``state`` [b, E, N] float32 is updated in place.  Returns y [b, E]."""
    import torch

    lib = load_library()
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("state must be a [b, E, N] tensor")
    device = state.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU device, got {device}")
    b, E, N = state.shape
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    io = x.dtype
    code = _dtype_code(torch, io)
    _check(torch, "state", state, (b, E, N), torch.float32, device)
    _check(torch, "x", x, (b, E), io, device)
    _check(torch, "delta", delta, (b, E), io, device)
    _check(torch, "A", A, (E, N), torch.float32, device)
    _check(torch, "B", B, (b, N), io, device)
    _check(torch, "C", C, (b, N), io, device)
    _check(torch, "D", D, (E,), torch.float32, device, optional=True)
    _check(torch, "z", z, (b, E), io, device, optional=True)
    _check(torch, "delta_bias", delta_bias, (E,), torch.float32, device, optional=True)
    if y is None:
        y = torch.empty((b, E), dtype=io, device=device)
    else:
        _check(torch, "y", y, (b, E), io, device)
    with _on(torch, device):
        status = lib.ssm_state_update(_ptr(state), _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                      _ptr(z), _ptr(delta_bias), int(bool(softplus)), _ptr(y), b, E, N, code,
                                      _stream_of(torch, device))
    _raise_on("ssm_state_update", status)
    return y


def ssm_conv_fwd(v, weight, conv_bias=None, state_in=None, x=None, state_out=None, return_state=True):
    """Causal depthwise convolution + SiLU over [b, L, E] on the GPU.  Returns ``(x, state_out)``.

    ``state_in`` [b, E, K] holds the K samples before the sequence (oldest first);
    None pads with zeros.  ``state_out`` receives the K most recent samples.
    """
    import torch

    lib = load_library()
    if not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError("v must be a [b, L, E] tensor")
    device = v.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU device, got {device}")
    b, L, E = v.shape
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be an [E, K] tensor")
    K = weight.shape[1]
    io = v.dtype
    code = _dtype_code(torch, io)
    _check(torch, "v", v, (b, L, E), io, device)
    _check(torch, "weight", weight, (E, K), torch.float32, device)
    _check(torch, "conv_bias", conv_bias, (E,), torch.float32, device, optional=True)
    _check(torch, "state_in", state_in, (b, E, K), io, device, optional=True)
    if x is None:
        x = torch.empty((b, L, E), dtype=io, device=device)
    else:
        _check(torch, "x", x, (b, L, E), io, device)
    if state_out is None and return_state:
        state_out = torch.empty((b, E, K), dtype=io, device=device)
    elif state_out is not None:
        _check(torch, "state_out", state_out, (b, E, K), io, device)
    if state_in is not None and state_out is not None and state_in.data_ptr() == state_out.data_ptr():
        raise ValueError("state_in must not be the state_out buffer")
    with _on(torch, device):
        status = lib.ssm_conv_fwd(_ptr(v), _ptr(weight), _ptr(conv_bias), _ptr(state_in), _ptr(x), _ptr(state_out),
                                  b, L, E, K, code, _stream_of(torch, device))
    _raise_on("ssm_conv_fwd", status)
    return x, state_out


def ssm_conv_update(conv_state, v, weight, conv_bias=None, x=None):
    """One token of the convolution; ``conv_state`` [b, E, K] is updated in place.  Returns x [b, E]."""
    import torch

    lib = load_library()
    if not isinstance(conv_state, torch.Tensor) or conv_state.dim() != 3:
        raise ValueError("conv_state must be a [b, E, K] tensor")
    device = conv_state.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU device, got {device}")
    b, E, K = conv_state.shape
    io = conv_state.dtype
    code = _dtype_code(torch, io)
    _check(torch, "conv_state", conv_state, (b, E, K), io, device)
    _check(torch, "v", v, (b, E), io, device)
    _check(torch, "weight", weight, (E, K), torch.float32, device)
    _check(torch, "conv_bias", conv_bias, (E,), torch.float32, device, optional=True)
    if x is None:
        x = torch.empty((b, E), dtype=io, device=device)
    else:
        _check(torch, "x", x, (b, E), io, device)
    with _on(torch, device):
        status = lib.ssm_conv_update(_ptr(conv_state), _ptr(v), _ptr(weight), _ptr(conv_bias), _ptr(x), b, E, K, code,
                                     _stream_of(torch, device))
    _raise_on("ssm_conv_update", status)
    return x


# ---------------------------------------------------------------------------
# linear attention with a decay for each head
# ---------------------------------------------------------------------------
def ssm_linattn_workspace(b, L, H, G, Dk, Dv, dtype="bf16", backward=False):
    """Bytes of workspace of ``ssm_linattn_fwd`` or ``ssm_linattn_bwd`` at these sizes (host-only query)."""
    code = {"f32": SSM_F32, "bf16": SSM_BF16}.get(dtype, dtype)
    n = load_library().ssm_linattn_workspace(int(b), int(L), int(H), int(G), int(Dk), int(Dv), int(code),
                                             int(bool(backward)))
    _raise_on("ssm_linattn_workspace", min(n, 0))
    return n


def _workspace(torch, n, device):
    """A workspace of n bytes from the allocator of PyTorch, on its current stream of ``device`` (None for 0)."""
    return torch.empty((n,), dtype=torch.uint8, device=device) if n else None


def _linattn_sizes(torch, q, k, v, g, A, lengths, tokens):
    """Checks the inputs of linear attention over ``tokens`` leading axes (2: [b, L], 1: [b]);
    returns (b, L, H, G, Dk, Dv, io dtype, code, device)."""
    shape = "[b, L, G, Dk]" if tokens == 2 else "[b, G, Dk]"
    if not isinstance(q, torch.Tensor) or q.dim() != tokens + 2:
        raise ValueError(f"q must be a {shape} tensor")
    if not isinstance(v, torch.Tensor) or v.dim() != tokens + 2:
        raise ValueError(f"v must be a {shape.replace('G, Dk', 'H, Dv')} tensor")
    device = q.device
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU device, got {device}")
    lead = tuple(q.shape[:tokens])
    G, Dk = q.shape[tokens:]
    H, Dv = v.shape[tokens:]
    if G == 0 and H > 0 or G > 0 and H % G:
        raise ValueError(f"the {H} heads of v must be a multiple of the {G} of q and k")
    io = q.dtype
    code = _dtype_code(torch, io)
    _check(torch, "q", q, (*lead, G, Dk), io, device)
    _check(torch, "k", k, (*lead, G, Dk), io, device)
    _check(torch, "v", v, (*lead, H, Dv), io, device)
    _check(torch, "g", g, (*lead, H), io, device, optional=True)
    _check(torch, "A", A, (H,), torch.float32, device, optional=True)
    _check(torch, "lengths", lengths, lead[:1], torch.int32, device, optional=True)
    return lead[0], lead[1] if tokens == 2 else 1, H, G, Dk, Dv, io, code, device


def _scale(scale, Dk):
    return (Dk or 1) ** -0.5 if scale is None else float(scale)  # a width of zero is refused by the library


def ssm_linattn_fwd(q, k, v, g=None, A=None, scale=None, lengths=None, initial_state=None, y=None, last_state=None,
                    return_last_state=True):
    """Linear attention with a decay for each head: ``(y, last_state)`` (None if not requested).

    ``S = exp(A[h] + g[b, t, h]) S + k v^T``, ``y = scale S^T q`` for every token, from
    ``initial_state`` (None: zero).  q, k [b, L, G, Dk]; v, y [b, L, H, Dv], each group of
    H / G heads sharing a row of q and k; g [b, L, H] in the streamed dtype, A [H] float32 (None:
    zero); ``scale`` None is Dk ** -0.5; ``lengths`` [b] int32 are the tokens of each batch row
    (None: all L): the others are not read, and their rows of y are zero.
    """
    import torch

    lib = load_library()
    b, L, H, G, Dk, Dv, io, code, device = _linattn_sizes(torch, q, k, v, g, A, lengths, 2)
    f32 = torch.float32
    _check(torch, "initial_state", initial_state, (b, H, Dk, Dv), f32, device, optional=True)
    if y is None:
        y = torch.empty((b, L, H, Dv), dtype=io, device=device)
    else:
        _check(torch, "y", y, (b, L, H, Dv), io, device)
    if last_state is None and return_last_state:
        last_state = torch.empty((b, H, Dk, Dv), dtype=f32, device=device)
    elif last_state is not None:
        _check(torch, "last_state", last_state, (b, H, Dk, Dv), f32, device)
    if b * H and initial_state is not None and last_state is not None and (
            initial_state.data_ptr() == last_state.data_ptr()):
        raise ValueError("initial_state must not be the last_state buffer")
    n = lib.ssm_linattn_workspace(b, L, H, G, Dk, Dv, code, 0)
    _raise_on("ssm_linattn_fwd", min(n, 0))
    ws = _workspace(torch, n, device)
    with _on(torch, device):
        status = lib.ssm_linattn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(A), _ptr(lengths), _scale(scale, Dk),
                                     _ptr(initial_state), _ptr(y), _ptr(last_state), b, L, H, G, Dk, Dv, code,
                                     _ptr(ws), n, _stream_of(torch, device))
    _raise_on("ssm_linattn_fwd", status)
    return y, last_state


def ssm_linattn_bwd(q, k, v, dy, g=None, A=None, scale=None, lengths=None, initial_state=None, d_last_state=None):
    """Gradients of sum(dy * y) + sum(d_last_state * last_state) for ``ssm_linattn_fwd``'s arguments.

    Returns a dict: dq, dk [b, L, G, Dk], dv [b, L, H, Dv] and dg [b, L, H] (None without g) in the
    streamed dtype, d_initial_state [b, H, Dk, Dv] float32 (None without initial_state).
    """
    import torch

    lib = load_library()
    b, L, H, G, Dk, Dv, io, code, device = _linattn_sizes(torch, q, k, v, g, A, lengths, 2)
    f32 = torch.float32
    _check(torch, "dy", dy, (b, L, H, Dv), io, device)
    _check(torch, "initial_state", initial_state, (b, H, Dk, Dv), f32, device, optional=True)
    _check(torch, "d_last_state", d_last_state, (b, H, Dk, Dv), f32, device, optional=True)
    out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
           "dg": None if g is None else torch.empty_like(g),
           "d_initial_state": None if initial_state is None else torch.empty_like(initial_state)}
    n = lib.ssm_linattn_workspace(b, L, H, G, Dk, Dv, code, 1)
    _raise_on("ssm_linattn_bwd", min(n, 0))
    ws = _workspace(torch, n, device)
    with _on(torch, device):
        status = lib.ssm_linattn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(A), _ptr(lengths), _scale(scale, Dk),
                                     _ptr(initial_state), _ptr(dy), _ptr(d_last_state), _ptr(out["dq"]),
                                     _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]), _ptr(out["d_initial_state"]),
                                     b, L, H, G, Dk, Dv, code, _ptr(ws), n, _stream_of(torch, device))
    _raise_on("ssm_linattn_bwd", status)
    return out


def ssm_linattn_update(state, q, k, v, g=None, A=None, scale=None, lengths=None, y=None):
    """One token of ``ssm_linattn_fwd``: ``state`` [b, H, Dk, Dv] float32 is updated in place; returns ``y``.

    q, k [b, G, Dk]; v, y [b, H, Dv]; g [b, H].  A batch row whose ``lengths`` is zero takes no step:
    its state stays and its row of y is zero.
    """
    import torch

    lib = load_library()
    b, _, H, G, Dk, Dv, io, code, device = _linattn_sizes(torch, q, k, v, g, A, lengths, 1)
    _check(torch, "state", state, (b, H, Dk, Dv), torch.float32, device)
    if y is None:
        y = torch.empty((b, H, Dv), dtype=io, device=device)
    else:
        _check(torch, "y", y, (b, H, Dv), io, device)
    with _on(torch, device):
        status = lib.ssm_linattn_update(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(A), _ptr(lengths),
                                        _scale(scale, Dk), _ptr(y), b, H, G, Dk, Dv, code, _stream_of(torch, device))
    _raise_on("ssm_linattn_update", status)
    return y


# ---------------------------------------------------------------------------
# the gated delta rule
# ---------------------------------------------------------------------------
def ssm_deltarule_workspace(b, L, H, G, Dk, Dv, dtype="bf16", backward=False):
    """Bytes of workspace of ``ssm_deltarule_fwd`` or ``ssm_deltarule_bwd`` at these sizes (host-only query)."""
    code = {"f32": SSM_F32, "bf16": SSM_BF16}.get(dtype, dtype)
    n = load_library().ssm_deltarule_workspace(int(b), int(L), int(H), int(G), int(Dk), int(Dv), int(code),
                                               int(bool(backward)))
    _raise_on("ssm_deltarule_workspace", min(n, 0))
    return n


def _deltarule_sizes(torch, q, k, v, beta, g, A, lengths, tokens):
    """As ``_linattn_sizes``, with beta."""
    sizes = _linattn_sizes(torch, q, k, v, g, A, lengths, tokens)
    _check(torch, "beta", beta, v.shape[:-1], q.dtype, q.device, optional=True)
    return sizes


def ssm_deltarule_fwd(q, k, v, beta=None, g=None, A=None, scale=None, lengths=None, initial_state=None, y=None,
                      last_state=None, return_last_state=True):
    """The gated delta rule: ``(y, last_state)`` (None if not requested).

    ``u = beta[b, t, h] (v - r S^T k)``, ``S = r S + k u^T``, ``y = scale S^T q`` for every token, with
    ``r = exp(A[h] + g[b, t, h])``, from ``initial_state`` (None: zero).  beta [b, L, H] in the streamed dtype
    (None: one); the others as in ``ssm_linattn_fwd``.  Keys are to be of length one.
    """
    import torch

    lib = load_library()
    b, L, H, G, Dk, Dv, io, code, device = _deltarule_sizes(torch, q, k, v, beta, g, A, lengths, 2)
    f32 = torch.float32
    _check(torch, "initial_state", initial_state, (b, H, Dk, Dv), f32, device, optional=True)
    if y is None:
        y = torch.empty((b, L, H, Dv), dtype=io, device=device)
    else:
        _check(torch, "y", y, (b, L, H, Dv), io, device)
    if last_state is None and return_last_state:
        last_state = torch.empty((b, H, Dk, Dv), dtype=f32, device=device)
    elif last_state is not None:
        _check(torch, "last_state", last_state, (b, H, Dk, Dv), f32, device)
    if b * H and initial_state is not None and last_state is not None and (
            initial_state.data_ptr() == last_state.data_ptr()):
        raise ValueError("initial_state must not be the last_state buffer")
    n = lib.ssm_deltarule_workspace(b, L, H, G, Dk, Dv, code, 0)
    _raise_on("ssm_deltarule_fwd", min(n, 0))
    ws = _workspace(torch, n, device)
    with _on(torch, device):
        status = lib.ssm_deltarule_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(A), _ptr(lengths),
                                       _scale(scale, Dk), _ptr(initial_state), _ptr(y), _ptr(last_state), b, L, H, G, Dk,
                                       Dv, code, _ptr(ws), n, _stream_of(torch, device))
    _raise_on("ssm_deltarule_fwd", status)
    return y, last_state


def ssm_deltarule_bwd(q, k, v, dy, beta=None, g=None, A=None, scale=None, lengths=None, initial_state=None,
                      d_last_state=None):
    """Gradients of sum(dy * y) + sum(d_last_state * last_state) for ``ssm_deltarule_fwd``'s arguments.

    Returns a dict: dq, dk [b, L, G, Dk], dv [b, L, H, Dv], dbeta and dg [b, L, H] (None without beta, g) in
    the streamed dtype, d_initial_state [b, H, Dk, Dv] float32 (None without initial_state).
    """
    import torch

    lib = load_library()
    b, L, H, G, Dk, Dv, io, code, device = _deltarule_sizes(torch, q, k, v, beta, g, A, lengths, 2)
    f32 = torch.float32
    _check(torch, "dy", dy, (b, L, H, Dv), io, device)
    _check(torch, "initial_state", initial_state, (b, H, Dk, Dv), f32, device, optional=True)
    _check(torch, "d_last_state", d_last_state, (b, H, Dk, Dv), f32, device, optional=True)
    out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
           "dbeta": None if beta is None else torch.empty_like(beta), "dg": None if g is None else torch.empty_like(g),
           "d_initial_state": None if initial_state is None else torch.empty_like(initial_state)}
    n = lib.ssm_deltarule_workspace(b, L, H, G, Dk, Dv, code, 1)
    _raise_on("ssm_deltarule_bwd", min(n, 0))
    ws = _workspace(torch, n, device)
    with _on(torch, device):
        status = lib.ssm_deltarule_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(A), _ptr(lengths),
                                       _scale(scale, Dk), _ptr(initial_state), _ptr(dy), _ptr(d_last_state),
                                       _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dbeta"]),
                                       _ptr(out["dg"]), _ptr(out["d_initial_state"]), b, L, H, G, Dk, Dv, code, _ptr(ws),
                                       n, _stream_of(torch, device))
    _raise_on("ssm_deltarule_bwd", status)
    return out


def ssm_deltarule_update(state, q, k, v, beta=None, g=None, A=None, scale=None, lengths=None, y=None):
    """One token of ``ssm_deltarule_fwd``: ``state`` [b, H, Dk, Dv] float32 is updated in place; returns ``y``.

    q, k [b, G, Dk]; v, y [b, H, Dv]; beta, g [b, H].  A batch row whose ``lengths`` is zero takes no step:
    its state stays and its row of y is zero.
    """
    import torch

    lib = load_library()
    b, _, H, G, Dk, Dv, io, code, device = _deltarule_sizes(torch, q, k, v, beta, g, A, lengths, 1)
    _check(torch, "state", state, (b, H, Dk, Dv), torch.float32, device)
    if y is None:
        y = torch.empty((b, H, Dv), dtype=io, device=device)
    else:
        _check(torch, "y", y, (b, H, Dv), io, device)
    with _on(torch, device):
        status = lib.ssm_deltarule_update(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(A),
                                          _ptr(lengths), _scale(scale, Dk), _ptr(y), b, H, G, Dk, Dv, code,
                                          _stream_of(torch, device))
    _raise_on("ssm_deltarule_update", status)
    return y


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
def ssm_layernorm_workspace(rows, H, W, dtype="bf16"):
    """Bytes of workspace of ``ssm_layernorm_bwd`` at these sizes (host-only query)."""
    code = {"f32": SSM_F32, "bf16": SSM_BF16}.get(dtype, dtype)
    n = load_library().ssm_layernorm_workspace(int(rows), int(H), int(W), int(code))
    _raise_on("ssm_layernorm_workspace", min(n, 0))
    return n


def _norm_sizes(torch, x, par):
    """(parameter shape, rows, H, W, code, device) of a layer norm of x with parameters like ``par``: a tensor [W], or
    [H, W] for x [..., H, W]; a number of heads H; or None for [W]."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be a [..., W] tensor")
    if x.device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU device, got {x.device}")
    if isinstance(par, int):
        par = (par, *x.shape[-1:])
    elif par is not None:
        if not isinstance(par, torch.Tensor):
            raise TypeError("weight and bias must be a torch.Tensor each")
        par = tuple(par.shape)
    else:
        par = tuple(x.shape[-1:])
    if len(par) not in (1, 2) or len(par) > x.dim() or par != tuple(x.shape[x.dim() - len(par):]):
        raise ValueError(f"parameters of shape {par} do not fit x of shape {tuple(x.shape)}: [W] or [H, W] of its last axes")
    H, W = (1, par[0]) if len(par) == 1 else par
    if W == 0:
        raise ValueError("x has rows of no elements")
    code = _dtype_code(torch, x.dtype)
    _check(torch, "x", x, x.shape, x.dtype, x.device)
    return par, x.numel() // (H * W) if H else 0, H, W, code, x.device


def ssm_layernorm_fwd(x, weight=None, bias=None, eps=1e-5, y=None):
    """Layer norm over the last axis of x [..., W]: ``(y, mean, rstd)``, mean and rstd [...] float32 for the backward.

    weight and bias are float32, [W], or [H, W] for x [..., H, W] (each head's channels with the head's
    own parameters); None is one and zero.
    """
    import torch

    lib = load_library()
    par, rows, H, W, code, device = _norm_sizes(torch, x, weight if weight is not None else bias)
    _check(torch, "weight", weight, par, torch.float32, device, optional=True)
    _check(torch, "bias", bias, par, torch.float32, device, optional=True)
    if y is None:
        y = torch.empty_like(x)
    else:
        _check(torch, "y", y, x.shape, x.dtype, device)
    mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=device)
    rstd = torch.empty_like(mean)
    with _on(torch, device):
        status = lib.ssm_layernorm_fwd(_ptr(x), _ptr(weight), _ptr(bias), float(eps), _ptr(y), _ptr(mean), _ptr(rstd),
                                       rows, H, W, code, _stream_of(torch, device))
    _raise_on("ssm_layernorm_fwd", status)
    return y, mean, rstd


def ssm_layernorm_bwd(x, dy, mean, rstd, weight=None, heads=None, param_grads=True):
    """Gradients of sum(dy * y) of ``ssm_layernorm_fwd``: a dict of dx (x's dtype) and dweight, dbias (float32).

    mean and rstd are the forward's.  The parameters' shape is weight's; without a weight it is [W], or
    [heads, W] where ``heads`` is given.  ``param_grads=False`` leaves dweight and dbias None.
    """
    import torch

    lib = load_library()
    par, rows, H, W, code, device = _norm_sizes(torch, x, weight if weight is not None else None if heads is None else int(heads))
    f32 = torch.float32
    _check(torch, "dy", dy, x.shape, x.dtype, device)
    _check(torch, "mean", mean, x.shape[:-1], f32, device)
    _check(torch, "rstd", rstd, x.shape[:-1], f32, device)
    _check(torch, "weight", weight, par, f32, device, optional=True)
    out = {"dx": torch.empty_like(x),
           "dweight": torch.empty(par, dtype=f32, device=device) if param_grads else None,
           "dbias": torch.empty(par, dtype=f32, device=device) if param_grads else None}
    n = lib.ssm_layernorm_workspace(rows, H, W, code) if param_grads else 0
    _raise_on("ssm_layernorm_bwd", min(n, 0))
    ws = _workspace(torch, n, device)
    with _on(torch, device):
        status = lib.ssm_layernorm_bwd(_ptr(x), _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(dy), _ptr(out["dx"]),
                                       _ptr(out["dweight"]), _ptr(out["dbias"]), rows, H, W, code, _ptr(ws), n,
                                       _stream_of(torch, device))
    _raise_on("ssm_layernorm_bwd", status)
    return out


# ---------------------------------------------------------------------------
# the norms around a block
# ---------------------------------------------------------------------------
_NORMS = {"post": 1, "pre": 2, "both": 3}


def ssm_blocknorm_workspace(rows, H, W, dtype="bf16", residual_dtype=None):
    """Bytes of workspace of ``ssm_blocknorm_bwd`` at these sizes (host-only query); the residual is of ``dtype`` (None)."""
    names = {"f32": SSM_F32, "bf16": SSM_BF16}
    code = names.get(dtype, dtype)
    rcode = code if residual_dtype is None else names.get(residual_dtype, residual_dtype)
    n = load_library().ssm_blocknorm_workspace(int(rows), int(H), int(W), int(code), int(rcode))
    _raise_on("ssm_blocknorm_workspace", min(n, 0))
    return n


def _blocknorm_sizes(torch, x, post_weight, z, scale, residual, pre_weight, norms, heads):
    """Checks the inputs of the norms around a block; returns (parameters' shape, rows, H, W, codes, the norms' flags,
    the residual's dtype)."""
    if norms not in _NORMS:
        raise ValueError(f"norms must be one of {sorted(_NORMS)}, got {norms!r}")
    if post_weight is not None and norms == "pre":
        raise ValueError("post_weight is given, but norms has no norm after the block")
    if pre_weight is not None and norms == "post":
        raise ValueError("pre_weight is given, but norms has no norm before the next block")
    like = next((p for p in (post_weight, scale, pre_weight) if p is not None), None if heads is None else int(heads))
    par, rows, H, W, code, device = _norm_sizes(torch, x, like)
    for name, p in (("post_weight", post_weight), ("scale", scale), ("pre_weight", pre_weight)):
        _check(torch, name, p, par, torch.float32, device, optional=True)
    _check(torch, "z", z, x.shape, x.dtype, device, optional=True)
    rdt = x.dtype
    if residual is not None:
        if not isinstance(residual, torch.Tensor):
            raise TypeError("residual must be a torch.Tensor")
        rdt = residual.dtype if residual.dtype == torch.float32 else x.dtype
        _check(torch, "residual", residual, x.shape, rdt, device)
    return par, rows, H, W, code, _dtype_code(torch, rdt), device, _NORMS[norms], rdt


def ssm_blocknorm_fwd(x, post_weight=None, z=None, scale=None, residual=None, pre_weight=None, norms="both", eps=1e-5,
                      return_h=True, h=None, n=None, heads=None):
    """RMS norm after a block, gate, scale, residual, RMS norm before the next: ``(h, n, rstd_post, rstd_pre)``.

    ``u = x rstd_post post_weight silu(z)``, ``h = residual + scale u``, ``n = h rstd_pre pre_weight``; ``norms`` is
    "post", "pre" or "both", a norm that is not there leaves its rstd (and n) None; z, scale and residual None leave
    their step out.  x, z, n [..., W] in the streamed dtype; residual and h in it or in float32; the parameters are
    float32, [W], or [H, W] for x [..., H, W] (None: one; ``heads`` says H where there are none).  ``return_h=False``
    does not compute h where n is what is wanted.  rstd_post, rstd_pre [...] float32 are for the backward.
    """
    import torch

    lib = load_library()
    par, rows, H, W, code, rcode, device, flags, rdt = _blocknorm_sizes(torch, x, post_weight, z, scale, residual, pre_weight,
                                                                       norms, heads)
    if h is not None:
        _check(torch, "h", h, x.shape, rdt, device)
    elif return_h or not flags & 2:
        h = torch.empty(x.shape, dtype=rdt, device=device)
    if n is not None:
        if not flags & 2:
            raise ValueError("n is given, but norms has no norm before the next block")
        _check(torch, "n", n, x.shape, x.dtype, device)
    elif flags & 2:
        n = torch.empty_like(x)
    rstd = [torch.empty(x.shape[:-1], dtype=torch.float32, device=device) if flags & f else None for f in (1, 2)]
    with _on(torch, device):
        status = lib.ssm_blocknorm_fwd(_ptr(x), _ptr(post_weight), _ptr(z), _ptr(scale), _ptr(residual), _ptr(pre_weight),
                                       float(eps), flags, _ptr(h), _ptr(n), _ptr(rstd[0]), _ptr(rstd[1]), rows, H, W, code,
                                       rcode, _stream_of(torch, device))
    _raise_on("ssm_blocknorm_fwd", status)
    return h, n, rstd[0], rstd[1]


def ssm_blocknorm_bwd(x, rstd_post=None, rstd_pre=None, dh=None, dn=None, post_weight=None, z=None, scale=None, residual=None,
                      pre_weight=None, norms="both", param_grads=True, heads=None):
    """Gradients of sum(dh * h) + sum(dn * n) of ``ssm_blocknorm_fwd``, from its inputs and its rstd.

    dh may be None where there is a norm before the next block, and is of the residual's dtype.  Returns a dict: dx, dz
    (None without z), dresidual (None without residual) and, float32, dpost_weight, dscale, dpre_weight (None without
    the parameter, or with ``param_grads=False``).
    """
    import torch

    lib = load_library()
    par, rows, H, W, code, rcode, device, flags, rdt = _blocknorm_sizes(torch, x, post_weight, z, scale, residual, pre_weight,
                                                                       norms, heads)
    f32 = torch.float32
    lead = x.shape[:-1]
    _check(torch, "rstd_post", rstd_post, lead, f32, device, optional=not flags & 1)
    _check(torch, "rstd_pre", rstd_pre, lead, f32, device, optional=not flags & 2)
    _check(torch, "dn", dn, x.shape, x.dtype, device, optional=not flags & 2)
    _check(torch, "dh", dh, x.shape, rdt, device, optional=bool(flags & 2))
    grad = lambda p: torch.empty_like(p) if p is not None and param_grads else None  # noqa: E731
    out = {"dx": torch.empty_like(x), "dz": None if z is None else torch.empty_like(z),
           "dresidual": None if residual is None else torch.empty_like(residual),
           "dpost_weight": grad(post_weight), "dscale": grad(scale), "dpre_weight": grad(pre_weight)}
    params = any(out[k] is not None for k in ("dpost_weight", "dscale", "dpre_weight"))
    size = lib.ssm_blocknorm_workspace(rows, H, W, code, rcode) if params else 0
    _raise_on("ssm_blocknorm_bwd", min(size, 0))
    ws = _workspace(torch, size, device)
    with _on(torch, device):
        status = lib.ssm_blocknorm_bwd(_ptr(x), _ptr(post_weight), _ptr(z), _ptr(scale), _ptr(residual), _ptr(pre_weight), flags,
                                       _ptr(rstd_post), _ptr(rstd_pre), _ptr(dh), _ptr(dn), _ptr(out["dx"]), _ptr(out["dz"]),
                                       _ptr(out["dresidual"]), _ptr(out["dpost_weight"]), _ptr(out["dscale"]),
                                       _ptr(out["dpre_weight"]), rows, H, W, code, rcode, _ptr(ws), size,
                                       _stream_of(torch, device))
    _raise_on("ssm_blocknorm_bwd", status)
    return out
