"""Thin ctypes binding of libcanopy.so (include/canopy.h).

Argument marshalling only: every step of the path runs in the library's
CUDA kernels.  (The calls of a few microseconds, step, prefill, accept, qk_prep,
attend and cache_commit, go through the native _marshal.so, which checks their arguments, allocates their
outputs and makes the call; the Python code here is for what it turns down, and
for all of them where that file is missing or built for another torch.)
Tensors are torch CUDA tensors (torch provides device memory
and the current stream), contiguous and on 16 bytes: a slice that starts
elsewhere is "invalid argument" and wants a clone().  The calls are enqueued on
``torch.cuda.current_stream()`` and return without synchronising.  If the
library has not been built, loading fails loudly: there is no fallback.
"""

from __future__ import annotations

import ctypes
import os
import warnings

import torch

from .build import marshal_tag

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcanopy.so")

OK, ERR_ARG, ERR_TREE, ERR_UNSUPPORTED, ERR_CUDA = 0, 1, 2, 3, 4
F32, BF16 = 0, 1
SOLVE = {"fwdsub": 0, "neumann": 1, "squaring": 2, "split": 3}
DEVERR_TREE, DEVERR_GATE, DEVERR_ACCEPTED, DEVERR_TIMEOUT, DEVERR_LENGTH = 0x1, 0x2, 0x4, 0x8, 0x10
DEVERR_TOKEN, DEVERR_PAGE = 0x20, 0x40
VERIFY_INPUTS_READY = 0x1
VERIFY_STATE_READY = 0x2
VERIFY_CLOSED_FORM = 0x4
VERIFY_PATH_REPLAY = 0x8
PLAN = {"none": -1, "path_replay": 0, "tc_block": 1, "tc_neumann": 2, "tc_blocked": 3, "fp32": 4, "variant": 5}
FORCE = {None: 0, "closed_form": VERIFY_CLOSED_FORM, "path_replay": VERIFY_PATH_REPLAY}
COMMIT_STATE_READY = 0x1
PREFILL_FORCE = {None: 0, "scan": 0x1, "chunked": 0x2}
PREFILL_PLAN = {"none": -1, "scan": 0, "chunked": 1}
ATTEND_PLAN = {"none": -1, "fp32": 0, "few": 1, "tiles": 2}
NORM = {"none": 0, "rms": 1, "l2": 2}
PAIRS = {"half": 0, "adjacent": 1}
ACT = {"none": 0, "silu": 1}
WS_REGION = {"err": 0, "l": 1, "depth": 2, "mask": 3, "order": 4, "u": 5}

# name -> (restype, argtypes); mirrors include/canopy.h
_P, _I, _S, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_L = ctypes.c_int64
SIGNATURES = {
    "canopy_workspace_bytes": (_S, [_I, _I, _I, _I, _I]),
    "canopy_workspace_init": (_I, [_P, _S, _P]),
    "canopy_workspace_offset": (_S, [_I, _I, _I, _I, _I, _I]),
    "canopy_tree_prep": (_I, [_P, _P, _I, _I, _I, _P, _P]),
    "canopy_tree_verify": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P, _I,
                                _P, ctypes.c_uint, _P]),
    "canopy_verify_plan": (_I, [_I, _I, _I, _I, _I, _I, _I, _I, ctypes.c_uint, _I]),
    "canopy_commit": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, ctypes.c_uint, _P]),
    "canopy_snapshot_bytes": (_S, [_I, _I, _I, _I, _I]),
    "canopy_serial_replay": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _I, _P, _P,
                                  _P]),
    "canopy_serial_replay_static": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _I, _P,
                                         _P]),
    "canopy_prefill_workspace_bytes": (_S, [_I, _I, _I, _I, _I]),
    "canopy_prefill": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _I, _P, _P,
                            ctypes.c_uint, _P]),
    "canopy_prefill_plan": (_I, [_I, _I, _I, _I, _I, _I, _I, ctypes.c_uint]),
    "canopy_step": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _I, _P, _P]),
    "canopy_accept": (_I, [_P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P]),
    "canopy_qk_prep": (_I, [_P, _P, _P, _I, _L, _L, _L, _I, _P, _P, _F, _P, _I, _P, _I, _L, _L, _P, _I, _I, _I, _I,
                            _I, _I, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P]),
    "canopy_attend_workspace_bytes": (_S, [_I, _I, _I, _I, _I]),
    "canopy_attend_plan": (_I, [_I, _I, _I, _I, _I, _I]),
    "canopy_attend": (_I, [_P, _I, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P,
                           _P]),
    "canopy_cache_commit": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _P, _I, _I, _I, _I, _P, _P, _P]),
    "canopy_tree_conv": (_I, [_P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P]),
    "canopy_conv_commit": (_I, [_P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "canopy_read_device_error": (_I, [_P, ctypes.POINTER(ctypes.c_int32), _P]),
    "canopy_status_string": (ctypes.c_char_p, [_I]),
    "canopy_version": (_I, []),
}

_lib = None
_marshal = None


class CanopyError(RuntimeError):
    pass


class _NoMarshal:
    """In place of _marshal.so: turns every call down."""

    @staticmethod
    def _none(*args):
        return None

    bind = step = prefill = accept = bind_attention = qk_prep = attend = cache_commit = _none


def _native():
    """_marshal.so, or where it does not load, or was built for another Python or torch, what stands in for it."""
    try:
        from . import _marshal as marshal
        built_for = getattr(marshal, "built_for", "something else")
        if built_for == marshal_tag():
            return marshal
        why = f"was built for {built_for}, not {marshal_tag()}"
    except ImportError as e:
        why = f"does not load ({e})"
    warnings.warn(f"_marshal.so {why}: step, prefill and accept take 10 us more of host time a call; "
                  "gated_deltanet_linear_tree_gb300.build.build() builds it")
    return _NoMarshal


def load(path: str = LIB_PATH):
    """Load the shared library (no CUDA call is made by loading)."""
    global _lib, _marshal
    if _lib is None:
        if not os.path.exists(path):
            raise CanopyError(f"{path} is missing: build it with gated_deltanet_linear_tree_gb300.build.build()")
        marshal = _native()
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        marshal.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.canopy_step, lib.canopy_prefill, lib.canopy_prefill_workspace_bytes, lib.canopy_accept)),
            torch.bfloat16, torch.float32)
        marshal.bind_attention(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.canopy_qk_prep, lib.canopy_attend, lib.canopy_attend_workspace_bytes, lib.canopy_cache_commit)))
        _lib, _marshal = lib, marshal
    return _lib


def _short_call(name: str, r):
    """A native call's outputs, or its status raised."""
    if r.__class__ is int:
        _check(r, name)
    return r


def _check(status: int, what: str):
    if status != OK:
        msg = load().canopy_status_string(status).decode()
        raise CanopyError(f"{what}: {msg} (status {status})")


def _ptr(t: torch.Tensor):
    return ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise CanopyError(f"unsupported dtype {t.dtype}")


def _need(t: torch.Tensor, name: str, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise CanopyError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise CanopyError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise CanopyError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise CanopyError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def workspace_bytes(B: int, T: int, HV: int, d: int) -> int:
    """Workspace bytes for B streams of T nodes and HV value heads."""
    return int(load().canopy_workspace_bytes(B, T, HV, d, d))


def _new_workspace(n: int, cleared: int, device) -> torch.Tensor:
    """n bytes on `device`, the first of them cleared on its own current stream (the calls' one)."""
    with torch.cuda.device(device):
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        _check(load().canopy_workspace_init(_ptr(ws), cleared, _stream()), "canopy_workspace_init")
    return ws


def workspace(B: int, T: int, HV: int, d: int, device="cuda") -> torch.Tensor:
    n = workspace_bytes(B, T, HV, d)
    if n == 0:
        raise CanopyError("unsupported sizes for the workspace")
    return _new_workspace(n, n, device)


def workspace_views(ws, B: int, T: int, HV: int, d: int) -> dict:
    """Views of the workspace regions a caller may read (canopy_ws_region):
    l fp32 [B, T, HV], depth int32 [B, T], mask int32 [B, T, ceil(T/32)]
    (the uint32 words' bits), order int32 [B, T], U fp32 [B, T, HV, d]."""
    _need(ws, "workspace", torch.uint8)
    W = (T + 31) // 32
    shapes = {"l": ((B, T, HV), torch.float32), "depth": ((B, T), torch.int32),
              "mask": ((B, T, W), torch.int32), "order": ((B, T), torch.int32),
              "u": ((B, T, HV, d), torch.float32)}
    out = {}
    for name, (shape, dt) in shapes.items():
        off = int(load().canopy_workspace_offset(B, T, HV, d, d, WS_REGION[name]))
        n = 1
        for x in shape:
            n *= x
        if off == ctypes.c_size_t(-1).value or off + 4 * n > ws.numel():
            raise CanopyError(f"workspace too small or sizes unsupported for region {name}")
        out[name] = ws[off:off + 4 * n].view(dt).view(shape)
    return out


def tree_prep(parent, g, ws):
    B, T = parent.shape
    HV = g.shape[-1]
    _need(parent, "parent", torch.int32)
    _need(g, "g", torch.float32, (B, T, HV))
    _check(load().canopy_tree_prep(_ptr(parent), _ptr(g), T, B, HV, _ptr(ws), _stream()), "canopy_tree_prep")


def _heads(q, k, v, g, beta, S0, parent):
    """Check the shapes of one verify call's inputs: q, k [B, T, H, dk]
    (key heads), v [B, T, HV, dv], g, beta [B, T, HV], S0 [B, HV, dv, dk]."""
    _need(q, "q")
    B, T, H, dk = q.shape
    _need(k, "k", q.dtype, q.shape)
    _need(v, "v", q.dtype)
    if v.dim() != 4 or v.shape[:2] != q.shape[:2]:
        raise CanopyError(f"v must have shape ({B}, {T}, HV, dv), got {tuple(v.shape)}")
    HV, dv = v.shape[2], v.shape[3]
    if HV % H:
        raise CanopyError(f"value heads {HV} are not a multiple of key heads {H}")
    _need(g, "g", torch.float32, (B, T, HV))
    _need(beta, "beta", torch.float32, (B, T, HV))
    _need(S0, "S0", torch.float32, (B, HV, dv, dk))
    _need(parent, "parent", torch.int32, (B, T))
    return B, T, H, HV, dk, dv


def _lengths(lengths, B):
    if lengths is None:
        return None
    _need(lengths, "lengths", torch.int32, (B,))
    return _ptr(lengths)


def verify(q, k, v, g, beta, S0, parent, ws, solve: str = "fwdsub", o_dtype=torch.float32, out=None,
           inputs_ready: bool = False, state_ready: bool = False, scale: float = 1.0, lengths=None, force=None):
    """o [B, T, HV, dv] for every node of every stream's tree; q and k carry
    H key heads, v, g, beta and S0 HV value heads (a multiple of H), and
    scale multiplies q.  solve: "fwdsub" (every size and dtype), or
    "neumann", "squaring", "split" (bf16 q/k/v, dk = dv = 128).  inputs_ready: q, k, v, g, beta and parent are not
    written by the kernel launched just before this call on the current
    stream (CANOPY_VERIFY_INPUTS_READY); state_ready (with inputs_ready): nor
    is S0 (CANOPY_VERIFY_STATE_READY).  lengths: int32 [B] CUDA tensor of
    per-stream tree sizes (ragged batches), or None for T everywhere; rows of
    o past a stream's length are left as they were.  force: None (the
    library's dispatch), "closed_form" or "path_replay" (forward substitution
    only; the path replay takes trees of up to 8 nodes)."""
    B, T, H, HV, dk, dv = _heads(q, k, v, g, beta, S0, parent)
    _need(ws, "workspace", torch.uint8)
    if out is None:
        out = torch.empty((B, T, HV, dv), dtype=o_dtype, device=q.device)
    _need(out, "o", None, (B, T, HV, dv))
    st = load().canopy_tree_verify(_ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(g), _ptr(beta), _ptr(S0),
                                   _ptr(parent), _lengths(lengths, B), T, B, H, HV, dk, dv, float(scale),
                                   SOLVE[solve], _ptr(out), _dt(out),
                                   _ptr(ws), (VERIFY_INPUTS_READY if inputs_ready else 0)
                                   | (VERIFY_STATE_READY if state_ready else 0) | FORCE[force], _stream())
    _check(st, "canopy_tree_verify")
    return out


def verify_plan(T: int, B: int, H: int, HV: int, bf16: bool, d: int, solve: str = "fwdsub", force=None,
                lengths: bool = False) -> str:
    """Which path canopy_tree_verify takes for these sizes (a PLAN name)."""
    code = load().canopy_verify_plan(T, B, H, HV, BF16 if bf16 else F32, d, d, SOLVE[solve], FORCE[force],
                                     int(bool(lengths)))
    return {v: k for k, v in PLAN.items()}[code]


def commit(accepted, S0, k, parent, ws, out=None, state_ready: bool = False, lengths=None):
    """S_new [B, HV, dv, dk] for the accepted node of every stream, from the
    preceding verify call's k (H key heads), parent and workspace.
    state_ready: S0, accepted, k and parent are not written by the kernel
    launched just before this call on the current stream
    (CANOPY_COMMIT_STATE_READY).  lengths: the verify call's, or None."""
    _need(S0, "S0", torch.float32)
    _need(parent, "parent", torch.int32)
    _need(k, "k")
    B, HV, dv, dk = S0.shape
    if parent.dim() != 2 or parent.shape[0] != B:
        raise CanopyError(f"parent must have shape ({B}, T), got {tuple(parent.shape)}")
    T = parent.shape[1]
    if k.dim() != 4 or k.shape[0] != B or k.shape[1] != T or k.shape[3] != dk or HV % k.shape[2]:
        raise CanopyError(f"k must have shape ({B}, {T}, H, {dk}) with H dividing {HV}, got {tuple(k.shape)}")
    H = k.shape[2]
    _need(accepted, "accepted", torch.int32, (B,))
    if out is None:
        out = torch.empty_like(S0)
    _need(out, "S_new", torch.float32, S0.shape)
    st = load().canopy_commit(_ptr(accepted), _ptr(S0), _ptr(out), _ptr(k), _ptr(parent), _lengths(lengths, B),
                              _dt(k), T, B, H, HV, dk, dv, _ptr(ws), COMMIT_STATE_READY if state_ready else 0,
                              _stream())
    _check(st, "canopy_commit")
    return out


def snapshot_bytes(B: int, T: int, HV: int, d: int) -> int:
    return int(load().canopy_snapshot_bytes(B, T, HV, d, d))


def serial_replay(q, k, v, g, beta, S0, parent, ws, snapshot=None, o_dtype=torch.float32, out=None,
                  scale: float = 1.0):
    B, T, H, HV, dk, dv = _heads(q, k, v, g, beta, S0, parent)
    if snapshot is None:
        snapshot = torch.empty(snapshot_bytes(B, T, HV, dk), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty((B, T, HV, dv), dtype=o_dtype, device=q.device)
    _need(out, "o", None, (B, T, HV, dv))
    st = load().canopy_serial_replay(_ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(g), _ptr(beta), _ptr(S0),
                                     _ptr(parent), T, B, H, HV, dk, dv, float(scale), _ptr(out), _dt(out),
                                     _ptr(snapshot), _ptr(ws), _stream())
    _check(st, "canopy_serial_replay")
    return out


def serial_replay_static(q, k, v, g, beta, S0, parent, err=None, o_dtype=torch.float32, out=None,
                         scale: float = 1.0):
    """Serial replay whose snapshots live in the library's fixed device array
    (no workspace, no snapshot buffer); err is an optional int32 CUDA tensor
    of one element that receives the device error bits (OR-ed)."""
    B, T, H, HV, dk, dv = _heads(q, k, v, g, beta, S0, parent)
    if out is None:
        out = torch.empty((B, T, HV, dv), dtype=o_dtype, device=q.device)
    _need(out, "o", None, (B, T, HV, dv))
    errp = _ptr(err) if err is not None else None
    st = load().canopy_serial_replay_static(_ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(g), _ptr(beta), _ptr(S0),
                                            _ptr(parent), T, B, H, HV, dk, dv, float(scale), _ptr(out), _dt(out),
                                            errp, _stream())
    _check(st, "canopy_serial_replay_static")
    return out


def _need_all(dev: int, *specs):
    """_need for (tensor, name, dtype, shape) specs, all on device `dev`."""
    for t, name, dtype, shape in specs:
        _need(t, name, dtype, shape)
        if t.get_device() != dev:
            raise CanopyError(f"{name} must be on the same device as the other tensors")


def _need_given(dev: int, *specs):
    """_need_all for those of the tensors that are not None."""
    _need_all(dev, *(spec for spec in specs if spec[0] is not None))


def _need_ints(*sizes):
    """The library takes sizes as int; ctypes would drop what is beyond."""
    if max(sizes) > 0x7FFFFFFF:
        raise CanopyError(f"unsupported sizes {tuple(sizes)}")


def _raw_stream(dev: int) -> int:
    """The current stream's handle on CUDA device `dev`."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _opt(t):
    return None if t is None else t.data_ptr()


def _heads3(q, v):
    """Sizes of q [n, H, dk] and v [n, HV, dv], their dtype's code, and v's shape."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise CanopyError("q must have shape (n, H, dk)")
    n, H, dk = q.shape
    if not isinstance(v, torch.Tensor) or v.dim() != 3 or v.shape[0] != n:
        raise CanopyError(f"v must have shape ({n}, HV, dv)")
    _, HV, dv = v.shape
    return n, H, HV, dk, dv


def prefill_workspace(N: int, B: int, HV: int, d: int, device="cuda") -> torch.Tensor:
    """Workspace of prefill calls over up to N packed tokens of B sequences
    with HV value heads."""
    n = int(load().canopy_prefill_workspace_bytes(N, B, HV, d, d))
    if n == 0:
        raise CanopyError("unsupported sizes for the prefill workspace")
    return _new_workspace(n, 256, device)


def prefill(q, k, v, g, beta, S0, starts, ws, o_dtype=torch.float32, out=None, S_out=None, scale: float = 1.0,
            force=None):
    """The layer over packed prompts: (o [N, HV, dv], S_new [B, HV, dv, dk]).
    q, k [N, H, dk] and v [N, HV, dv] hold the tokens of B sequences one
    after the other; sequence b is tokens starts[b] .. starts[b+1] - 1
    (starts int32 [B+1], CUDA) and starts from S0[b] (fp32 [B, HV, dv, dk], or
    None for zero states).  S_out may be S0.  ws: prefill_workspace for at
    least these sizes.  force: None (the library's dispatch), "scan" or
    "chunked" (bf16, d = 128)."""
    if _marshal is None:
        load()
    r = _marshal.prefill(q, k, v, g, beta, S0, starts, ws, o_dtype, out, S_out, scale, PREFILL_FORCE[force])
    if r is not None:
        return _short_call("canopy_prefill", r)
    N, H, HV, dk, dv = _heads3(q, v)
    if not isinstance(starts, torch.Tensor) or starts.dim() != 1 or starts.shape[0] < 2:
        raise CanopyError("starts must have shape (B + 1,)")
    B = starts.shape[0] - 1
    _need_ints(N, B, H, HV, dk, dv)
    state = (B, HV, dv, dk)
    dt, f32, dev = q.dtype, torch.float32, q.get_device()
    _need_all(dev, (q, "q", dt, q.shape), (k, "k", dt, q.shape), (v, "v", dt, v.shape), (g, "g", f32, (N, HV)),
              (beta, "beta", f32, (N, HV)), (starts, "starts", torch.int32, starts.shape),
              (ws, "workspace", torch.uint8, ws.shape))
    _need_given(dev, (S0, "S0", f32, state), (out, "o", None, v.shape), (S_out, "S_new", f32, state))
    lib = load()
    if ws.numel() < lib.canopy_prefill_workspace_bytes(N, B, HV, dk, dv):
        raise CanopyError("the workspace is too small for these sizes")
    with torch.cuda.device(dev):
        if out is None:
            out = torch.empty(v.shape, dtype=o_dtype, device=q.device)
        if S_out is None:
            S_out = torch.empty(state, dtype=f32, device=q.device)
        st = lib.canopy_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), _dt(q), g.data_ptr(), beta.data_ptr(),
                                _opt(S0), starts.data_ptr(), N, B, H, HV, dk, dv, scale, out.data_ptr(), _dt(out),
                                S_out.data_ptr(), ws.data_ptr(), PREFILL_FORCE[force], _raw_stream(dev))
    _check(st, "canopy_prefill")
    return out, S_out


def prefill_plan(N: int, B: int, H: int, HV: int, bf16: bool, d: int, force=None) -> str:
    """Which path canopy_prefill takes for these sizes (a PREFILL_PLAN name)."""
    code = load().canopy_prefill_plan(N, B, H, HV, BF16 if bf16 else F32, d, d, PREFILL_FORCE[force])
    return {v: k for k, v in PREFILL_PLAN.items()}[code]


def step(q, k, v, g, beta, S, o_dtype=torch.float32, out=None, S_out=None, scale: float = 1.0, err=None):
    """One token of every stream: (o [B, HV, dv], S_new [B, HV, dv, dk]).
    q, k [B, H, dk]; v [B, HV, dv]; g, beta fp32 [B, HV]; S fp32
    [B, HV, dv, dk].  S_out may be S (in place).  err: an optional int32 CUDA
    tensor of one element that receives device error bits (OR-ed)."""
    if _marshal is None:
        load()
    r = _marshal.step(q, k, v, g, beta, S, o_dtype, out, S_out, scale, err)
    if r is not None:
        return _short_call("canopy_step", r)
    B, H, HV, dk, dv = _heads3(q, v)
    _need_ints(B, H, HV, dk, dv)
    state = (B, HV, dv, dk)
    dt, f32, dev = q.dtype, torch.float32, q.get_device()
    _need_all(dev, (q, "q", dt, q.shape), (k, "k", dt, q.shape), (v, "v", dt, v.shape), (g, "g", f32, (B, HV)),
              (beta, "beta", f32, (B, HV)), (S, "S", f32, state))
    _need_given(dev, (out, "o", None, v.shape), (S_out, "S_new", f32, state), (err, "err", torch.int32, (1,)))
    lib = load()
    with torch.cuda.device(dev):
        if out is None:
            out = torch.empty(v.shape, dtype=o_dtype, device=q.device)
        if S_out is None:
            S_out = torch.empty_like(S)
        st = lib.canopy_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), _dt(q), g.data_ptr(), beta.data_ptr(),
                             S.data_ptr(), S_out.data_ptr(), B, H, HV, dk, dv, scale, out.data_ptr(), _dt(out),
                             _opt(err), _raw_stream(dev))
    _check(st, "canopy_step")
    return out, S_out


def accept(p, tokens, parent, u, noise, q=None, lengths=None, err=None):
    """The accepted node of every stream's draft tree, from the target's
    probabilities and given random numbers: (accepted int32 [B], out_tokens
    int32 [B, T], counts int32 [B]).  p [B, T, V]: the target's distribution
    after each node; q: the draft's that each node's children were drawn from
    (same shape and dtype), or None where the candidates are fixed choices;
    tokens, parent int32 [B, T] (node 0 is the last emitted token); u fp32
    [B, T] uniform in [0, 1); noise fp32 [B, V] exponential variates.
    out_tokens: the accepted tokens in path order, the next token after them,
    then -1; counts: how many; accepted is what commit and conv_commit take."""
    if _marshal is None:
        load()
    r = _marshal.accept(p, tokens, parent, u, noise, q, lengths, err)
    if r is not None:
        return _short_call("canopy_accept", r)
    if not isinstance(p, torch.Tensor) or p.dim() != 3:
        raise CanopyError("p must have shape (B, T, V)")
    B, T, V = p.shape
    _need_ints(B, T, V)
    i32, f32, dev = torch.int32, torch.float32, p.get_device()
    _need_all(dev, (p, "p", p.dtype, p.shape), (tokens, "tokens", i32, (B, T)), (parent, "parent", i32, (B, T)),
              (u, "u", f32, (B, T)), (noise, "noise", f32, (B, V)))
    _need_given(dev, (q, "q", p.dtype, p.shape), (lengths, "lengths", i32, (B,)), (err, "err", i32, (1,)))
    lib = load()
    with torch.cuda.device(dev):
        accepted = torch.empty((B,), dtype=i32, device=p.device)
        out_tokens = torch.empty_like(tokens)
        counts = torch.empty_like(accepted)
        st = lib.canopy_accept(p.data_ptr(), _opt(q), _dt(p), tokens.data_ptr(), parent.data_ptr(), _opt(lengths),
                               u.data_ptr(), noise.data_ptr(), T, B, V, accepted.data_ptr(), out_tokens.data_ptr(),
                               counts.data_ptr(), _opt(err), _raw_stream(dev))
    _check(st, "canopy_accept")
    return accepted, out_tokens, counts


def _rows_shape(q, starts, lengths, what: str):
    """Leading sizes of an attention layer's rows q [N, H, d] (packed, or one token of each stream) or
    [B, T, H, d], and N."""
    if not isinstance(q, torch.Tensor) or q.dim() not in (3, 4):
        raise CanopyError(f"{what} must have shape (N, H, d) or (B, T, H, d)")
    lead = tuple(q.shape[:-2])
    if q.dim() == 4 and starts is not None:
        raise CanopyError("starts come with packed rows, not with (B, T, H, d)")
    if q.dim() == 3 and lengths is not None:
        raise CanopyError("lengths come with (B, T, H, d), not with packed rows")
    return lead, lead[0] * (lead[1] if q.dim() == 4 else 1)


def _need_rows(t, name: str, dev: int, dtype, shape) -> int:
    """Rows whose heads are dense but whose tokens may lie apart; elements from a token to the next."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise CanopyError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise CanopyError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != dev:
        raise CanopyError(f"{name} must be on the same device as the other tensors")
    H, d = shape[-2:]
    ld = t.stride(-3) if shape[-3] > 1 else t.stride(0) if len(shape) == 4 and shape[0] > 1 else H * d
    if d > 1 and t.stride(-1) != 1 or H > 1 and t.stride(-2) != d or \
            len(shape) == 4 and shape[0] > 1 and t.stride(0) != ld * shape[1]:
        raise CanopyError(f"{name} must have dense heads and tokens at one distance")
    return ld


def _cache(k_cache, v_cache, page_table, context, dtype, HKV, d, dev):
    """Check a paged cache: k_cache, v_cache [pages, HKV, page_size, d], page_table int32 [B, max_pages], context
    int32 [B]; (B, pages, page_size, max_pages)."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4 or k_cache.shape[1] != HKV or \
            k_cache.shape[3] != d:
        raise CanopyError(f"k_cache must have shape (pages, {HKV}, page_size, {d})")
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise CanopyError("page_table must have shape (B, max_pages)")
    B = page_table.shape[0]
    _need_all(dev, (k_cache, "k_cache", dtype, k_cache.shape), (v_cache, "v_cache", dtype, k_cache.shape),
              (page_table, "page_table", torch.int32, page_table.shape), (context, "context", torch.int32, (B,)))
    sizes = (k_cache.shape[0], k_cache.shape[2], page_table.shape[1])
    _need_ints(B, HKV, d, *sizes)
    return (B, *sizes)


def _streams(lead, B, starts):
    """Whether rows of these leading sizes are those of B streams."""
    if len(lead) == 2 and lead[0] != B or len(lead) == 1 and starts is None and lead[0] != B:
        raise CanopyError(f"{lead} rows do not fit {B} streams: (B, T, H, d), one token of each, or packed with starts")


def qk_prep(q, k, v=None, norm: str = "rms", q_weight=None, k_weight=None, eps: float = 1e-6, freqs=None,
            positions=None, axis=None, pairs: str = "half", q_out=None, k_out=None, k_cache=None, v_cache=None,
            page_table=None, context=None, starts=None, lengths=None, err=None):
    """Queries and keys of a layer in one pass: (q_out, k_out).  Every head's
    row normed ("rms", "l2" for unit rows, or "none"; weights fp32 [d] or
    None), the first 2 len(freqs) columns rotated by position (freqs fp32;
    positions int32 of the rows' shape, or [axes, ...] (expanded or transposed
    ones too) with axis int32 [len(freqs)] each pair's axis, or None for the place in the cache; pairs
    "half" (j, j + R/2) or "adjacent" (2j, 2j + 1)), rounded once.
    q [N, HQ, d], k, v [N, HKV, d]: packed sequences at starts int32 [B+1], or
    one token of each stream; or [B, T, heads, d], of which lengths int32 [B] (or
    all) are there.  Tokens may lie apart (slices of one projection), their heads
    dense.  With k_cache and v_cache [pages, HKV, page_size, d], page_table int32
    [B, max_pages] and context int32 [B], row i's key and value go to place
    context[b] + i of its stream and k_out is None.  q_out may be q and k_out k.
    err: an optional int32 CUDA tensor of one element for device error bits."""
    if _marshal is None:
        load()
    r = _marshal.qk_prep(q, k, v, NORM[norm], q_weight, k_weight, eps, freqs, positions, axis, PAIRS[pairs], q_out,
                         k_out, k_cache, v_cache, page_table, context, starts, lengths, err)
    if r is not None:
        return _short_call("canopy_qk_prep", r)
    lead, N = _rows_shape(q, starts, lengths, "q")
    HQ, d = q.shape[-2:]
    if not isinstance(k, torch.Tensor) or k.dim() != q.dim():
        raise CanopyError("k must have the rows of q")
    HKV = k.shape[-2]
    _need_ints(N, HQ, HKV, d)
    dt, f32, i32, dev = q.dtype, torch.float32, torch.int32, q.get_device()
    code = _dt(q)
    ldq = _need_rows(q, "q", dev, dt, (*lead, HQ, d))
    ldk = _need_rows(k, "k", dev, dt, (*lead, HKV, d))
    R = ldv = B = pages = page_size = max_pages = 0
    axes, axis_step, row_step = 1, 0, 1
    if k_cache is not None:
        B, pages, page_size, max_pages = _cache(k_cache, v_cache, page_table, context, dt, HKV, d, dev)
        _streams(lead, B, starts)
        ldv = _need_rows(v, "v", dev, dt, (*lead, HKV, d))
        _need_given(dev, (starts, "starts", i32, (B + 1,)), (lengths, "lengths", i32, (B,)))
        if k_out is not None:
            raise CanopyError("k_out comes without a cache")
    elif any(x is not None for x in (v, v_cache, page_table, context, starts, lengths)):
        raise CanopyError("v, v_cache, page_table, context, starts and lengths come with k_cache")
    _need_given(dev, (q_weight, "q_weight", f32, (d,)), (k_weight, "k_weight", f32, (d,)),
                (q_out, "q_out", dt, (*lead, HQ, d)), (k_out, "k_out", dt, (*lead, HKV, d)), (err, "err", i32, (1,)))
    if freqs is not None:
        _need_all(dev, (freqs, "freqs", f32, freqs.shape if isinstance(freqs, torch.Tensor) else ()))
        if freqs.dim() != 1:
            raise CanopyError("freqs must have shape (R / 2,)")
        R = 2 * freqs.shape[0]
    if positions is not None:
        if not isinstance(positions, torch.Tensor) or \
                tuple(positions.shape) not in (lead, (*positions.shape[:1], *lead)):
            raise CanopyError(f"positions must have shape {lead} or (axes, *{lead})")
        if not positions.is_cuda or positions.dtype != i32:
            raise CanopyError("positions must be an int32 CUDA tensor")
        if positions.get_device() != dev:
            raise CanopyError("positions must be on the same device as the other tensors")
        if positions.dim() > len(lead):
            axes, axis_step = positions.shape[0], positions.stride(0)
        two = len(lead) == 2 and lead[0] > 1
        row_step = positions.stride(-1) if lead[-1] > 1 else positions.stride(-2) if two else 1
        if two and positions.stride(-2) != row_step * lead[-1]:
            raise CanopyError("positions must have their tokens at one distance")
    _need_given(dev, (axis, "axis", i32, (R // 2,)))
    lib = load()
    with torch.cuda.device(dev):
        if q_out is None:
            q_out = torch.empty((*lead, HQ, d), dtype=dt, device=q.device)
        if k_out is None and k_cache is None:
            k_out = torch.empty((*lead, HKV, d), dtype=dt, device=q.device)
        st = lib.canopy_qk_prep(q.data_ptr(), k.data_ptr(), _opt(v), code, ldq, ldk, ldv, NORM[norm], _opt(q_weight),
                                _opt(k_weight), eps, _opt(freqs), R, _opt(positions), axes, axis_step, row_step,
                                _opt(axis), PAIRS[pairs], N, B, HQ, HKV, d, q_out.data_ptr(), _opt(k_out),
                                _opt(k_cache), _opt(v_cache),
                                _opt(page_table), pages, page_size, max_pages, _opt(context), _opt(starts),
                                _opt(lengths), _opt(err), _raw_stream(dev))
    _check(st, "canopy_qk_prep")
    return q_out, k_out


def attend_workspace(N: int, B: int, HQ: int, HKV: int, d: int, device="cuda") -> torch.Tensor:
    """Workspace of attend calls over up to N rows of B sequences with these
    heads.  Calls that may run at the same time need one each."""
    n = int(load().canopy_attend_workspace_bytes(N, B, HQ, HKV, d))
    if n == 0:
        raise CanopyError("unsupported sizes for the attend workspace")
    return _new_workspace(n, 4096, device)


def attend_plan(N: int, B: int, HQ: int, HKV: int, bf16: bool, d: int) -> str:
    """Which path canopy_attend takes for these sizes (an ATTEND_PLAN name)."""
    code = load().canopy_attend_plan(N, B, HQ, HKV, BF16 if bf16 else F32, d)
    return {v: k for k, v in ATTEND_PLAN.items()}[code]


def attend(q, k_cache, v_cache, page_table, context, ws, starts=None, parent=None, lengths=None, window: int = 0,
           sinks: int = 0, scale=None, out=None):
    """Attention of new rows over a paged cache that holds their keys and
    values already (qk_prep): o of q's shape and dtype.
    q [N, HQ, d]: packed sequences at starts int32 [B+1], or one token of each
    stream; or [B, T, HQ, d], with parent int32 [B, T] the nodes of draft trees
    (T <= 256), of which lengths int32 [B] (or all) are there; rows that are not
    there are left as they were.  Row i of a sequence sees the context[b] tokens
    before it and the new ones up to itself, or on its root path; with window > 0
    only those less than window positions before it and the first `sinks`.
    k_cache, v_cache [pages, HKV, page_size, d], page_table int32
    [B, max_pages].  scale: d ** -0.5 unless given.  out lies apart from q and the
    caches.  ws: attend_workspace for at least these sizes."""
    if _marshal is None:
        load()
    r = _marshal.attend(q, k_cache, v_cache, page_table, context, ws, starts, parent, lengths, window, sinks, scale,
                        out)
    if r is not None:
        return _short_call("canopy_attend", r)
    lead, N = _rows_shape(q, starts, lengths, "q")
    HQ, d = q.shape[-2:]
    dt, i32, dev = q.dtype, torch.int32, q.get_device()
    code = _dt(q)
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise CanopyError("k_cache must have shape (pages, HKV, page_size, d)")
    HKV = k_cache.shape[1]
    B, pages, page_size, max_pages = _cache(k_cache, v_cache, page_table, context, dt, HKV, d, dev)
    _need_ints(N, HQ, window, sinks)
    _streams(lead, B, starts)
    if parent is not None and len(lead) != 2:
        raise CanopyError("parent comes with (B, T, HQ, d)")
    _need_all(dev, (q, "q", dt, q.shape), (ws, "workspace", torch.uint8, ws.shape))
    _need_given(dev, (starts, "starts", i32, (B + 1,)), (parent, "parent", i32, lead), (out, "o", dt, q.shape),
                (lengths, "lengths", i32, (B,)))
    lib = load()
    if ws.numel() < lib.canopy_attend_workspace_bytes(N, B, HQ, HKV, d):
        raise CanopyError("the workspace is too small for these sizes")
    with torch.cuda.device(dev):
        if out is None:
            out = torch.empty(q.shape, dtype=dt, device=q.device)
        st = lib.canopy_attend(q.data_ptr(), code, k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), pages,
                               page_size, max_pages, context.data_ptr(), _opt(starts), _opt(parent), _opt(lengths), N,
                               B, HQ, HKV, d, window, sinks, d ** -0.5 if scale is None else scale, out.data_ptr(),
                               ws.data_ptr(), _raw_stream(dev))
    _check(st, "canopy_attend")
    return out


def cache_commit(accepted, parent, k_cache, v_cache, page_table, context, lengths=None, err=None):
    """The paged cache after accepting node accepted[b] of every stream's draft
    tree (int32 [B], as commit takes it; parent int32 [B, T]): the keys and
    values of its root path, at places context[b] + node, move to context[b] +
    depth, in place.  Returns the new lengths, int32 [B].  err: an optional int32
    CUDA tensor of one element for device error bits."""
    if _marshal is None:
        load()
    r = _marshal.cache_commit(accepted, parent, k_cache, v_cache, page_table, context, lengths, err)
    if r is not None:
        return _short_call("canopy_cache_commit", r)
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise CanopyError("k_cache must have shape (pages, HKV, page_size, d)")
    _, HKV, _, d = k_cache.shape
    i32, dev = torch.int32, k_cache.get_device()
    code = _dt(k_cache)
    B, pages, page_size, max_pages = _cache(k_cache, v_cache, page_table, context, k_cache.dtype, HKV, d, dev)
    if not isinstance(parent, torch.Tensor) or parent.dim() != 2 or parent.shape[0] != B:
        raise CanopyError(f"parent must have shape ({B}, T)")
    T = parent.shape[1]
    _need_ints(T)
    _need_all(dev, (parent, "parent", i32, (B, T)), (accepted, "accepted", i32, (B,)))
    _need_given(dev, (lengths, "lengths", i32, (B,)), (err, "err", i32, (1,)))
    lib = load()
    with torch.cuda.device(dev):
        new = torch.empty((B,), dtype=i32, device=k_cache.device)
        st = lib.canopy_cache_commit(accepted.data_ptr(), parent.data_ptr(), _opt(lengths), k_cache.data_ptr(),
                                     v_cache.data_ptr(), code, page_table.data_ptr(), pages, page_size, max_pages,
                                     context.data_ptr(), T, B, HKV, d, new.data_ptr(), _opt(err), _raw_stream(dev))
    _check(st, "canopy_cache_commit")
    return new


def tree_conv(x, conv_state, weight, parent, bias=None, act: str = "silu", err=None, out=None):
    """Tree-aware short causal convolution: y [B, T, C] in x's dtype.
    x [B, T, C] (bf16 or fp32); conv_state fp32 [B, C, K-1]; weight fp32
    [C, K]; bias fp32 [C] or None; parent int32 [B, T]; err an optional int32
    CUDA tensor of one element that receives device error bits (OR-ed)."""
    _need(x, "x")
    B, T, C = x.shape
    _need(weight, "weight", torch.float32)
    if weight.dim() != 2 or weight.shape[0] != C:
        raise CanopyError(f"weight must have shape ({C}, K), got {tuple(weight.shape)}")
    K = weight.shape[1]
    _need(conv_state, "conv_state", torch.float32, (B, C, K - 1))
    _need(parent, "parent", torch.int32, (B, T))
    if bias is not None:
        _need(bias, "bias", torch.float32, (C,))
    if out is None:
        out = torch.empty_like(x)
    _need(out, "y", x.dtype, x.shape)
    st = load().canopy_tree_conv(_ptr(x), _dt(x), _ptr(conv_state), _ptr(weight),
                                 _ptr(bias) if bias is not None else None, _ptr(parent), T, B, C, K, ACT[act],
                                 _ptr(out), _ptr(err) if err is not None else None, _stream())
    _check(st, "canopy_tree_conv")
    return out


def conv_commit(accepted, x, parent, conv_state, out=None, err=None):
    """The convolution state after accepting node accepted[b] of every
    stream's tree: [B, C, K-1] fp32 (out may be conv_state itself)."""
    _need(x, "x")
    B, T, C = x.shape
    _need(conv_state, "conv_state", torch.float32)
    if conv_state.dim() != 3 or conv_state.shape[:2] != (B, C):
        raise CanopyError(f"conv_state must have shape ({B}, {C}, K-1), got {tuple(conv_state.shape)}")
    K = conv_state.shape[2] + 1
    _need(accepted, "accepted", torch.int32, (B,))
    _need(parent, "parent", torch.int32, (B, T))
    if out is None:
        out = torch.empty_like(conv_state)
    _need(out, "conv_state_new", torch.float32, conv_state.shape)
    st = load().canopy_conv_commit(_ptr(accepted), _ptr(x), _dt(x), _ptr(parent), _ptr(conv_state), _ptr(out), T, B,
                                   C, K, _ptr(err) if err is not None else None, _stream())
    _check(st, "canopy_conv_commit")
    return out


def read_device_error(ws) -> int:
    """Synchronise the current stream of the workspace's device, return and
    clear the device error word."""
    err = ctypes.c_int32(0)
    with torch.cuda.device(ws.device):
        _check(load().canopy_read_device_error(_ptr(ws), ctypes.byref(err), _stream()), "canopy_read_device_error")
    return int(err.value)
