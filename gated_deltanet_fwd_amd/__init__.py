"""Python binding of the MI355X gated-delta-rule training kernel (libgdn.so, include/gdn.h).

Argument marshalling only: every step of the computation runs in the HIP kernels behind the C
ABI. PyTorch supplies device memory and streams: the launch stream (torch's current stream unless
one is given) and, for problems whose longest document runs apart from the others, an auxiliary
stream that this module keeps per device and names in the problem descriptor. Buffers that a call
allocates are allocated on its launch stream. The functions carry the C names:

    gdn_saved_bytes(problem)                      -> int
    gdn_workspace_bytes(problem, op)              -> int
    gdn_fwd(problem, q, k, v, g, beta, cu, ...)   -> (o, ht, saved)
    gdn_fwd_recompute(problem, q, k, v, g, beta, cu, ...) -> saved
    gdn_bwd(problem, q, k, v, g, beta, cu, saved, dO, ...) -> dict of gradients
    gdn_status(problem, op, workspace)            -> int (synchronises the stream)
    gdn_conv_fwd(conv_problem, x, weight, bias, cu, ...)      -> list of outputs (one per group)
    gdn_conv_bwd(conv_problem, x, weight, bias, cu, dys, ...) -> dict dx, dweight, dbias
    gdn_recurrent(recurrent_problem, q, k, v, g, beta, states, slot_in, slot_out, ...) -> o
    gdn_conv_step(conv_step_problem, x, weight, bias, windows, slot_in, slot_out, ...) -> list of outputs
    gdn_rope_frequencies(rotary_dim, ...)         -> (int64 tensor on the CPU, magnitude)
    gdn_qk_rope_fwd(rope_problem, q, k, positions, freqs, ...) -> (q_out, k_out)
    gdn_qk_rope_bwd(rope_problem, q, k, positions, freqs, dq_out, dk_out, ...) -> dict of gradients

gdn_recurrent, gdn_conv_step, gdn_qk_rope_fwd and gdn_qk_rope_bwd check their tensors (shape, type,
layout, device) before the call and raise GdnError; their marshalling is native (csrc/gdn_binding.cpp),
since a decoding step is shorter than it would take in Python.

A missing or unloadable library raises ImportError-like errors at first use; there is no other
code path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

GDN_OK, GDN_EINVAL, GDN_EUNSUPPORTED, GDN_ESAVED, GDN_EWORKSPACE, GDN_EHIP = range(6)
DTYPE_BF16, DTYPE_F32 = 0, 1
SAVE_LIGHT, SAVE_FULL, SAVE_TAPE = 0, 1, 2
OP_FWD, OP_RECOMPUTE, OP_BWD = 0, 1, 2
ABI_VERSION = 2

EXPORTS = ("gdn_saved_bytes", "gdn_workspace_bytes", "gdn_fwd", "gdn_fwd_recompute", "gdn_bwd", "gdn_status",
           "gdn_fwd_noalloc", "gdn_conv_workspace_bytes", "gdn_conv_fwd", "gdn_conv_bwd", "gdn_last_error",
           "gdn_abi_version", "gdn_recurrent", "gdn_conv_step", "gdn_rope_frequencies", "gdn_qk_rope_workspace_bytes",
           "gdn_qk_rope_fwd", "gdn_qk_rope_bwd")
NORMS = {"none": 0, "l2": 1, "rms": 2}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


class GdnError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__("gdn error %d: %s" % (code, msg))
        self.code = code


class _Problem(ctypes.Structure):
    _fields_ = [
        ("n_seqs", ctypes.c_int32),
        ("h_qk", ctypes.c_int32),
        ("h_v", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("n_tokens", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("l2norm_qk", ctypes.c_int32),
        ("has_h0", ctypes.c_int32),
        ("want_ht", ctypes.c_int32),
        ("save_mode", ctypes.c_int32),
        ("deterministic", ctypes.c_int32),
        ("cu_seqlens_host", ctypes.POINTER(ctypes.c_int32)),
        ("aux_stream", ctypes.c_void_p),
        ("segments", ctypes.c_int32),
        ("reserved0", ctypes.c_int32),
    ]


class _ConvProblem(ctypes.Structure):
    _fields_ = [
        ("n_seqs", ctypes.c_int32),
        ("channels", ctypes.c_int32),
        ("n_tokens", ctypes.c_int64),
        ("width", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("silu", ctypes.c_int32),
        ("n_groups", ctypes.c_int32),
        ("group_channels", ctypes.c_int32 * 4),
        ("cu_seqlens_host", ctypes.POINTER(ctypes.c_int32)),
    ]


class _RecurrentProblem(ctypes.Structure):
    _fields_ = [
        ("n_seqs", ctypes.c_int32),
        ("h_qk", ctypes.c_int32),
        ("h_v", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("n_tokens", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("l2norm_qk", ctypes.c_int32),
        ("n_slots", ctypes.c_int32),
        ("reserved0", ctypes.c_int32),
        ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64),
        ("cu_seqlens_host", ctypes.POINTER(ctypes.c_int32)),
    ]


class _ConvStepProblem(ctypes.Structure):
    _fields_ = [
        ("n_seqs", ctypes.c_int32),
        ("channels", ctypes.c_int32),
        ("n_tokens", ctypes.c_int64),
        ("width", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("silu", ctypes.c_int32),
        ("n_groups", ctypes.c_int32),
        ("group_channels", ctypes.c_int32 * 4),
        ("n_slots", ctypes.c_int32),
        ("reserved0", ctypes.c_int32),
        ("x_stride", ctypes.c_int64),
        ("cu_seqlens_host", ctypes.POINTER(ctypes.c_int32)),
    ]


class _QkRopeProblem(ctypes.Structure):
    _fields_ = [
        ("n_tokens", ctypes.c_int64),
        ("h_q", ctypes.c_int32),
        ("h_k", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("norm", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("magnitude", ctypes.c_float),
        ("reserved0", ctypes.c_int32),
        ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64),
        ("qo_stride", ctypes.c_int64),
        ("ko_stride", ctypes.c_int64),
        ("dq_stride", ctypes.c_int64),
        ("dk_stride", ctypes.c_int64),
    ]


class _RopeScaling(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32),
        ("base", ctypes.c_double),
        ("factor", ctypes.c_double),
        ("original_length", ctypes.c_double),
        ("fast", ctypes.c_double),
        ("slow", ctypes.c_double),
    ]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libgdn.so once. Raises OSError if it was not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError("libgdn.so not found at %s: build it with `python -m gated_deltanet_fwd_amd.build`" % path)
    lib = ctypes.CDLL(path)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    pp = ctypes.POINTER(_Problem)
    lib.gdn_saved_bytes.argtypes = [pp]
    lib.gdn_saved_bytes.restype = Z
    lib.gdn_workspace_bytes.argtypes = [pp, I]
    lib.gdn_workspace_bytes.restype = Z
    lib.gdn_fwd.argtypes = [pp] + [P] * 11 + [Z, P]
    lib.gdn_fwd.restype = I
    lib.gdn_fwd_recompute.argtypes = [pp] + [P] * 9 + [Z, P]
    lib.gdn_fwd_recompute.restype = I
    lib.gdn_bwd.argtypes = [pp] + [P] * 17 + [Z, P]
    lib.gdn_bwd.restype = I
    lib.gdn_status.argtypes = [pp, I, P, P]
    lib.gdn_status.restype = I
    lib.gdn_fwd_noalloc.argtypes = [pp] + [P] * 10 + [P]
    lib.gdn_fwd_noalloc.restype = I
    cp = ctypes.POINTER(_ConvProblem)
    lib.gdn_conv_workspace_bytes.argtypes = [cp]
    lib.gdn_conv_workspace_bytes.restype = Z
    lib.gdn_conv_fwd.argtypes = [cp, P, P, P, P, P, P]
    lib.gdn_conv_fwd.restype = I
    lib.gdn_conv_bwd.argtypes = [cp, P, P, P, P, P, P, P, P, P, Z, P]
    lib.gdn_conv_bwd.restype = I
    lib.gdn_recurrent.argtypes = [ctypes.POINTER(_RecurrentProblem)] + [P] * 12
    lib.gdn_recurrent.restype = I
    lib.gdn_conv_step.argtypes = [ctypes.POINTER(_ConvStepProblem)] + [P] * 10
    lib.gdn_conv_step.restype = I
    lib.gdn_rope_frequencies.argtypes = [ctypes.POINTER(_RopeScaling), P, ctypes.POINTER(ctypes.c_float)]
    lib.gdn_rope_frequencies.restype = I
    rp = ctypes.POINTER(_QkRopeProblem)
    lib.gdn_qk_rope_workspace_bytes.argtypes = [rp]
    lib.gdn_qk_rope_workspace_bytes.restype = Z
    lib.gdn_qk_rope_fwd.argtypes = [rp] + [P] * 9
    lib.gdn_qk_rope_fwd.restype = I
    lib.gdn_qk_rope_bwd.argtypes = [rp] + [P] * 13 + [Z, P]
    lib.gdn_qk_rope_bwd.restype = I
    lib.gdn_last_error.argtypes = []
    lib.gdn_last_error.restype = ctypes.c_char_p
    lib.gdn_abi_version.argtypes = []
    lib.gdn_abi_version.restype = I
    if lib.gdn_abi_version() != ABI_VERSION:
        raise OSError("libgdn.so has ABI version %d, this binding expects %d: rebuild it" %
                      (lib.gdn_abi_version(), ABI_VERSION))
    _lib = lib
    return lib


class Problem:
    """A gdn_problem descriptor plus the host copy of cu_seqlens it points to."""

    def __init__(self, cu_seqlens_host, h_qk: int, h_v: int, d: int, dtype=torch.bfloat16, l2norm: bool = True,
                 has_h0: bool = False, want_ht: bool = False, save_mode: int = SAVE_LIGHT,
                 deterministic: bool = True, use_aux_stream=True, segments: int = 0):
        self.cu = np.ascontiguousarray(np.asarray(cu_seqlens_host, dtype=np.int32))
        self.dtype = dtype
        # True: the module's auxiliary stream of the device; False: one stream; or a stream object
        self.use_aux_stream = use_aux_stream
        self.st = _Problem(
            n_seqs=int(self.cu.shape[0] - 1),
            h_qk=int(h_qk),
            h_v=int(h_v),
            d=int(d),
            n_tokens=int(self.cu[-1]),
            dtype=DTYPE_BF16 if dtype == torch.bfloat16 else DTYPE_F32,
            l2norm_qk=int(bool(l2norm)),
            has_h0=int(bool(has_h0)),
            want_ht=int(bool(want_ht)),
            save_mode=int(save_mode),
            deterministic=int(bool(deterministic)),
            cu_seqlens_host=self.cu.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
            aux_stream=None,
            segments=int(segments),
            reserved0=0,
        )

    @property
    def T(self) -> int:
        return int(self.st.n_tokens)

    @property
    def N(self) -> int:
        return int(self.st.n_seqs)

    def ref(self):
        return ctypes.byref(self.st)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _torch_stream(stream, device) -> torch.cuda.Stream:
    if stream is None:
        return torch.cuda.current_stream(device)
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream), device=device)


_aux_streams: Dict[int, torch.cuda.Stream] = {}


def aux_stream(device) -> torch.cuda.Stream:
    """The auxiliary stream this module names in problems on `device` (created on first use, kept
    for the life of the process, default priority)."""
    idx = torch.device(device).index
    idx = torch.cuda.current_device() if idx is None else idx
    if idx not in _aux_streams:
        _aux_streams[idx] = torch.cuda.Stream(device=idx)
    return _aux_streams[idx]


class _Call:
    """Launch context of one call: the launch stream, allocations on it, and the problem's auxiliary
    stream set for the call."""

    def __init__(self, p: "Problem", device, stream):
        self.p = p
        self.device = device
        self.stream = _torch_stream(stream, device)
        u = p.use_aux_stream
        aux = u if isinstance(u, torch.cuda.Stream) else aux_stream(device) if u else None
        p.st.aux_stream = None if aux is None or aux.cuda_stream == self.stream.cuda_stream else aux.cuda_stream

    def empty(self, *shape, dtype):
        with torch.cuda.stream(self.stream):
            return torch.empty(*shape, dtype=dtype, device=self.device)

    def empty_like(self, t):
        with torch.cuda.stream(self.stream):
            return torch.empty_like(t)

    def handle(self) -> ctypes.c_void_p:
        return ctypes.c_void_p(self.stream.cuda_stream)


def _check(rc: int):
    if rc != GDN_OK:
        raise GdnError(rc, load_library().gdn_last_error().decode())


def gdn_saved_bytes(p: Problem) -> int:
    n = load_library().gdn_saved_bytes(p.ref())
    if n == 0:
        raise GdnError(GDN_EINVAL, load_library().gdn_last_error().decode())
    return int(n)


def gdn_workspace_bytes(p: Problem, op: int) -> int:
    n = load_library().gdn_workspace_bytes(p.ref(), int(op))
    if n == 0:
        raise GdnError(GDN_EINVAL, load_library().gdn_last_error().decode())
    return int(n)


def gdn_fwd(p: Problem, q, k, v, g, beta, cu_seqlens, h0=None, o=None, ht=None, saved=None, workspace=None,
            stream=None):
    """Forward: returns (o, ht or None, saved)."""
    lib = load_library()
    c = _Call(p, q.device, stream)
    T, HV, d = p.T, p.st.h_v, p.st.d
    if o is None:
        o = c.empty((T, HV, d), dtype=q.dtype)
    if p.st.want_ht and ht is None:
        ht = c.empty((p.N, HV, d, d), dtype=torch.float32)
    if saved is None:
        saved = c.empty(gdn_saved_bytes(p), dtype=torch.uint8)
    if workspace is None:
        workspace = c.empty(gdn_workspace_bytes(p, OP_FWD), dtype=torch.uint8)
    _check(lib.gdn_fwd(p.ref(), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), _ptr(h0), _ptr(o),
                       _ptr(ht), _ptr(saved), _ptr(workspace), workspace.numel(), c.handle()))
    return o, ht, saved


def gdn_fwd_recompute(p: Problem, q, k, v, g, beta, cu_seqlens, h0=None, saved=None, workspace=None, stream=None):
    """Checkpoint re-run of the forward: returns the saved set only."""
    lib = load_library()
    c = _Call(p, q.device, stream)
    if saved is None:
        saved = c.empty(gdn_saved_bytes(p), dtype=torch.uint8)
    if workspace is None:
        workspace = c.empty(gdn_workspace_bytes(p, OP_RECOMPUTE), dtype=torch.uint8)
    _check(lib.gdn_fwd_recompute(p.ref(), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens),
                                 _ptr(h0), _ptr(saved), _ptr(workspace), workspace.numel(), c.handle()))
    return saved


def gdn_bwd(p: Problem, q, k, v, g, beta, cu_seqlens, saved, dO, h0=None, dht=None, grads=None, workspace=None,
            stream=None) -> Dict[str, torch.Tensor]:
    """Backward: returns dict dq, dk, dv, dg, dbeta, dh0 (dh0 None without h0)."""
    lib = load_library()
    c = _Call(p, q.device, stream)
    if grads is None:
        grads = dict(dq=c.empty_like(q), dk=c.empty_like(k), dv=c.empty_like(v), dg=c.empty_like(g),
                     dbeta=c.empty_like(beta),
                     dh0=c.empty_like(h0) if (p.st.has_h0 and h0 is not None) else None)
    if workspace is None:
        workspace = c.empty(gdn_workspace_bytes(p, OP_BWD), dtype=torch.uint8)
    _check(lib.gdn_bwd(p.ref(), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), _ptr(h0),
                       _ptr(saved), _ptr(dO), _ptr(dht), _ptr(grads["dq"]), _ptr(grads["dk"]), _ptr(grads["dv"]),
                       _ptr(grads["dg"]), _ptr(grads["dbeta"]), _ptr(grads.get("dh0")), _ptr(workspace),
                       workspace.numel(), c.handle()))
    return grads


def gdn_fwd_noalloc(p: Problem, q, k, v, g, beta, cu_seqlens, h0=None, o=None, ht=None, saved=None, stream=None):
    """Forward whose workspace is the library's fixed device scratch array (no workspace
    argument; the library allocates nothing). Returns (o, ht or None, saved); o, ht and saved are
    allocated here when not given."""
    lib = load_library()
    c = _Call(p, q.device, stream)
    T, HV, d = p.T, p.st.h_v, p.st.d
    if o is None:
        o = c.empty((T, HV, d), dtype=q.dtype)
    if p.st.want_ht and ht is None:
        ht = c.empty((p.N, HV, d, d), dtype=torch.float32)
    if saved is None:
        saved = c.empty(gdn_saved_bytes(p), dtype=torch.uint8)
    _check(lib.gdn_fwd_noalloc(p.ref(), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(cu_seqlens), _ptr(h0),
                               _ptr(o), _ptr(ht), _ptr(saved), c.handle()))
    return o, ht, saved


def gdn_status(p: Problem, op: int, workspace, stream=None) -> int:
    """Device-side status of the last call of `op` on this workspace: GDN_OK, GDN_EINVAL or
    GDN_ESAVED (synchronises the launch stream)."""
    c = _Call(p, workspace.device, stream)
    return int(load_library().gdn_status(p.ref(), int(op), _ptr(workspace), c.handle()))


def problem_for(w, save_mode: int = SAVE_LIGHT, deterministic: Optional[bool] = None, l2norm: Optional[bool] = None,
                want_ht: Optional[bool] = None, use_aux_stream=True, segments: int = 0) -> Problem:
    """Problem descriptor for a synthetic workload description (see synthetic.Workload)."""
    cu = np.zeros(w.N + 1, dtype=np.int32)
    cu[1:] = np.cumsum(np.asarray(w.lengths, dtype=np.int64))
    return Problem(cu, w.H, w.HV, w.d, dtype=w.torch_dtype, l2norm=w.l2norm if l2norm is None else l2norm,
                   has_h0=w.has_h0, want_ht=w.want_ht if want_ht is None else want_ht, save_mode=save_mode,
                   deterministic=w.deterministic if deterministic is None else deterministic,
                   use_aux_stream=use_aux_stream, segments=segments)


class ConvProblem:
    """A gdn_conv_problem descriptor: the causal conv1d + SiLU front-end over [T, sum(groups)]
    channels with a `width`-tap window, its output split into the groups' tensors."""

    def __init__(self, cu_seqlens_host, group_channels, width: int = 4, dtype=torch.bfloat16, silu: bool = True):
        self.cu = np.ascontiguousarray(np.asarray(cu_seqlens_host, dtype=np.int32))
        self.groups = [int(c) for c in group_channels]
        self.dtype = dtype
        gc = (ctypes.c_int32 * 4)(*(self.groups + [0] * (4 - len(self.groups))))
        self.st = _ConvProblem(n_seqs=int(self.cu.shape[0] - 1), channels=int(sum(self.groups)),
                               n_tokens=int(self.cu[-1]), width=int(width),
                               dtype=DTYPE_BF16 if dtype == torch.bfloat16 else DTYPE_F32, silu=int(bool(silu)),
                               n_groups=len(self.groups), group_channels=gc,
                               cu_seqlens_host=self.cu.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))

    @property
    def T(self) -> int:
        return int(self.st.n_tokens)

    def ref(self):
        return ctypes.byref(self.st)


def _ptr_array(ts):
    return (ctypes.c_void_p * 4)(*([t.data_ptr() for t in ts] + [0] * (4 - len(ts))))


def gdn_conv_workspace_bytes(p: ConvProblem) -> int:
    n = load_library().gdn_conv_workspace_bytes(p.ref())
    if n == 0:
        raise GdnError(GDN_EINVAL, load_library().gdn_last_error().decode())
    return int(n)


def gdn_conv_fwd(p: ConvProblem, x, weight, bias, cu_seqlens, outs=None, stream=None):
    """Forward of the conv front-end: returns the list of output tensors, [T, group_channels[g]]."""
    lib = load_library()
    dev = x.device
    s = _torch_stream(stream, dev)
    if outs is None:
        with torch.cuda.stream(s):
            outs = [torch.empty((p.T, c), dtype=x.dtype, device=dev) for c in p.groups]
    _check(lib.gdn_conv_fwd(p.ref(), _ptr(x), _ptr(weight), _ptr(bias), _ptr(cu_seqlens), _ptr_array(outs),
                            ctypes.c_void_p(s.cuda_stream)))
    return outs


def gdn_conv_bwd(p: ConvProblem, x, weight, bias, cu_seqlens, dys, dx=None, dweight=None, dbias=None,
                 workspace=None, stream=None) -> Dict[str, torch.Tensor]:
    """Backward of the conv front-end: returns dict dx [T, C], dweight [C, W], dbias [C] (None when
    bias is None)."""
    lib = load_library()
    dev = x.device
    s = _torch_stream(stream, dev)
    with torch.cuda.stream(s):
        if dx is None:
            dx = torch.empty_like(x)
        if dweight is None:
            dweight = torch.empty_like(weight)
        if dbias is None and bias is not None:
            dbias = torch.empty_like(bias)
        if workspace is None:
            workspace = torch.empty(gdn_conv_workspace_bytes(p), dtype=torch.uint8, device=dev)
    _check(lib.gdn_conv_bwd(p.ref(), _ptr(x), _ptr(weight), _ptr(bias), _ptr(cu_seqlens), _ptr_array(dys), _ptr(dx),
                            _ptr(dweight), _ptr(dbias), _ptr(workspace), workspace.numel(),
                            ctypes.c_void_p(s.cuda_stream)))
    return dict(dx=dx, dweight=dweight, dbias=dbias)


# ------------------------------------------------------------------- serving steps, q/k rotation


def _io_dtype(dtype) -> int:
    if dtype not in (torch.bfloat16, torch.float32):
        raise GdnError(GDN_EUNSUPPORTED, "unsupported dtype %s" % (dtype,))
    return DTYPE_BF16 if dtype == torch.bfloat16 else DTYPE_F32


_marshal = None


def _native():
    """The native argument marshalling of the functions below (csrc/gdn_binding.cpp), bound to the
    loaded library. Raises OSError if it was not built."""
    global _marshal
    if _marshal is None:
        lib = load_library()
        try:
            from . import _binding
        except ImportError as e:
            raise OSError("_binding.so not loadable (%s): build it with `python -m gated_deltanet_fwd_amd.build`" % e)
        _binding.init(GdnError, *(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in
                                  ("gdn_recurrent", "gdn_conv_step", "gdn_qk_rope_fwd", "gdn_qk_rope_bwd",
                                   "gdn_qk_rope_workspace_bytes", "gdn_last_error")))
        _marshal = _binding
    return _marshal


def _call(name: str, device_of, stream, *args):
    """A native call on torch's current stream, or with `stream` as the current one (the launch stream
    and the one that buffers are allocated on)."""
    f = getattr(_marshal or _native(), name)
    if stream is None:
        return f(*args)
    with torch.cuda.stream(_torch_stream(stream, device_of.device)):
        return f(*args)


def _step_lengths(cu_seqlens_host, n_seqs):
    """(host copy of cu_seqlens or None, its pointer or None, token count)."""
    if cu_seqlens_host is None:
        return None, None, int(n_seqs)
    cu = np.ascontiguousarray(np.asarray(cu_seqlens_host, dtype=np.int32))
    if cu.shape != (n_seqs + 1,):
        raise GdnError(GDN_EINVAL, "cu_seqlens_host has shape %s, expected (%d,)" % (cu.shape, n_seqs + 1))
    return cu, cu.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), int(cu[-1])


class RecurrentProblem:
    """A gdn_recurrent_problem descriptor: `n_seqs` sequences on a cache of `n_slots` states, one
    token each, or as many as the host copy of cu_seqlens says."""

    def __init__(self, n_seqs: int, h_qk: int, h_v: int, d: int, n_slots: int, cu_seqlens_host=None,
                 dtype=torch.bfloat16, l2norm: bool = True):
        self.cu, ptr, tokens = _step_lengths(cu_seqlens_host, n_seqs)
        self.dtype = dtype
        self.st = _RecurrentProblem(n_seqs=int(n_seqs), h_qk=int(h_qk), h_v=int(h_v), d=int(d), n_tokens=tokens,
                                    dtype=_io_dtype(dtype),
                                    l2norm_qk=int(bool(l2norm)), n_slots=int(n_slots), cu_seqlens_host=ptr)
        self.at = ctypes.addressof(self.st)

    def ref(self):
        return ctypes.byref(self.st)


def gdn_recurrent(p: RecurrentProblem, q, k, v, g, beta, states, slot_in, slot_out, slot_tok=None, cu_seqlens=None,
                  o=None, stream=None):
    """One serving step of the recurrent rule: runs every sequence's tokens from states[slot_in] (-1:
    zero), leaves its state in states[slot_out] (-1: nowhere) and, with slot_tok, the state after each
    token in states[slot_tok]. q, k and v may be parts of one row (a token's heads contiguous).
    Returns o; `states` is updated in place. Rows that the lengths on the device leave to no sequence are
    not written: with `o` given they keep its values, without they are uninitialised."""
    return _call("recurrent", v, stream, p.at, q, k, v, g, beta, states, slot_in, slot_out, slot_tok, cu_seqlens, o)


class ConvStepProblem:
    """A gdn_conv_step_problem descriptor: the conv1d + SiLU front-end on `n_seqs` sequences with a
    cache of `n_slots` windows, one token each, or as many as the host copy of cu_seqlens says."""

    def __init__(self, n_seqs: int, group_channels, n_slots: int, cu_seqlens_host=None, width: int = 4,
                 dtype=torch.bfloat16, silu: bool = True):
        self.cu, ptr, tokens = _step_lengths(cu_seqlens_host, n_seqs)
        self.dtype = dtype
        self.groups = [int(c) for c in group_channels]
        if not 1 <= len(self.groups) <= 4:
            raise GdnError(GDN_EINVAL, "n_groups must be 1..4 (got %d)" % len(self.groups))
        channels, width = sum(self.groups), int(width)
        self.st = _ConvStepProblem(n_seqs=int(n_seqs), channels=channels, n_tokens=tokens, width=width,
                                   dtype=_io_dtype(dtype), silu=int(bool(silu)),
                                   n_groups=len(self.groups),
                                   group_channels=(ctypes.c_int32 * 4)(*self.groups),
                                   n_slots=int(n_slots), cu_seqlens_host=ptr)
        self.at = ctypes.addressof(self.st)

    def ref(self):
        return ctypes.byref(self.st)


def gdn_conv_step(p: ConvStepProblem, x, weight, bias, windows, slot_in, slot_out, slot_tok=None, cu_seqlens=None,
                  outs=None, stream=None):
    """One serving step of the conv front-end on cached windows (slots as in gdn_recurrent). Returns
    the list of outputs, [T, group_channels[g]]; `windows` is updated in place (None at width 1). Rows of
    no sequence are as in gdn_recurrent. The outputs of a short call (up to 1 MiB together) are parts of
    one storage, as those of gdn_qk_rope_fwd and _bwd: one part keeps all of the memory and torch.save
    of it writes all, and resize_ to more elements grows a part over the ones behind it, as with the
    parts of torch.split. Clone a part before either, or give the outputs."""
    return _call("conv_step", x, stream, p.at, x, weight, bias, windows, slot_in, slot_out, slot_tok, cu_seqlens,
                 None if outs is None else list(outs))


def gdn_rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                         original_length: float = 0.0, fast: float = 32.0, slow: float = 1.0):
    """Frequencies of the rotation as 64-bit fractions of a turn (an int64 tensor of rotary_dim / 2 on
    the CPU: move it to the GPU once) and the magnitude. `scaling`: "none", "linear", "ntk", "yarn" or
    "bands" (see gdn.h)."""
    if scaling not in ROPE_SCALINGS:
        raise GdnError(GDN_EINVAL, "unknown scaling %r" % (scaling,))
    s = _RopeScaling(kind=ROPE_SCALINGS[scaling], rotary_dim=int(rotary_dim), base=float(base), factor=float(factor),
                     original_length=float(original_length), fast=float(fast), slow=float(slow))
    out = torch.zeros(max(int(rotary_dim) // 2, 1), dtype=torch.int64)
    m = ctypes.c_float()
    _check(load_library().gdn_rope_frequencies(ctypes.byref(s), out.data_ptr(), ctypes.byref(m)))
    return out, float(m.value)


class QkRopeProblem:
    """A gdn_qk_rope_problem descriptor: norms ("rms", "l2" or "none") of h_q q heads and h_k k heads
    of n_tokens tokens and the rotation of each head's first rotary_dim values (None: all)."""

    def __init__(self, n_tokens: int, h_q: int, h_k: int, d: int, dtype=torch.bfloat16, norm: str = "rms",
                 rotary_dim: Optional[int] = None, interleaved: bool = False, eps: float = 1e-6,
                 magnitude: float = 1.0):
        if norm not in NORMS:
            raise GdnError(GDN_EINVAL, "unknown norm %r" % (norm,))
        rotary = int(d if rotary_dim is None else rotary_dim)
        self.dtype = dtype
        self.st = _QkRopeProblem(n_tokens=int(n_tokens), h_q=int(h_q), h_k=int(h_k), d=int(d),
                                 dtype=_io_dtype(dtype), norm=NORMS[norm],
                                 rotary_dim=rotary, interleaved=int(bool(interleaved)), eps=float(eps),
                                 magnitude=float(magnitude))
        self.at = ctypes.addressof(self.st)

    def ref(self):
        return ctypes.byref(self.st)


def gdn_qk_rope_workspace_bytes(p: QkRopeProblem) -> int:
    n = load_library().gdn_qk_rope_workspace_bytes(p.ref())
    if n == 0:
        raise GdnError(GDN_EINVAL, load_library().gdn_last_error().decode())
    return int(n)


def gdn_qk_rope_fwd(p: QkRopeProblem, q, k, positions, freqs, q_weight=None, k_weight=None, q_out=None, k_out=None,
                    stream=None):
    """Norms and rotation of q [T, h_q, d] and k [T, h_k, d] (None when h_k = 0), which may be parts of
    one row, with positions int32 [T] and the frequencies of gdn_rope_frequencies on the device.
    Returns (q_out, k_out); they may be given, also as q and k themselves."""
    return _call("rope_fwd", q, stream, p.at, q, k, positions, freqs, q_weight, k_weight, q_out, k_out)


def gdn_qk_rope_bwd(p: QkRopeProblem, q, k, positions, freqs, dq_out, dk_out, q_weight=None, k_weight=None, grads=None,
                    workspace=None, stream=None) -> Dict[str, torch.Tensor]:
    """Backward of gdn_qk_rope_fwd (q and k may be None with norm "none"): returns dict dq, dk,
    dq_weight, dk_weight (None without the weight). `grads` may name any of the buffers."""
    g = grads or {}
    dq, dk, dwq, dwk = _call("rope_bwd", dq_out, stream, p.at, q, k, positions, freqs, q_weight, k_weight, dq_out, dk_out,
                             g.get("dq"), g.get("dk"), g.get("dq_weight"), g.get("dk_weight"), workspace)
    return dict(dq=dq, dk=dk, dq_weight=dwq, dk_weight=dwk)
