"""Plans of the sequence operators (the C ABI in include/seq.h).

``CausalConvPlan`` is the short causal depthwise convolution, ``ScanPlan`` the
selective state-space scan, ``BlockNormPlan`` the norms around a block with
its gate and residual scale: what a selective state-space layer runs between
its matrix products.  Each runs forwards (``run``) and backwards
(``backward``); the first two also advance single tokens against a cache of
states (``step``).

The computation runs in the library's CUDA kernels, PyTorch supplies memory
and streams, and there is no CPU fallback.  Tensors are checked and calls made
in ``bind/seq_bind.cpp`` (a Python module of its own: for single tokens the
checks in Python would take longer than the kernels).  Activations are
token-major, channels innermost; rows may be slices of wider tensors (any
strides, channels contiguous).  Sizes in a plan are the largest that its calls
may bring, and size its workspace: device memory of its own, outside PyTorch's
allocator (``workspace_bytes``; the gradients' share is taken by the first
``backward``, after ``torch.cuda.empty_cache`` where there is no room).  A call allocates the outputs that it is not given.  With an
explicit ``stream`` (a torch.cuda.Stream) it runs, and allocates, on that
stream, and the tensors it is given are recorded there.

As with ``Plan``, results carry no autograd graph, whether or not the inputs
require gradients: training wraps ``run`` and ``backward`` in a
``torch.autograd.Function`` (``examples/selective_layer.py``).  Tensors that a
call is given to write (caches, states, outputs) count as changed in place.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import warnings
from collections import namedtuple

from . import build as _build
from .binding import DgradError, load_library

DTYPE = {"fp32": 0, "fp16": 1, "bf16": 2}
OUT_OF_MEMORY = 5   # DGRAD_ERR_OOM
ACT = {"none": 0, "silu": 1, "sigmoid": 2}

# Every function declared in include/seq.h (checked by the CPU tests).
SEQ_EXPORTS = ("seq_conv_plan", "seq_conv_run", "seq_conv_backward", "seq_conv_step", "seq_conv_check",
               "seq_conv_workspace_bytes", "seq_conv_destroy", "seq_scan_plan", "seq_scan_checkpoint_bytes",
               "seq_scan_run", "seq_scan_backward", "seq_scan_step", "seq_scan_check", "seq_scan_workspace_bytes",
               "seq_scan_destroy", "seq_norm_plan", "seq_norm_run", "seq_norm_backward", "seq_norm_workspace_bytes",
               "seq_norm_destroy")

ConvGrads = namedtuple("ConvGrads", "x weight bias state")
ScanGrads = namedtuple("ScanGrads", "u dt A B C D z dt_bias state")
NormGrads = namedtuple("NormGrads", "y gate residual post_weight scale next_weight")

_LIB = _BIND = None


def _library():
    """The C library, with the functions that are called through ctypes declared, and the call module."""
    global _LIB, _BIND
    if _LIB is None:
        import torch  # noqa: F401 (the call module links against it)
        lib = load_library()
        if not _build.bind_up_to_date():
            try:
                _build.build_bind()
            except Exception as e:
                if not _build.bind_fits():
                    raise RuntimeError("the sequence operators' call module is missing, or was built for another "
                                       f"PyTorch or Python, and could not be built: {e}") from e
                warnings.warn(f"{_build.BIND} is older than its source and could not be rebuilt: {e}", RuntimeWarning,
                              stacklevel=2)
        i, q, vp, f = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p, ctypes.c_float
        lib.seq_conv_plan.argtypes = [q, q, q, i, i, i, ctypes.POINTER(vp)]
        lib.seq_scan_plan.argtypes = [q, q, q, i, i, i, ctypes.POINTER(vp)]
        lib.seq_norm_plan.argtypes = [q, q, i, i, i, f, ctypes.POINTER(vp)]
        for name in ("seq_conv", "seq_scan", "seq_norm"):
            getattr(lib, name + "_plan").restype = i
            getattr(lib, name + "_destroy").argtypes = [vp]
            getattr(lib, name + "_destroy").restype = None
            getattr(lib, name + "_workspace_bytes").argtypes = [vp, i]
            getattr(lib, name + "_workspace_bytes").restype = ctypes.c_size_t
            if name != "seq_norm":
                getattr(lib, name + "_check").argtypes = [vp]
                getattr(lib, name + "_check").restype = i
        loader = importlib.machinery.ExtensionFileLoader("_seq_bind", _build.BIND)
        spec = importlib.util.spec_from_file_location("_seq_bind", _build.BIND, loader=loader)
        bind = importlib.util.module_from_spec(spec)
        loader.exec_module(bind)
        bind.set_error(DgradError)
        _LIB, _BIND = lib, bind
    return _LIB


class _SeqPlan:
    """What the three plans share: the handle, and calls on an explicit stream."""

    _kind = ""

    def _open(self, *args, dtype, residual=None, batch, length, channels, inner, groups, gated=False):
        import torch
        self._torch = torch
        self._lib = _library()
        self._h = ctypes.c_void_p()
        self.dtype = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}[dtype]

        def make():
            st = getattr(self._lib, f"seq_{self._kind}_plan")(*args, ctypes.byref(self._h))
            if st != 0:
                raise DgradError(st, f"seq_{self._kind}_plan")

        self._with_room(make)
        self.device = torch.cuda.current_device()
        self._c = _BIND.open_plan(self._h.value, self.device, DTYPE[dtype], DTYPE[residual or dtype], batch, length,
                                  channels, inner, groups, gated)

    def _alive(self):
        if not self._h:
            raise ValueError("the plan is closed")

    def _with_room(self, call, *args):
        """The call; where the plan's workspace found no memory, once more after PyTorch has given back what it holds
        unused."""
        try:
            return call(*args)
        except DgradError as e:
            if e.status != OUT_OF_MEMORY:
                raise
        self._torch.cuda.empty_cache()
        return call(*args)

    def _backward(self, call, args, stream):
        if stream is not None:
            return self._with_room(self._on, stream, call, *args)
        return self._with_room(call, self._c, *args)

    def workspace_bytes(self, gradients=True):
        """Device memory that the plan holds for itself, without or with backward calls."""
        self._alive()
        return getattr(self._lib, f"seq_{self._kind}_workspace_bytes")(self._h, int(bool(gradients)))

    def _on(self, stream, call, *args):
        """The call on an explicit stream, which is told which tensors it uses."""
        torch = self._torch
        for t in args:
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)
        with torch.cuda.stream(stream):
            return call(self._c, *args)

    def check(self):
        """Raise if a kernel of this plan recorded an error (call after synchronising)."""
        self._alive()
        st = getattr(self._lib, f"seq_{self._kind}_check")(self._h)
        if st != 0:
            raise DgradError(st, f"seq_{self._kind}_check")

    def close(self):
        if getattr(self, "_h", None):
            getattr(self._lib, f"seq_{self._kind}_destroy")(self._h)
            self._h = ctypes.c_void_p()
            self._c = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class CausalConvPlan(_SeqPlan):
    """The short causal depthwise convolution, bound to the current CUDA device.

    CausalConvPlan(batch, length, channels, width, dtype="bf16" | "fp16" | "fp32", activation="silu" | "none")

    run(x, weight, bias=None, lengths=None, state=None, out=None, final_state=None) -> y
        x, y [batch, length, channels]; weight [channels, width] and bias [channels] fp32; lengths [batch] int32;
        state, final_state [batch, width - 1, channels]: the inputs before the first token, and the last ones.
    backward(grad_out, x, weight, ..., grad_final_state=None) -> ConvGrads(x, weight, bias, state)
    step(x, weight, cache, bias=None, slots=None, write_slots=None, out=None) -> y [batch, channels]
        cache [n_slots, width - 1, channels]; row i reads slot slots[i] (negative: padding) and writes
        write_slots[i] (default: the slot it read).
    """

    _kind = "conv"

    def __init__(self, batch, length, channels, width, dtype="bf16", activation="silu"):
        if dtype not in DTYPE or activation not in ("none", "silu"):
            raise ValueError(f"unknown dtype {dtype!r} or activation {activation!r}")
        self.batch, self.length, self.channels, self.width = batch, length, channels, width
        self._open(batch, length, channels, width, DTYPE[dtype], ACT[activation], dtype=dtype, batch=batch,
                   length=length, channels=channels, inner=width, groups=1)

    def run(self, x, weight, bias=None, lengths=None, state=None, out=None, final_state=None, stream=None):
        if stream is not None:
            return self._on(stream, _BIND.conv_run, x, weight, bias, lengths, state, out, final_state)
        return _BIND.conv_run(self._c, x, weight, bias, lengths, state, out, final_state)

    def backward(self, grad_out, x, weight, bias=None, lengths=None, state=None, grad_final_state=None, grad_x=None,
                 stream=None):
        args = (grad_out, x, weight, bias, lengths, state, grad_final_state, grad_x)
        return ConvGrads._make(self._backward(_BIND.conv_backward, args, stream))

    def step(self, x, weight, cache, bias=None, slots=None, write_slots=None, out=None, stream=None):
        if stream is not None:
            return self._on(stream, _BIND.conv_step, x, weight, cache, bias, slots, write_slots, out)
        return _BIND.conv_step(self._c, x, weight, cache, bias, slots, write_slots, out)


class ScanPlan(_SeqPlan):
    """The selective state-space scan, bound to the current CUDA device.

    ScanPlan(batch, length, channels, states, groups=1, dtype="bf16" | "fp16" | "fp32")

    run(u, dt, A, B, C, D=None, z=None, dt_bias=None, lengths=None, state=None, out=None, final_state=None,
        checkpoints=None) -> out
        u, dt, z, out [batch, length, channels]; B, C [batch, length, groups, states]; A [channels, states], D,
        dt_bias [channels] fp32; lengths [batch] int32; state, final_state [batch, channels, states] fp32;
        checkpoints from checkpoints(): filled for backward.
    backward(grad_out, u, dt, A, B, C, checkpoints, ..., grad_final_state=None, grad_u=None, grad_z=None)
        -> ScanGrads(u, dt, A, B, C, D, z, dt_bias, state)
    step(u, dt, A, B, C, cache, D=None, z=None, dt_bias=None, slots=None, write_slots=None, out=None) -> out
        one token: u, dt, z [batch, channels]; B, C [batch, groups, states]; cache [n_slots, channels, states] fp32,
        slots as in CausalConvPlan.step.
    """

    _kind = "scan"

    def __init__(self, batch, length, channels, states, groups=1, dtype="bf16"):
        if dtype not in DTYPE:
            raise ValueError(f"unknown dtype {dtype!r}")
        self.batch, self.length, self.channels = batch, length, channels
        self.states, self.groups = states, groups
        self._open(batch, length, channels, states, groups, DTYPE[dtype], dtype=dtype, batch=batch, length=length,
                   channels=channels, inner=states, groups=groups)

    def checkpoints(self, batch=None, length=None):
        """A buffer for run and backward: the states at every 8th token of a batch (default: the plan's)."""
        return _BIND.scan_checkpoints(self._c, batch, length)

    def run(self, u, dt, A, B, C, D=None, z=None, dt_bias=None, lengths=None, state=None, out=None,
            final_state=None, checkpoints=None, stream=None):
        args = (u, dt, A, B, C, D, z, dt_bias, lengths, state, out, final_state, checkpoints)
        if stream is not None:
            return self._on(stream, _BIND.scan_run, *args)
        return _BIND.scan_run(self._c, *args)

    def backward(self, grad_out, u, dt, A, B, C, checkpoints, D=None, z=None, dt_bias=None, lengths=None, state=None,
                 grad_final_state=None, grad_u=None, grad_z=None, stream=None):
        args = (grad_out, u, dt, A, B, C, checkpoints, D, z, dt_bias, lengths, state, grad_final_state, grad_u, grad_z)
        return ScanGrads._make(self._backward(_BIND.scan_backward, args, stream))

    def step(self, u, dt, A, B, C, cache, D=None, z=None, dt_bias=None, slots=None, write_slots=None, out=None,
             stream=None):
        args = (u, dt, A, B, C, cache, D, z, dt_bias, slots, write_slots, out)
        if stream is not None:
            return self._on(stream, _BIND.scan_step, *args)
        return _BIND.scan_step(self._c, *args)


class BlockNormPlan(_SeqPlan):
    """The norms around a block, bound to the current CUDA device.

    BlockNormPlan(rows, channels, dtype="bf16" | "fp16" | "fp32", residual_dtype=None (dtype) | "fp32",
                  gate="none" | "silu" | "sigmoid", eps=1e-5)

    run(y, residual, next_weight, post_weight=None, gate=None, scale=None, residual_out=None, out=None)
        -> (residual_out, out)
        residual_out = residual + scale * act(gate) * norm(y) * post_weight   (post_weight None: y itself)
        out = norm(residual_out) * next_weight
        y, gate, residual, out [rows, channels]; weights and scale [channels] fp32.
    backward(grad_residual_out, grad_out, y, residual, next_weight, ...) -> NormGrads(y, gate, residual,
        post_weight, scale, next_weight); grad_residual_out None: zeros.
    """

    _kind = "norm"

    def __init__(self, rows, channels, dtype="bf16", residual_dtype=None, gate="none", eps=1e-5):
        if dtype not in DTYPE or gate not in ACT or (residual_dtype or dtype) not in DTYPE:
            raise ValueError(f"unknown dtype {dtype!r}, residual_dtype {residual_dtype!r} or gate {gate!r}")
        self.rows, self.channels, self.gated = rows, channels, gate != "none"
        self._open(rows, channels, DTYPE[dtype], DTYPE[residual_dtype or dtype], ACT[gate], eps, dtype=dtype,
                   residual=residual_dtype, batch=rows, length=1, channels=channels, inner=1, groups=1,
                   gated=self.gated)

    def check(self):
        """The block norm's kernels have nothing to record."""

    def run(self, y, residual, next_weight, post_weight=None, gate=None, scale=None, residual_out=None, out=None,
            stream=None):
        args = (y, residual, next_weight, post_weight, gate, scale, residual_out, out)
        if stream is not None:
            return self._on(stream, _BIND.norm_run, *args)
        return _BIND.norm_run(self._c, *args)

    def backward(self, grad_residual_out, grad_out, y, residual, next_weight, post_weight=None, gate=None, scale=None,
                 grad_y=None, grad_gate=None, grad_residual=None, stream=None):
        args = (grad_residual_out, grad_out, y, residual, next_weight, post_weight, gate, scale, grad_y, grad_gate,
                grad_residual)
        return NormGrads._make(self._backward(_BIND.norm_backward, args, stream))
