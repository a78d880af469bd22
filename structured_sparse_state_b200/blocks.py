"""Binding of the operators around the PD-SSM scan in a pre-norm block: the
decay scan (linear attention with a decay for each head) and its single step,
the root-mean-square norm with the residual's addition, and the balance loss
of the hard selection.  As in the package's other entry points, a function
here checks and marshals tensors into the C ABI of ``include/pdssm.h``, where
the formulas, layouts and limits stand; the kernels do the arithmetic.  The
checks and allocations run natively (``csrc/blocks_py.cpp``): these calls are
short.

Every tensor of a call lies on one CUDA device, which need not be the current
one; work goes to that device's current stream, or to ``stream``, whose order
with the streams that made the inputs and read the results is the caller's to
keep (``stream.wait_stream``).  Inputs may be dropped after the call.  A wrong
argument raises ValueError, a status of the library PdssmError.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from contextlib import contextmanager

import torch

from . import (PDSSM_BF16, PDSSM_F32, DecayDims, PdssmError, _check, _lib, _ptr, _stream, lib,
               pdssm_ws_status)

BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_blocks.so")
LAYOUTS = {"bhl": False, "blh": True}


class _Native:
    """Loads _blocks.so on first use (the build step imports this package
    before it exists); any call without it raises."""

    def __getattr__(self, name):
        if not os.path.exists(BINDING_PATH):
            raise ImportError(
                f"{BINDING_PATH} is missing: build it with "
                "`python -m structured_sparse_state_b200.build` (there is no fallback)")
        lib()
        loader = importlib.machinery.ExtensionFileLoader(__package__ + "._blocks", BINDING_PATH)
        module = importlib.util.module_from_spec(
            importlib.util.spec_from_loader(loader.name, loader))
        loader.exec_module(module)
        for key, value in vars(module).items():
            if not key.startswith("_"):
                setattr(self, key, value)
        return getattr(module, name)


_native = _Native()


@contextmanager
def _enter(stream):
    with torch.cuda.device(stream.device), torch.cuda.stream(stream):
        yield


def _layout(layout):
    if layout not in tuple(LAYOUTS):
        raise ValueError(f"layout must be one of {tuple(LAYOUTS)}")
    return LAYOUTS[layout]


def _call(fn, x, stream, *args):
    """fn on the current stream of the tensors' device, or on `stream`: then
    what it allocates belongs to that stream, and what it was given is not
    handed out again before that stream is done with it."""
    if stream is None:
        return fn(*args)
    if isinstance(x, torch.Tensor) and x.is_cuda and stream.device != x.device:
        raise ValueError(f"stream is on {stream.device}, expected {x.device}")
    with _enter(stream):
        result = fn(*args)
    for t in args:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    return result


# ----------------------------------------------------------------------------
# decay scan
# ----------------------------------------------------------------------------
def pdssm_decay_workspace_bytes(B, H, G, L, N, P, dtype=torch.float32, for_bwd=False) -> int:
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"dtype {dtype}, expected float32 or bfloat16")
    code = PDSSM_BF16 if dtype == torch.bfloat16 else PDSSM_F32
    n = _lib.pdssm_decay_workspace_bytes(ctypes.byref(DecayDims(B, H, G, L, N, P)), code,
                                         int(bool(for_bwd)))
    if n == 0:
        raise PdssmError(1, "pdssm_decay_workspace_bytes")
    return int(n)


def pdssm_decay_scan_fwd(c, b, x, log_a, h0=None, lengths=None, layout="bhl", for_bwd=False,
                         ws=None, y=None, h_last=None, stream=None):
    """Linear attention with a decay for each head, over whole sequences:
    S_t = exp(log_a_t) S_{t-1} + b_t x_t^T, y_t = S_t^T c_t.

    c, b [B, G, L, N], x [B, H, L, P] (layout "bhl") or [B, L, G, N],
    [B, L, H, P] ("blh"), fp32 or bf16, H a multiple of G; log_a fp32 per step
    ([B, H, L] / [B, L, H]) or per head ([H]); h0 fp32 [B, H, N, P] or None;
    lengths int32 [B] or None.  Returns (y like x, h_last fp32 [B, H, N, P],
    ws); for_bwd=True makes ws serve pdssm_decay_scan_bwd."""
    return _call(_native.decay_scan_fwd, x, stream, c, b, x, log_a, h0, lengths, _layout(layout),
                 bool(for_bwd), ws, y, h_last)


def pdssm_decay_scan_bwd(c, b, x, log_a, h0, g_y, ws, g_hlast=None, lengths=None, layout="bhl",
                         out=None, stream=None):
    """Exact adjoint of pdssm_decay_scan_fwd; ws is the forward's (made with
    for_bwd=True).  Returns (g_c, g_b, g_x, g_log_a, g_h0)."""
    return _call(_native.decay_scan_bwd, x, stream, c, b, x, log_a, h0, g_y, ws, g_hlast, lengths,
                 _layout(layout), *(out if out is not None else (None,) * 5))


def pdssm_decay_wait_selftest(B, H, L, N, for_bwd=False):
    """The bf16 forward with its copies held back: its bounded waits give up
    after 2 s.  Returns (status of ws, y, h_last, ws): PDSSM_ERR_TIMEOUT (5)
    and NaN everywhere expected.  Synchronises."""
    dev = torch.device("cuda", torch.cuda.current_device())
    ws = torch.zeros(pdssm_decay_workspace_bytes(B, H, H, L, N, N, torch.bfloat16, for_bwd),
                     dtype=torch.uint8, device=dev)
    log_a = torch.zeros(B, H, L, device=dev)
    y = torch.zeros(B, H, L, N, dtype=torch.bfloat16, device=dev)
    h_last = torch.zeros(B, H, N, N, device=dev)
    _check(_lib.pdssm_decay_wait_selftest(ctypes.byref(DecayDims(B, H, H, L, N, N)), _ptr(log_a), _ptr(y),
                                          _ptr(h_last), int(bool(for_bwd)), _ptr(ws), ws.numel(), _stream(None)),
           "pdssm_decay_wait_selftest")
    return pdssm_ws_status(ws), y, h_last, ws


def pdssm_decay_step(c, b, x, log_a, state, slots=None, y=None, stream=None):
    """One step for single tokens: c, b [B, G, N], x [B, H, P], log_a [B, H]
    or [H]; state fp32 [slots, H, N, P] is updated in place, row r in slot
    slots[r] (int32 [B]; outside the pool: an empty row, y zero), or slot r.
    Returns y [B, H, P]."""
    return _call(_native.decay_step, x, stream, c, b, x, log_a, state, slots, y)


# ----------------------------------------------------------------------------
# residual addition and root-mean-square norm
# ----------------------------------------------------------------------------
def pdssm_add_rmsnorm_fwd(x, residual, weight, eps=1e-6, out_dtype=None, out=None, res_out=None,
                          rstd=None, scale=None, stream=None):
    """res_out = x + residual (rounded to residual's type; residual None: x),
    out = res_out * rstd * weight with rstd = 1 / sqrt(mean(res_out^2) + eps)
    over the last dimension.  x, residual [..., D] fp32 or bf16, weight [D];
    out_dtype fp32, bf16 or float8_e4m3fn (default x's), the last with one
    fp32 scale per row.  Returns (out, res_out, rstd, scale or None)."""
    return _call(_native.add_rmsnorm_fwd, x, stream, x, residual, weight, eps, out_dtype, out,
                 res_out, rstd, scale)


def pdssm_add_rmsnorm_bwd(g_out, res_out, weight, rstd, g_res=None, g_x=None, g_weight=None,
                          scratch=None, stream=None):
    """Backward of pdssm_add_rmsnorm_fwd from its res_out and rstd: (g_x,
    g_weight fp32), g_x in res_out's type, the gradient of x and residual
    alike; g_res is the gradient that reaches res_out itself."""
    return _call(_native.add_rmsnorm_bwd, res_out, stream, g_out, res_out, weight, rstd, g_res, g_x,
                 g_weight, scratch)


# ----------------------------------------------------------------------------
# balance of the hard selection
# ----------------------------------------------------------------------------
def pdssm_select_balance_fwd(u, W_sel, k, inv_tau=1.0, lengths=None, scratch=None, stream=None):
    """Balance of a hard selection k [B, H, L] made from u [B, L, D_in] and
    W_sel [H, K, D_in]: loss[h] = K sum_j (counts[h, j] / T) probs[h, j] over
    the T steps (those in front of lengths [B], if given), with probs the mean
    of softmax(inv_tau W_sel u).  Returns (loss fp32 [H], counts int32 [H, K],
    probs fp32 [H, K])."""
    return _call(_native.select_balance_fwd, u, stream, u, W_sel, k, inv_tau, lengths, scratch)


def pdssm_select_balance_bwd(u, W_sel, counts, g_loss, inv_tau=1.0, lengths=None, scratch=None,
                             stream=None):
    """Gradients of sum_h g_loss[h] loss[h] with the counts held fixed:
    (g_u like u, g_W like W_sel)."""
    return _call(_native.select_balance_bwd, u, stream, u, W_sel, counts, g_loss, inv_tau, lengths,
                 scratch)
