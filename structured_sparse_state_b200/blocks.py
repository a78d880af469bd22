"""Binding of the operators around the PD-SSM scan in a pre-norm block: the
decay scan (linear attention with a decay for each head) and its single step,
the root-mean-square norm with the residual's addition, and the balance loss
of the hard selection.  As in the package's other entry points, a function
here checks and marshals tensors into the C ABI of ``include/pdssm.h``, where
the formulas, layouts and limits stand; the kernels do the arithmetic.

Every tensor of a call lies on one CUDA device, which need not be the current
one; work goes to that device's current stream, or to ``stream``.
"""
from __future__ import annotations

import ctypes
from contextlib import contextmanager, nullcontext

import torch

from . import (PDSSM_BF16, PDSSM_E4M3, PDSSM_F32, DecayDims, PdssmError, _check, _lib, _ptr, dims)

_FLOATS = (torch.float32, torch.bfloat16)
_CODE = {torch.float32: PDSSM_F32, torch.bfloat16: PDSSM_BF16, torch.float8_e4m3fn: PDSSM_E4M3}
LAYOUTS = {"bhl": 0, "blh": 1}


# ----------------------------------------------------------------------------
# checks
# ----------------------------------------------------------------------------
def _arg(t, name, dtypes, shape=None, device=None):
    """A contiguous CUDA tensor of one of `dtypes`, of `shape`, on `device`."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _opt(t, name, dtypes, shape, device):
    return None if t is None else _arg(t, name, dtypes, shape, device)


@contextmanager
def _enter(device, stream):
    with torch.cuda.device(device):
        with torch.cuda.stream(stream) if stream is not None else nullcontext():
            yield


_HERE = nullcontext()


def _on(device, stream):
    """The call's device and stream, for its allocations and its launches."""
    if stream is None and device.index == torch.cuda.current_device():
        return _HERE
    if stream is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, expected {device}")
    return _enter(device, stream)


def _cur() -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _out(t, name, dtype, shape, device):
    """A caller's output buffer, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _arg(t, name, (dtype,), shape, device)


# ----------------------------------------------------------------------------
# decay scan
# ----------------------------------------------------------------------------
def _decay_shapes(c, b, x, log_a, layout):
    """(dims, per_step) of a scan's inputs."""
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be one of {tuple(LAYOUTS)}")
    _arg(x, "x", _FLOATS)
    dev = x.device
    if x.dim() != 4:
        raise ValueError("x must have four dimensions")
    if layout == "bhl":
        B, H, L, P = x.shape
    else:
        B, L, H, P = x.shape
    _arg(c, "c", (x.dtype,), None, dev)
    if c.dim() != 4:
        raise ValueError("c must have four dimensions")
    G, N = (c.shape[1] if layout == "bhl" else c.shape[2]), c.shape[3]
    keys = (B, G, L, N) if layout == "bhl" else (B, L, G, N)
    _arg(c, "c", (x.dtype,), keys, dev)
    _arg(b, "b", (x.dtype,), keys, dev)
    if G == 0 or H % G:
        raise ValueError(f"{H} heads cannot share {G} groups of c and b")
    _arg(log_a, "log_a", (torch.float32,), None, dev)
    per_step = log_a.dim() != 1
    _arg(log_a, "log_a", (torch.float32,),
         ((B, H, L) if layout == "bhl" else (B, L, H)) if per_step else (H,), dev)
    return DecayDims(B, H, G, L, N, P), per_step


def pdssm_decay_workspace_bytes(B, H, G, L, N, P, dtype=torch.float32, for_bwd=False) -> int:
    n = _lib.pdssm_decay_workspace_bytes(ctypes.byref(DecayDims(B, H, G, L, N, P)),
                                         _CODE[dtype], int(bool(for_bwd)))
    if n == 0:
        raise PdssmError(1, "pdssm_decay_workspace_bytes")
    return int(n)


def _decay_ws(dm, dtype, for_bwd):
    n = _lib.pdssm_decay_workspace_bytes(ctypes.byref(dm), _CODE[dtype], int(for_bwd))
    if n == 0:      # sizes outside the limits: let the call itself say which
        n = 256
    return n


def pdssm_decay_scan_fwd(c, b, x, log_a, h0=None, lengths=None, layout="bhl", for_bwd=False,
                         ws=None, y=None, h_last=None, stream=None):
    """Linear attention with a decay for each head, over whole sequences:
    S_t = exp(log_a_t) S_{t-1} + b_t x_t^T, y_t = S_t^T c_t.

    c, b [B, G, L, N], x [B, H, L, P] (layout "bhl") or [B, L, G, N],
    [B, L, H, P] ("blh"), fp32 or bf16, H a multiple of G; log_a fp32 per step
    ([B, H, L] / [B, L, H]) or per head ([H]); h0 fp32 [B, H, N, P] or None;
    lengths int32 [B] or None.  Returns (y like x, h_last fp32 [B, H, N, P],
    ws); for_bwd=True makes ws serve pdssm_decay_scan_bwd."""
    dm, per_step = _decay_shapes(c, b, x, log_a, layout)
    dev = x.device
    state = (dm.B, dm.H, dm.N, dm.P)
    _opt(h0, "h0", (torch.float32,), state, dev)
    _opt(lengths, "lengths", (torch.int32,), (dm.B,), dev)
    with _on(dev, stream):
        if ws is None:
            ws = torch.empty(_decay_ws(dm, x.dtype, for_bwd), dtype=torch.uint8, device=dev)
        _arg(ws, "ws", (torch.uint8,), None, dev)
        y = _out(y, "y", x.dtype, x.shape, dev)
        h_last = _out(h_last, "h_last", torch.float32, state, dev)
        _check(_lib.pdssm_decay_scan_fwd(
            ctypes.byref(dm), _ptr(c), _ptr(b), _ptr(x), _CODE[x.dtype], LAYOUTS[layout],
            _ptr(log_a), int(per_step), _ptr(h0), _ptr(lengths), _ptr(y), _ptr(h_last),
            int(bool(for_bwd)), _ptr(ws), ws.numel(), _cur()), "pdssm_decay_scan_fwd")
    return y, h_last, ws


def pdssm_decay_scan_bwd(c, b, x, log_a, h0, g_y, ws, g_hlast=None, lengths=None, layout="bhl",
                         out=None, stream=None):
    """Exact adjoint of pdssm_decay_scan_fwd; ws is the forward's (made with
    for_bwd=True).  Returns (g_c, g_b, g_x, g_log_a, g_h0)."""
    dm, per_step = _decay_shapes(c, b, x, log_a, layout)
    dev = x.device
    state = (dm.B, dm.H, dm.N, dm.P)
    _opt(h0, "h0", (torch.float32,), state, dev)
    _opt(g_hlast, "g_hlast", (torch.float32,), state, dev)
    _opt(lengths, "lengths", (torch.int32,), (dm.B,), dev)
    _arg(g_y, "g_y", (x.dtype,), x.shape, dev)
    _arg(ws, "ws", (torch.uint8,), None, dev)
    with _on(dev, stream):
        g_c, g_b, g_x, g_la, g_h0 = out if out is not None else (None,) * 5
        g_c = _out(g_c, "g_c", x.dtype, c.shape, dev)
        g_b = _out(g_b, "g_b", x.dtype, c.shape, dev)
        g_x = _out(g_x, "g_x", x.dtype, x.shape, dev)
        g_la = _out(g_la, "g_log_a", torch.float32, log_a.shape, dev)
        g_h0 = _out(g_h0, "g_h0", torch.float32, state, dev)
        _check(_lib.pdssm_decay_scan_bwd(
            ctypes.byref(dm), _ptr(c), _ptr(b), _ptr(x), _CODE[x.dtype], LAYOUTS[layout],
            _ptr(log_a), int(per_step), _ptr(h0), _ptr(lengths), _ptr(g_y), _ptr(g_hlast),
            _ptr(g_c), _ptr(g_b), _ptr(g_x), _ptr(g_la), _ptr(g_h0), _ptr(ws), ws.numel(),
            _cur()), "pdssm_decay_scan_bwd")
    return g_c, g_b, g_x, g_la, g_h0


def pdssm_decay_step(c, b, x, log_a, state, slots=None, y=None, stream=None):
    """One step for single tokens: c, b [B, G, N], x [B, H, P], log_a [B, H]
    or [H]; state fp32 [slots, H, N, P] is updated in place, row r in slot
    slots[r] (int32 [B]; outside the pool: an empty row, y zero), or slot r.
    Returns y [B, H, P]."""
    _arg(x, "x", _FLOATS)
    dev = x.device
    if x.dim() != 3 or not isinstance(c, torch.Tensor) or c.dim() != 3:
        raise ValueError("x and c must have three dimensions")
    B, H, P = x.shape
    G, N = c.shape[1], c.shape[2]
    _arg(c, "c", (x.dtype,), (B, G, N), dev)
    _arg(b, "b", (x.dtype,), (B, G, N), dev)
    if G == 0 or H % G:
        raise ValueError(f"{H} heads cannot share {G} groups of c and b")
    _arg(log_a, "log_a", (torch.float32,), None, dev)
    per_step = log_a.dim() != 1
    _arg(log_a, "log_a", (torch.float32,), (B, H) if per_step else (H,), dev)
    _arg(state, "state", (torch.float32,), None, dev)
    n_slots = state.shape[0] if state.dim() == 4 else -1
    _arg(state, "state", (torch.float32,), (n_slots, H, N, P), dev)
    _opt(slots, "slots", (torch.int32,), (B,), dev)
    dm = DecayDims(B, H, G, 1, N, P)
    with _on(dev, stream):
        y = _out(y, "y", x.dtype, x.shape, dev)
        _check(_lib.pdssm_decay_step(
            ctypes.byref(dm), _ptr(c), _ptr(b), _ptr(x), _CODE[x.dtype], _ptr(log_a),
            int(per_step), _ptr(state), n_slots, _ptr(slots), _ptr(y), _cur()),
            "pdssm_decay_step")
    return y


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
    _arg(x, "x", _FLOATS)
    dev = x.device
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    D = x.shape[-1]
    lead = x.shape[:-1]
    _opt(residual, "residual", _FLOATS, x.shape, dev)
    _arg(weight, "weight", _FLOATS, (D,), dev)
    res_dtype = x.dtype if residual is None else residual.dtype
    out_dtype = x.dtype if out_dtype is None else out_dtype
    if out_dtype not in _CODE:
        raise ValueError(f"out_dtype {out_dtype}, expected one of {tuple(_CODE)}")
    rows = 1
    for n in lead:
        rows *= n
    with _on(dev, stream):
        out = _out(out, "out", out_dtype, x.shape, dev)
        res_out = _out(res_out, "res_out", res_dtype, x.shape, dev)
        rstd = _out(rstd, "rstd", torch.float32, lead, dev)
        if out_dtype == torch.float8_e4m3fn:
            scale = _out(scale, "scale", torch.float32, lead, dev)
        elif scale is not None:
            raise ValueError("scale goes with an 8-bit output only")
        _check(_lib.pdssm_add_rmsnorm_fwd(
            rows, D, _ptr(x), _CODE[x.dtype], _ptr(residual), _CODE[res_dtype], _ptr(weight),
            _CODE[weight.dtype], float(eps), _ptr(out), _CODE[out_dtype], _ptr(res_out),
            _ptr(rstd), _ptr(scale), _cur()), "pdssm_add_rmsnorm_fwd")
    return out, res_out, rstd, scale


def pdssm_add_rmsnorm_bwd(g_out, res_out, weight, rstd, g_res=None, g_x=None, g_weight=None,
                          scratch=None, stream=None):
    """Backward of pdssm_add_rmsnorm_fwd from its res_out and rstd: (g_x,
    g_weight fp32), g_x in res_out's type, the gradient of x and residual
    alike; g_res is the gradient that reaches res_out itself."""
    _arg(res_out, "res_out", _FLOATS)
    dev = res_out.device
    if res_out.dim() < 1:
        raise ValueError("res_out must have at least one dimension")
    D, lead = res_out.shape[-1], res_out.shape[:-1]
    _arg(g_out, "g_out", _FLOATS, res_out.shape, dev)
    _arg(weight, "weight", _FLOATS, (D,), dev)
    _arg(rstd, "rstd", (torch.float32,), lead, dev)
    _opt(g_res, "g_res", (res_out.dtype,), res_out.shape, dev)
    rows = rstd.numel()
    with _on(dev, stream):
        g_x = _out(g_x, "g_x", res_out.dtype, res_out.shape, dev)
        g_weight = _out(g_weight, "g_weight", torch.float32, (D,), dev)
        if scratch is None:
            n = int(_lib.pdssm_add_rmsnorm_scratch_bytes(rows, D)) or 256
            scratch = torch.empty(n, dtype=torch.uint8, device=dev)
        _arg(scratch, "scratch", (torch.uint8,), None, dev)
        _check(_lib.pdssm_add_rmsnorm_bwd(
            rows, D, _ptr(g_out), _CODE[g_out.dtype], _ptr(res_out), _CODE[res_out.dtype],
            _ptr(weight), _CODE[weight.dtype], _ptr(rstd), _ptr(g_res), _ptr(g_x),
            _ptr(g_weight), _ptr(scratch), scratch.numel(), _cur()), "pdssm_add_rmsnorm_bwd")
    return g_x, g_weight


# ----------------------------------------------------------------------------
# balance of the hard selection
# ----------------------------------------------------------------------------
def _balance_shapes(u, W_sel, lengths):
    _arg(u, "u", _FLOATS)
    dev = u.device
    if u.dim() != 3:
        raise ValueError("u must be [B, L, D_in]")
    B, L, D = u.shape
    _arg(W_sel, "W_sel", (torch.float32,), None, dev)
    if W_sel.dim() != 3 or W_sel.shape[2] != D:
        raise ValueError("W_sel must be [H, K, D_in]")
    _opt(lengths, "lengths", (torch.int32,), (B,), dev)
    return dims(B, W_sel.shape[0], L, 0, W_sel.shape[1], D), dev


def _balance_scratch(dm, scratch, dev):
    if scratch is None:
        n = int(_lib.pdssm_select_balance_scratch_bytes(ctypes.byref(dm))) or 256
        scratch = torch.empty(n, dtype=torch.uint8, device=dev)
    return _arg(scratch, "scratch", (torch.uint8,), None, dev)


def pdssm_select_balance_fwd(u, W_sel, k, inv_tau=1.0, lengths=None, scratch=None, stream=None):
    """Balance of a hard selection k [B, H, L] made from u [B, L, D_in] and
    W_sel [H, K, D_in]: loss[h] = K sum_j (counts[h, j] / T) probs[h, j] over
    the T steps (those in front of lengths [B], if given), with probs the mean
    of softmax(inv_tau W_sel u).  Returns (loss fp32 [H], counts int32 [H, K],
    probs fp32 [H, K])."""
    dm, dev = _balance_shapes(u, W_sel, lengths)
    _arg(k, "k", (torch.int32,), (dm.B, dm.H, dm.L), dev)
    with _on(dev, stream):
        loss = torch.empty((dm.H,), dtype=torch.float32, device=dev)
        counts = torch.empty((dm.H, dm.K), dtype=torch.int32, device=dev)
        probs = torch.empty((dm.H, dm.K), dtype=torch.float32, device=dev)
        scratch = _balance_scratch(dm, scratch, dev)
        _check(_lib.pdssm_select_balance_fwd(
            ctypes.byref(dm), _ptr(u), _CODE[u.dtype], _ptr(W_sel), _ptr(k), float(inv_tau),
            _ptr(lengths), _ptr(loss), _ptr(counts), _ptr(probs), _ptr(scratch), scratch.numel(),
            _cur()), "pdssm_select_balance_fwd")
    return loss, counts, probs


def pdssm_select_balance_bwd(u, W_sel, counts, g_loss, inv_tau=1.0, lengths=None, scratch=None,
                             stream=None):
    """Gradients of sum_h g_loss[h] loss[h] with the counts held fixed:
    (g_u like u, g_W like W_sel)."""
    dm, dev = _balance_shapes(u, W_sel, lengths)
    _arg(counts, "counts", (torch.int32,), (dm.H, dm.K), dev)
    _arg(g_loss, "g_loss", (torch.float32,), (dm.H,), dev)
    with _on(dev, stream):
        g_u, g_W = torch.empty_like(u), torch.empty_like(W_sel)
        scratch = _balance_scratch(dm, scratch, dev)
        _check(_lib.pdssm_select_balance_bwd(
            ctypes.byref(dm), _ptr(u), _CODE[u.dtype], _ptr(W_sel), _ptr(counts), float(inv_tau),
            _ptr(lengths), _ptr(g_loss), _ptr(g_u), _ptr(g_W), _ptr(scratch), scratch.numel(),
            _cur()), "pdssm_select_balance_bwd")
    return g_u, g_W
