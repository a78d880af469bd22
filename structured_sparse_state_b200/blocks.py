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

from . import (PDSSM_BF16, PDSSM_E4M3, PDSSM_F32, DecayDims, Dims, PdssmError, _check, _lib)

_FLOATS = (torch.float32, torch.bfloat16)
_F32 = (torch.float32,)
_I32 = (torch.int32,)
_U8 = (torch.uint8,)
_CODE = {torch.float32: PDSSM_F32, torch.bfloat16: PDSSM_BF16, torch.float8_e4m3fn: PDSSM_E4M3}
LAYOUTS = {"bhl": 0, "blh": 1}

_current_device = torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream
_ref = ctypes.byref
_fns = {}


# ----------------------------------------------------------------------------
# checks (these calls are short: a decoded token's step runs for microseconds,
# so the host's part is kept lean)
# ----------------------------------------------------------------------------
def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = _fns[name] = getattr(_lib, name)
    return f


def _arg(t, name, dtypes, shape=None, index=None):
    """The device pointer of a contiguous CUDA tensor of one of `dtypes`, of
    `shape`, on device `index`."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path)")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    return t.data_ptr()


def _opt(t, name, dtypes, shape, index):
    return None if t is None else _arg(t, name, dtypes, shape, index)


@contextmanager
def _enter(index, stream):
    with torch.cuda.device(index):
        with torch.cuda.stream(stream) if stream is not None else nullcontext():
            yield


_HERE = nullcontext()


def _on(index, stream):
    """The call's device and stream, for its allocations and its launches."""
    if stream is None:
        return _HERE if index == _current_device() else _enter(index, None)
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, expected cuda:{index}")
    return _enter(index, stream)


def _out(t, name, dtype, shape, like, index):
    """A caller's output buffer, checked, or a new one; and its pointer."""
    if t is None:
        t = (torch.empty_like(like, dtype=dtype) if shape == like.shape
             else like.new_empty(shape, dtype=dtype))
        return t, t.data_ptr()
    return t, _arg(t, name, (dtype,), shape, index)


def _room(t, name, nbytes, like, index):
    """A caller's workspace or a new one: (tensor, pointer, bytes)."""
    if t is None:
        t = like.new_empty(nbytes, dtype=torch.uint8)
        return t, t.data_ptr(), nbytes
    return t, _arg(t, name, _U8, None, index), t.numel()


# ----------------------------------------------------------------------------
# decay scan
# ----------------------------------------------------------------------------
def _decay_shapes(c, b, x, log_a, layout):
    """(dims, per_step, device index, pointers of c, b, x, log_a)."""
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be one of {tuple(LAYOUTS)}")
    px = _arg(x, "x", _FLOATS)
    at = x.get_device()
    if x.dim() != 4 or not isinstance(c, torch.Tensor) or c.dim() != 4:
        raise ValueError("x and c must have four dimensions")
    if layout == "bhl":
        B, H, L, P = x.shape
        G, N = c.shape[1], c.shape[3]
        keys, gate = (B, G, L, N), (B, H, L)
    else:
        B, L, H, P = x.shape
        G, N = c.shape[2], c.shape[3]
        keys, gate = (B, L, G, N), (B, L, H)
    own = (x.dtype,)
    pc = _arg(c, "c", own, keys, at)
    pb = _arg(b, "b", own, keys, at)
    if G == 0 or H % G:
        raise ValueError(f"{H} heads cannot share {G} groups of c and b")
    per_step = not isinstance(log_a, torch.Tensor) or log_a.dim() != 1
    pla = _arg(log_a, "log_a", _F32, gate if per_step else (H,), at)
    return DecayDims(B, H, G, L, N, P), per_step, at, pc, pb, px, pla


def pdssm_decay_workspace_bytes(B, H, G, L, N, P, dtype=torch.float32, for_bwd=False) -> int:
    n = _fn("pdssm_decay_workspace_bytes")(_ref(DecayDims(B, H, G, L, N, P)), _CODE[dtype],
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
    dm, per_step, at, pc, pb, px, pla = _decay_shapes(c, b, x, log_a, layout)
    code, state, bwd = _CODE[x.dtype], (dm.B, dm.H, dm.N, dm.P), int(bool(for_bwd))
    ph0 = _opt(h0, "h0", _F32, state, at)
    pn = _opt(lengths, "lengths", _I32, (dm.B,), at)
    with _on(at, stream):
        # sizes outside the limits need 0 bytes: the call itself then says which
        n = _fn("pdssm_decay_workspace_bytes")(_ref(dm), code, bwd) if ws is None else 0
        ws, pws, n = _room(ws, "ws", n or 256, x, at)
        y, py = _out(y, "y", x.dtype, x.shape, x, at)
        h_last, ph = _out(h_last, "h_last", torch.float32, state, x, at)
        _check(_fn("pdssm_decay_scan_fwd")(
            _ref(dm), pc, pb, px, code, LAYOUTS[layout], pla, int(per_step), ph0, pn, py, ph, bwd,
            pws, n, _raw_stream(at)), "pdssm_decay_scan_fwd")
    return y, h_last, ws


def pdssm_decay_scan_bwd(c, b, x, log_a, h0, g_y, ws, g_hlast=None, lengths=None, layout="bhl",
                         out=None, stream=None):
    """Exact adjoint of pdssm_decay_scan_fwd; ws is the forward's (made with
    for_bwd=True).  Returns (g_c, g_b, g_x, g_log_a, g_h0)."""
    dm, per_step, at, pc, pb, px, pla = _decay_shapes(c, b, x, log_a, layout)
    state, own = (dm.B, dm.H, dm.N, dm.P), x.dtype
    ph0 = _opt(h0, "h0", _F32, state, at)
    pgh = _opt(g_hlast, "g_hlast", _F32, state, at)
    pn = _opt(lengths, "lengths", _I32, (dm.B,), at)
    pgy = _arg(g_y, "g_y", (own,), x.shape, at)
    pws = _arg(ws, "ws", _U8, None, at)
    with _on(at, stream):
        g_c, g_b, g_x, g_la, g_h0 = out if out is not None else (None,) * 5
        g_c, p1 = _out(g_c, "g_c", own, c.shape, x, at)
        g_b, p2 = _out(g_b, "g_b", own, c.shape, x, at)
        g_x, p3 = _out(g_x, "g_x", own, x.shape, x, at)
        g_la, p4 = _out(g_la, "g_log_a", torch.float32, log_a.shape, x, at)
        g_h0, p5 = _out(g_h0, "g_h0", torch.float32, state, x, at)
        _check(_fn("pdssm_decay_scan_bwd")(
            _ref(dm), pc, pb, px, _CODE[own], LAYOUTS[layout], pla, int(per_step), ph0, pn, pgy,
            pgh, p1, p2, p3, p4, p5, pws, ws.numel(), _raw_stream(at)), "pdssm_decay_scan_bwd")
    return g_c, g_b, g_x, g_la, g_h0


def pdssm_decay_step(c, b, x, log_a, state, slots=None, y=None, stream=None):
    """One step for single tokens: c, b [B, G, N], x [B, H, P], log_a [B, H]
    or [H]; state fp32 [slots, H, N, P] is updated in place, row r in slot
    slots[r] (int32 [B]; outside the pool: an empty row, y zero), or slot r.
    Returns y [B, H, P]."""
    px = _arg(x, "x", _FLOATS)
    at = x.get_device()
    if x.dim() != 3 or not isinstance(c, torch.Tensor) or c.dim() != 3:
        raise ValueError("x and c must have three dimensions")
    B, H, P = x.shape
    G, N = c.shape[1], c.shape[2]
    own, keys = (x.dtype,), (B, G, N)
    pc = _arg(c, "c", own, keys, at)
    pb = _arg(b, "b", own, keys, at)
    if G == 0 or H % G:
        raise ValueError(f"{H} heads cannot share {G} groups of c and b")
    per_step = not isinstance(log_a, torch.Tensor) or log_a.dim() != 1
    pla = _arg(log_a, "log_a", _F32, (B, H) if per_step else (H,), at)
    ps = _arg(state, "state", _F32, None, at)
    n_slots = state.shape[0] if state.dim() else 0
    if state.shape != (n_slots, H, N, P):
        raise ValueError(f"state has shape {tuple(state.shape)}, expected (slots, {H}, {N}, {P})")
    pslots = _opt(slots, "slots", _I32, (B,), at)
    with _on(at, stream):
        y, py = _out(y, "y", x.dtype, x.shape, x, at)
        _check(_fn("pdssm_decay_step")(
            _ref(DecayDims(B, H, G, 1, N, P)), pc, pb, px, _CODE[x.dtype], pla, int(per_step), ps,
            n_slots, pslots, py, _raw_stream(at)), "pdssm_decay_step")
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
    px = _arg(x, "x", _FLOATS)
    at, shape = x.get_device(), x.shape
    if not shape:
        raise ValueError("x must have at least one dimension")
    D, lead = shape[-1], shape[:-1]
    pr = _opt(residual, "residual", _FLOATS, shape, at)
    pw = _arg(weight, "weight", _FLOATS, (D,), at)
    res_dtype = x.dtype if residual is None else residual.dtype
    out_dtype = x.dtype if out_dtype is None else out_dtype
    if out_dtype not in _CODE:
        raise ValueError(f"out_dtype {out_dtype}, expected one of {tuple(_CODE)}")
    with _on(at, stream):
        out, po = _out(out, "out", out_dtype, shape, x, at)
        res_out, ps = _out(res_out, "res_out", res_dtype, shape, x, at)
        rstd, pd = _out(rstd, "rstd", torch.float32, lead, x, at)
        pc = None
        if out_dtype == torch.float8_e4m3fn:
            scale, pc = _out(scale, "scale", torch.float32, lead, x, at)
        elif scale is not None:
            raise ValueError("scale goes with an 8-bit output only")
        _check(_fn("pdssm_add_rmsnorm_fwd")(
            rstd.numel(), D, px, _CODE[x.dtype], pr, _CODE[res_dtype], pw, _CODE[weight.dtype],
            eps, po, _CODE[out_dtype], ps, pd, pc, _raw_stream(at)), "pdssm_add_rmsnorm_fwd")
    return out, res_out, rstd, scale


def pdssm_add_rmsnorm_bwd(g_out, res_out, weight, rstd, g_res=None, g_x=None, g_weight=None,
                          scratch=None, stream=None):
    """Backward of pdssm_add_rmsnorm_fwd from its res_out and rstd: (g_x,
    g_weight fp32), g_x in res_out's type, the gradient of x and residual
    alike; g_res is the gradient that reaches res_out itself."""
    ps = _arg(res_out, "res_out", _FLOATS)
    at, shape, own = res_out.get_device(), res_out.shape, res_out.dtype
    if not shape:
        raise ValueError("res_out must have at least one dimension")
    D, lead = shape[-1], shape[:-1]
    pg = _arg(g_out, "g_out", _FLOATS, shape, at)
    pw = _arg(weight, "weight", _FLOATS, (D,), at)
    pd = _arg(rstd, "rstd", _F32, lead, at)
    pr = _opt(g_res, "g_res", (own,), shape, at)
    rows = rstd.numel()
    with _on(at, stream):
        g_x, px = _out(g_x, "g_x", own, shape, res_out, at)
        g_weight, pgw = _out(g_weight, "g_weight", torch.float32, (D,), res_out, at)
        n = _fn("pdssm_add_rmsnorm_scratch_bytes")(rows, D) if scratch is None else 0
        scratch, pc, n = _room(scratch, "scratch", n or 256, res_out, at)
        _check(_fn("pdssm_add_rmsnorm_bwd")(
            rows, D, pg, _CODE[g_out.dtype], ps, _CODE[own], pw, _CODE[weight.dtype], pd, pr, px,
            pgw, pc, n, _raw_stream(at)), "pdssm_add_rmsnorm_bwd")
    return g_x, g_weight


# ----------------------------------------------------------------------------
# balance of the hard selection
# ----------------------------------------------------------------------------
def _balance_shapes(u, W_sel, lengths):
    """(dims, device index, pointers of u, W_sel, lengths)."""
    pu = _arg(u, "u", _FLOATS)
    at = u.get_device()
    if u.dim() != 3:
        raise ValueError("u must be [B, L, D_in]")
    B, L, D = u.shape
    pw = _arg(W_sel, "W_sel", _F32, None, at)
    if W_sel.dim() != 3 or W_sel.shape[2] != D:
        raise ValueError("W_sel must be [H, K, D_in]")
    pn = _opt(lengths, "lengths", _I32, (B,), at)
    H, K, _ = W_sel.shape
    return Dims(B, H, L, 0, K, D), at, pu, pw, pn


def pdssm_select_balance_fwd(u, W_sel, k, inv_tau=1.0, lengths=None, scratch=None, stream=None):
    """Balance of a hard selection k [B, H, L] made from u [B, L, D_in] and
    W_sel [H, K, D_in]: loss[h] = K sum_j (counts[h, j] / T) probs[h, j] over
    the T steps (those in front of lengths [B], if given), with probs the mean
    of softmax(inv_tau W_sel u).  Returns (loss fp32 [H], counts int32 [H, K],
    probs fp32 [H, K])."""
    dm, at, pu, pw, pn = _balance_shapes(u, W_sel, lengths)
    H, K = dm.H, dm.K
    pk = _arg(k, "k", _I32, (dm.B, H, dm.L), at)
    with _on(at, stream):
        loss = u.new_empty((H,), dtype=torch.float32)
        counts = u.new_empty((H, K), dtype=torch.int32)
        probs = u.new_empty((H, K), dtype=torch.float32)
        n = _fn("pdssm_select_balance_scratch_bytes")(_ref(dm)) if scratch is None else 0
        scratch, pc, n = _room(scratch, "scratch", n or 256, u, at)
        _check(_fn("pdssm_select_balance_fwd")(
            _ref(dm), pu, _CODE[u.dtype], pw, pk, inv_tau, pn, loss.data_ptr(), counts.data_ptr(),
            probs.data_ptr(), pc, n, _raw_stream(at)), "pdssm_select_balance_fwd")
    return loss, counts, probs


def pdssm_select_balance_bwd(u, W_sel, counts, g_loss, inv_tau=1.0, lengths=None, scratch=None,
                             stream=None):
    """Gradients of sum_h g_loss[h] loss[h] with the counts held fixed:
    (g_u like u, g_W like W_sel)."""
    dm, at, pu, pw, pn = _balance_shapes(u, W_sel, lengths)
    pk = _arg(counts, "counts", _I32, (dm.H, dm.K), at)
    pg = _arg(g_loss, "g_loss", _F32, (dm.H,), at)
    with _on(at, stream):
        g_u, g_W = torch.empty_like(u), torch.empty_like(W_sel)
        n = _fn("pdssm_select_balance_scratch_bytes")(_ref(dm)) if scratch is None else 0
        scratch, pc, n = _room(scratch, "scratch", n or 256, u, at)
        _check(_fn("pdssm_select_balance_bwd")(
            _ref(dm), pu, _CODE[u.dtype], pw, pk, inv_tau, pn, pg, g_u.data_ptr(), g_W.data_ptr(),
            pc, n, _raw_stream(at)), "pdssm_select_balance_bwd")
    return g_u, g_W
