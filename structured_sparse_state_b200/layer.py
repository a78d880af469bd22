"""Multi-head Flash PD-SSM layer over the C ABI.

Flash PD-SSM technical summary, Methodology §4: the SSM sits in a standard
pre-norm architecture as a multi-head layer, and the heads share the dense
dictionary matrices (which amortises their parameters); §1: the dictionary
is the column hardmax of those matrices and each step selects one entry by
the argmax of K linear scores; §2: the backward replaces the discrete
choices by tempered softmaxes (straight-through).

``PDSSMFunction`` is the differentiable core, every step in the library's
kernels: the dictionary (pdssm_dict_hardmax), the selection (pdssm_select),
the single-pass forward (pdssm_scan_fwd), the exact adjoint for d, b, c and
h0 (pdssm_scan_bwd) and the surrogate gradients for W_sel and the dictionary
matrices (pdssm_surrogate_bwd).  The one product outside the library is the
gradient with respect to u, g_u = g_logits . W_sel, a plain GEMM.

``PDSSMLayer`` wraps it in a pre-norm residual block with its projections
(RMS norm, linear maps for u, d, b, c and the output), which are ordinary
library operations.

The operators around the scan have differentiable forms here too:
``add_rmsnorm`` (residual addition and norm in one pass), ``decay_scan``
(linear attention with a decay for each head) and ``select_balance`` (the
balance loss of the hard selection).  ``DecayLayer`` is the decay scan's
pre-norm block, with its single step for served tokens, and ``ResidualStack``
chains blocks of both kinds over one residual stream, each block's addition
fused into the next one's norm.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (pdssm_add_rmsnorm_bwd, pdssm_add_rmsnorm_fwd, pdssm_decay_scan_bwd,
               pdssm_decay_scan_fwd, pdssm_decay_step, pdssm_dict_hardmax, pdssm_scan_bwd,
               pdssm_scan_fwd, pdssm_select, pdssm_select_balance_bwd, pdssm_select_balance_fwd,
               pdssm_surrogate_bwd)


class PDSSMFunction(torch.autograd.Function):
    """(u, W_sel, A, d, b, c, h0) -> (y, h_last) of the hard model."""

    @staticmethod
    def forward(ctx, u, W_sel, A, d, b, c, h0, chunk, inv_tau_s, inv_tau_a, k=None):
        pi = pdssm_dict_hardmax(A)
        if k is None:
            k = pdssm_select(u, W_sel)
        y, h_last, ws = pdssm_scan_fwd(pi, k, d, b, c, h0, chunk=chunk, for_bwd=True)
        ctx.save_for_backward(u, W_sel, A, d, b, c, h0, pi, k, ws)
        ctx.chunk, ctx.inv_tau_s, ctx.inv_tau_a = chunk, inv_tau_s, inv_tau_a
        return y, h_last

    @staticmethod
    def backward(ctx, g_y, g_hlast):
        u, W_sel, A, d, b, c, h0, pi, k, ws = ctx.saved_tensors
        g_y = torch.zeros_like(k, dtype=torch.float32) if g_y is None else g_y.float().contiguous()
        g_hl = None if g_hlast is None else g_hlast.float().contiguous()
        g_b, g_d, g_c, g_h0 = pdssm_scan_bwd(pi, k, d, b, c, h0, g_y, ws, chunk=ctx.chunk,
                                             g_hlast=g_hl)
        g_l, g_W, g_A = pdssm_surrogate_bwd(u, W_sel, A, pi, k, d, b, h0, g_b, ws, ctx.chunk,
                                            ctx.inv_tau_s, ctx.inv_tau_a)
        # dl/du[b, t, :] = sum_{h, k} g_logits[b, h, t, k] W_sel[h, k, :]
        B, H, L, K = g_l.shape
        g_u = torch.matmul(g_l.permute(0, 2, 1, 3).reshape(B, L, H * K),
                           W_sel.reshape(H * K, -1))
        return (g_u.to(u.dtype), g_W, g_A, g_d.to(d.dtype), g_b.to(b.dtype), g_c.to(c.dtype),
                g_h0 if h0 is not None else None, None, None, None, None)


def pdssm(u, W_sel, A, d, b, c, h0=None, chunk=128, inv_tau_s=1.0, inv_tau_a=1.0, k=None):
    """Differentiable hard-selection PD-SSM: returns (y [B, H, L], h_last).
    k: the selection pdssm_select(u, W_sel), if the caller has it already."""
    return PDSSMFunction.apply(u, W_sel, A, d, b, c, h0, chunk, inv_tau_s, inv_tau_a, k)


class AddRMSNormFunction(torch.autograd.Function):
    """(x, residual, weight) -> (out, residual stream) of pdssm_add_rmsnorm_fwd."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps, out_dtype):
        if out_dtype not in (None, torch.float32, torch.bfloat16):
            raise ValueError(f"add_rmsnorm gives float32 or bfloat16, not {out_dtype}: 8-bit rows "
                             "come with their scales from pdssm_add_rmsnorm_fwd")
        out, res_out, rstd, _ = pdssm_add_rmsnorm_fwd(
            x.contiguous(), None if residual is None else residual.contiguous(), weight, eps,
            out_dtype)
        ctx.save_for_backward(res_out, weight, rstd)
        ctx.types = x.dtype, None if residual is None else residual.dtype
        ctx.set_materialize_grads(False)
        return out, res_out

    @staticmethod
    @once_differentiable
    def backward(ctx, g_out, g_res):
        res_out, weight, rstd = ctx.saved_tensors
        x_dtype, r_dtype = ctx.types
        if g_out is None:
            if g_res is None:
                return None, None, None, None, None
            return g_res.to(x_dtype), None if r_dtype is None else g_res, None, None, None
        g_res = None if g_res is None else g_res.contiguous()
        g_s, g_w = pdssm_add_rmsnorm_bwd(g_out.contiguous(), res_out, weight, rstd, g_res)
        return (g_s.to(x_dtype), None if r_dtype is None else g_s, g_w.to(weight.dtype), None,
                None)


def add_rmsnorm(x, residual, weight, eps=1e-6, out_dtype=None):
    """s = x + residual (residual None: s = x) and its root-mean-square norm:
    returns (norm(s) * weight in out_dtype, s in residual's type).  out_dtype is
    float32, bfloat16 or None (x's); ValueError otherwise.  x and residual may
    have any strides."""
    return AddRMSNormFunction.apply(x, residual, weight, eps, out_dtype)


class DecayScanFunction(torch.autograd.Function):
    """(c, b, x, log_a, h0) -> (y, h_last) of pdssm_decay_scan_fwd."""

    @staticmethod
    def forward(ctx, c, b, x, log_a, h0, lengths, layout):
        grads = any(ctx.needs_input_grad)
        y, h_last, ws = pdssm_decay_scan_fwd(c, b, x, log_a, h0, lengths=lengths, layout=layout,
                                             for_bwd=grads)
        if grads:
            ctx.save_for_backward(c, b, x, log_a, h0, lengths, ws)
        ctx.layout = layout
        ctx.set_materialize_grads(False)
        return y, h_last

    @staticmethod
    @once_differentiable
    def backward(ctx, g_y, g_hlast):
        c, b, x, log_a, h0, lengths, ws = ctx.saved_tensors
        if g_y is None and g_hlast is None:
            return None, None, None, None, None, None, None
        g_y = torch.zeros_like(x) if g_y is None else g_y.contiguous()
        g_hlast = None if g_hlast is None else g_hlast.contiguous()
        g_c, g_b, g_x, g_la, g_h0 = pdssm_decay_scan_bwd(
            c, b, x, log_a, h0, g_y, ws, g_hlast=g_hlast, lengths=lengths, layout=ctx.layout)
        return g_c, g_b, g_x, g_la, g_h0 if h0 is not None else None, None, None


def decay_scan(c, b, x, log_a, h0=None, lengths=None, layout="bhl"):
    """Differentiable linear attention with a decay for each head: returns
    (y like x, h_last); arguments as pdssm_decay_scan_fwd."""
    return DecayScanFunction.apply(c, b, x, log_a, h0, lengths, layout)


class SelectBalanceFunction(torch.autograd.Function):
    """(u, W_sel) -> loss [H] of a selection k; counts and mean probabilities
    come along without gradients."""

    @staticmethod
    def forward(ctx, u, W_sel, k, inv_tau, lengths):
        loss, counts, probs = pdssm_select_balance_fwd(u, W_sel, k, inv_tau, lengths)
        ctx.save_for_backward(u, W_sel, counts, lengths)
        ctx.inv_tau = inv_tau
        ctx.mark_non_differentiable(counts, probs)
        return loss, counts, probs

    @staticmethod
    @once_differentiable
    def backward(ctx, g_loss, _counts, _probs):
        u, W_sel, counts, lengths = ctx.saved_tensors
        g_u, g_W = pdssm_select_balance_bwd(u, W_sel, counts, g_loss.float().contiguous(),
                                            ctx.inv_tau, lengths)
        return g_u, g_W, None, None, None


def select_balance(u, W_sel, k=None, inv_tau=1.0, lengths=None):
    """Balance loss of the hard selection, per head (1 when even, K when all
    steps fall on one entry), with the counts of every entry and the mean
    probabilities: (loss [H], counts [H, K], probs [H, K])."""
    if k is None:
        with torch.no_grad():
            k = pdssm_select(u, W_sel)
    return SelectBalanceFunction.apply(u, W_sel, k, inv_tau, lengths)


class PDSSMLayer(torch.nn.Module):
    """Pre-norm residual multi-head PD-SSM block:
        x -> x + W_out y,  y = PD-SSM(u, d, b, c) of RMSNorm(x),
    u = W_u x_n (selection input), d = sigmoid(W_d x_n), b = W_b x_n,
    c = W_c x_n per head, a dictionary of K dense N x N matrices shared by
    the heads.  Inputs [B, L, d_model]; d, b, c in `state_dtype`."""

    def __init__(self, d_model, n_heads, n_state, n_dict, d_select=None, chunk=128,
                 inv_tau_s=1.0, inv_tau_a=1.0, state_dtype=torch.float32, device=None):
        super().__init__()
        d_select = d_select or d_model
        self.H, self.N, self.K, self.D = n_heads, n_state, n_dict, d_select
        self.chunk, self.inv_tau_s, self.inv_tau_a = chunk, inv_tau_s, inv_tau_a
        self.state_dtype = state_dtype
        f = dict(device=device, dtype=torch.float32)
        self.norm = torch.nn.RMSNorm(d_model, **f)
        self.proj_u = torch.nn.Linear(d_model, d_select, bias=False, **f)
        self.proj_d = torch.nn.Linear(d_model, n_heads * n_state, **f)
        self.proj_b = torch.nn.Linear(d_model, n_heads * n_state, bias=False, **f)
        self.proj_c = torch.nn.Linear(d_model, n_heads * n_state, bias=False, **f)
        self.W_sel = torch.nn.Parameter(torch.randn(n_heads, n_dict, d_select, **f) /
                                        d_select ** 0.5)
        self.A = torch.nn.Parameter(torch.randn(n_dict, n_state, n_state, **f))
        self.proj_out = torch.nn.Linear(n_heads, d_model, bias=False, **f)
        with torch.no_grad():
            self.proj_d.bias.fill_(2.0)   # decays start near sigmoid(2)

    def _heads(self, t, B, L):
        return t.view(B, L, self.H, self.N).permute(0, 2, 1, 3).contiguous().to(self.state_dtype)

    def mix(self, xn, balance=False):
        """The mixer on normed inputs: out [B, L, d_model], or with balance
        also the selection's balance loss per head."""
        B, L, _ = xn.shape
        u = self.proj_u(xn)
        if self.state_dtype == torch.bfloat16:
            u = u.to(torch.bfloat16)
        d = self._heads(torch.sigmoid(self.proj_d(xn)), B, L)
        b = self._heads(self.proj_b(xn), B, L)
        c = self._heads(self.proj_c(xn), B, L)
        u = u.contiguous()
        k = None
        if balance:
            with torch.no_grad():
                k = pdssm_select(u, self.W_sel)
        y, _ = pdssm(u, self.W_sel, self.A, d, b, c, None, self.chunk, self.inv_tau_s,
                     self.inv_tau_a, k)
        out = self.proj_out(y.permute(0, 2, 1))
        if not balance:
            return out
        return out, select_balance(u, self.W_sel, k, self.inv_tau_s)[0]

    def forward(self, x):
        return x + self.mix(self.norm(x))

    def block(self, delta, residual=None, balance=False):
        """The block over a residual stream: adds delta to it, norms the sum in
        the same pass, and returns (what the next block adds, the stream) and
        with balance the selection's loss per head."""
        eps = torch.finfo(torch.float32).eps if self.norm.eps is None else self.norm.eps
        xn, residual = add_rmsnorm(delta, residual, self.norm.weight, eps)
        out = self.mix(xn, balance)
        return (out[0], residual, out[1]) if balance else (out, residual)


class DecayLayer(torch.nn.Module):
    """Pre-norm residual multi-head block of the decay scan:
        x -> x + W_out y,  y = decay_scan(c, b, v, log_a) of RMSNorm(x),
    c, b of n_groups groups of heads, v and a decay per head and step,
    log_a = -exp(A_log) softplus(W_a x_n + bias).  Inputs [B, L, d_model];
    the projections' rows are used as they lie (layout "blh"), in
    `state_dtype`; the states are fp32 [B, H, n_state, head_dim]."""

    def __init__(self, d_model, n_heads, n_state, head_dim, n_groups=1, state_dtype=torch.float32,
                 device=None):
        super().__init__()
        if n_heads % n_groups:
            raise ValueError("n_heads must be a multiple of n_groups")
        self.H, self.G, self.N, self.P = n_heads, n_groups, n_state, head_dim
        self.state_dtype = state_dtype
        f = dict(device=device, dtype=torch.float32)
        self.norm = torch.nn.RMSNorm(d_model, **f)
        self.proj_c = torch.nn.Linear(d_model, n_groups * n_state, bias=False, **f)
        self.proj_b = torch.nn.Linear(d_model, n_groups * n_state, bias=False, **f)
        self.proj_v = torch.nn.Linear(d_model, n_heads * head_dim, bias=False, **f)
        self.proj_a = torch.nn.Linear(d_model, n_heads, **f)
        self.A_log = torch.nn.Parameter(torch.linspace(-1.0, 1.0, n_heads, **f))
        self.proj_out = torch.nn.Linear(n_heads * head_dim, d_model, bias=False, **f)
        with torch.no_grad():
            self.proj_a.bias.fill_(-3.0)   # decays start near exp(-softplus(-3))

    def _inputs(self, xn):
        lead, t = xn.shape[:-1], self.state_dtype
        c = self.proj_c(xn).view(*lead, self.G, self.N).to(t) * self.N ** -0.5
        b = self.proj_b(xn).view(*lead, self.G, self.N).to(t)
        v = self.proj_v(xn).view(*lead, self.H, self.P).to(t)
        log_a = -torch.exp(self.A_log) * torch.nn.functional.softplus(self.proj_a(xn))
        return c, b, v, log_a

    def mix(self, xn, h0=None, lengths=None):
        """(out [B, L, d_model], last state) on normed inputs."""
        y, h_last = decay_scan(*self._inputs(xn), h0, lengths, "blh")
        return self.proj_out(y.flatten(-2).to(xn.dtype)), h_last

    def forward(self, x, h0=None, lengths=None):
        return x + self.mix(self.norm(x), h0, lengths)[0]

    def _eps(self):
        return torch.finfo(torch.float32).eps if self.norm.eps is None else self.norm.eps

    def block(self, delta, residual=None, h0=None, lengths=None):
        """As PDSSMLayer.block, from states h0 and up to lengths: (what the next
        block adds, the stream, last state)."""
        xn, residual = add_rmsnorm(delta, residual, self.norm.weight, self._eps())
        out, h_last = self.mix(xn, h0, lengths)
        return out, residual, h_last

    @torch.no_grad()
    def step(self, delta, residual, state, slots=None):
        """One token of each stream: delta, residual [B, d_model], state
        [slots, H, N, P] updated in place.  Returns (what the next block adds,
        the stream)."""
        xn, residual = add_rmsnorm(delta, residual, self.norm.weight, self._eps())
        y = pdssm_decay_step(*self._inputs(xn), state, slots)
        return self.proj_out(y.flatten(-2).to(xn.dtype)), residual


class ResidualStack(torch.nn.Module):
    """Blocks (PDSSMLayer or DecayLayer) over one residual stream with a final
    norm; a block's output is added to the stream inside the next norm.
    (It calls their `block`, so forward hooks of blocks and norms do not run.)
    balance=True also returns the mean balance loss of the selecting blocks."""

    def __init__(self, blocks, d_model, device=None):
        super().__init__()
        self.blocks = torch.nn.ModuleList(blocks)
        self.norm = torch.nn.RMSNorm(d_model, device=device, dtype=torch.float32)

    def forward(self, x, balance=False):
        delta, residual, losses = x, None, []
        for block in self.blocks:
            if isinstance(block, PDSSMLayer):
                out = block.block(delta, residual, balance)
                losses += out[2:]
            else:
                out = block.block(delta, residual)
            delta, residual = out[0], out[1]
        eps = torch.finfo(torch.float32).eps if self.norm.eps is None else self.norm.eps
        out, _ = add_rmsnorm(delta, residual, self.norm.weight, eps)
        if not balance:
            return out
        if not losses:
            raise ValueError("no block of this stack selects")
        return out, torch.stack([loss.mean() for loss in losses]).mean()
