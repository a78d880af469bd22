"""Plain 64-bit implementations of the operators around the scan, step by step
from their definitions, and the sums of their terms' magnitudes that the error
bounds of the tests are multiples of.

Every bound here is counted, not fitted: a result that is a sum of terms, each
with at most `n` roundings to fp32 on its way (products, decays and the chain
of additions it passes through), is off by at most n 2^-24 times the sum of
the terms' magnitudes (to first order), and a rounding to bf16 on the way adds
2^-8 of it.
"""
import torch

U32, UBF = 2.0 ** -24, 2.0 ** -8


def unit(dtype):
    return UBF if dtype == torch.bfloat16 else U32


def _steps_first(v, layout):
    v = v.double()
    return v.permute(2, 0, 1, *range(3, v.dim())) if layout == "bhl" else v.transpose(0, 1)


def _back(v, layout):
    return (v.permute(1, 2, 0, *range(3, v.dim())) if layout == "bhl" else v.transpose(0, 1)).contiguous()


def decay_scan(c, b, x, log_a, h0=None, lengths=None, layout="bhl", g_y=None, g_hlast=None,
               magnitudes=False):
    """The recurrence and, with g_y, its adjoint, in 64 bits.  magnitudes=True
    takes the absolute values of every input: the sums of magnitudes."""
    f = torch.abs if magnitudes else (lambda v: v)
    c, b, x = (f(_steps_first(v, layout)) for v in (c, b, x))
    L, B, G, N = c.shape
    H, P = x.shape[2], x.shape[3]
    dev = x.device
    rep = H // G
    c, b = c.repeat_interleave(rep, 2), b.repeat_interleave(rep, 2)
    on = torch.ones(L, B, dtype=torch.bool, device=dev)
    if lengths is not None:
        on = torch.arange(L, device=dev)[:, None] < lengths.to(dev)
    if log_a.dim() == 1:
        a = log_a.double().exp().expand(L, B, H)
    else:
        a = _steps_first(log_a, layout).exp()
    a = torch.where(on[..., None], a, torch.ones((), dtype=torch.float64, device=dev))
    zero = torch.zeros((), dtype=torch.float64, device=dev)
    c, b, x = (torch.where(on[..., None, None], v, zero) for v in (c, b, x))
    S = f(h0.double()) if h0 is not None else torch.zeros(B, H, N, P, dtype=torch.float64, device=dev)
    kept, ys = [S], []
    for t in range(L):
        S = a[t][..., None, None] * S + b[t][..., None] * x[t][..., None, :]
        ys.append((c[t][..., None] * S).sum(-2))
        kept.append(S)
    y = torch.stack(ys) if L else torch.zeros(0, B, H, P, dtype=torch.float64, device=dev)
    out = dict(y=_back(y, layout), h_last=S)
    if g_y is None:
        return out
    gy = torch.where(on[..., None, None], f(_steps_first(g_y, layout)), zero)
    R = f(g_hlast.double()) if g_hlast is not None else torch.zeros_like(S)
    gc, gb, gx, gla = [None] * L, [None] * L, [None] * L, [None] * L
    for t in range(L - 1, -1, -1):
        R = R + c[t][..., None] * gy[t][..., None, :]
        gc[t] = (kept[t + 1] * gy[t][..., None, :]).sum(-1)
        gb[t] = (R * x[t][..., None, :]).sum(-1)
        gx[t] = (R * b[t][..., None]).sum(-2)
        R = a[t][..., None, None] * R
        gla[t] = (R * kept[t]).sum((-1, -2))
    if L:
        gc, gb, gx, gla = (torch.stack(v) for v in (gc, gb, gx, gla))
        gc, gb, gx = (torch.where(on[..., None, None], v, zero) for v in (gc, gb, gx))
        gla = torch.where(on[..., None], gla, zero)
    else:
        gc, gb = torch.zeros_like(c), torch.zeros_like(b)
        gx, gla = torch.zeros_like(x), torch.zeros(0, B, H, dtype=torch.float64, device=dev)
    share = lambda v: _back(v.reshape(L, B, G, rep, N).sum(3), layout)  # noqa: E731
    per_pair = (gy * y.abs()).sum(-1) if L else gla     # [L, B, H]
    out.update(g_c=share(gc), g_b=share(gb), g_x=_back(gx, layout),
               g_log_a=gla.sum((0, 1)) if log_a.dim() == 1 else _back(gla, layout), g_h0=R,
               pairs=per_pair)
    return out


def decay_bounds(dtype, N, P, L, mag, roundings):
    """{output: largest error}, elementwise, from the sums of magnitudes.

    fp32 roundings of a term: the chain of additions over a chunk's steps (at
    most 64: 32 one by one, or on the tensor cores 128 in eight additions of
    each of three parts, truncated and so of two units) and over the widths N and P, the decay (exponent rounded to fp32:
    at most 126 ln 2 units before the decay underflows, plus 4), once per
    chunk on the way 4 more, and 16 for the products around them.
    `roundings` bf16 roundings where the tensor cores take a decayed score or
    a state; the output's own rounding is added to bf16 outputs."""
    n = 64 + N + P + 90 + 16 + 4 * (L // 32 + 1)
    tol32 = n * U32
    low = roundings * UBF if dtype == torch.bfloat16 else 0.0
    own = unit(dtype)
    out = {}
    for k, v in mag.items():
        if k in ("y", "g_c", "g_b", "g_x"):
            out[k] = (tol32 + low + own) * v + 1e-37
        elif k in ("h_last", "g_h0"):
            out[k] = tol32 * v + 1e-37
    if "g_log_a" in mag:
        # the pair products of a whole chunk are added up before those that do
        # not straddle step t cancel
        whole = mag["pairs"].sum(0)                      # [B, H], all steps: no smaller than any chunk
        if mag["g_log_a"].dim() == 1:
            out["g_log_a"] = tol32 * (mag["g_log_a"] + L * whole.sum(0)) + 1e-37
        else:
            out["g_log_a"] = (mag["g_log_a"], tol32 * whole, tol32)
    return out


def add_rmsnorm(x, residual, weight, eps, res_dtype):
    s = x.double() if residual is None else x.double() + residual.double()
    s = s.to(torch.float32).to(res_dtype).double() if res_dtype == torch.bfloat16 else s.to(torch.float32).double()
    rstd = 1.0 / (s.square().mean(-1) + eps).sqrt()
    return s, rstd, s * rstd[..., None] * weight.double()


def add_rmsnorm_bwd(g_out, s, weight, rstd, g_res):
    s, g, w, r = s.double(), g_out.double(), weight.double(), rstd.double()[..., None]
    hat = s * r
    gw = g * w
    g_x = r * (gw - hat * (gw * hat).mean(-1, keepdim=True))
    if g_res is not None:
        g_x = g_x + g_res.double()
    return g_x, (g * hat).reshape(-1, s.shape[-1]).sum(0)


def balance(u, W, k, inv_tau, lengths=None, g_loss=None):
    B, L, D = u.shape
    H, K, _ = W.shape
    on = torch.ones(B, L, dtype=torch.bool, device=u.device)
    if lengths is not None:
        on = torch.arange(L, device=u.device) < lengths[:, None]
    T = int(on.sum())
    inv = 1.0 / T if T else 0.0
    ud, Wd = u.double(), W.double()
    p = torch.softmax(inv_tau * torch.einsum("bld,hkd->bhlk", ud, Wd), -1)
    p = torch.where(on[:, None, :, None], p, torch.zeros((), dtype=torch.float64, device=u.device))
    hit = (k[..., None] == torch.arange(K, device=u.device)) & on[:, None, :, None]
    counts = hit.sum((0, 2))
    f, m = counts.double() * inv, p.sum((0, 2)) * inv
    out = dict(loss=K * (f * m).sum(-1), counts=counts.to(torch.int32), probs=m)
    if g_loss is not None:
        gp = f[None, :, None, :] * (g_loss.double() * K * inv)[None, :, None, None]
        gz = inv_tau * p * (gp - (p * gp).sum(-1, keepdim=True))
        mag = inv_tau * p * (gp.abs() + (p * gp.abs()).sum(-1, keepdim=True))
        ud = torch.where(on[..., None], ud, torch.zeros((), dtype=torch.float64, device=u.device))
        out.update(g_u=torch.einsum("bhlk,hkd->bld", gz, Wd), g_W=torch.einsum("bhlk,bld->hkd", gz, ud),
                   mag_u=torch.einsum("bhlk,hkd->bld", mag, Wd.abs()),
                   mag_W=torch.einsum("bhlk,bld->hkd", mag, ud.abs()))
    return out
