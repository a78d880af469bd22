"""The operators of a multi-head state-space block around the PD-SSM scan, as cases to be timed and compared.

Three groups that one pre-norm block uses together:

* the decay scan (linear attention with a decay for each head), the matrix-state sibling of the PD-SSM scan: over whole
  prompts and training sequences, and one step for single tokens;
* the root-mean-square norm with the residual's addition, forward (16-, 32- or 8-bit output) and backward;
* the balance loss of the hard selection, with the counts of every dictionary entry and its gradients.

A case's "op" says which one; run() makes the calls of the package where `own` is true and computes the same in
elementary torch operations, in 32 bits, where it is false.
"""
import math

import torch

own = False

_T = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}
_CHUNK = 128          # steps per block of the plain scan
_FLOOR = -200.0       # exp(-200) is 0 in 32 bits: a log decay below it acts as a reset


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------
def listed():
    return [
        # prompts of a served batch: the sizes of the library's bf16 selection-and-forward workload
        dict(name="scan prompts", op="scan", B=8, H=16, G=16, L=16384, N=64, P=64, dtype="bf16", layout="bhl",
             decay="step", h0=False, ragged=False),
        # one long document, keys shared by groups of heads, rows as the projections leave them
        dict(name="scan one document", op="scan", B=1, H=32, G=4, L=32768, N=128, P=64, dtype="bf16", layout="blh",
             decay="step", h0=True, ragged=False),
        # a short padded batch that goes on from earlier states, odd widths, a fixed decay for each head
        dict(name="scan short padded", op="scan", B=3, H=5, G=5, L=77, N=12, P=20, dtype="f32", layout="bhl",
             decay="head", h0=True, ragged=True),
        # a training step of the layer: forward and backward
        dict(name="train", op="train", B=2, H=16, G=16, L=16384, N=64, P=64, dtype="bf16", layout="bhl",
             decay="step", h0=False, ragged=False),
        # a small training step in 32 bits, odd length, shared keys
        dict(name="train small f32", op="train", B=2, H=4, G=2, L=1501, N=32, P=48, dtype="f32", layout="blh",
             decay="step", h0=True, ragged=False),
        # single tokens of a full batch of streams, states in slots of a pool
        dict(name="step full batch", op="step", B=256, S=272, H=16, G=16, N=64, P=64, dtype="bf16", decay="step"),
        # a single token of two streams: latency
        dict(name="step two streams", op="step", B=2, S=4, H=8, G=2, N=64, P=64, dtype="f32", decay="head"),
        # the residual stream of a training batch
        dict(name="norm batch", op="norm", T=65536, D=1024, x="bf16", res="bf16", out="bf16"),
        # the same in front of an 8-bit projection, a few decoded tokens: latency
        dict(name="norm tokens 8-bit", op="norm", T=24, D=2048, x="bf16", res="f32", out="e4m3"),
        # backward of the norm on a 32-bit residual stream
        dict(name="norm backward", op="norm_bwd", T=16384, D=2048, x="bf16", res="f32", out="bf16"),
        # balance of the selection at the sizes of the bf16 selection-and-forward workload
        dict(name="balance", op="balance", B=8, L=16384, H=16, K=16, D=128, dtype="bf16", inv_tau=1.0, ragged=False),
        # the same in 32 bits for a small padded batch
        dict(name="balance small f32", op="balance", B=4, L=501, H=3, K=8, D=64, dtype="f32", inv_tau=1.5, ragged=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["scan", "train", "step", "norm", "norm_bwd", "balance"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("scan", "train", "step"):
        G = rng.choice([1, 2, 3, 4, 8, 16])
        H = G * rng.choice([1, 1, 2, 4])
        N, P = rng.choice([16, 31, 32, 48, 64, 64, 64, 96, 128]), rng.choice([16, 31, 32, 48, 64, 64, 64, 96, 128])
        decay = rng.choice(["step", "step", "head"])
        if op == "step":
            B = _log(rng, 1, max(1, (256 * 16 * 64 * 64) // (H * N * P)))
            return dict(op=op, B=B, S=B + rng.randint(0, 16), H=H, G=G, N=N, P=P, dtype=dtype, decay=decay)
        B = rng.choice([1, 1, 2, 3, 4, 8])
        most = (1 << 20) if op == "scan" else (1 << 18)      # steps of all heads
        width = max(N, P) / 64
        L = _log(rng, 1, min(65536 if op == "scan" else 16384, max(1, int(most / (B * H * width * width)))))
        return dict(op=op, B=B, H=H, G=G, L=L, N=N, P=P, dtype=dtype, layout=rng.choice(["bhl", "blh"]), decay=decay,
                    h0=rng.random() < 0.5, ragged=rng.random() < 0.3)
    if op in ("norm", "norm_bwd"):
        D = rng.choice([_log(rng, 33, 8192), 96, 512, 1024, 2048, 4096])
        T = _log(rng, 1, min(65536, (1 << 25) // D))
        x = rng.choice(["bf16", "bf16", "f32"])
        res = rng.choice([x, "f32"])
        out = rng.choice([x, "bf16", "e4m3"]) if op == "norm" else x
        return dict(op=op, T=T, D=D, x=x, res=res, out=out)
    K, H = rng.choice([2, 4, 7, 8, 16, 32]), rng.choice([1, 2, 3, 4, 8, 16])
    D = rng.choice([16, 24, 33, 64, 96, 128, 200, 256])
    B = rng.choice([1, 2, 3, 4, 8])
    L = _log(rng, 1, min(16384, (1 << 21) // (B * H)))
    return dict(op=op, B=B, L=L, H=H, K=K, D=D, dtype=dtype, inv_tau=rng.choice([0.5, 1.0, 2.0]), ragged=rng.random() < 0.3)


def work(c):
    op = c["op"]
    if op in ("scan", "train", "step"):
        es, B, H, G, N, P = _SIZE[c["dtype"]], c["B"], c["H"], c["G"], c["N"], c["P"]
        L = 1 if op == "step" else c["L"]
        keys, vals = B * G * L * N * es, B * H * L * P * es
        la = B * H * L * 4 if c["decay"] == "step" else H * 4
        st = B * H * N * P * 4
        if op == "step":
            return {"bytes": 2 * keys + 2 * vals + la + 2 * st + 4 * B, "flops": 5 * B * H * N * P}
        n = B * H * L * N * P
        if op == "scan":
            return {"bytes": 2 * keys + 2 * vals + la + (2 if c["h0"] else 1) * st, "flops": 5 * n}
        # c, b, x, log a, g_y in; y, g_c, g_b, g_x, g_log_a, states out; the forward's own products and the gradients'
        return {"bytes": 4 * keys + 4 * vals + 2 * la + (5 if c["h0"] else 3) * st, "flops": 16 * n}
    if op == "norm":
        n = c["T"] * c["D"]
        return {"bytes": n * (_SIZE[c["x"]] + 2 * _SIZE[c["res"]] + _SIZE[c["out"]]) + 4 * c["D"] + 4 * c["T"], "flops": 6 * n}
    if op == "norm_bwd":
        n = c["T"] * c["D"]
        return {"bytes": n * (_SIZE[c["out"]] + 3 * _SIZE[c["res"]]) + 8 * c["D"] + 4 * c["T"], "flops": 10 * n}
    T, HK, D = c["B"] * c["L"], c["H"] * c["K"], c["D"]
    return {"bytes": 2 * T * D * _SIZE[c["dtype"]] + T * c["H"] * 4 + 2 * HK * D * 4, "flops": 6 * T * HK * D}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------
def _lengths(case, g):
    if not case["ragged"]:
        return None
    n = torch.randint(0, case["L"] + 1, (case["B"],), generator=g, device="cuda", dtype=torch.int32)
    n[0] = case["L"]
    return n


def _log_decay(case, g, lead):
    """Heads from short to long memory, steps around them, as a softplus gate gives."""
    H = case["H"]
    base = torch.linspace(-1.0, -7.0, H, device="cuda")
    if case["decay"] == "head":
        return -torch.nn.functional.softplus(base + 0.3 * torch.randn(H, generator=g, device="cuda"))
    z = torch.randn(*lead, generator=g, device="cuda")
    shape = [1] * len(lead)
    shape[1 if case.get("layout", "bhl") == "bhl" else 2] = H
    return -torch.nn.functional.softplus(base.view(shape) + z)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def normal(*shape, dtype=torch.float32, by=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * by).to(dtype)

    s = dict(case=case)
    if op in ("scan", "train", "step"):
        t = _T[case["dtype"]]
        B, H, G, N, P = case["B"], case["H"], case["G"], case["N"], case["P"]
        if op == "step":
            s["c"], s["b"], s["x"] = normal(B, G, N, dtype=t), normal(B, G, N, dtype=t, by=N ** -0.5), normal(B, H, P, dtype=t)
            s["log_a"] = _log_decay(case, g, (B, H))
            s["state"] = normal(case["S"], H, N, P)
            slots = torch.randperm(case["S"], generator=g, device="cuda")[:B].to(torch.int32)
            if B > 4:
                slots[B // 2] = -1               # an empty row of the batch
            s["slots"] = slots
            return s
        L = case["L"]
        keys, vals, gate = ((B, G, L, N), (B, H, L, P), (B, H, L)) if case["layout"] == "bhl" else ((B, L, G, N), (B, L, H, P), (B, L, H))
        s["c"], s["b"], s["x"] = normal(*keys, dtype=t), normal(*keys, dtype=t, by=N ** -0.5), normal(*vals, dtype=t)
        s["log_a"] = _log_decay(case, g, gate)
        s["h0"] = normal(B, H, N, P) if case["h0"] else None
        s["lengths"] = _lengths(case, g)
        if op == "train":
            s["g_y"] = normal(*vals, dtype=t)
            s["g_hlast"] = normal(B, H, N, P) if case["h0"] else None
        return s
    if op in ("norm", "norm_bwd"):
        T, D = case["T"], case["D"]
        s["weight"] = 1.0 + normal(D, by=0.1)
        s["eps"] = 1e-5
        if op == "norm":
            s["x"], s["residual"] = normal(T, D, dtype=_T[case["x"]]), normal(T, D, dtype=_T[case["res"]], by=2.0)
            return s
        s["g_out"], s["g_res"] = normal(T, D, dtype=_T[case["out"]]), normal(T, D, dtype=_T[case["res"]])
        s["res_out"] = normal(T, D, dtype=_T[case["res"]], by=2.0)
        s["rstd"] = torch.rsqrt(s["res_out"].float().square().mean(-1) + s["eps"])
        return s
    B, L, H, K, D = case["B"], case["L"], case["H"], case["K"], case["D"]
    s["u"] = normal(B, L, D, dtype=_T[case["dtype"]])
    s["W_sel"] = normal(H, K, D, by=D ** -0.5)
    # a selection that leans to its first entries, as one that has begun to collapse
    s["k"] = (torch.rand(B, H, L, generator=g, device="cuda").square() * K).to(torch.int32).clamp_(max=K - 1)
    s["g_loss"] = normal(H)
    s["lengths"] = _lengths(case, g)
    return s


# ---------------------------------------------------------------------------------------------------------------
# plain forms, in 32 bits
# ---------------------------------------------------------------------------------------------------------------
def _valid(s, L):
    n = s["lengths"]
    return None if n is None else torch.arange(L, device="cuda") < n[:, None]


def _blocks(s):
    """The scan's inputs as [B, H, blocks, steps, width] in 32 bits, log decays in 64, the last block filled up."""
    case = s["case"]
    H, G, L = case["H"], case["G"], case["L"]
    n = -(-L // _CHUNK)
    live = _valid(s, L)

    def block(v, heads):
        v = v if case["layout"] == "bhl" else v.transpose(1, 2)
        v = v if live is None else v * (live[:, None, :, None] if v.dim() == 4 else live[:, None])
        v = v if heads == H else v.repeat_interleave(H // heads, 1)
        pad = n * _CHUNK - L
        v = torch.nn.functional.pad(v, (0, 0, 0, pad) if v.dim() == 4 else (0, pad))
        return v.reshape(v.shape[0], H, n, _CHUNK, *v.shape[3:])

    la = s["log_a"].double().clamp(min=_FLOOR)
    if case["decay"] == "head":
        la = la.view(1, -1, 1).expand(case["B"], H, L)
        la = la if case["layout"] == "bhl" else la.transpose(1, 2)
    la = block(la, H)
    return block(s["c"].float(), G), block(s["b"].float(), G), block(s["x"].float(), H), la


def _carries(loc, tot, first):
    """State before each block and after the last: first * decays + sum over earlier blocks of loc * decays."""
    B, H, n = tot.shape
    T = torch.cat([torch.zeros_like(tot[..., :1]), tot.cumsum(-1)], -1)              # [B, H, n + 1]
    M = T[..., :, None] - T[..., None, 1:]                                           # into block i from after block j
    i, j = torch.arange(n + 1, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
    M = M.masked_fill(j >= i, -math.inf).exp().float()
    S = M @ loc.flatten(-2)
    if first is not None:
        S = S + T.exp().float()[..., None] * first.flatten(-2)[:, :, None]
    return S.view(B, H, n + 1, *loc.shape[-2:])


def _unblock(v, case, heads, live):
    """Back to the caller's layout, gradients of shared keys summed over their heads."""
    L, H = case["L"], case["H"]
    v = v.flatten(2, 3)[:, :, :L]
    if heads != H:
        v = v.view(v.shape[0], heads, H // heads, *v.shape[2:]).sum(2)
    if live is not None:
        v = v * (live[:, None, :, None] if v.dim() == 4 else live[:, None])
    return (v if case["layout"] == "bhl" else v.transpose(1, 2)).contiguous()


def _plain_scan(s):
    case = s["case"]
    c, b, x, la = _blocks(s)
    live = _valid(s, case["L"])
    cum = la.cumsum(-1)
    D = (cum[..., :, None] - cum[..., None, :]).masked_fill(~torch.ones(_CHUNK, _CHUNK, dtype=torch.bool, device="cuda").tril(), -math.inf).exp().float()
    into, out = cum.exp().float()[..., None], (cum[..., -1:] - cum).exp().float()[..., None]
    Pm = (c @ b.transpose(-1, -2)) * D
    S = _carries((b * out).transpose(-1, -2) @ x, cum[..., -1], s["h0"])
    y = Pm @ x + into * (c @ S[:, :, :-1])
    t = _T[case["dtype"]]
    outs = dict(y=_unblock(y, case, case["H"], live).to(t), h_last=S[:, :, -1].contiguous())
    if case["op"] == "scan":
        return outs
    H, G, L = case["H"], case["G"], case["L"]
    gy = s["g_y"].float() if case["layout"] == "bhl" else s["g_y"].float().transpose(1, 2)
    gy = gy if live is None else gy * live[:, None, :, None]
    gy = torch.nn.functional.pad(gy, (0, 0, 0, la.shape[2] * _CHUNK - L)).view_as(x)
    # gradient of the state after each block: the same recurrence backwards
    R = _carries(((c * into).transpose(-1, -2) @ gy).flip(2), cum[..., -1].flip(2), s["g_hlast"]).flip(2)
    g_h0, R = R[:, :, 0], R[:, :, 1:]
    V = gy @ x.transpose(-1, -2)
    E = (Pm * V).tril(-1).double()
    Q = V * D
    c_in, b_out = into * (gy @ S[:, :, :-1].transpose(-1, -2)), out * (x @ R.transpose(-1, -2))
    g_c, g_b = Q @ b + c_in, Q.transpose(-1, -2) @ c + b_out
    g_x = Pm.transpose(-1, -2) @ gy + out * (b @ R)
    after = (E.sum(-1) + (c * c_in).sum(-1).double() - E.sum(-2)).flip(-1).cumsum(-1).flip(-1)
    v = (b * b_out).sum(-1).double()
    through = cum[..., -1].exp() * (S[:, :, :-1] * R).double().sum((-1, -2))
    g_la = (after + v.cumsum(-1) - v + through[..., None]).float()
    g_la = _unblock(g_la, case, H, live)
    if case["decay"] == "head":
        g_la = g_la.double().sum((0, 2) if case["layout"] == "bhl" else (0, 1)).float()
    return dict(outs, g_c=_unblock(g_c, case, G, live).to(t), g_b=_unblock(g_b, case, G, live).to(t),
                g_x=_unblock(g_x, case, H, live).to(t), g_log_a=g_la, g_h0=g_h0.contiguous())


def _plain_step(s):
    case = s["case"]
    r = case["H"] // case["G"]
    slots, state = s["slots"].long(), s["state"]
    live = slots >= 0
    c, b, x = s["c"].float().repeat_interleave(r, 1), s["b"].float().repeat_interleave(r, 1), s["x"].float()
    a = s["log_a"].exp().expand(case["B"], case["H"])
    h = a[..., None, None] * state[slots.clamp(min=0)] + b[..., None] * x[..., None, :]
    y = (c[..., None] * h).sum(-2) * live[:, None, None]
    # an empty row writes to a slot behind the pool's last
    room = torch.cat([state, state[:1]])
    room[torch.where(live, slots, case["S"])] = h
    state.copy_(room[:-1])
    return dict(y=y.to(s["x"].dtype), state=state)


def _plain_norm(s):
    case = s["case"]
    total = (s["x"].float() + s["residual"].float()).to(_T[case["res"]])
    h = total.float()
    rstd = (h.square().mean(-1) + s["eps"]).rsqrt()
    y = h * rstd[:, None] * s["weight"]
    if case["out"] != "e4m3":
        return dict(out=y.to(_T[case["out"]]), res_out=total, rstd=rstd)
    top = y.abs().amax(-1)
    scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    return dict(out=(y / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), res_out=total, rstd=rstd, scale=scale)


def _plain_norm_bwd(s):
    h, gw = s["res_out"].float(), s["g_out"].float()
    hat = h * s["rstd"][:, None]
    g = gw * s["weight"]
    g_s = (g - hat * (g * hat).mean(-1, keepdim=True)) * s["rstd"][:, None] + s["g_res"].float()
    return dict(g_x=g_s.to(s["res_out"].dtype), g_weight=(gw * hat).sum(0))


def _plain_balance(s):
    case = s["case"]
    B, L, H, K, D = (case[n] for n in ("B", "L", "H", "K", "D"))
    live = _valid(s, L)
    live = torch.ones(B, L, dtype=torch.bool, device="cuda") if live is None else live
    u, W = s["u"].float(), s["W_sel"]
    z = (u.view(B * L, D) @ W.view(H * K, D).t()).view(B, L, H, K) * case["inv_tau"]
    e = (z - z.amax(-1, keepdim=True)).exp()
    p = e / e.sum(-1, keepdim=True) * live[..., None, None]
    T = live.sum().clamp(min=1)
    hit = (s["k"].transpose(1, 2)[..., None] == torch.arange(K, device="cuda")) & live[..., None, None]
    counts = hit.sum((0, 1))
    f = counts.float() / T
    probs = p.sum((0, 1)) / T
    loss = K * (f * probs).sum(-1)
    g_z = (s["g_loss"] * (K * case["inv_tau"]) / T)[:, None] * p * (f - (p * f).sum(-1, keepdim=True))
    g_z = g_z.view(B * L, H * K)
    return dict(loss=loss, counts=counts.to(torch.int32), probs=probs,
                g_u=(g_z @ W.view(H * K, D)).view(B, L, D).to(s["u"].dtype), g_W=(g_z.t() @ u.view(B * L, D)).view(H, K, D))


_PLAIN = dict(scan=_plain_scan, train=_plain_scan, step=_plain_step, norm=_plain_norm, norm_bwd=_plain_norm_bwd, balance=_plain_balance)


# ---------------------------------------------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------------------------------------------
def _own(s):
    import structured_sparse_state_b200 as pd
    case = s["case"]
    op = case["op"]
    if op == "scan":
        y, h_last, _ = pd.pdssm_decay_scan_fwd(s["c"], s["b"], s["x"], s["log_a"], s["h0"], lengths=s["lengths"], layout=case["layout"])
        return dict(y=y, h_last=h_last)
    if op == "train":
        y, h_last, ws = pd.pdssm_decay_scan_fwd(s["c"], s["b"], s["x"], s["log_a"], s["h0"], lengths=s["lengths"],
                                                layout=case["layout"], for_bwd=True)
        g = pd.pdssm_decay_scan_bwd(s["c"], s["b"], s["x"], s["log_a"], s["h0"], s["g_y"], ws, g_hlast=s["g_hlast"],
                                    lengths=s["lengths"], layout=case["layout"])
        return dict(y=y, h_last=h_last, g_c=g[0], g_b=g[1], g_x=g[2], g_log_a=g[3], g_h0=g[4])
    if op == "step":
        y = pd.pdssm_decay_step(s["c"], s["b"], s["x"], s["log_a"], s["state"], slots=s["slots"])
        return dict(y=y, state=s["state"])
    if op == "norm":
        out, res_out, rstd, scale = pd.pdssm_add_rmsnorm_fwd(s["x"], s["residual"], s["weight"], eps=s["eps"], out_dtype=_T[case["out"]])
        return dict(out=out, res_out=res_out, rstd=rstd, **({} if scale is None else dict(scale=scale)))
    if op == "norm_bwd":
        g_x, g_weight = pd.pdssm_add_rmsnorm_bwd(s["g_out"], s["res_out"], s["weight"], s["rstd"], g_res=s["g_res"])
        return dict(g_x=g_x, g_weight=g_weight)
    loss, counts, probs = pd.pdssm_select_balance_fwd(s["u"], s["W_sel"], s["k"], inv_tau=case["inv_tau"], lengths=s["lengths"])
    g_u, g_W = pd.pdssm_select_balance_bwd(s["u"], s["W_sel"], counts, s["g_loss"], inv_tau=case["inv_tau"], lengths=s["lengths"])
    return dict(loss=loss, counts=counts, probs=probs, g_u=g_u, g_W=g_W)


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------
def _exact_scan(s):
    """The recurrence step by step: S_t = a_t S_{t-1} + b_t x_t^T, y_t = S_t^T c_t; its adjoint in reverse."""
    case = s["case"]
    B, H, G, L, N, P = (case[n] for n in ("B", "H", "G", "L", "N", "P"))
    train = case["op"] == "train"
    if L > 200000 or (train and L * B * H * N * P * 8 > 60e9):
        return None
    first = (lambda v: v.double().permute(2, 0, 1, *range(3, v.dim()))) if case["layout"] == "bhl" else (lambda v: v.double().transpose(0, 1))
    share = lambda v: v.unsqueeze(3).expand(L, B, G, H // G, N).reshape(L, B, H, N)  # noqa: E731
    c, b, x = share(first(s["c"])), share(first(s["b"])), first(s["x"])
    a = (s["log_a"].double().exp().expand(L, B, H) if case["decay"] == "head" else first(s["log_a"]).exp()).contiguous()
    n = s["lengths"]
    on = torch.ones(L, B, dtype=torch.bool, device="cuda") if n is None else torch.arange(L, device="cuda")[:, None] < n
    a = torch.where(on[..., None], a, torch.ones_like(a))
    b, c = b * on[..., None, None], c * on[..., None, None]
    S = s["h0"].double() if s["h0"] is not None else torch.zeros(B, H, N, P, dtype=torch.float64, device="cuda")
    y = torch.empty(L, B, H, P, dtype=torch.float64, device="cuda")
    kept = torch.empty(L + 1, B, H, N, P, dtype=torch.float64, device="cuda") if train else None
    if train:
        kept[0] = S
    a4 = a[..., None, None]
    for t in range(L):
        S = torch.addcmul(a4[t] * S, b[t][..., None], x[t][..., None, :])
        torch.sum(c[t][..., None] * S, -2, out=y[t])
        if train:
            kept[t + 1] = S

    def back(v):
        return v.permute(1, 2, 0, *range(3, v.dim())) if case["layout"] == "bhl" else v.transpose(0, 1)

    outs = dict(y=back(y), h_last=S)
    if not train:
        return outs
    gy = first(s["g_y"]) * on[..., None, None]
    gS = s["g_hlast"].double() if s["g_hlast"] is not None else torch.zeros_like(S)
    gc, gb, gx, gla = torch.empty_like(c), torch.empty_like(b), torch.empty_like(x), torch.empty_like(a)
    for t in range(L - 1, -1, -1):
        gS = torch.addcmul(gS, c[t][..., None], gy[t][..., None, :])
        gc[t] = (kept[t + 1] * gy[t][..., None, :]).sum(-1)
        gb[t] = (gS * x[t][..., None, :]).sum(-1)
        gx[t] = (gS * b[t][..., None]).sum(-2)
        gS = a4[t] * gS
        gla[t] = (gS * kept[t]).sum((-1, -2))
    gc, gb, gla = gc * on[..., None, None], gb * on[..., None, None], gla * on[..., None]
    over = lambda v: back(v.reshape(L, B, G, H // G, N).sum(3))  # noqa: E731
    return dict(outs, g_c=over(gc), g_b=over(gb), g_x=back(gx), g_log_a=gla.sum((0, 1)) if case["decay"] == "head" else back(gla), g_h0=gS)


def _exact_step(s):
    case = s["case"]
    state = s["state"].double()
    y = torch.zeros(case["B"], case["H"], case["P"], dtype=torch.float64, device="cuda")
    a = s["log_a"].double().exp().expand(case["B"], case["H"])
    r = case["H"] // case["G"]
    for i, at in enumerate(s["slots"].tolist()):
        if at >= 0:
            b, c = s["b"][i].double().repeat_interleave(r, 0), s["c"][i].double().repeat_interleave(r, 0)
            state[at] = a[i, :, None, None] * state[at] + torch.einsum("hn,hp->hnp", b, s["x"][i].double())
            y[i] = torch.einsum("hn,hnp->hp", c, state[at])
    return dict(y=y, state=state)


def _exact_norm(s):
    case = s["case"]
    total = (s["x"].double() + s["residual"].double()).to(_T[case["res"]]).double()
    rms = torch.sqrt(torch.einsum("td,td->t", total, total) / case["D"] + s["eps"])
    y = total / rms[:, None] * s["weight"].double()
    if case["out"] != "e4m3":
        return dict(out=y, res_out=s["x"].double() + s["residual"].double(), rstd=1 / rms)
    scale = y.abs().amax(-1) / 448
    return dict(out=y / scale[:, None], res_out=s["x"].double() + s["residual"].double(), rstd=1 / rms, scale=scale)


def _exact_norm_bwd(s):
    h, g, r, w = s["res_out"].double(), s["g_out"].double(), s["rstd"].double(), s["weight"].double()
    D = h.shape[1]
    dot = torch.einsum("td,td,d->t", g, h, w)
    g_x = r[:, None] * (g * w) - h * (r ** 3 * dot / D)[:, None] + s["g_res"].double()
    return dict(g_x=g_x, g_weight=torch.einsum("td,td,t->d", g, h, r))


def _exact_balance(s):
    case = s["case"]
    B, L, H, K, D = (case[n] for n in ("B", "L", "H", "K", "D"))
    n = s["lengths"]
    rows = torch.ones(B, L, dtype=torch.bool, device="cuda") if n is None else torch.arange(L, device="cuda") < n[:, None]
    u, T = s["u"][rows].double(), max(1, int(rows.sum()))
    loss, counts, probs, g_W, g_u = [], [], [], [], torch.zeros(B, L, D, dtype=torch.float64, device="cuda")
    for h in range(H):
        W = s["W_sel"][h].double()
        p = torch.softmax(case["inv_tau"] * torch.einsum("td,kd->tk", u, W), -1)
        count = torch.bincount(s["k"][:, h][rows].long(), minlength=K)
        f, m = count.double() / T, p.sum(0) / T
        gp = s["g_loss"][h].double() * K / T * f                       # gradient of every row's probabilities
        gz = case["inv_tau"] * p * (gp - (p * gp).sum(-1, keepdim=True))
        loss.append(K * (f * m).sum())
        counts.append(count)
        probs.append(m)
        g_W.append(gz.t() @ u)
        g_u[rows] += gz @ W
    return dict(loss=torch.stack(loss), counts=torch.stack(counts).to(torch.int32), probs=torch.stack(probs), g_u=g_u, g_W=torch.stack(g_W))


def exact(case, seed):
    return dict(scan=_exact_scan, train=_exact_scan, step=_exact_step, norm=_exact_norm, norm_bwd=_exact_norm_bwd,
                balance=_exact_balance)[case["op"]](prepare(case, seed))
