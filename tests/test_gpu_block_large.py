"""GPU checks of the block operators on tensors of more than 2^31 elements: the
last rows, heads and slots against the same work done on a small copy."""
import pytest
import torch

import block_ref as ref
import structured_sparse_state_b200 as pd

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    yield
    torch.cuda.empty_cache()


BF, F32 = torch.bfloat16, torch.float32


def normal(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


@pytest.mark.parametrize("dtype,P,L", [(BF, 64, 530_000), (F32, 64, 530_000), (BF, 33, 1_100_000)], ids=str)
def test_decay_scan(dtype, P, L):
    """The last head of 64 that share one key against that head by itself:
    each is within the counted bound of the exact result, so the two differ by
    at most twice as much."""
    H, N = 64, 8
    assert H * L * P > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    c, b = normal(g, 1, L, 1, N, dtype=dtype), normal(g, 1, L, 1, N, dtype=dtype)
    x = normal(g, 1, L, H, P, dtype=dtype)
    la = -0.05 - 0.5 * torch.rand(H, generator=g, device="cuda")
    y, h_last, ws = pd.pdssm_decay_scan_fwd(c, b, x, la, layout="blh", for_bwd=True)
    one = x[:, :, -1:].contiguous()
    y1, h1, ws1 = pd.pdssm_decay_scan_fwd(c, b, one, la[-1:], layout="blh", for_bwd=True)
    my, mh, _ = pd.pdssm_decay_scan_fwd(c.abs().float(), b.abs().float(), one.abs().float(), la[-1:], layout="blh")
    bound = ref.decay_bounds(dtype, N, P, L, dict(y=my, h_last=mh), 2)
    assert ((y[:, :, -1:].float() - y1.float()).abs() <= 2.01 * bound["y"]).all()
    assert ((h_last[:, -1:] - h1).abs() <= 2.01 * bound["h_last"]).all()
    del y
    # a gradient in the last head alone
    g_y = torch.zeros_like(x)
    g_y[:, :, -1:] = normal(g, 1, L, 1, P, dtype=dtype)
    got = pd.pdssm_decay_scan_bwd(c, b, x, la, None, g_y, ws, layout="blh")
    want = pd.pdssm_decay_scan_bwd(c, b, one, la[-1:], None, g_y[:, :, -1:].contiguous(), ws1, layout="blh")
    assert (got[2][:, :, :-1] == 0).all()
    # magnitudes of the gradients: those of the adjoint of the magnitudes
    m = [v.abs().float().contiguous() for v in (c, b, one)]
    _, _, wsm = pd.pdssm_decay_scan_fwd(*m, la[-1:], layout="blh", for_bwd=True)
    mag = pd.pdssm_decay_scan_bwd(*m, la[-1:], None, g_y[:, :, -1:].abs().float().contiguous(), wsm, layout="blh")
    bound = ref.decay_bounds(dtype, N, P, L, dict(g_c=mag[0], g_b=mag[1], g_x=mag[2]), 2)
    for k, (p, q) in dict(g_c=(got[0], want[0]), g_b=(got[1], want[1]), g_x=(got[2][:, :, -1:], want[2])).items():
        assert ((p.float() - q.float()).abs() <= 2.01 * bound[k]).all(), k


def test_decay_step_in_the_last_slot():
    S, H, N, P = 33_000, 16, 64, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    state = torch.zeros(S, H, N, P, device="cuda")
    assert state.numel() > 2 ** 31
    state[-1] = normal(g, H, N, P)
    small = state[-1:].clone()
    c, b, x = normal(g, 2, H, N), normal(g, 2, H, N), normal(g, 2, H, P)
    la = -torch.rand(2, H, generator=g, device="cuda")
    y = pd.pdssm_decay_step(c, b, x, la, state, slots=torch.tensor([0, S - 1], dtype=torch.int32, device="cuda"))
    want = pd.pdssm_decay_step(c[1:].contiguous(), b[1:].contiguous(), x[1:].contiguous(), la[1:].contiguous(), small)
    assert torch.equal(y[1:], want) and torch.equal(state[-1:], small)
    assert (state[0] != 0).any() and (state[1:-1].view(-1)[:: 4097] == 0).all()


@pytest.mark.parametrize("D", [1000, 1001, 1024])
def test_norm(D):
    rows = 2 ** 31 // D + 5000
    g = torch.Generator(device="cuda").manual_seed(3)
    x, res, w = normal(g, rows, D, dtype=BF), normal(g, rows, D, dtype=BF), normal(g, D)
    out, s, rstd, _ = pd.pdssm_add_rmsnorm_fwd(x, res, w)
    # the same row parities, so that pieces and pairs fall alike
    n = 4000 + rows % 8
    tail = slice(rows - n, rows)
    a = pd.pdssm_add_rmsnorm_fwd(x[tail].clone(), res[tail].clone(), w)
    assert torch.equal(s[tail], a[1])
    # another order of a row's additions: 45 units each (rstd), the output's rounding
    assert ((rstd[tail] - a[2]).abs() <= 90 * ref.U32 * a[2]).all()
    assert ((out[tail].float() - a[0].float()).abs() <= 2 * (ref.UBF + 50 * ref.U32) * a[0].float().abs()).all()
    g_x, _ = pd.pdssm_add_rmsnorm_bwd(x, s, w, rstd, g_res=res)
    b, _ = pd.pdssm_add_rmsnorm_bwd(x[tail].clone(), s[tail].clone(), w, rstd[tail].clone(), g_res=res[tail].clone())
    assert torch.equal(g_x[tail], b)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_balance(dtype):
    L, D, K = 2 ** 23 + 333, 256, 4
    g = torch.Generator(device="cuda").manual_seed(4)
    u = normal(g, 1, L, D, dtype=dtype)
    W = normal(g, 1, K, D) * D ** -0.5
    k = torch.randint(0, K, (1, 1, L), generator=g, device="cuda", dtype=torch.int32)
    loss, counts, probs = pd.pdssm_select_balance_fwd(u, W, k)
    assert torch.equal(counts[0].long(), torch.bincount(k.view(-1), minlength=K))
    g_u, g_W = pd.pdssm_select_balance_bwd(u, W, counts, torch.ones(1, device="cuda") * L)
    # the last rows' gradients by the formula in 64 bits
    p = torch.softmax(u[0, -999:].double() @ W[0].double().T, -1)
    f = counts[0].double() / L
    terms = K * p * (f - (p * f).sum(-1, keepdim=True))
    want = terms @ W[0].double()
    # logits of 256 products (fp32; the tensor cores' W has 16 bits for g_u), the
    # softmax's few roundings, and one (fp32: none) of the gradients to bf16
    mag = (K * p * (f + (p * f).sum(-1, keepdim=True))) @ W[0].double().abs()
    size = (u[0, -999:].double().abs() @ W[0].double().abs().T).amax(-1, keepdim=True)
    logit = (2 * 260 * ref.U32 + (2.0 ** -17 if dtype == BF else 0.0)) * size
    tol = 4 * logit + 64 * ref.U32 + (ref.UBF if dtype == BF else 0.0)
    assert ((g_u[0, -999:].double() - want).abs() <= tol * mag + ref.unit(dtype) * want.abs()).all()
    assert torch.isfinite(g_W).all() and abs(probs.sum().item() - 1) <= 1e-5


@pytest.mark.parametrize("dtype", [BF, F32])
def test_balance_weights_gradient(dtype):
    """g_W over 2^23 rows against the formula in 64 bits, by its norm: units as in
    the balance's own test of it, and 12 for the sums over a CTA's hundreds of
    tiles (each addition of them off by half a unit at most, in squares)."""
    L, D, K = 2 ** 23 + 333, 256, 4
    g = torch.Generator(device="cuda").manual_seed(5)
    u, W = normal(g, 1, L, D, dtype=dtype), normal(g, 1, K, D) * D ** -0.5
    k = (torch.rand(1, 1, L, generator=g, device="cuda").square() * K).to(torch.int32).clamp_(max=K - 1)
    _, counts, probs = pd.pdssm_select_balance_fwd(u, W, k)
    _, g_W = pd.pdssm_select_balance_bwd(u, W, counts, torch.ones(1, device="cuda"))
    f = counts[0].double() / L
    want, mean = torch.zeros(K, D, dtype=torch.float64, device="cuda"), torch.zeros(K, dtype=torch.float64, device="cuda")
    for part in u[0].split(1 << 20):
        p = torch.softmax(part.double() @ W[0].double().T, -1)
        want += (K / L * p * (f - (p * f).sum(-1, keepdim=True))).T @ part.double()
        mean += p.sum(0) / L
    units = 1.5 * (D / 16 + 8 + 8) + 12
    assert (g_W[0].double() - want).norm() <= units * ref.U32 * want.norm()
    assert (probs[0].double() - mean).norm() <= units * ref.U32 * mean.norm()
