"""GPU checks of the selection's balance loss, counts and gradients against a
64-bit implementation with counted bounds."""
import pytest
import torch

import block_ref as ref
import structured_sparse_state_b200 as pd

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


BF, F32 = torch.bfloat16, torch.float32
# dtype, B, L, H, K, D, inv_tau, ragged
CASES = [
    (F32, 1, 1, 1, 1, 1, 1.0, False),
    (F32, 2, 63, 3, 7, 33, 1.5, True),
    (F32, 3, 100, 2, 32, 256, 0.5, False),
    (F32, 1, 1000, 5, 8, 64, 2.0, False),
    # several groups of heads, split over CTAs or not; many tiles per CTA
    (F32, 1, 1, 16, 32, 64, 1.0, False),
    (F32, 2, 30, 19, 7, 24, 1.0, True),
    (F32, 4, 1200, 16, 8, 200, 1.0, False),
    (F32, 1, 30000, 3, 2, 128, 1.0, False),
    (F32, 3, 50, 5, 31, 250, 0.5, False),
    (BF, 2, 64, 4, 16, 128, 1.0, False),
    (BF, 1, 65, 1, 2, 16, 1.0, False),
    (BF, 4, 301, 3, 16, 96, 1.0, True),
    (BF, 2, 257, 16, 32, 256, 1.0, False),
    (BF, 3, 130, 2, 5, 31, 0.7, True),
    (BF, 2, 3000, 16, 16, 128, 1.0, False),
    (BF, 2, 500, 3, 4, 200, 1.0, False),
    # several tiles per CTA at every width of the weights' ring
    (BF, 3, 14000, 2, 8, 256, 1.0, False),
    (BF, 2, 13000, 3, 16, 160, 1.0, True),
    (BF, 1, 25000, 12, 32, 192, 1.0, False),
    (BF, 2, 20000, 4, 16, 64, 1.0, False),
]


def make(dtype, B, L, H, K, D, inv_tau, ragged, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.randn(B, L, D, generator=g, device="cuda").to(dtype)
    W = torch.randn(H, K, D, generator=g, device="cuda") * D ** -0.5
    k = (torch.rand(B, H, L, generator=g, device="cuda") * K).to(torch.int32).clamp_(max=K - 1)
    n = None
    if ragged:
        n = torch.randint(0, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        n[-1] = 0
    return u, W, k, torch.randn(H, generator=g, device="cuda"), n


def close(name, got, want, bound):
    err = (got.double() - want).abs()
    worst = (err - bound).max().item()
    assert worst <= 0, f"{name}: off by {err.max().item():.3g}, {worst:.3g} more than counted"


def logit_error(u, W, inv_tau):
    """Largest relative error of exp(logit): D additions of products, twice
    (the logit and the maximum that is subtracted)."""
    D = u.shape[-1]
    top = inv_tau * (u.double().abs().amax(0).amax(0) * W.double().abs().amax(0).amax(0)).sum().item()
    return 2 * (D + 4) * ref.U32 * min(top, inv_tau * u.double().norm(dim=-1).max().item() *
                                       W.double().norm(dim=-1).max().item())


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_loss_counts_and_gradients(case):
    u, W, k, g_loss, n = make(*case)
    K, inv_tau = case[4], case[6]
    want = ref.balance(u, W, k, inv_tau, n, g_loss)
    loss, counts, probs = pd.pdssm_select_balance_fwd(u, W, k, inv_tau=inv_tau, lengths=n)
    assert torch.equal(counts, want["counts"])
    rows = case[1] * case[2]
    # a probability: its logit, K additions of the norm, exp and division; the
    # sum over the steps: at most one chain over all of them
    e = logit_error(u, W, inv_tau) + (K + 12) * ref.U32
    tol = e + rows * ref.U32
    close("probs", probs, want["probs"], tol * want["probs"])
    close("loss", loss, want["loss"], (tol + 2 * ref.U32) * want["loss"])
    g_u, g_W = pd.pdssm_select_balance_bwd(u, W, counts, g_loss, inv_tau=inv_tau, lengths=n)
    # a logit's gradient: three probabilities, K additions
    tol = 3 * e + (K + 16) * ref.U32
    HK = case[3] * K
    # bf16: a logit's gradient is rounded on its way to g_u (2^-8 of each term),
    # W to 16 bits (2^-16), and g_u itself is rounded
    low = 2 * ref.UBF + 2.0 ** -16 if u.dtype == BF else ref.U32
    close("g_u", g_u, want["g_u"], (tol + HK * ref.U32 + low) * want["mag_u"] + 1e-37)
    close("g_W", g_W, want["g_W"], (tol + rows * ref.U32) * want["mag_W"] + 1e-37)


@pytest.mark.parametrize("D", [64, 33, 200])
@pytest.mark.parametrize("L", [1, 31, 33, 127, 159, 170])
def test_the_last_rows_of_a_tile(L, D):
    """B L rows that end inside a warp's 32, and lengths that do."""
    u, W, k, g_loss, _ = make(BF, 2, L, 3, 8, D, 1.0, False, seed=L)
    for n in (None, torch.tensor([L, L // 2], dtype=torch.int32, device="cuda")):
        want = ref.balance(u, W, k, 1.0, n, g_loss)
        loss, counts, probs = pd.pdssm_select_balance_fwd(u, W, k, lengths=n)
        g_u, g_W = pd.pdssm_select_balance_bwd(u, W, counts, g_loss, lengths=n)
        assert torch.equal(counts, want["counts"])
        e = logit_error(u, W, 1.0) + 20 * ref.U32
        tol = e + 2 * L * ref.U32
        close("probs", probs, want["probs"], tol * want["probs"])
        close("loss", loss, want["loss"], (tol + 2 * ref.U32) * want["loss"])
        # as in test_loss_counts_and_gradients
        tol = 3 * e + 24 * ref.U32
        close("g_u", g_u, want["g_u"], (tol + 24 * ref.U32 + 2 * ref.UBF + 2.0 ** -16) * want["mag_u"] + 1e-37)
        close("g_W", g_W, want["g_W"], (tol + 2 * L * ref.U32) * want["mag_W"] + 1e-37)


@pytest.mark.parametrize("case", [
    (BF, 2, 3000, 16, 16, 128, 1.0, False), (BF, 2, 20000, 4, 16, 64, 1.0, False), (BF, 3, 14000, 2, 8, 256, 1.0, False),
    (BF, 2, 257, 16, 32, 256, 1.0, False), (F32, 4, 1200, 16, 8, 200, 1.0, False), (F32, 1, 30000, 3, 2, 128, 1.0, False)],
    ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_weights_gradient_in_norm(case):
    """Tighter than the counted sums of worst cases: a lost bf16 part of the
    weights or of the logits' gradients (2.7e-6 in the mean square) would show.

    In units of 2^-24: a product's additions are truncated, by one unit on
    average: D / 16 of a logit (of size one), 8 of a tile's g_W; the roundings
    of exp (4), its argument (4), the division (2), the norm (4) and the factors
    (3) add up in squares, to 8.  With half as much again for the sums over
    tiles (fp32: for the chains over D and the rows)."""
    u, W, k, g_loss, _ = make(*case)
    want = ref.balance(u, W, k, case[6], None, g_loss)
    loss, counts, probs = pd.pdssm_select_balance_fwd(u, W, k, inv_tau=case[6])
    _, g_W = pd.pdssm_select_balance_bwd(u, W, counts, g_loss, inv_tau=case[6])
    units = 1.5 * (max(case[5], 64) / 16 + 8 + 8)
    for n, got in (("probs", probs), ("loss", loss), ("g_W", g_W)):
        err = ((got.double() - want[n]).norm() / want[n].norm()).item()
        assert err <= units * ref.U32, (n, err / ref.U32)


def test_gradients_against_differences():
    u, W, k, g_loss, n = make(F32, 2, 40, 2, 6, 24, 1.3, False, seed=1)
    _, counts, _ = pd.pdssm_select_balance_fwd(u, W, k, inv_tau=1.3)
    g_u, g_W = pd.pdssm_select_balance_bwd(u, W, counts, g_loss, inv_tau=1.3)
    g = torch.Generator(device="cuda").manual_seed(2)
    d = [torch.randn(v.shape, generator=g, device="cuda", dtype=torch.float64) for v in (u, W)]
    loss = lambda h: (ref.balance(u.double() + h * d[0], W.double() + h * d[1], k, 1.3)["loss"] *  # noqa: E731
                      g_loss.double()).sum().item()
    numeric = (loss(1e-5) - loss(-1e-5)) / 2e-5
    terms = [g_u.double() * d[0], g_W.double() * d[1]]
    mag = sum(t.abs().sum().item() for t in terms)
    assert abs(sum(t.sum().item() for t in terms) - numeric) <= 200 * ref.U32 * mag + 1e-8 * mag


def test_even_and_collapsed_selections():
    u = torch.zeros(2, 64, 16, device="cuda")
    W = torch.zeros(1, 4, 16, device="cuda")
    k = (torch.arange(128, device="cuda") % 4).to(torch.int32).view(2, 1, 64)
    loss, counts, probs = pd.pdssm_select_balance_fwd(u, W, k)
    assert loss.item() == 1.0 and (counts == 32).all() and (probs == 0.25).all()
    u[..., 0], W[0, 2, 0] = 1.0, 200.0       # all the weight on entry 2
    loss, counts, probs = pd.pdssm_select_balance_fwd(u, W, torch.full_like(k, 2))
    assert loss.item() == 4.0 and counts[0].tolist() == [0, 0, 128, 0]


def test_indices_outside_the_dictionary_are_not_counted():
    u, W, k, g_loss, _ = make(F32, 1, 100, 2, 4, 8, 1.0, False, seed=3)
    k[:, :, ::2] = -1
    k[:, :, 1::4] = 4
    _, counts, _ = pd.pdssm_select_balance_fwd(u, W, k)
    assert torch.equal(counts, ref.balance(u, W, k, 1.0)["counts"]) and counts.sum() == 2 * 25


def test_no_steps():
    u, W, k, g_loss, _ = make(BF, 2, 0, 2, 4, 32, 1.0, False)
    loss, counts, probs = pd.pdssm_select_balance_fwd(u, W, k)
    assert (loss == 0).all() and (counts == 0).all() and (probs == 0).all()
    g_u, g_W = pd.pdssm_select_balance_bwd(u, W, counts, g_loss)
    assert (g_W == 0).all()
    u, W, k, g_loss, _ = make(BF, 2, 70, 2, 4, 32, 1.0, False)
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    u.fill_(float("nan"))
    loss, counts, probs = pd.pdssm_select_balance_fwd(u, W, k, lengths=n)
    g_u, g_W = pd.pdssm_select_balance_bwd(u, W, counts, g_loss, lengths=n)
    for v in (loss, counts, probs, g_u, g_W):
        assert (v == 0).all()


def test_padding_is_not_read():
    u, W, k, g_loss, _ = make(BF, 3, 130, 4, 16, 64, 1.0, False, seed=4)
    n = torch.tensor([130, 64, 17], dtype=torch.int32, device="cuda")
    run = lambda: (*pd.pdssm_select_balance_fwd(u, W, k, lengths=n),)  # noqa: E731
    first = run()
    g = pd.pdssm_select_balance_bwd(u, W, first[1], g_loss, lengths=n)
    behind = torch.arange(130, device="cuda") >= n[:, None]
    u[behind] = float("nan")
    k.masked_fill_(behind[:, None], 1 << 30)
    for a, b in zip(first + g, run() + pd.pdssm_select_balance_bwd(u, W, first[1], g_loss, lengths=n)):
        assert torch.equal(a, b)
    assert (g[0][behind] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_same_bits_again_and_in_a_graph(dtype):
    u, W, k, g_loss, _ = make(dtype, 2, 2000, 4, 16, 128, 1.0, False, seed=5)

    def both():
        out = pd.pdssm_select_balance_fwd(u, W, k)
        return (*out, *pd.pdssm_select_balance_bwd(u, W, out[1], g_loss))

    first, again = both(), both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for v in held:
        v.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, again, held):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,L", [(31, 9), (32, 9), (33, 9), (1025, 3), (5000, 5)])
def test_many_ragged_sequences(dtype, B, L):
    """Up to as many lengths as a warp has lanes, and thousands; some negative or
    beyond L."""
    u, W, k, g_loss, n = make(dtype, B, L, 5, 16, 48, 1.0, True, seed=B)
    n[1], n[2] = L + 7, -3
    want = ref.balance(u, W, k, 1.0, n.clamp(0, L), g_loss)
    loss, counts, probs = pd.pdssm_select_balance_fwd(u, W, k, lengths=n)
    g_u, g_W = pd.pdssm_select_balance_bwd(u, W, counts, g_loss, lengths=n)
    assert torch.equal(counts, want["counts"])
    # as in test_loss_counts_and_gradients
    e = logit_error(u, W, 1.0) + 28 * ref.U32
    tol = e + B * L * ref.U32
    close("probs", probs, want["probs"], tol * want["probs"])
    close("loss", loss, want["loss"], (tol + 2 * ref.U32) * want["loss"])
    tol = 3 * e + 32 * ref.U32
    low = 2 * ref.UBF + 2.0 ** -16 if dtype == BF else ref.U32
    close("g_u", g_u, want["g_u"], (tol + 80 * ref.U32 + low) * want["mag_u"] + 1e-37)
    close("g_W", g_W, want["g_W"], (tol + B * L * ref.U32) * want["mag_W"] + 1e-37)


def test_selection_then_balance():
    """The selection's own indices: what the layer does."""
    u, W, _, g_loss, _ = make(BF, 2, 300, 4, 16, 64, 1.0, False, seed=6)
    k = pd.pdssm_select(u, W)
    loss, counts, probs = pd.pdssm_select_balance_fwd(u, W, k)
    want = ref.balance(u, W, k, 1.0)
    assert torch.equal(counts, want["counts"]) and counts.sum() == 2 * 300 * 4
