"""GPU checks of the residual addition with root-mean-square norm, forward and
backward, against 64-bit implementations with counted bounds."""
import math

import pytest
import torch

import block_ref as ref
import structured_sparse_state_b200 as pd

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
WIDTHS = [1, 7, 96, 512, 513, 1000, 1024, 1032, 2048, 4096, 4100, 5120, 8192, 9000, 16384,
          # odd widths, around the sizes where a row takes more threads
          9, 1018, 1023, 2047, 4091, 16373, 16379]


def normal(g, *shape, dtype=F32, by=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * by).to(dtype)


def close(name, got, want, bound):
    err = (got.double() - want).abs()
    worst = (err - bound).max().item()
    assert worst <= 0, f"{name}: off by {err.max().item():.3g}, {worst:.3g} more than counted"


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("types", [(F32, F32, F32), (BF, BF, BF), (BF, F32, BF), (BF, F32, E4), (F32, None, E4),
                                   (BF, None, F32)], ids=str)
def test_forward(D, types):
    x_t, r_t, o_t = types
    g = torch.Generator(device="cuda").manual_seed(D)
    rows, eps = 5, 1e-5
    x = normal(g, rows, D, dtype=x_t)
    res = None if r_t is None else normal(g, rows, D, dtype=r_t, by=2.0)
    w = (1 + normal(g, D, by=0.2)).to(BF if D % 2 else F32)
    out, s, rstd, scale = pd.pdssm_add_rmsnorm_fwd(x, res, w, eps=eps, out_dtype=o_t)
    s_ref, r_ref, y_ref = ref.add_rmsnorm(x, res, w, eps, x_t if r_t is None else r_t)
    assert s.dtype == (x_t if r_t is None else r_t) and torch.equal(s.double(), s_ref)
    # the mean of squares: a chain of at most 32 additions per thread and 42
    # over threads and warps, halved by the root; division, root, eps: 8
    tol = 45 * ref.U32
    close("rstd", rstd, r_ref, tol * r_ref)
    if o_t is not E4:
        assert scale is None
        close("out", out, y_ref, (tol + 2 * ref.U32 + ref.unit(o_t)) * y_ref.abs())
        return
    top = y_ref.abs().amax(-1)
    close("scale", scale, top / 448, (tol + 4 * ref.U32) * top / 448)
    # e4m3: half a step of 2^-4 relative, or of the smallest subnormal 2^-9
    val = out.float().double() * scale.double()[:, None]
    close("out", val, y_ref, (2.0 ** -4 + 2 * tol) * y_ref.abs() + 2.0 ** -10 * scale.double()[:, None])


def test_rows_of_zeros_and_non_finite_rows():
    x = torch.zeros(4, 256, device="cuda")
    x[1, 3], x[2, 5] = math.nan, math.inf
    x[3] = 1.0
    w = torch.ones(256, device="cuda")
    out, s, rstd, scale = pd.pdssm_add_rmsnorm_fwd(x, None, w, eps=1e-5, out_dtype=E4)
    assert (out[0].float() == 0).all() and scale[0] == 1.0
    assert not math.isfinite(scale[1].item()) and not math.isfinite(scale[2].item())
    assert (out[3].float() == 448).all()
    out, _, _, _ = pd.pdssm_add_rmsnorm_fwd(x, None, w, eps=1e-5)
    assert (out[0] == 0).all() and torch.isnan(out[1]).all() and torch.isfinite(out[3]).all()


@pytest.mark.parametrize("rows", [0, 1, 3, 4, 5, 300])
def test_row_counts(rows):
    g = torch.Generator(device="cuda").manual_seed(rows)
    for D in (64, 2048):
        x, res, w = normal(g, rows, D), normal(g, rows, D), normal(g, D)
        out, s, rstd, _ = pd.pdssm_add_rmsnorm_fwd(x, res, w)
        assert out.shape == x.shape and torch.equal(s, x + res)
        g_x, g_w = pd.pdssm_add_rmsnorm_bwd(normal(g, rows, D), s, w, rstd)
        assert g_x.shape == x.shape and torch.isfinite(g_w).all()
        if rows == 0:
            assert (g_w == 0).all()


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("types", [(F32, F32), (BF, BF), (BF, F32)], ids=str)
@pytest.mark.parametrize("with_res", [False, True])
def test_backward(D, types, with_res):
    check_backward(37, D, *types, with_res)


@pytest.mark.parametrize("D", [96, 640, 1001, 1024, 2048])
@pytest.mark.parametrize("types", [(F32, F32), (BF, BF)], ids=str)
def test_backward_of_many_rows(D, types):
    """Several turns of every CTA, the last one with fewer rows."""
    check_backward(3001, D, *types, True)


def check_backward(rows, D, g_t, r_t, with_res):
    g = torch.Generator(device="cuda").manual_seed(D + 1)
    s, g_out = normal(g, rows, D, dtype=r_t, by=2.0), normal(g, rows, D, dtype=g_t)
    w = (1 + normal(g, D, by=0.2)).to(BF if D % 2 else F32)
    rstd = (s.double().square().mean(-1) + 1e-5).rsqrt().float()
    g_res = normal(g, rows, D, dtype=r_t) if with_res else None
    g_x, g_w = pd.pdssm_add_rmsnorm_bwd(g_out, s, w, rstd, g_res=g_res)
    x_ref, w_ref = ref.add_rmsnorm_bwd(g_out, s, w, rstd, g_res)
    hat = s.double().abs() * rstd.double()[:, None]
    gw = g_out.double().abs() * w.double().abs()
    mag = rstd.double()[:, None] * (gw + hat * (gw * hat).mean(-1, keepdim=True))
    if with_res:
        mag = mag + g_res.double().abs()
    close("g_x", g_x, x_ref, 64 * ref.U32 * mag + ref.unit(r_t) * x_ref.abs())
    close("g_weight", g_w, w_ref, (rows + 8) * ref.U32 * (g_out.double().abs() * hat).sum(0))


def test_gradients_against_differences():
    """A direction of x, residual and weight, differences in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x, res, w = normal(g, 6, 200), normal(g, 6, 200), 1 + normal(g, 200, by=0.1)
    go, gr = normal(g, 6, 200), normal(g, 6, 200)
    out, s, rstd, _ = pd.pdssm_add_rmsnorm_fwd(x, res, w, eps=1e-5)
    g_x, g_w = pd.pdssm_add_rmsnorm_bwd(go, s, w, rstd, g_res=gr)
    d = [torch.randn(v.shape, generator=g, device="cuda", dtype=torch.float64) for v in (x, res, w)]

    def loss(h):
        a, b, c = (v.double() + h * e for v, e in zip((x, res, w), d))
        t = a + b
        y = t / (t.square().mean(-1, keepdim=True) + 1e-5).sqrt() * c
        return ((y * go.double()).sum() + (t * gr.double()).sum()).item()

    numeric = (loss(1e-5) - loss(-1e-5)) / 2e-5
    terms = [(g_x.double() * (d[0] + d[1])), (g_w.double() * d[2])]
    mag = sum(t.abs().sum().item() for t in terms)
    assert abs(sum(t.sum().item() for t in terms) - numeric) <= 100 * ref.U32 * mag + 1e-8 * mag


def test_in_place_and_same_bits():
    g = torch.Generator(device="cuda").manual_seed(4)
    for D in (96, 1000, 1001, 2048, 4099):
        x, res, w = normal(g, 50, D, dtype=BF), normal(g, 50, D, dtype=BF), normal(g, D)
        out, s, rstd, _ = pd.pdssm_add_rmsnorm_fwd(x, res, w)
        x2, r2 = x.clone(), res.clone()
        pd.pdssm_add_rmsnorm_fwd(x2, r2, w, out=x2, res_out=r2)
        assert torch.equal(x2, out) and torch.equal(r2, s)
        go, gr = normal(g, 50, D, dtype=BF), normal(g, 50, D, dtype=BF)
        a = pd.pdssm_add_rmsnorm_bwd(go, s, w, rstd, g_res=gr)
        b = pd.pdssm_add_rmsnorm_bwd(go, s, w, rstd, g_res=gr, g_x=gr)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_unaligned_rows_and_leading_dimensions():
    g = torch.Generator(device="cuda").manual_seed(6)
    room = normal(g, 2 * 3 * 64 + 1)
    x = room[1:].view(2, 3, 64)
    res, w = normal(g, 2, 3, 64), normal(g, 64)
    out, s, rstd, _ = pd.pdssm_add_rmsnorm_fwd(x, res, w)
    want = pd.pdssm_add_rmsnorm_fwd(x.clone(), res, w)
    assert rstd.shape == (2, 3)
    for a, b in zip((out, s, rstd), want):
        # another order of the additions: the rows are still within the count
        assert (a - b).abs().max() <= 100 * ref.U32 * b.abs().max()


def test_in_a_graph_and_on_a_given_stream():
    g = torch.Generator(device="cuda").manual_seed(7)
    x, res, w, go = normal(g, 40, 512), normal(g, 40, 512), normal(g, 512), normal(g, 40, 512)

    def both(stream=None):
        out, s, rstd, _ = pd.pdssm_add_rmsnorm_fwd(x, res, w, stream=stream)
        return (out, s, *pd.pdssm_add_rmsnorm_bwd(go, s, w, rstd, stream=stream))

    want = both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for v in held:
        v.fill_(0)
    graph.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = both(side)
    torch.cuda.synchronize()
    for a, b, c in zip(want, held, other):
        assert torch.equal(a, b) and torch.equal(a, c)
