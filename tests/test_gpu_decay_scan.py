"""GPU checks of the decay scan (linear attention with a decay for each head):
forward, adjoint and single step against a step-by-step 64-bit implementation,
with counted error bounds (tests/block_ref.py)."""
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


BF, F32 = torch.bfloat16, torch.float32

# dtype, B, H, G, L, N, P, layout, decay, h0, ragged
CASES = [
    (F32, 1, 1, 1, 1, 1, 1, "bhl", "step", True, False),
    (F32, 2, 3, 3, 31, 12, 20, "bhl", "head", False, False),
    (F32, 2, 2, 1, 32, 32, 32, "blh", "step", True, False),
    (F32, 3, 4, 2, 33, 33, 17, "blh", "step", True, True),
    (F32, 1, 2, 2, 700, 64, 48, "bhl", "step", True, False),
    (F32, 2, 2, 2, 130, 128, 100, "bhl", "head", True, True),
    (F32, 1, 1, 1, 1500, 16, 128, "blh", "step", False, False),
    (BF, 1, 1, 1, 1, 64, 64, "bhl", "step", True, False),
    (BF, 2, 3, 3, 63, 64, 64, "bhl", "step", True, False),
    (BF, 2, 2, 2, 64, 32, 64, "blh", "head", False, False),
    (BF, 2, 4, 1, 65, 64, 32, "blh", "step", True, True),
    (BF, 1, 2, 2, 1100, 64, 64, "bhl", "step", True, False),
    (BF, 3, 2, 2, 257, 31, 63, "bhl", "step", True, True),
    (BF, 1, 4, 2, 300, 128, 64, "blh", "step", True, False),
    (BF, 2, 2, 2, 200, 64, 128, "bhl", "head", True, True),
    (BF, 1, 2, 1, 513, 128, 128, "bhl", "step", False, False),
    (BF, 1, 1, 1, 3000, 48, 40, "bhl", "step", True, False),
    # widths in different units of 32 and 64, several segments, odd widths
    (F32, 1, 2, 2, 300, 128, 32, "bhl", "step", True, False),
    (F32, 2, 2, 1, 250, 40, 128, "blh", "step", True, True),
    (F32, 1, 3, 3, 140, 24, 50, "bhl", "head", False, False),
    (BF, 2, 4, 2, 1500, 100, 72, "blh", "step", True, True),
    (BF, 1, 2, 2, 1300, 128, 128, "bhl", "head", True, False),
    (BF, 1, 2, 1, 1200, 65, 31, "blh", "step", True, False),
    (BF, 2, 2, 2, 700, 17, 127, "bhl", "step", False, True),
    (BF, 3, 3, 1, 1, 1, 1, "blh", "head", True, False),
    (BF, 1, 2, 2, 640, 64, 9, "blh", "step", True, False),
]


def make(dtype, B, H, G, L, N, P, layout, decay, h0, ragged, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s, dtype=F32, by=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * by).to(dtype)

    keys, vals, gate = ((B, G, L, N), (B, H, L, P), (B, H, L)) if layout == "bhl" else \
        ((B, L, G, N), (B, L, H, P), (B, L, H))
    t = dict(c=normal(*keys, dtype=dtype), b=normal(*keys, dtype=dtype, by=N ** -0.5),
             x=normal(*vals, dtype=dtype))
    if decay == "head":
        t["log_a"] = -torch.rand(H, generator=g, device="cuda") * 0.3
    else:
        t["log_a"] = -torch.nn.functional.softplus(normal(*gate) - 3.0)
    t["h0"] = normal(B, H, N, P) if h0 else None
    t["lengths"] = None
    if ragged:
        n = torch.randint(0, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        n[-1] = 0
        t["lengths"] = n
    t["g_y"] = normal(*vals, dtype=dtype)
    t["g_hlast"] = normal(B, H, N, P) if h0 else None
    return t


def within(name, got, want, bound):
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all(), name
    worst = (err - bound).max().item() if err.numel() else 0.0
    assert worst <= 0, f"{name}: off by {err.max().item():.3g}, {worst:.3g} more than counted"


def check_all(t, got, layout, names):
    args = (t["c"], t["b"], t["x"], t["log_a"], t["h0"], t["lengths"], layout)
    grads = "g_c" in names
    extra = (t["g_y"], t["g_hlast"]) if grads else (None, None)
    want = ref.decay_scan(*args, *extra)
    mag = ref.decay_scan(*args, *extra, magnitudes=True)
    N, P = t["c"].shape[-1], t["x"].shape[-1]
    L = t["x"].shape[2 if layout == "bhl" else 1]
    # bf16: a score or a state is rounded on the way to an output, and the
    # decayed weights of a score at most once more
    bound = ref.decay_bounds(t["x"].dtype, N, P, L, mag, 2)
    for name in names:
        b = bound[name]
        if isinstance(b, tuple):
            m, whole, tol = b
            w = whole[:, :, None] if layout == "bhl" else whole[:, None, :]
            b = tol * m + w + 1e-37
        within(name, got[name], want[name], b)


def fwd_bwd(t, layout):
    y, h_last, ws = pd.pdssm_decay_scan_fwd(t["c"], t["b"], t["x"], t["log_a"], t["h0"],
                                            lengths=t["lengths"], layout=layout, for_bwd=True)
    g = pd.pdssm_decay_scan_bwd(t["c"], t["b"], t["x"], t["log_a"], t["h0"], t["g_y"], ws,
                                g_hlast=t["g_hlast"], lengths=t["lengths"], layout=layout)
    return dict(y=y, h_last=h_last, g_c=g[0], g_b=g[1], g_x=g[2], g_log_a=g[3], g_h0=g[4])


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_forward(case):
    t = make(*case)
    y, h_last, _ = pd.pdssm_decay_scan_fwd(t["c"], t["b"], t["x"], t["log_a"], t["h0"],
                                           lengths=t["lengths"], layout=case[7])
    check_all(t, dict(y=y, h_last=h_last), case[7], ("y", "h_last"))


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_forward_and_adjoint(case):
    t = make(*case, seed=1)
    check_all(t, fwd_bwd(t, case[7]), case[7],
              ("y", "h_last", "g_c", "g_b", "g_x", "g_log_a", "g_h0"))


# The counted bounds above are sums of worst cases.  These are of a result's norm,
# in units of 2^-24, and tight enough that a lost bf16 part of a split operand
# shows (two parts of three: each rounding leaves (1 / sqrt 12) 2^-7 / 1.36 =
# 1.66e-3 in the mean square, so 2.7e-6 of the operand).
#   last state, bf16: the largest part's eight additions of a chunk, truncated (2
#   units each at most), decay of a step (ex2: 4, its argument: 4), split, sum: 26
#   first state's gradient, bf16: twelve such additions (three parts of four), 34
#   fp32: 32 additions of a chunk, decay and sum, 40
STATE_UNITS = {("h_last", BF): 26, ("g_h0", BF): 34, ("h_last", F32): 40, ("g_h0", F32): 40}
#   g_log_a: 128 additions over a width, 32 over a chunk, 8 around them; and a
#   chunk's pairs that do not straddle the step cancel (twice as many at most)
DECAY_UNITS = 2 * 168

NORMS = [
    (BF, 1, 2, 2, 1100, 64, 64, "bhl", "step", True, False),
    (BF, 2, 4, 2, 1500, 100, 72, "blh", "step", True, True),
    (BF, 1, 2, 2, 1300, 128, 128, "bhl", "step", True, False),
    (BF, 1, 1, 1, 3000, 48, 40, "bhl", "step", True, False),
    (BF, 1, 2, 1, 513, 128, 128, "bhl", "step", True, False),
    (F32, 1, 1, 1, 1500, 16, 128, "blh", "step", True, False),
    (F32, 1, 2, 2, 700, 64, 48, "bhl", "step", True, False),
    (F32, 2, 2, 2, 330, 128, 100, "bhl", "step", True, False),
]


def heads_of(v, layout):
    """[B, H, L] of a per-step log decay's gradient."""
    return v.double() if layout == "bhl" else v.double().transpose(1, 2)


@pytest.mark.parametrize("case", NORMS, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_states_and_decay_gradients_in_norm(case):
    dtype, layout = case[0], case[7]
    t = make(*case, seed=15)
    got = fwd_bwd(t, layout)
    want = ref.decay_scan(t["c"], t["b"], t["x"], t["log_a"], t["h0"], t["lengths"], layout, t["g_y"], t["g_hlast"])
    for n in ("h_last", "g_h0"):
        err = (got[n].double() - want[n]).norm() / want[n].norm()
        assert err <= STATE_UNITS[n, dtype] * ref.U32, (n, err.item() / ref.U32)
    a, w = heads_of(got["g_log_a"], layout), heads_of(want["g_log_a"], layout)
    err, size = (a - w).norm(dim=-1), w.norm(dim=-1)
    assert (err <= DECAY_UNITS * ref.U32 * size).all(), (err / size).max().item() / ref.U32
    live = torch.full((case[1],), case[4], device="cuda") if t["lengths"] is None else t["lengths"]
    assert (size[live > 0] > 0).all()       # nothing but an empty sequence's could be zero


@pytest.mark.parametrize("dtype,L,N,P", [(BF, 1300, 128, 128), (BF, 1100, 64, 64), (F32, 1100, 32, 48)], ids=str)
def test_decays_gradient_of_a_head_against_its_steps_and_differences(dtype, L, N, P):
    """A decay for each head over several segments: the sum of the steps'
    gradients, and the difference of the loss in 64 bits."""
    t = make(dtype, 2, 3, 3, L, N, P, "bhl", "head", True, True, seed=16)
    got = fwd_bwd(t, "bhl")["g_log_a"].double()

    def at(h):
        la = t["log_a"].double() + h
        return ref.decay_scan(t["c"], t["b"], t["x"], la[None, :, None].expand(2, 3, L), t["h0"], t["lengths"], "bhl",
                              t["g_y"], t["g_hlast"])

    steps = at(0.0)["g_log_a"]
    bound = DECAY_UNITS * ref.U32 * steps.abs().sum((0, 2))
    want = steps.sum((0, 2))
    assert ((got - want).abs() <= bound).all()
    assert (want.abs() > bound).all()       # a zero would not pass

    def loss(h):
        o = at(h)
        return ((o["y"] * t["g_y"].double()).sum((0, 2, 3)) + (o["h_last"] * t["g_hlast"].double()).sum((0, 2, 3)))

    h = 1e-5        # a head's loss depends on its own decay alone
    numeric = (loss(h) - loss(-h)) / (2 * h)
    # the difference's own error: h^2 / 6 of a third derivative, of at most (1 / (1 - a))^2 the first's
    memory = (1 / (1 - t["log_a"].double().exp())).clamp(max=L)
    assert ((got - numeric).abs() <= bound + h * h * memory ** 2 * steps.abs().sum((0, 2)) + 1e-9 * numeric.abs()).all()


@pytest.mark.parametrize("widths", [(64, 64), (31, 63), (128, 64), (96, 128)], ids=str)
@pytest.mark.parametrize("L", [1, 15, 33, 62, 95, 97, 126, 161, 287])
def test_the_last_rows_of_a_tile(L, widths):
    """Sequences that end inside a warp's 32 rows, at every width of the
    tensor-core kernels."""
    t = make(BF, 1, 2, 1, L, *widths, "blh", "step", True, False, seed=L)
    check_all(t, fwd_bwd(t, "blh"), "blh", ("y", "h_last", "g_c", "g_b", "g_x", "g_log_a", "g_h0"))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_adjoint_against_differences(dtype):
    """<g, dx> against (f(x + dx) - f(x - dx)) / 2 in 64 bits on a direction of
    the inputs: the adjoint is that of the definition, not only of the
    reference's formulas."""
    case = (dtype, 1, 2, 1, 97, 24, 40, "bhl", "step", True, False)
    t = make(*case, seed=2)
    got = fwd_bwd(t, "bhl")
    g = torch.Generator(device="cuda").manual_seed(5)
    names = ("c", "b", "x", "log_a", "h0")
    d = {n: torch.randn(t[n].shape, generator=g, device="cuda", dtype=torch.float64) for n in names}

    def loss(h):
        v = {n: t[n].double() + h * d[n] for n in names}
        o = ref.decay_scan(v["c"], v["b"], v["x"], v["log_a"], v["h0"], None, "bhl")
        return ((o["y"] * t["g_y"].double()).sum() + (o["h_last"] * t["g_hlast"].double()).sum()).item()

    h = 1e-5
    numeric = (loss(h) - loss(-h)) / (2 * h)
    mags = {n: (got["g_" + n].double().abs() * d[n].abs()).sum().item() for n in names}
    analytic = sum((got["g_" + n].double() * d[n]).sum().item() for n in names)
    # each gradient element within its counted bound; here their sum
    tol = (3 * ref.UBF if dtype == BF else 0) + 400 * ref.U32
    assert abs(analytic - numeric) <= tol * sum(mags.values()) + 1e-6 * abs(numeric)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_minus_infinity_separates_packed_sequences(dtype):
    """Sequences packed one behind another with log_a = -inf at each first
    step give what they give alone, forward and backward."""
    cuts = [0, 1, 40, 104, 168, 230]
    t = make(dtype, 1, 2, 2, cuts[-1], 32, 32, "bhl", "step", False, False, seed=3)
    t["log_a"][:, :, cuts[:-1]] = -math.inf
    got = fwd_bwd(t, "bhl")
    for lo, hi in zip(cuts, cuts[1:]):
        part = {n: (v[:, :, lo:hi].contiguous() if v is not None and n != "h0" and v.dim() >= 3 else None)
                for n, v in t.items()}
        part["h0"] = part["g_hlast"] = part["lengths"] = None
        want = ref.decay_scan(part["c"], part["b"], part["x"], part["log_a"], None, None, "bhl", part["g_y"])
        mag = ref.decay_scan(part["c"], part["b"], part["x"], part["log_a"], None, None, "bhl", part["g_y"],
                             magnitudes=True)
        bound = ref.decay_bounds(dtype, 32, 32, cuts[-1], mag, 2)
        for n in ("y", "g_c", "g_b", "g_x"):
            within(n, got[n][:, :, lo:hi], want[n], bound[n])
    assert (got["g_log_a"][:, :, cuts[:-1]] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_strong_and_absent_decay(dtype):
    t = make(dtype, 1, 3, 3, 200, 16, 16, "bhl", "step", True, False, seed=4)
    t["log_a"][:, 0] = 0.0                  # a = 1: plain linear attention
    t["log_a"][:, 1] = -150.0               # each step forgets what went before
    t["log_a"][:, 2] = -9.0
    check_all(t, fwd_bwd(t, "bhl"), "bhl", ("y", "h_last", "g_c", "g_b", "g_x", "g_log_a", "g_h0"))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_growing_states(dtype):
    """log_a of either sign, and a head that grows by e^77 over a chunk."""
    t = make(dtype, 1, 3, 3, 300, 32, 64, "bhl", "step", True, False, seed=17)
    g = torch.Generator(device="cuda").manual_seed(18)
    t["log_a"] = 0.3 * torch.randn(1, 3, 300, generator=g, device="cuda")
    t["log_a"][:, 1] = -0.6
    t["log_a"][:, 1, 128:256] = 0.6
    t["log_a"][:, 2] = 0.05
    check_all(t, fwd_bwd(t, "bhl"), "bhl", ("y", "h_last", "g_c", "g_b", "g_x", "g_log_a", "g_h0"))


def test_the_status_of_a_scan_of_no_steps():
    t = make(BF, 2, 2, 1, 0, 8, 8, "blh", "head", True, False)
    ws = torch.full((1 << 16,), 255, dtype=torch.uint8, device="cuda")
    pd.pdssm_decay_scan_fwd(t["c"], t["b"], t["x"], t["log_a"], t["h0"], layout="blh", ws=ws)
    assert pd.pdssm_ws_status(ws) == 0


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("layout", ["bhl", "blh"])
def test_nothing_behind_a_length_is_read(dtype, layout):
    t = make(dtype, 3, 2, 2, 150, 64, 64, layout, "step", True, False, seed=5)
    t["lengths"] = torch.tensor([0, 64, 101], dtype=torch.int32, device="cuda")
    clean = fwd_bwd(t, layout)
    axis = 2 if layout == "bhl" else 1
    behind = torch.arange(150, device="cuda") >= t["lengths"][:, None]
    for n in ("c", "b", "x", "g_y", "log_a"):
        v = t[n]
        m = behind[:, None] if axis == 2 else behind[:, :, None]
        m = m[..., None] if v.dim() == 4 else m
        t[n] = torch.where(m, torch.full((), math.nan, dtype=v.dtype, device="cuda"), v).contiguous()
    got = fwd_bwd(t, layout)
    for n in clean:
        assert torch.equal(got[n], clean[n]), n
    y = got["y"] if layout == "bhl" else got["y"].transpose(1, 2)
    assert (y[0] == 0).all() and (y[1, :, 64:] == 0).all() and (y[2, :, 101:] == 0).all()
    assert torch.equal(got["h_last"][0], t["h0"][0])
    # lengths beyond L count as L, negative ones as 0
    t2 = make(dtype, 2, 2, 2, 70, 32, 32, layout, "step", True, False, seed=6)
    t2["lengths"] = torch.tensor([1000, -5], dtype=torch.int32, device="cuda")
    a = fwd_bwd(t2, layout)
    t2["lengths"] = torch.tensor([70, 0], dtype=torch.int32, device="cuda")
    b = fwd_bwd(t2, layout)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_no_steps():
    for layout in ("bhl", "blh"):
        t = make(F32, 2, 2, 1, 0, 8, 8, layout, "head", True, False)
        got = fwd_bwd(t, layout)
        assert torch.equal(got["h_last"], t["h0"]) and torch.equal(got["g_h0"], t["g_hlast"])
        assert (got["g_log_a"] == 0).all() and got["y"].numel() == 0
    y, h_last, _ = pd.pdssm_decay_scan_fwd(t["c"], t["b"], t["x"], t["log_a"], layout=layout)
    assert (h_last == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_same_bits_again_and_on_other_streams_and_graphs(dtype):
    t = make(dtype, 2, 4, 2, 700, 64, 64, "blh", "head", True, False, seed=7)
    first = fwd_bwd(t, "blh")
    again = fwd_bwd(t, "blh")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = fwd_bwd(t, "blh")
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = fwd_bwd(t, "blh")
    for v in held.values():
        v.fill_(0)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for n in first:
        assert torch.equal(first[n], again[n]), n
        assert torch.equal(first[n], other[n]), n
        assert torch.equal(first[n], held[n]), n


def test_the_adjoint_may_run_twice_on_one_workspace():
    t = make(BF, 1, 2, 2, 900, 64, 64, "bhl", "step", True, False, seed=8)
    y, h_last, ws = pd.pdssm_decay_scan_fwd(t["c"], t["b"], t["x"], t["log_a"], t["h0"], for_bwd=True)
    a = pd.pdssm_decay_scan_bwd(t["c"], t["b"], t["x"], t["log_a"], t["h0"], t["g_y"], ws)
    b = pd.pdssm_decay_scan_bwd(t["c"], t["b"], t["x"], t["log_a"], t["h0"], t["g_y"], ws)
    for u, v in zip(a, b):
        assert torch.equal(u, v)


def test_a_given_stream_owns_the_call():
    t = make(BF, 1, 2, 2, 300, 64, 64, "bhl", "step", True, False, seed=9)
    want = fwd_bwd(t, "bhl")["y"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, _, _ = pd.pdssm_decay_scan_fwd(t["c"], t["b"], t["x"], t["log_a"], t["h0"], stream=side)
    side.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("offset", [1, 2, 3])
def test_pointers_off_the_16_byte_grid(offset):
    """Contiguous tensors that start inside a storage."""
    t = make(BF, 1, 2, 2, 130, 64, 64, "bhl", "step", True, False, seed=10)
    want = fwd_bwd(t, "bhl")
    for n in ("c", "b", "x", "g_y"):
        room = torch.empty(t[n].numel() + 8, dtype=BF, device="cuda")
        v = room[offset:offset + t[n].numel()].view(t[n].shape)
        v.copy_(t[n])
        t[n] = v
    got = fwd_bwd(t, "bhl")
    for n in want:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("offset", [1, 2, 3])
@pytest.mark.parametrize("case", [
    (BF, 1, 2, 2, 130, 64, 64, "bhl", "step", True, False), (BF, 2, 2, 1, 130, 128, 100, "blh", "head", True, True),
    (BF, 1, 1, 1, 1100, 32, 64, "bhl", "step", True, False), (BF, 1, 2, 2, 1, 16, 4, "blh", "step", True, False),
    (F32, 1, 2, 2, 130, 64, 64, "bhl", "step", True, False), (F32, 1, 2, 1, 300, 40, 96, "blh", "head", True, True)],
    ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_every_buffer_off_the_16_byte_grid(case, offset):
    """Inputs, states and the caller's own outputs that start inside a storage,
    each 1 to 3 values off: the same bits, and nothing around them is written."""
    t, layout = make(*case, seed=13), case[7]
    want = fwd_bwd(t, layout)

    def off(v, fill=None):
        room = torch.full((v.numel() + 8,), 7.0, dtype=v.dtype, device="cuda")
        at = room[offset:offset + v.numel()].view(v.shape)
        at.copy_(v) if fill is None else at.fill_(fill)
        return room, at

    moved = {n: v if v is None or n == "lengths" else off(v)[1] for n, v in t.items()}
    rooms = {n: off(v, math.nan) for n, v in want.items()}
    out = {n: v[1] for n, v in rooms.items()}
    _, _, ws = pd.pdssm_decay_scan_fwd(*(moved[n] for n in ("c", "b", "x", "log_a", "h0")), lengths=t["lengths"],
                                       layout=layout, for_bwd=True, y=out["y"], h_last=out["h_last"])
    pd.pdssm_decay_scan_bwd(*(moved[n] for n in ("c", "b", "x", "log_a", "h0", "g_y")), ws, g_hlast=moved["g_hlast"],
                            lengths=t["lengths"], layout=layout,
                            out=[out[n] for n in ("g_c", "g_b", "g_x", "g_log_a", "g_h0")])
    for n in want:
        assert torch.equal(out[n], want[n]), n
        room = rooms[n][0]
        assert (room[:offset] == 7).all() and (room[offset + want[n].numel():] == 7).all(), n


def test_odd_widths_at_other_addresses_in_the_adjoint():
    """The adjoint of rows of odd width, with inputs that the forward saw at
    addresses off the 16-byte grid."""
    t = make(BF, 2, 2, 1, 130, 31, 24, "blh", "step", True, False, seed=12)
    want = fwd_bwd(t, "blh")
    moved = dict(t)
    for n in ("c", "b", "x"):
        room = torch.empty(t[n].numel() + 8, dtype=BF, device="cuda")
        moved[n] = room[1:1 + t[n].numel()].view(t[n].shape)
        moved[n].copy_(t[n])
    y, _, ws = pd.pdssm_decay_scan_fwd(moved["c"], moved["b"], moved["x"], t["log_a"], t["h0"],
                                       layout="blh", for_bwd=True)
    assert torch.equal(y, want["y"])
    g = pd.pdssm_decay_scan_bwd(t["c"], t["b"], t["x"], t["log_a"], t["h0"], t["g_y"], ws,
                                g_hlast=t["g_hlast"], layout="blh")
    for got, n in zip(g, ("g_c", "g_b", "g_x", "g_log_a", "g_h0")):
        assert torch.equal(got, want[n]), n


@pytest.mark.parametrize("N,L,for_bwd", [(64, 200, False), (128, 200, True), (64, 1100, True)])
def test_a_wait_that_gives_up_leaves_no_result(N, L, for_bwd):
    """Copies held back: the status word says so, and y, the last state and the
    states for the adjoint are NaN (one segment, and two); the context stays
    usable."""
    st, y, h_last, ws = pd.pdssm_decay_wait_selftest(1, 2, L, N, for_bwd)
    assert st == 5 and torch.isnan(y).all() and torch.isnan(h_last).all()
    t = make(BF, 1, 2, 2, L, N, N, "bhl", "step", False, False, seed=14)
    if for_bwd:         # a gradient that rests on a state is NaN too (the first 64 steps' rest on none)
        g = pd.pdssm_decay_scan_bwd(t["c"], t["b"], t["x"], t["log_a"], None, t["g_y"], ws)
        assert torch.isnan(g[0][:, :, 64:]).all()
    check_all(t, fwd_bwd(t, "bhl"), "bhl", ("y", "h_last", "g_c", "g_b", "g_x", "g_log_a", "g_h0"))


# ----------------------------------------------------------------------------
# single tokens
# ----------------------------------------------------------------------------
STEPS = [
    # dtype, B, S, H, G, N, P, decay
    (F32, 1, 1, 1, 1, 1, 1, "step"),
    (F32, 3, 5, 4, 2, 12, 20, "head"),
    (BF, 7, 9, 3, 1, 64, 64, "step"),
    (BF, 130, 140, 2, 2, 32, 63, "step"),
    (BF, 2, 2, 2, 2, 128, 128, "head"),
    (F32, 4, 4, 2, 2, 100, 7, "step"),
    # several heads per CTA, the last one with fewer
    (F32, 5, 6, 7, 7, 8, 16, "step"),
    (BF, 9, 9, 18, 6, 16, 64, "step"),
    (F32, 2, 3, 40, 8, 1, 4, "head"),
    (BF, 3, 5, 33, 11, 16, 8, "head"),
    (F32, 2, 2, 9, 3, 5, 3, "step"),
    (BF, 600, 601, 3, 3, 16, 64, "step"),
]


def make_step(dtype, B, S, H, G, N, P, decay, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    la = -torch.rand(*((B, H) if decay == "step" else (H,)), generator=g, device="cuda")
    slots = torch.randperm(S, generator=g, device="cuda")[:B].to(torch.int32)
    return dict(c=r(B, G, N).to(dtype), b=r(B, G, N).to(dtype), x=r(B, H, P).to(dtype), log_a=la,
                state=r(S, H, N, P), slots=slots)


def step_ref(t, magnitudes=False):
    f = torch.abs if magnitudes else (lambda v: v)
    B, H, P = t["x"].shape
    rep = H // t["c"].shape[1]
    state = f(t["state"].double()).clone()
    y = torch.zeros(B, H, P, dtype=torch.float64, device="cuda")
    a = t["log_a"].double().exp().expand(B, H)
    seen = set()
    for r, s in enumerate(t["slots"].tolist()):
        if not 0 <= s < state.shape[0] or s in seen:
            continue
        seen.add(s)
        b, c = (f(t[n][r].double()).repeat_interleave(rep, 0) for n in ("b", "c"))
        state[s] = a[r, :, None, None] * state[s] + b[..., None] * f(t["x"][r].double())[:, None, :]
        y[r] = (c[..., None] * state[s]).sum(1)
    return y, state


@pytest.mark.parametrize("case", STEPS, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
@pytest.mark.parametrize("empty", [False, True])
def test_step(case, empty):
    t = make_step(*case)
    if empty:
        t["slots"][0] = -1
        t["slots"][-1] = t["state"].shape[0]
        if len(t["slots"]) > 3:
            t["slots"][2] = t["slots"][1]           # the earlier row has it
    want_y, want_s = step_ref(t)
    mag_y, mag_s = step_ref(t, True)
    y = pd.pdssm_decay_step(t["c"], t["b"], t["x"], t["log_a"], t["state"], t["slots"])
    # a state element: two products, an addition, the decay; y: N additions
    within("state", t["state"], want_s, 8 * ref.U32 * mag_s)
    within("y", y, want_y, ((case[5] + 16) * ref.U32 + ref.unit(case[0])) * mag_y)


def test_step_without_slots_and_in_a_graph():
    t = make_step(BF, 6, 8, 4, 2, 64, 64, "step")
    t["slots"] = torch.arange(6, dtype=torch.int32, device="cuda")
    start = t["state"].clone()
    y0 = pd.pdssm_decay_step(t["c"], t["b"], t["x"], t["log_a"], t["state"], t["slots"])
    after = t["state"].clone()
    t["state"].copy_(start)
    y1 = pd.pdssm_decay_step(t["c"], t["b"], t["x"], t["log_a"], t["state"])
    assert torch.equal(y0, y1) and torch.equal(after, t["state"])
    assert torch.equal(after[6:], start[6:])
    t["state"].copy_(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2 = pd.pdssm_decay_step(t["c"], t["b"], t["x"], t["log_a"], t["state"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y0, y2) and torch.equal(after, t["state"])


def test_step_resets_on_minus_infinity():
    t = make_step(F32, 2, 2, 2, 2, 16, 16, "step")
    t["log_a"][:] = -math.inf
    t["slots"] = torch.arange(2, dtype=torch.int32, device="cuda")
    pd.pdssm_decay_step(t["c"], t["b"], t["x"], t["log_a"], t["state"])
    assert torch.equal(t["state"], t["b"][..., None] * t["x"][:, :, None, :])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_steps_continue_a_prompt(dtype):
    """A prompt by the scan, then tokens by the step: what the scan gives for
    the whole."""
    L, cut = 90, 77
    t = make(dtype, 2, 4, 2, L, 64, 48, "blh", "step", True, False, seed=11)
    head = lambda v: v[:, :cut].contiguous()  # noqa: E731
    y, state, _ = pd.pdssm_decay_scan_fwd(head(t["c"]), head(t["b"]), head(t["x"]), head(t["log_a"]),
                                          t["h0"], layout="blh")
    ys = [y]
    for i in range(cut, L):
        at = lambda v: v[:, i].contiguous()  # noqa: E731
        ys.append(pd.pdssm_decay_step(at(t["c"]), at(t["b"]), at(t["x"]), at(t["log_a"]), state)[:, None])
    check_all(t, dict(y=torch.cat(ys, 1), h_last=state), "blh", ("y", "h_last"))
