"""GPU checks of the block operators as they are used together: the
differentiable forms, the decay layer (prompts, single tokens) and a stack of
selecting and decaying blocks over one residual stream, against the same
formulas in 64 bits or against the unfused path."""
import copy

import pytest
import torch

import block_ref as ref
import structured_sparse_state_b200 as pd
from structured_sparse_state_b200.layer import (DecayLayer, PDSSMLayer, ResidualStack, add_rmsnorm,
                                                decay_scan, select_balance)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def rel(a, b):
    return ((a.double() - b.double()).norm() / b.double().norm().clamp(min=1e-300)).item()


def rand(*s, seed=0, by=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*s, generator=g, device="cuda") * by


def decay_layer_64(layer, x, h0=None):
    """DecayLayer.forward in 64 bits, torch operations and autograd only."""
    xn = x / (x.square().mean(-1, keepdim=True) + torch.finfo(torch.float32).eps).sqrt() * layer.norm.weight
    c, b, v, log_a = layer._inputs(xn)
    B, L = x.shape[:2]
    rep = layer.H // layer.G
    c, b = c.repeat_interleave(rep, 2), b.repeat_interleave(rep, 2)
    S = x.new_zeros(B, layer.H, layer.N, layer.P) if h0 is None else h0
    ys = []
    for t in range(L):
        S = log_a[:, t].exp()[..., None, None] * S + b[:, t][..., None] * v[:, t][:, :, None, :]
        ys.append((c[:, t][..., None] * S).sum(-2))
    return x + layer.proj_out(torch.stack(ys, 1).flatten(-2)), S


def test_decay_layer_and_its_gradients():
    torch.manual_seed(0)
    layer = DecayLayer(96, 4, 32, 24, n_groups=2, device="cuda")
    big = copy.deepcopy(layer).double()
    big.state_dtype = torch.float64
    x = rand(2, 70, 96, seed=1).requires_grad_()
    xd = x.detach().double().requires_grad_()
    g = rand(2, 70, 96, seed=2)
    layer(x).backward(g)
    want, _ = decay_layer_64(big, xd)
    want.backward(g.double())
    # products of 96 terms in fp32 on both sides of a scan: 2^-24 times a few
    # hundred additions, in the norm
    assert rel(layer(x.detach()), want) < 400 * ref.U32
    assert rel(x.grad, xd.grad) < 400 * ref.U32
    for (name, p), q in zip(layer.named_parameters(), big.parameters()):
        assert rel(p.grad, q.grad) < 1000 * ref.U32, name


@pytest.mark.parametrize("state_dtype", [torch.float32, torch.bfloat16])
def test_prompt_then_single_tokens(state_dtype):
    """A served stream: the prompt by the scan, each further token by the step,
    gives what the scan gives over the whole."""
    torch.manual_seed(1)
    layer = DecayLayer(64, 4, 64, 32, n_groups=2, state_dtype=state_dtype, device="cuda")
    x = rand(3, 50, 64, seed=3)
    with torch.no_grad():
        whole, stream, last = layer.block(x)
        head, _, state = layer.block(x[:, :41].contiguous())
        pool = rand(5, 4, 64, 32, seed=4)
        slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
        pool[slots.long()] = state
        outs = [head]
        for t in range(41, 50):
            out, res = layer.step(x[:, t].contiguous(), None, pool, slots)
            assert torch.equal(res, x[:, t])
            outs.append(out[:, None])
    # bf16: y is rounded, and so are the scores and states behind it (2^-8 each)
    tol = 3 * ref.UBF if state_dtype == torch.bfloat16 else 400 * ref.U32
    assert rel(torch.cat(outs, 1), whole) < tol
    assert rel(pool[slots.long()], last) < 400 * ref.U32


def test_padded_prompts_stop_at_their_lengths():
    torch.manual_seed(2)
    layer = DecayLayer(64, 2, 16, 16, device="cuda")
    x = rand(2, 40, 64, seed=5)
    n = torch.tensor([40, 23], dtype=torch.int32, device="cuda")
    with torch.no_grad():
        _, _, state = layer.block(x, lengths=n)
        _, _, alone = layer.block(x[1:, :23].contiguous())
    # the projections' products run on other shapes: another order of additions
    assert rel(state[1:], alone) < 100 * ref.U32


def unfused(stack, x):
    for block in stack.blocks:
        x = block(x)
    return stack.norm(x)


def make_stack(state_dtype, seed=3):
    torch.manual_seed(seed)
    blocks = [PDSSMLayer(96, 4, 32, 8, d_select=64, chunk=64, state_dtype=state_dtype, device="cuda"),
              DecayLayer(96, 4, 32, 48, n_groups=2, state_dtype=state_dtype, device="cuda"),
              PDSSMLayer(96, 2, 16, 4, d_select=32, chunk=64, state_dtype=state_dtype, device="cuda")]
    return ResidualStack(blocks, 96, device="cuda")


def test_a_stack_equals_its_unfused_blocks():
    """Sums and norms in one pass against torch's, over selecting and decaying
    blocks: the same selections (else nothing below would be close), outputs and
    gradients within fp32 rounding."""
    stack = make_stack(torch.float32)
    x = rand(2, 130, 96, seed=6)
    g = rand(2, 130, 96, seed=7)
    out = stack(x)
    out.backward(g)
    grads = {n: p.grad.clone() for n, p in stack.named_parameters()}
    stack.zero_grad()
    want = unfused(stack, x)
    want.backward(g)
    assert rel(out, want) < 2000 * ref.U32
    for n, p in stack.named_parameters():
        assert rel(grads[n], p.grad) < 20000 * ref.U32, n


@pytest.mark.parametrize("state_dtype", [torch.float32, torch.bfloat16])
def test_a_training_step_of_the_stack(state_dtype):
    """Runs, with the balance loss, and reaches every parameter with finite
    gradients; the selections' weights get the balance's share."""
    stack = make_stack(state_dtype)
    x = rand(2, 200, 96, seed=8)
    out, balance = stack(x, balance=True)
    assert out.shape == x.shape and 1.0 - 1e-6 <= balance.item() <= 8.0
    (out.square().mean() + 0.1 * balance).backward()
    for n, p in stack.named_parameters():
        assert p.grad is not None and torch.isfinite(p.grad).all(), n
    with_balance = stack.blocks[0].W_sel.grad.clone()
    stack.zero_grad()
    stack(x).square().mean().backward()
    assert not torch.equal(with_balance, stack.blocks[0].W_sel.grad)


def test_a_whole_training_step_in_a_graph():
    """Forward, loss and backward captured once and replayed on new inputs
    give the eager step's gradients, bit for bit."""
    stack = make_stack(torch.bfloat16)
    x = rand(2, 150, 96, seed=9)

    def step():
        for p in stack.parameters():
            p.grad = None
        out, balance = stack(x, balance=True)
        (out.square().mean() + 0.1 * balance).backward()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for p in stack.parameters():
        p.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, balance = stack(x, balance=True)
        (out.square().mean() + 0.1 * balance).backward()
    held = {n: p.grad for n, p in stack.named_parameters()}
    x.copy_(rand(2, 150, 96, seed=10))
    graph.replay()
    torch.cuda.synchronize()
    got = {n: v.clone() for n, v in held.items()}
    del out, balance
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    for n, p in stack.named_parameters():
        assert torch.equal(got[n], p.grad), n


def test_missing_gradients_and_inference():
    x, w = rand(4, 64, seed=11).requires_grad_(), torch.ones(64, device="cuda", requires_grad=True)
    res = rand(4, 64, seed=12).requires_grad_()
    out, s = add_rmsnorm(x, res, w)
    s.sum().backward()                          # nothing reaches out
    assert (x.grad == 1).all() and (res.grad == 1).all() and w.grad is None
    x.grad = None
    out, s = add_rmsnorm(x, None, w)
    out.sum().backward()                        # nothing reaches the stream
    assert x.grad is not None and w.grad is not None
    c = rand(1, 2, 40, 16, seed=13).requires_grad_()
    v = rand(1, 2, 40, 16, seed=14)
    la = torch.full((2,), -0.1, device="cuda")
    y, last = decay_scan(c, c.detach(), v, la)
    last.sum().backward()                       # only the last state's gradient
    assert (c.grad == 0).all()                  # c does not reach the state
    with torch.no_grad():
        y2, _ = decay_scan(c, c, v, la)
    assert torch.equal(y, y2)
    u, W = rand(1, 30, 16, seed=15).requires_grad_(), rand(2, 4, 16, seed=16).requires_grad_()
    loss, counts, probs = select_balance(u, W)
    assert not counts.requires_grad and not probs.requires_grad
    loss.sum().backward()
    assert torch.isfinite(u.grad).all() and torch.isfinite(W.grad).all()


def test_blocks_and_steps_take_any_strides():
    """What forward accepts, block, step and a stack accept too: a token cut out
    of a batch, a transposed batch, and their gradients."""
    torch.manual_seed(4)
    layer = DecayLayer(64, 2, 16, 16, device="cuda")
    x = rand(3, 20, 64, seed=30)
    state = torch.zeros(3, 2, 16, 16, device="cuda")
    for t in range(3):
        a, s = state.clone(), state.clone()
        res = rand(3, 20, 64, seed=31)
        got = layer.step(x[:, t], res[:, t], a)
        want = layer.step(x[:, t].contiguous(), res[:, t].contiguous(), s)
        assert all(torch.equal(u, v) for u, v in zip(got, want)) and torch.equal(a, s)
        state = a
    xt = rand(20, 3, 64, seed=32).requires_grad_()
    xc = xt.detach().transpose(0, 1).contiguous().requires_grad_()
    for model in (layer, ResidualStack([layer], 64, device="cuda")):
        call = model.block if model is layer else (lambda v: (model(v),))
        got, want = call(xt.transpose(0, 1))[0], call(xc)[0]
        g = rand(*got.shape, seed=33)
        assert torch.equal(got, want)
        gt, = torch.autograd.grad(got, xt, g)
        gc, = torch.autograd.grad(want, xc, g)
        assert torch.equal(gt.transpose(0, 1), gc)


def calls_on_a_stream():
    """{name: (input, call of it on a stream)}, for two calls each."""
    x, w = rand(4096, 256, seed=20), rand(256, seed=21)
    rstd = x[:, 0].abs()
    k = torch.zeros(1, 2, 4096, dtype=torch.int32, device="cuda")
    W, c, log_a = rand(2, 4, 256, seed=22), rand(1, 1, 4096, 16, seed=23), -rand(4, seed=25).abs()
    token = c.view(4096, 1, 16)
    state = rand(4096, 4, 16, 64, seed=24)
    states = [state, state.clone()]
    return dict(
        norm=(x, lambda t, s: pd.pdssm_add_rmsnorm_fwd(t, None, w, stream=s)[0]),
        norm_backward=(x, lambda t, s: pd.pdssm_add_rmsnorm_bwd(t, x, w, rstd, stream=s)[0]),
        balance=(x.view(1, 4096, 256), lambda t, s: pd.pdssm_select_balance_fwd(t, W, k, stream=s)[2]),
        scan=(x.view(1, 4, 4096, 64), lambda t, s: pd.pdssm_decay_scan_fwd(c, c, t, log_a, stream=s)[0]),
        step=(x.view(4096, 4, 64), lambda t, s: pd.pdssm_decay_step(token, token, t, log_a, states.pop(), stream=s)))


@pytest.mark.parametrize("call", ["norm", "norm_backward", "balance", "scan", "step"])
def test_an_input_dropped_after_a_call_on_another_stream(call):
    """Its memory is not handed out again while that stream has yet to read it."""
    src, run = calls_on_a_stream()[call]
    want = run(src, None)
    side = torch.cuda.Stream()
    t = src.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)          # about 50 ms
    got = run(t, side)
    del t
    others = [torch.full_like(src, float("nan")) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(others) == 3


@pytest.mark.parametrize("call", ["norm", "norm_backward", "balance", "scan"])
def test_a_given_stream_inside_a_capture(call):
    """stream= named in a captured call, its inputs dropped before the replay of
    what it made from them."""
    src, run = calls_on_a_stream()[call]
    want = run(src, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t = src * 1.0
        got = run(t, torch.cuda.current_stream())
        del t
        later = torch.full_like(src, float("nan"))
    got.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.isnan(later).all()


@pytest.mark.parametrize("call", ["norm", "norm_backward", "balance", "scan"])
def test_calls_from_several_threads(call):
    """Each thread on a stream of its own, at the same time."""
    import threading

    src, run = calls_on_a_stream()[call]
    want, got, start = run(src, None), [None] * 4, threading.Barrier(4)
    torch.cuda.synchronize()

    def work(i):
        side = torch.cuda.Stream()
        start.wait()
        for _ in range(20):
            got[i] = run(src, side)
        side.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for g in got:
        assert torch.equal(g, want)
