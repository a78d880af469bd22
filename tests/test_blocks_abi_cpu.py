"""Host-side checks of the operators around the scan that need no GPU: what
their C entry points and their binding refuse, before anything is launched."""
import ctypes

import pytest
import torch

import structured_sparse_state_b200 as pd

P = ctypes.c_void_p(4096)
BIG = 1 << 40


def dd(**kw):
    d = dict(B=2, H=4, G=2, L=100, N=16, P=24)
    d.update(kw)
    return pd.DecayDims(**d)


def decay_fwd(dm, dtype=0, layout=0, c=P, log_a=P, y=P, ws=P, ws_bytes=BIG, for_bwd=0):
    return pd.lib().pdssm_decay_scan_fwd(ctypes.byref(dm) if dm else None, c, P, P, dtype, layout, log_a, 1, None,
                                         None, y, None, for_bwd, ws, ws_bytes, None)


BAD_SIZES = [(dict(B=0), 1), (dict(H=0), 1), (dict(G=0), 1), (dict(G=3), 1), (dict(L=-1), 1), (dict(N=0), 1),
             (dict(P=0), 1), (dict(N=129), 2), (dict(P=129), 2), (dict(B=1 << 30), 2), (dict(L=1 << 40), 2)]


@pytest.mark.parametrize("bad,code", BAD_SIZES)
def test_decay_scan_refuses_sizes(bad, code):
    dm = dd(**bad)
    assert decay_fwd(dm) == code and pd.last_error() != ""
    assert pd.lib().pdssm_decay_workspace_bytes(ctypes.byref(dm), 0, 0) == 0
    st = pd.lib().pdssm_decay_scan_bwd(ctypes.byref(dm), P, P, P, 0, 0, P, 1, None, None, P, None, P, P, P, P, None,
                                       P, BIG, None)
    assert st == code


def test_decay_scan_refuses_arguments():
    dm = dd()
    assert decay_fwd(None) == 1
    assert decay_fwd(dm, dtype=2) == 1 and decay_fwd(dm, dtype=9) == 1
    assert decay_fwd(dm, layout=2) == 1 and "layout" in pd.last_error()
    assert decay_fwd(dm, c=None) == 1
    assert decay_fwd(dm, log_a=None) == 1
    assert decay_fwd(dm, y=None) == 1
    assert decay_fwd(dm, ws=None) == 1
    assert decay_fwd(dm, ws=ctypes.c_void_p(4096 + 128)) == 1 and "aligned" in pd.last_error()
    need = pd.pdssm_decay_workspace_bytes(2, 4, 2, 100, 16, 24, for_bwd=True)
    assert decay_fwd(dm, ws_bytes=need - 1, for_bwd=1) == 6
    lib = pd.lib()

    def bwd(g_c=P, g_la=P, ws_bytes=BIG):
        return lib.pdssm_decay_scan_bwd(ctypes.byref(dm), P, P, P, 0, 0, P, 1, None, None, P, None, g_c, P, P, g_la,
                                        None, P, ws_bytes, None)

    assert bwd(g_c=None) == 1 and bwd(g_la=None) == 1
    assert bwd(ws_bytes=pd.pdssm_decay_workspace_bytes(2, 4, 2, 100, 16, 24)) == 6     # the plain forward's


def test_decay_workspace_grows_as_documented():
    small = pd.pdssm_decay_workspace_bytes(2, 4, 4, 4096, 64, 64, torch.bfloat16)
    back = pd.pdssm_decay_workspace_bytes(2, 4, 4, 4096, 64, 64, torch.bfloat16, for_bwd=True)
    shared = pd.pdssm_decay_workspace_bytes(2, 4, 2, 4096, 64, 64, torch.bfloat16, for_bwd=True)
    assert 0 < small < back < shared
    assert pd.pdssm_decay_workspace_bytes(1, 1, 1, 0, 1, 1) > 0
    with pytest.raises(pd.PdssmError):
        pd.pdssm_decay_workspace_bytes(1, 1, 1, 10, 200, 1)


def test_decay_step_refuses_arguments():
    lib = pd.lib()

    def step(dm, c=P, state=P, n=8, slots=P, y=P, la=P, dtype=0):
        return lib.pdssm_decay_step(ctypes.byref(dm), c, P, P, dtype, la, 1, state, n, slots, y, None)

    for bad, code in BAD_SIZES:
        if "L" not in bad:
            assert step(dd(**bad)) == code
    dm = dd()
    assert step(dm, c=None) == 1 and step(dm, y=None) == 1 and step(dm, la=None) == 1 and step(dm, dtype=2) == 1
    assert step(dm, state=None) == 1
    assert step(dm, n=-1) == 1 and step(dm, n=1 << 40) == 1
    assert step(dm, n=1, slots=None) == 1 and "n_slots" in pd.last_error()


def test_add_rmsnorm_refuses_arguments():
    lib = pd.lib()

    def fwd(rows=4, D=64, x=P, xt=0, rt=0, wt=0, eps=1e-6, out=P, ot=0, scale=None, w=P):
        return lib.pdssm_add_rmsnorm_fwd(rows, D, x, xt, P, rt, w, wt, eps, out, ot, P, P, scale, None)

    assert fwd(rows=-1) == 1 and fwd(D=0) == 1
    assert fwd(D=16385) == 2 and fwd(rows=1 << 31) == 2
    assert fwd(x=None) == 1 and fwd(out=None) == 1 and fwd(w=None) == 1
    assert fwd(xt=2) == 1 and fwd(rt=2) == 1 and fwd(wt=5) == 1 and fwd(ot=3) == 1
    assert fwd(eps=-1.0) == 1 and fwd(eps=float("nan")) == 1 and fwd(eps=float("inf")) == 1
    assert fwd(ot=2) == 1 and "scale" in pd.last_error()       # 8 bits need scales
    assert fwd(scale=P) == 1                                   # and nothing else has them
    assert fwd(rows=0) == 0                                    # nothing to do

    def bwd(rows=4, D=64, g=P, gt=0, rt=0, rstd=P, gw=P, scratch=P, n=BIG):
        return lib.pdssm_add_rmsnorm_bwd(rows, D, g, gt, P, rt, P, 0, rstd, None, P, gw, scratch, n, None)

    assert bwd(D=0) == 1 and bwd(D=16385) == 2 and bwd(gt=2) == 1 and bwd(rt=2) == 1
    assert bwd(g=None) == 1 and bwd(rstd=None) == 1 and bwd(gw=None) == 1
    assert bwd(scratch=None) == 1 and bwd(scratch=ctypes.c_void_p(4096 + 64)) == 1
    assert bwd(n=pd.lib().pdssm_add_rmsnorm_scratch_bytes(4, 64) - 1) == 6
    assert pd.lib().pdssm_add_rmsnorm_scratch_bytes(4, 0) == 0


def test_select_balance_refuses_arguments():
    lib = pd.lib()

    def dm(**kw):
        d = dict(B=2, H=3, L=50, N=0, K=8, D_in=32)
        d.update(kw)
        return pd.dims(**d)

    def fwd(d, u=P, ut=0, W=P, k=P, tau=1.0, loss=P, scratch=P, n=BIG):
        return lib.pdssm_select_balance_fwd(ctypes.byref(d), u, ut, W, k, tau, None, loss, P, P, scratch, n, None)

    def bwd(d, counts=P, g=P, scratch=P, n=BIG):
        return lib.pdssm_select_balance_bwd(ctypes.byref(d), P, 0, P, counts, 1.0, None, g, P, P, scratch, n, None)

    for bad, code in ((dict(B=0), 1), (dict(H=0), 1), (dict(K=0), 1), (dict(D_in=0), 1), (dict(L=-1), 1),
                      (dict(K=33), 2), (dict(D_in=257), 2), (dict(B=1 << 16, L=1 << 16), 2)):
        assert fwd(dm(**bad)) == code and bwd(dm(**bad)) == code
        assert lib.pdssm_select_balance_scratch_bytes(ctypes.byref(dm(**bad))) == 0
    d = dm()
    assert fwd(d, u=None) == 1 and fwd(d, W=None) == 1 and fwd(d, k=None) == 1 and fwd(d, loss=None) == 1
    assert fwd(d, ut=2) == 1
    for tau in (0.0, -1.0, float("nan"), float("inf")):
        assert fwd(d, tau=tau) == 1
    assert fwd(d, scratch=None) == 1 and fwd(d, scratch=ctypes.c_void_p(4096 + 16)) == 1
    need = lib.pdssm_select_balance_scratch_bytes(ctypes.byref(d))
    assert need > 0 and fwd(d, n=need - 1) == 6 and bwd(d, n=need - 1) == 6
    assert bwd(d, counts=None) == 1 and bwd(d, g=None) == 1


def test_binding_refuses_cpu_tensors():
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        pd.pdssm_decay_scan_fwd(z(1, 1, 4, 8), z(1, 1, 4, 8), z(1, 1, 4, 8), z(1, 1, 4))
    with pytest.raises(ValueError, match="CUDA"):
        pd.pdssm_decay_step(z(1, 1, 8), z(1, 1, 8), z(1, 1, 8), z(1, 1), z(1, 1, 8, 8))
    with pytest.raises(ValueError, match="CUDA"):
        pd.pdssm_add_rmsnorm_fwd(z(2, 8), z(2, 8), z(8))
    with pytest.raises(ValueError, match="CUDA"):
        pd.pdssm_add_rmsnorm_bwd(z(2, 8), z(2, 8), z(8), z(2))
    with pytest.raises(ValueError, match="CUDA"):
        pd.pdssm_select_balance_fwd(z(1, 4, 8), z(1, 2, 8), z(1, 1, 4, dtype=torch.int32))
    with pytest.raises(ValueError, match="layout"):
        pd.pdssm_decay_scan_fwd(z(1, 1, 4, 8), z(1, 1, 4, 8), z(1, 1, 4, 8), z(1, 1, 4), layout="lbh")


@pytest.mark.parametrize("out_dtype", [torch.float8_e4m3fn, torch.float16, torch.float64], ids=str)
def test_differentiable_norm_refuses_types_whose_values_it_would_lose(out_dtype):
    """8-bit rows mean nothing without the scales that the raw call returns."""
    from structured_sparse_state_b200.layer import add_rmsnorm
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        add_rmsnorm(torch.zeros(2, 8), torch.zeros(2, 8), torch.ones(8), out_dtype=out_dtype)


def test_decay_wait_selftest_refuses_arguments():
    def run(dm, log_a=P, y=P, h=P, ws=P, n=BIG):
        return pd.lib().pdssm_decay_wait_selftest(ctypes.byref(dm), log_a, y, h, 0, ws, n, None)

    ok = dict(G=4, N=16, P=16)
    assert run(dd(**ok, B=0)) == 1
    assert run(dd(**{**ok, "G": 2})) == 1 and run(dd(**{**ok, "N": 24})) == 1 and run(dd(G=4, N=12, P=12)) == 1
    assert run(dd(**{**ok, "L": 0})) == 1
    for bad in (dict(log_a=None), dict(y=None), dict(h=None), dict(ws=None), dict(y=ctypes.c_void_p(4096 + 8))):
        assert run(dd(**ok), **bad) == 1
    assert run(dd(**ok), n=256) == 6


def test_wrong_arguments_are_value_errors():
    for dtype in (torch.float16, torch.float64, None, "bf16"):
        with pytest.raises(ValueError, match="dtype"):
            pd.pdssm_decay_workspace_bytes(1, 1, 1, 10, 16, 16, dtype)
    z = torch.zeros
    for layout in (None, 1, ["bhl"]):
        with pytest.raises(ValueError, match="layout"):
            pd.pdssm_decay_scan_fwd(z(1, 1, 4, 8), z(1, 1, 4, 8), z(1, 1, 4, 8), z(1, 1, 4), layout=layout)
