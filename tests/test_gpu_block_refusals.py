"""What the binding of the operators around the scan refuses on CUDA tensors:
shapes, types, strides and devices, with nothing launched."""
import pytest
import torch

import structured_sparse_state_b200 as pd

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def z(*s, dtype=torch.float32):
    return torch.zeros(*s, dtype=dtype, device="cuda")


def scan(**kw):
    a = dict(c=z(1, 2, 6, 8), b=z(1, 2, 6, 8), x=z(1, 4, 6, 8), log_a=z(1, 4, 6))
    a.update(kw)
    return pd.pdssm_decay_scan_fwd(**a)


@pytest.mark.parametrize("bad", [
    dict(c=lambda: z(1, 2, 7, 8)), dict(b=lambda: z(1, 2, 6, 9)), dict(c=lambda: z(1, 3, 6, 8)),
    dict(log_a=lambda: z(1, 6, 4)), dict(log_a=lambda: z(3)), dict(log_a=lambda: z(1, 4, 6, dtype=torch.bfloat16)),
    dict(x=lambda: z(1, 4, 6, 8, dtype=torch.float16)), dict(x=lambda: z(1, 4, 6, 8, dtype=torch.bfloat16)),
    dict(x=lambda: z(1, 4, 8, 6).transpose(2, 3)), dict(h0=lambda: z(1, 2, 8, 8)), dict(h0=lambda: torch.zeros(1, 4, 8, 8)),
    dict(lengths=lambda: z(1)), dict(lengths=lambda: z(2, dtype=torch.int32)), dict(y=lambda: z(1, 4, 6, 9)),
    dict(x=lambda: z(4, 6, 8)), dict(ws=lambda: z(4))], ids=lambda d: next(iter(d)))
def test_scan_inputs(bad):
    with pytest.raises(ValueError):
        scan(**{k: f() for k, f in bad.items()})


def test_sizes_that_the_library_refuses():
    with pytest.raises(pd.PdssmError, match="128"):
        scan(c=z(1, 2, 6, 130), b=z(1, 2, 6, 130))
    with pytest.raises(pd.PdssmError, match="workspace"):
        scan(ws=z(16, dtype=torch.uint8))
    with pytest.raises(pd.PdssmError):
        pd.pdssm_add_rmsnorm_fwd(z(1, 16385), None, z(16385))
    with pytest.raises(pd.PdssmError):
        pd.pdssm_select_balance_fwd(z(1, 4, 8), z(1, 33, 8), z(1, 1, 4, dtype=torch.int32))
    with pytest.raises(pd.PdssmError, match="inv_tau"):
        pd.pdssm_select_balance_fwd(z(1, 4, 8), z(1, 3, 8), z(1, 1, 4, dtype=torch.int32), inv_tau=0.0)


def test_a_plain_forward_has_no_workspace_for_the_adjoint():
    a = (z(1, 2, 300, 8), z(1, 2, 300, 8), z(1, 2, 300, 8), z(1, 2, 300))
    y, _, ws = pd.pdssm_decay_scan_fwd(*a)
    with pytest.raises(pd.PdssmError, match="workspace"):
        pd.pdssm_decay_scan_bwd(*a, None, y, ws)


def test_step_norm_and_balance_inputs():
    a = dict(c=z(3, 2, 8), b=z(3, 2, 8), x=z(3, 4, 8), log_a=z(3, 4), state=z(3, 4, 8, 8))
    pd.pdssm_decay_step(**a)
    for bad in (dict(state=z(3, 4, 8, 9)), dict(state=z(4, 8, 8)), dict(slots=z(3)), dict(slots=z(2, dtype=torch.int32)),
                dict(log_a=z(4, 3)), dict(c=z(3, 3, 8), b=z(3, 3, 8))):
        with pytest.raises(ValueError):
            pd.pdssm_decay_step(**{**a, **bad})
    with pytest.raises(pd.PdssmError, match="n_slots"):
        pd.pdssm_decay_step(**{**a, "state": z(2, 4, 8, 8)})
    for bad in ((z(2, 8), z(3, 8), z(8)), (z(2, 8), z(2, 8), z(9)), (z(2, 8), z(2, 8, dtype=torch.float16), z(8))):
        with pytest.raises(ValueError):
            pd.pdssm_add_rmsnorm_fwd(*bad)
    with pytest.raises(ValueError):
        pd.pdssm_add_rmsnorm_fwd(z(2, 8), None, z(8), out_dtype=torch.float16)
    with pytest.raises(ValueError, match="scale"):
        pd.pdssm_add_rmsnorm_fwd(z(2, 8), None, z(8), scale=z(2))
    k = z(1, 2, 4, dtype=torch.int32)
    for bad in ((z(1, 4, 8), z(2, 3, 9), k), (z(1, 4, 8), z(2, 3, 8), k.long()), (z(1, 5, 8), z(2, 3, 8), k)):
        with pytest.raises(ValueError):
            pd.pdssm_select_balance_fwd(*bad)
    with pytest.raises(ValueError):
        pd.pdssm_select_balance_bwd(z(1, 4, 8), z(2, 3, 8), z(2, 4, dtype=torch.int32), z(2))
