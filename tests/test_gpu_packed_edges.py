"""The packed operators where a batch has less to do than its buffers hold, and at shapes of their own.

Tolerances as in test_gpu_packed_scan.py and test_gpu_slots.py (relL2 1e-5 against 64 bits for fp32 outputs); where two
calls have the same arithmetic, their outputs are equal.
"""
import pytest
import torch

import mamba_selective_state_causal_b200 as ssd
import packed_ref as ref
from test_gpu_packed_scan import DEV, _data, _parts, _plan, _ref_in

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype,P,N", [(torch.bfloat16, 64, 128), (torch.float32, 16, 16)])
@pytest.mark.parametrize("total", [0, 5])
@pytest.mark.parametrize("refused", [False, True])
def test_gradients_of_a_batch_without_chunks(refused, total, dtype, P, N):
    """Nothing but empty sequences without a slot, or nothing but refused ones: the gradients of the weights and of what the
    sequences start from are zero, whatever the outputs held."""
    H, n, cch = 2, 3, 2 * P + 2 * N
    cu = torch.tensor([9, 10, 11, 12] if refused else [total] * 4, **I32)
    plan = ssd.packed_plan(cu, total, slots=torch.tensor([0, 1, 2] if refused else [-1] * 3, **I32), n_slots=3)
    v, dt = torch.randn(total, cch, device=DEV).to(dtype), torch.rand(total, H, device=DEV)
    x, B, C = v[:, :H * P], v[:, H * P:H * P + N], v[:, H * P + N:]
    A, D, dy = -torch.ones(H, device=DEV), torch.ones(H, device=DEV), torch.randn(total, H * P, device=DEV).to(dtype)
    nan = lambda *s: torch.full(s, float("nan"), device=DEV)  # noqa: E731
    o = ssd.packed_scan_backward(x, B, C, dt, A, D, dy, plan=plan, H=H, h_in=torch.ones(3, H, P, N, device=DEV),
                                 dh_out=torch.ones(n, H, P, N, device=DEV), out={"dh_in": nan(n, H, P, N), "dA": nan(H), "dD": nan(H)})
    c = ssd.packed_conv_backward(v, torch.ones(cch, 4, device=DEV), plan, o["dx"], o["dB"], o["dC"],
                                 tail_in=torch.ones(3, 3, cch, device=DEV, dtype=dtype), dtail_out=torch.ones(n, 3, cch, device=DEV),
                                 out={"dtail_in": nan(n, 3, cch), "dconv_w": nan(cch, 4), "dconv_bias": nan(cch)})
    torch.cuda.synchronize()
    if refused:
        with pytest.raises(ssd.SSDError) as e:
            ssd.sync_status()
        assert e.value.code == 10
    else:
        ssd.sync_status()
    for k in ("dh_in", "dA", "dD"):
        assert (o[k] == 0).all(), k
    for k in ("dtail_in", "dconv_w", "dconv_bias"):
        assert (c[k] == 0).all(), k
