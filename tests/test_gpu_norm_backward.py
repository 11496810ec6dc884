"""GPU gradient of the gated norm against its formula in 64 bits.

Tolerances.  dweight, and dy, dz in fp32: relL2 1e-5 (sums of up to 8192 fp32 products; exponentials 2^-21).
dy, dz in bf16, element by element: the rounding 2^-8 and fp32 errors of at most 2^-14 of the sum of the absolute values
of the two terms that dv is a difference of.
"""
import pytest
import torch

import mamba_selective_state_causal_b200 as ssd
import packed_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _data(rows, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    t = [torch.randn(rows, d, generator=g).to(dtype) for _ in range(3)]
    t[2] = (t[2].float() * 1.5).to(dtype)
    return t[0], t[1], t[2], 1 + 0.2 * torch.randn(d, generator=g)     # dout, y, z, weight


def _near(dout, y, z, w, eps, group, dtype):
    """Bounds of dy and dz."""
    dout, y, z, w = (t.double() for t in (dout, y, z, w))
    sg = 1 / (1 + torch.exp(-z))
    v = (y * z * sg).view(y.shape[0], -1, group)
    gg = (dout * w).view_as(v)
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    big = (r * (gg.abs() + v.abs() * r * r * (gg * v).abs().mean(-1, keepdim=True))).view_as(y)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    dy, dz, _ = ref.norm_grad(dout, y, z, w, eps, group)
    return half * dy.abs() + 2.0 ** -14 * big * (z * sg).abs(), half * dz.abs() + 2.0 ** -14 * big * y.abs() * (1 + z.abs()) * sg


CASES = [(1, 8, 0), (5, 256, 0), (33, 768, 256), (70, 2048, 0), (40, 2048, 512), (9, 1024, 8), (7, 1024, 64), (11, 240, 24),
         (6, 240, 0), (3, 5120, 640), (5, 8192, 0), (4, 8192, 256), (300, 64, 16), (13, 40, 40), (2, 4096, 128), (1500, 256, 0)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d,group", CASES)
def test_backward(rows, d, group, dtype):
    dout, y, z, w = _data(rows, d, dtype, 60)
    n = group or d
    dy, dz, dw = ref.norm_grad(dout, y, z, w, 1e-5, n)
    o = ssd.gated_rmsnorm_backward(dout.to(DEV), y.to(DEV), z.to(DEV), w.to(DEV), eps=1e-5, group_size=group)
    ssd.sync_status()
    assert ref.rel(o["dweight"], dw) <= 1e-5
    ny, nz = _near(dout, y, z, w, 1e-5, n, dtype)
    for k, r, near in (("dy", dy, ny), ("dz", dz, nz)):
        if dtype == torch.float32:
            assert ref.rel(o[k], r) <= 1e-5, k
        assert ((o[k].cpu().double() - r).abs() <= near + 1e-30).all(), k


def test_in_place_strided_and_no_rows():
    """dy over dout, dz over z; z a slice of a wider tensor; no rows leave a zero dweight."""
    dout, y, z, w = (t.to(DEV) for t in _data(37, 512, torch.bfloat16, 61))
    a = ssd.gated_rmsnorm_backward(dout, y, z, w, group_size=128)
    wide = torch.zeros(37, 1024, dtype=torch.bfloat16, device=DEV)
    zs = wide[:, 512:]
    zs.copy_(z)
    d2 = dout.clone()
    b = ssd.gated_rmsnorm_backward(d2, y, zs, w, group_size=128, out={"dy": d2, "dz": zs})
    ssd.sync_status()
    for k in ("dy", "dz", "dweight"):
        assert torch.equal(a[k], b[k])
    assert (wide[:, :512] == 0).all()
    e = ssd.gated_rmsnorm_backward(dout[:0], y[:0], z[:0], w)
    ssd.sync_status()
    assert (e["dweight"] == 0).all()


def test_saturated_gates_stay_finite():
    """Gates of +-200 and rows of zeros: sigma saturates, the norm of a zero row is eps alone."""
    dout, y, z, w = _data(8, 256, torch.float32, 62)
    z[0], z[1], y[2] = 200.0, -200.0, 0.0
    dy, dz, dw = ref.norm_grad(dout, y, z, w, 1e-5, 256)
    o = ssd.gated_rmsnorm_backward(dout.to(DEV), y.to(DEV), z.to(DEV), w.to(DEV))
    ssd.sync_status()
    for k, r in (("dy", dy), ("dz", dz), ("dweight", dw)):
        assert torch.isfinite(o[k]).all()
        assert ref.rel(o[k], r) <= 1e-5, k
    assert torch.isfinite(o["dz"]).all()


def test_differences():
    """Against central differences of the fp32 forward norm (1e-6 relative): within 2e-3 of the gradient's norm."""
    dout, y, z, w = (t.to(DEV) for t in _data(20, 256, torch.float32, 63))
    o = ssd.gated_rmsnorm_backward(dout, y, z, w, group_size=64)
    g = torch.Generator().manual_seed(64)
    args, grads = [y, z, w], [o["dy"], o["dz"], o["dweight"]]
    for j in range(3):
        s = torch.randn(args[j].shape, generator=g).to(DEV)
        f = lambda e: float((ssd.gated_rmsnorm(*[a + e * s if i == j else a for i, a in enumerate(args)], group_size=64).double()  # noqa: E731
                             * dout.double()).sum())
        diff, exact = (f(1e-2) - f(-1e-2)) / 2e-2, float((grads[j].double() * s.double()).sum())
        assert abs(diff - exact) <= 2e-3 * float(grads[j].double().norm()) + 1e-2, (j, diff, exact)
    ssd.sync_status()
