"""GPU convolution over packed sequences (forward and backward) against plain 64-bit statements, and against the layer's
own convolution, whose arithmetic it shares.

Tolerances.  bf16 v: one hardware tanh (relative error 2^-11, entering as h tanh(h) with |h tanh h| <= |z| / 2), four
fp32 sums (2^-22) and one rounding (2^-8): |v - exact| <= 2^-8 |exact| + 2^-11 |z| / 2 + 2^-20 sum|w u|.  fp32 v and all
gradients: relL2 at the framework's fp32 bound 1e-5; their worst term is the hardware exponential in sigma (2^-21) and the
sums of up to a few hundred fp32 products (300 * 2^-24 = 1.8e-5 of the absolute sum at worst, its square root of that
number in the 2-norm, 1e-6).
"""
import pytest
import torch

import mamba_selective_state_causal_b200 as ssd
import packed_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _data(lens, cch, dtype, seed=0, slots=None, resume=None, before=0, behind=0, n_slots=None, wide=0):
    g = torch.Generator().manual_seed(seed)
    cu, total, sl, rs = ref.batch(lens, slots=slots, resume=resume, before=before, behind=behind)
    n_slots = n_slots or len(lens) + 2
    d = dict(cu=cu, total=total, slots=sl, resume=rs, n_slots=n_slots)
    d["u"] = torch.randn(total, cch + wide, generator=g).to(dtype)[:, :cch]
    d["w"] = torch.rand(cch, 4, generator=g) - 0.5
    d["bias"] = torch.randn(cch, generator=g) * 0.1
    d["tail"] = torch.randn(n_slots, 3, cch, generator=g).to(dtype)
    return d


def _plan(d, slots=True, max_seqlen=0):
    i32 = dict(dtype=torch.int32, device=DEV)
    return ssd.packed_plan(torch.tensor(d["cu"], **i32), d["total"], slots=torch.tensor(d["slots"], **i32) if slots else None,
                           resume=torch.tensor(d["resume"], **i32), n_slots=d["n_slots"], max_seqlen=max_seqlen)


CASES = [
    ([1], 16, [1]),
    ([1, 2, 3, 4, 0, 5], 48, [1, 0, 1, 1, 1, 0]),
    ([64, 63, 65, 128, 1, 200], 96, [0, 1, 1, 0, 1, 1]),
    ([0, 0], 32, [1, 0]),
    ([700], 2304, [1]),
    ([3, 130, 2, 2], 2304, [1, 1, 1, 0]),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,cch,resume", CASES)
def test_forward(lens, cch, resume, dtype):
    n = len(lens)
    d = _data(lens, cch, dtype, 1, slots=list(range(n + 1, 1, -1)), resume=resume, before=3, behind=5, n_slots=n + 3, wide=16)
    mark = torch.full((d["total"], cch), 7.0, dtype=dtype)
    tmark = torch.full_like(d["tail"], -3.0)
    vr, tr = ref.conv(d["u"], d["w"], d["bias"], d["cu"], d["slots"], resume, d["tail"], tmark, mark)
    u = torch.zeros(d["total"], cch + 16, dtype=dtype, device=DEV)[:, :cch].copy_(d["u"])
    v, tail = ssd.packed_conv_forward(u, d["w"].to(DEV), _plan(d), d["bias"].to(DEV), d["tail"].to(DEV), tmark.to(DEV), mark.to(DEV))
    ssd.sync_status()
    assert torch.equal(tail.cpu().double(), tr)
    if dtype == torch.float32:
        assert ref.rel(v, vr) <= 1e-5
        a, b = d["cu"][0], d["cu"][-1]
        assert torch.equal(v[:a].cpu(), mark[:a]) and torch.equal(v[b:].cpu(), mark[b:])
    else:
        most = 0.5 * 4 * float(max(d["u"].abs().max(), d["tail"].abs().max())) + float(d["bias"].abs().max())   # >= |z|
        near = vr.abs() * 2.0 ** -8 + 2.0 ** -11 * most / 2 + 2.0 ** -20 * most
        assert ((v.cpu().double() - vr).abs() <= near).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_forward_is_the_layers_convolution(dtype):
    """Each packed sequence gets the v of ssd_conv_forward on it alone, bit for bit, in place of its buffer too."""
    lens = [5, 64, 1, 300, 2, 129]
    d = _data(lens, 2304, dtype, 2, slots=[4, 0, 3, 1, 5, 2], n_slots=6)
    pool = d["tail"].to(DEV)
    u, w, bias = d["u"].to(DEV), d["w"].to(DEV), d["bias"].to(DEV)
    plan = _plan(d)
    before = pool.clone()
    v, _ = ssd.packed_conv_forward(u, w, plan, bias, pool, pool)
    for i, k in enumerate(d["slots"]):
        a, b = d["cu"][i], d["cu"][i + 1]
        tail = torch.empty(1, 3, 2304, dtype=dtype, device=DEV)
        vi, _ = ssd.conv_forward(u[None, a:b].contiguous(), w, bias, before[k:k + 1].contiguous(), tail)
        assert torch.equal(v[a:b], vi[0])
        assert torch.equal(pool[k], tail[0])
    ssd.sync_status()


def test_forward_keeps_neighbours_apart():
    """NaN and infinite rows of one sequence, and rows of none, reach no other sequence; slot -1 keeps nothing."""
    lens = [70, 5, 64]
    d = _data(lens, 64, torch.bfloat16, 3, slots=[0, -1, 1], before=2, behind=4)
    u = d["u"].clone()
    u[d["cu"][1]:d["cu"][2]] = float("nan")
    u[:2] = float("inf")
    u[d["cu"][-1]:] = float("nan")
    pool = d["tail"].to(DEV)
    v, _ = ssd.packed_conv_forward(u.to(DEV), d["w"].to(DEV), _plan(d), d["bias"].to(DEV), pool, pool)
    ssd.sync_status()
    clean = d["tail"].to(DEV)
    good, _ = ssd.packed_conv_forward(torch.nan_to_num(d["u"]).to(DEV), d["w"].to(DEV), _plan(d), d["bias"].to(DEV), clean, clean)
    for i in (0, 2):
        a, b = d["cu"][i], d["cu"][i + 1]
        assert torch.equal(v[a:b], good[a:b])
    assert torch.equal(pool, clean)
    assert torch.equal(pool[2:], d["tail"][2:].to(DEV))


GRADS = [
    ([1], 16, 16, [1]),
    ([1, 2, 3, 4, 0, 5, 7], 32, 16, [1, 0, 1, 1, 1, 0, 1]),
    ([64, 63, 65, 128, 1, 200, 66], 64, 32, [0, 1, 1, 0, 1, 1, 1]),
    ([300, 2, 131], 2048, 128, [1, 1, 0]),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,hp,gn,resume", GRADS)
def test_backward(lens, hp, gn, resume, dtype):
    cch, n = hp + 2 * gn, len(lens)
    d = _data(lens, cch, dtype, 4, slots=list(range(n, 0, -1)), resume=resume, before=1, behind=3, n_slots=n + 1)
    g = torch.Generator().manual_seed(5)
    dv = torch.randn(d["total"], cch, generator=g)
    dto = torch.randn(n, 3, cch, generator=g)
    du, dt, dw, db = ref.conv_grad(d["u"], d["w"], d["bias"], d["cu"], d["slots"], resume, d["tail"], dv, dto)
    parts = [dv[:, :hp].contiguous().to(DEV), dv[:, hp:hp + gn].contiguous().to(DEV), dv[:, hp + gn:].contiguous().to(DEV)]
    o = ssd.packed_conv_backward(d["u"].to(DEV), d["w"].to(DEV), _plan(d), *parts, bias=d["bias"].to(DEV),
                                 tail_in=d["tail"].to(DEV), dtail_out=dto.to(DEV))
    ssd.sync_status()
    for k, r in (("du", du), ("dtail_in", dt), ("dconv_w", dw), ("dconv_bias", db)):
        assert ref.rel(o[k], r) <= 1e-5, k


def test_backward_differences():
    """The gradient along random directions against central differences of the forward: the loss is a sum of
    about 2e4 fp32 terms of size 1, each off by at most 2^-22 (its own rounding and the sum's, carried in 64 bits),
    so a difference over a step of 1e-2 is off by at most sqrt(2e4) 2^-22 / 2e-2 = 1.7e-3 and by the third
    derivative times 1e-4 / 6, below 1e-4 of the gradient's size (hundreds)."""
    lens, hp, gn = [90, 2, 61], 64, 16
    cch = hp + 2 * gn
    d = _data(lens, cch, torch.float32, 6)
    d["resume"] = [1, 1, 1]
    g = torch.Generator().manual_seed(7)
    dv = torch.randn(d["total"], cch, generator=g).to(DEV)
    plan = _plan(d)
    u, w, bias, tail = (d[k].to(DEV) for k in ("u", "w", "bias", "tail"))
    o = ssd.packed_conv_backward(u, w, plan, dv[:, :hp].contiguous(), dv[:, hp:hp + gn].contiguous(), dv[:, hp + gn:].contiguous(),
                                 bias=bias, tail_in=tail)

    def loss(u, w, bias, tail):
        v, _ = ssd.packed_conv_forward(u, w, plan, bias, tail)
        return float((v.double() * dv.double()).sum())

    args = [u, w, bias, tail]
    grads = [o["du"], o["dconv_w"], o["dconv_bias"], None]
    full = torch.zeros_like(tail)
    for i, k in enumerate(d["slots"]):
        full[k] = o["dtail_in"][i]
    grads[3] = full
    for j in range(4):
        s = torch.randn(args[j].shape, generator=g).to(DEV)
        e = 1e-2
        up = [a + e * s if i == j else a for i, a in enumerate(args)]
        dn = [a - e * s if i == j else a for i, a in enumerate(args)]
        diff = (loss(*up) - loss(*dn)) / (2 * e)
        exact = float((grads[j].double() * s.double()).sum())
        assert abs(diff - exact) <= 2e-3 * float(grads[j].double().norm()) + 5e-3, (j, diff, exact)
    ssd.sync_status()


def test_rows_of_no_sequence_stay():
    lens = [40, 3]
    d = _data(lens, 48, torch.float32, 8, before=2, behind=2)
    g = torch.Generator().manual_seed(9)
    dv = [torch.randn(d["total"], k, generator=g).to(DEV) for k in (16, 16, 16)]
    du = torch.full((d["total"], 48), 5.0, device=DEV)
    o = ssd.packed_conv_backward(d["u"].to(DEV), d["w"].to(DEV), _plan(d), *dv, out={"du": du})
    ssd.sync_status()
    assert (o["du"][:2] == 5.0).all() and (o["du"][-2:] == 5.0).all()
    assert torch.equal(o["dtail_in"], torch.zeros_like(o["dtail_in"]))
