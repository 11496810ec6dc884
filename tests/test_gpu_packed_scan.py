"""GPU selective scan over packed sequences (forward and backward) against plain 64-bit recurrences.

Tolerances.  States and gradients are fp32: relL2 at the framework's fp32 bound 1e-5.  On the tensor cores the product
that forms a state takes w x as two bf16 parts, off by 2^-16 of a term at most (2^-17.6 in the 2-norm), the decays come
from fp32 sums of dt A in chunks of 128 rows (about 1e-6 of a weight that matters), the accumulation is fp32.
y in fp32: 1e-5.  y in bf16 on the tensor cores, element by element: its own rounding 2^-8 |y|, and of every term of it
one rounding of the masked product or of the entering state (2^-8 each, a term has one of them) plus the fp32
errors above: at most 2^-8 |y| + (2^-8 + 2^-14) y_abs, where y_abs is the same recurrence on the absolute
values of x, B, C, D and the state.  The CUDA-core kernels round y once: 2^-8 |y| + 1e-4 y_abs.
"""
import pytest
import torch

import mamba_selective_state_causal_b200 as ssd
import packed_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64


def _data(lens, H, P, N, G, dtype, seed=0, slots=None, resume=None, before=0, behind=0, n_slots=None, dt_max=1e-1):
    g = torch.Generator().manual_seed(seed)
    cu, total, sl, rs = ref.batch(lens, slots=slots, resume=resume, before=before, behind=behind)
    n_slots = n_slots or len(lens) + 1
    cch = H * P + 2 * G * N
    d = dict(cu=cu, total=total, slots=sl, resume=rs, n_slots=n_slots, H=H, P=P, N=N, G=G, dtype=dtype)
    d["v"] = torch.nn.functional.silu(torch.randn(total, cch, generator=g)).to(dtype)
    d["dt"] = torch.exp(torch.rand(total, H, generator=g) * 4.0 + torch.tensor(dt_max).log() - 4.0)
    d["A"] = -torch.exp(torch.rand(H, generator=g) * 2.77)
    d["D"] = torch.randn(H, generator=g)
    d["h"] = torch.randn(n_slots, H, P, N, generator=g)
    return d


def _parts(d, v):
    H, P, N, G = (d[k] for k in "HPNG")
    return v[:, :H * P], v[:, H * P:H * P + G * N], v[:, H * P + G * N:]


def _ref_in(d):
    H, P, N, G = (d[k] for k in "HPNG")
    x, B, C = _parts(d, d["v"])
    return x.reshape(-1, H, P), B.reshape(-1, G, N), C.reshape(-1, G, N)


def _plan(d, slots=True, max_seqlen=0):
    i32 = dict(dtype=torch.int32, device=DEV)
    return ssd.packed_plan(torch.tensor(d["cu"], **i32), d["total"], slots=torch.tensor(d["slots"], **i32) if slots else None,
                           resume=torch.tensor(d["resume"], **i32), n_slots=d["n_slots"], max_seqlen=max_seqlen)


def _run(d, plan=None, h_in=None, h_out=None, y=None, v=None, **kw):
    x, B, C = _parts(d, d["v"].to(DEV) if v is None else v)
    return ssd.packed_scan_forward(x, B, C, kw.pop("dt", d["dt"]).to(DEV), d["A"].to(DEV), d["D"].to(DEV), plan=plan or _plan(d),
                                   H=d["H"], G=d["G"], h_in=h_in, h_out=h_out, y=y, **kw)


def _check(d, y, h, mark=7.0, hmark=-3.0, h_in="h", dt=None, tc=True):
    H, P, N = d["H"], d["P"], d["N"]
    hin = d["h"] if h_in == "h" else None
    dt = d["dt"] if dt is None else dt
    ym, hm = torch.full((d["total"], H, P), mark), torch.full((d["n_slots"], H, P, N), hmark)
    x, B, C = _ref_in(d)
    yr, hr = ref.scan(x, B, C, dt, d["A"], d["D"], d["cu"], d["slots"], d["resume"], hin, hm, ym, d["G"])
    assert ref.rel(h, hr) <= 1e-5
    assert torch.equal(h.cpu()[hr == hmark], hm[hr == hmark])          # slots of no sequence
    a, b = d["cu"][0], d["cu"][-1]
    assert (y[:a] == mark).all() and (y[b:] == mark).all()
    if d["dtype"] == torch.float32:
        assert ref.rel(y[a:b], yr[a:b]) <= 1e-5
        return
    ya, _ = ref.scan(x.abs(), B.abs(), C.abs(), dt, d["A"], d["D"].abs(), d["cu"], d["slots"], d["resume"],
                     hin.abs() if hin is not None else None, hm, ym, d["G"])
    near = 2.0 ** -8 * yr.abs() + ((2.0 ** -8 + 2.0 ** -14) if tc else 1e-4) * ya
    off = (y.cpu().to(F64) - yr).abs()[a:b]
    assert (off <= near[a:b]).all(), float((off / near[a:b].clamp_min(1e-30)).max())


def _fill(d):
    y = torch.full((d["total"], d["H"], d["P"]), 7.0, dtype=d["dtype"], device=DEV)
    h = torch.full((d["n_slots"], d["H"], d["P"], d["N"]), -3.0, device=DEV)
    return y, h


TC = [
    # lens, H, G, resume
    ([1], 2, 1, [1]),
    ([128], 2, 1, [0]),
    ([127, 129, 1, 0, 2, 256, 31], 4, 1, [1, 0, 1, 1, 0, 1, 1]),
    ([300, 5], 4, 2, [1, 1]),
    ([1500], 4, 1, [1]),
    ([17] * 40, 2, 1, [1, 0] * 20),
    ([900, 3, 640, 128, 77], 6, 1, [1, 1, 0, 1, 0]),
    ([0], 2, 1, [1]),
]


@pytest.mark.parametrize("lens,H,G,resume", TC)
def test_forward_tensor_cores(lens, H, G, resume):
    n = len(lens)
    d = _data(lens, H, 64, 128, G, torch.bfloat16, 11, slots=[(7 * i + 3) % n for i in range(n)] if n % 7 else list(range(n)),
              resume=resume, before=2, behind=3, n_slots=n + 2)
    y, h = _fill(d)
    y, h = _run(d, h_in=d["h"].to(DEV), h_out=h, y=y)
    ssd.sync_status()
    _check(d, y, h)


GENERIC = [
    ([1], 1, 16, 16, 1, [1]),
    ([64, 63, 65, 0, 1, 200], 2, 16, 16, 1, [1, 0, 1, 1, 0, 1]),
    ([300, 7], 3, 32, 64, 3, [1, 1]),
    ([150, 40], 2, 128, 128, 1, [0, 1]),
    ([90, 400], 4, 64, 16, 2, [1, 0]),
    ([70], 2, 64, 128, 2, [1]),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,H,P,N,G,resume", GENERIC)
def test_forward_cuda_cores(lens, H, P, N, G, resume, dtype):
    d = _data(lens, H, P, N, G, dtype, 12, resume=resume, before=1, behind=2, n_slots=len(lens) + 1)
    y, h = _fill(d)
    y, h = _run(d, h_in=d["h"].to(DEV), h_out=h, y=y)
    ssd.sync_status()
    _check(d, y, h, tc=False)


@pytest.mark.parametrize("dtype,P,N", [(torch.bfloat16, 64, 128), (torch.float32, 32, 16)])
def test_in_place_and_repeated(dtype, P, N):
    """States updated in their pool (also those of a sequence that spans many windows) are those written elsewhere, bit for
    bit; the same call twice gives the same; a plan made with a bound of the lengths gives the same."""
    lens = [2600, 5, 700, 130]
    d = _data(lens, 2, P, N, 1, dtype, 13, slots=[2, 0, 4, 1], n_slots=5)
    h0 = d["h"].to(DEV)
    ya, ha = _run(d, h_in=h0, h_out=h0.clone())
    yb, hb = _run(d, h_in=h0, h_out=h0.clone())
    assert torch.equal(ya, yb) and torch.equal(ha, hb)
    pool = h0.clone()
    yc, _ = _run(d, h_in=pool, h_out=pool)
    assert torch.equal(ya, yc) and torch.equal(pool, ha)
    yd, hd = _run(d, plan=_plan(d, max_seqlen=2600), h_in=h0, h_out=h0.clone())
    assert torch.equal(ya, yd) and torch.equal(ha, hd)
    ssd.sync_status()


def test_without_states_and_with_slot_minus_one():
    lens = [140, 30, 200]
    d = _data(lens, 2, 64, 128, 1, torch.bfloat16, 14, slots=[1, -1, 0], n_slots=3, resume=[1, 1, 1])
    y, h = _fill(d)
    _run(d, h_out=h, y=y)
    ssd.sync_status()
    _check(d, y, h, h_in=None)
    y2, _ = _fill(d)
    _run(d, y=y2)                     # nothing kept
    assert torch.equal(y, y2)
    y3, h3 = _fill(d)
    _run(d, h_in=d["h"].to(DEV), h_out=h3, y=y3)
    ssd.sync_status()
    _check(d, y3, h3)


@pytest.mark.parametrize("dtype,P,N", [(torch.bfloat16, 64, 128), (torch.float32, 16, 32)])
def test_neighbours_stay_apart(dtype, P, N):
    """NaN and infinite rows, dt and states of one sequence, and of rows that belong to none, reach no other."""
    lens = [100, 20, 300, 1]
    d = _data(lens, 2, P, N, 1, dtype, 15, before=3, behind=9)
    y, h = _fill(d)
    ya, ha = _run(d, h_in=d["h"].to(DEV), h_out=h, y=y)
    v, dt, h0 = d["v"].clone(), d["dt"].clone(), d["h"].clone()
    a, b = d["cu"][1], d["cu"][2]
    v[a:b], dt[a:b], h0[1] = float("nan"), float("inf"), float("nan")
    for s in (slice(0, 3), slice(d["cu"][-1], d["total"])):
        v[s], dt[s] = float("inf"), float("nan")
    y, h = _fill(d)
    yb, hb = _run(d, v=v.to(DEV), dt=dt, h_in=h0.to(DEV), h_out=h, y=y)
    ssd.sync_status()
    keep = [i for i in range(d["total"]) if not a <= i < b]
    assert torch.equal(ya[keep], yb[keep])
    for k in (0, 2, 3, 4):
        assert torch.equal(ha[k], hb[k])


@pytest.mark.parametrize("dtype,P,N", [(torch.bfloat16, 64, 128), (torch.float32, 16, 16)])
def test_dt_surroundings(dtype, P, N):
    """dt_bias, softplus and the clamp inside the scan: the GPU's softplus is off by a few 2^-23 relative, which the
    bounds of the states and of y hold."""
    d = _data([200, 33], 2, P, N, 1, dtype, 16)
    g = torch.Generator().manual_seed(17)
    raw, bias = torch.randn(d["total"], 2, generator=g) * 0.5, torch.randn(2, generator=g) * 0.3 - 3.5
    y, h = _fill(d)
    _run(d, h_in=d["h"].to(DEV), h_out=h, y=y, dt=raw, dt_bias=bias.to(DEV), dt_softplus=True, dt_limit=(1e-3, 1e-1))
    ssd.sync_status()
    _check(d, y, h, dt=ref.dt_used(raw, bias, True, (1e-3, 1e-1)), tc=P == 64)


def test_long_steps_underflow():
    """Steps up to 0.5 with A down to -16: decays underflow to zero and stay finite."""
    d = _data([260, 140], 4, 64, 128, 1, torch.bfloat16, 18, dt_max=0.5)
    d["A"] = torch.tensor([-16.0, -1.0, -7.0, -0.01])
    y, h = _fill(d)
    _run(d, h_in=d["h"].to(DEV), h_out=h, y=y)
    ssd.sync_status()
    _check(d, y, h)


def test_parts_of_a_sequence():
    """A prompt in three packed calls, resumed from its slot, is the prompt in one (the states to fp32 rounding: the
    chunks differ, 1e-5; y each to its own bound)."""
    d = _data([517], 4, 64, 128, 1, torch.bfloat16, 19, slots=[1], n_slots=3, resume=[0])
    y, h = _fill(d)
    _run(d, h_out=h, y=y)
    pool = torch.full_like(h, 5.0)
    at, ys = 0, []
    for i, m in enumerate((1, 300, 216)):
        e = dict(d, v=d["v"][at:at + m], dt=d["dt"][at:at + m], cu=[0, m], total=m, resume=[int(i > 0)])
        yi, _ = _run(e, h_in=pool, h_out=pool)
        ys.append(yi)
        at += m
    ssd.sync_status()
    assert ref.rel(pool[1], h[1].cpu()) <= 1e-5
    y2 = torch.cat(ys)
    _check(d, y2, torch.cat((torch.full_like(h[:1], -3.0), pool[1:2], torch.full_like(h[:1], -3.0))))


GRADS = [
    ([1], 2, 64, 128, 1, torch.bfloat16, [1]),
    ([64, 63, 65, 0, 130, 2], 2, 64, 128, 1, torch.bfloat16, [1, 0, 1, 1, 0, 1]),
    ([500, 77], 4, 64, 128, 2, torch.bfloat16, [0, 1]),
    ([64, 63, 65, 0, 130, 2], 2, 16, 16, 1, torch.float32, [1, 0, 1, 1, 0, 1]),
    ([200, 40], 4, 32, 64, 2, torch.float32, [1, 1]),
    ([90, 3], 2, 64, 128, 1, torch.float32, [1, 0]),
    ([90, 3], 3, 128, 32, 1, torch.bfloat16, [1, 0]),
]


@pytest.mark.parametrize("lens,H,P,N,G,dtype,resume", GRADS)
def test_backward(lens, H, P, N, G, dtype, resume):
    n = len(lens)
    d = _data(lens, H, P, N, G, dtype, 21, slots=list(range(n, 0, -1)), resume=resume, before=2, behind=5, n_slots=n + 1)
    g = torch.Generator().manual_seed(22)
    dy = torch.randn(d["total"], H * P, generator=g).to(dtype)
    dh = torch.randn(n, H, P, N, generator=g)
    x, B, C = _ref_in(d)
    r = ref.scan_grad(x, B, C, d["dt"], d["A"], d["D"], d["cu"], d["slots"], resume, d["h"], dy.view(-1, H, P), dh, G)
    xg, Bg, Cg = _parts(d, d["v"].to(DEV))
    o = ssd.packed_scan_backward(xg, Bg, Cg, d["dt"].to(DEV), d["A"].to(DEV), d["D"].to(DEV), dy.to(DEV), plan=_plan(d), H=H, G=G,
                                 h_in=d["h"].to(DEV), dh_out=dh.to(DEV))
    ssd.sync_status()
    for k in r:
        assert ref.rel(o[k], r[k]) <= 1e-5, (k, ref.rel(o[k], r[k]))


def test_backward_neighbours_and_rows_of_none():
    lens = [70, 20, 128]
    d = _data(lens, 2, 64, 128, 1, torch.bfloat16, 23, before=2, behind=3)
    g = torch.Generator().manual_seed(24)
    dy = torch.randn(d["total"], 128, generator=g).to(torch.bfloat16)

    def grads(v, dy, dt):
        xg, Bg, Cg = _parts(d, v.to(DEV))
        out = {"dx": torch.full((d["total"], 2, 64), 4.0, device=DEV), "ddt": torch.full((d["total"], 2), 4.0, device=DEV),
               "dB": torch.full((d["total"], 1, 128), 4.0, device=DEV)}
        return ssd.packed_scan_backward(xg, Bg, Cg, dt.to(DEV), d["A"].to(DEV), d["D"].to(DEV), dy.to(DEV), plan=_plan(d), H=2,
                                        out=out)

    a = grads(d["v"], dy, d["dt"])
    v, dy2, dt = d["v"].clone(), dy.clone(), d["dt"].clone()
    for s in (slice(0, 2), slice(d["cu"][1], d["cu"][2]), slice(d["cu"][-1], d["total"])):
        v[s], dy2[s], dt[s] = float("nan"), float("inf"), float("nan")
    b = grads(v, dy2, dt)
    ssd.sync_status()
    for s in (slice(d["cu"][0], d["cu"][1]), slice(d["cu"][2], d["cu"][3])):
        for k in ("dx", "dB", "dC", "ddt"):
            assert torch.equal(a[k][s], b[k][s]), k
    for k in ("dx", "dB", "ddt"):
        assert (a[k][:2] == 4.0).all() and (a[k][-3:] == 4.0).all()


def test_backward_differences():
    """Gradients along random directions against central differences of the fp32 forward (its y to 1e-6 relative, the loss
    a sum of 2.6e3 terms): within 2e-3 of the gradient's norm."""
    d = _data([70, 31], 2, 16, 16, 1, torch.float32, 25, dt_max=0.3)
    g = torch.Generator().manual_seed(26)
    dy = torch.randn(d["total"], 32, generator=g).to(DEV)
    dh = torch.randn(2, 2, 16, 16, generator=g).to(DEV)
    plan = _plan(d)
    x, B, C = (t.contiguous() for t in _parts(d, d["v"].to(DEV)))
    args = [x, B, C, d["dt"].to(DEV), d["A"].to(DEV), d["D"].to(DEV), d["h"].to(DEV)]
    o = ssd.packed_scan_backward(*args[:6], dy, plan=plan, H=2, h_in=args[6], dh_out=dh)
    grads = [o["dx"].flatten(1), o["dB"].flatten(1), o["dC"].flatten(1), o["ddt"], o["dA"], o["dD"], torch.zeros_like(args[6])]
    for i, k in enumerate(d["slots"]):
        grads[6][k] = o["dh_in"][i]

    def loss(*t):
        y, h = ssd.packed_scan_forward(*t[:6], plan=plan, H=2, h_in=t[6], h_out=torch.zeros_like(t[6]))
        return float((y.flatten(1).double() * dy.double()).sum() + sum((h[k].double() * dh[i].double()).sum() for i, k in enumerate(d["slots"])))

    for j, t in enumerate(args):
        s = torch.randn(t.shape, generator=g).to(DEV)
        e = 1e-3 if j == 3 else 1e-2
        diff = (loss(*[a + e * s if i == j else a for i, a in enumerate(args)]) -
                loss(*[a - e * s if i == j else a for i, a in enumerate(args)])) / (2 * e)
        exact = float((grads[j].double() * s.double()).sum())
        assert abs(diff - exact) <= 5e-3 * float(grads[j].double().norm()) + 1e-2, (j, diff, exact)
    ssd.sync_status()


@pytest.mark.parametrize("lens,H,P,N,dtype,resume", [
    ([700, 5, 1300, 128, 60, 384, 1, 900], 32, 64, 128, torch.bfloat16, [1, 0, 1, 1, 0, 1, 1, 0]),
    ([90] * 30, 48, 64, 128, torch.bfloat16, [1, 0, 0] * 10),
    ([500, 3, 640, 64, 33, 400], 80, 16, 16, torch.float32, [0, 1, 1, 0, 1, 1]),
])
def test_windows_of_several_chunks(lens, H, P, N, dtype, resume):
    """Enough heads that a CTA walks several chunks, of several sequences and of ones that reach into the next window
    (the 64-bit recurrence runs on the GPU)."""
    d = _data(lens, H, P, N, 1, dtype, 27, slots=list(range(len(lens)))[::-1], resume=resume, n_slots=len(lens) + 1)
    pool = d["h"].to(DEV)
    y, _ = _run(d, h_in=pool, h_out=pool)
    ssd.sync_status()
    x, B, C = (t.to(DEV) for t in _ref_in(d))
    hin, dt, A, D = d["h"].to(DEV), d["dt"].to(DEV), d["A"].to(DEV), d["D"].to(DEV)
    zero = torch.zeros(d["total"], H, P, device=DEV)
    args = (d["cu"], d["slots"], resume)

    def on_gpu(x, B, C, D, hin):
        h0 = hin.to(F64)
        out, yy = h0.clone(), zero.to(F64).clone()
        for i, k in enumerate(args[1]):
            h = h0[k] * resume[i]
            for t in range(args[0][i], args[0][i + 1]):
                h = h * torch.exp(dt[t].to(F64) * A.to(F64))[:, None, None] + (dt[t].to(F64)[:, None] * x[t].to(F64))[..., None] * B[t].to(F64)
                yy[t] = (h * C[t].to(F64)).sum(-1) + D.to(F64)[:, None] * x[t].to(F64)
            out[k] = h
        return yy, out

    yr, hr = on_gpu(x, B, C, D, hin)
    assert ref.rel(pool, hr) <= 1e-5
    for k in range(len(lens) + 1):
        assert ref.rel(pool[k], hr[k].cpu()) <= 2e-5, k       # each on its own: twice the bound of all
    if dtype == torch.float32:
        assert ref.rel(y, yr) <= 1e-5
        return
    ya, _ = on_gpu(x.abs(), B.abs(), C.abs(), D.abs(), hin.abs())
    near = 2.0 ** -8 * yr.abs() + (2.0 ** -8 + 2.0 ** -14) * ya
    assert ((y.to(F64) - yr).abs() <= near).all()
