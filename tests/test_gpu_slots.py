"""GPU single-token step over a pool of slots, and a run of the packed operators as serving and training use them, against
plain 64-bit statements.

Tolerances.  States are fp32: relL2 1e-5 (exponentials 2^-22, a handful of fp32 operations).  The buffer is copied: equal.
y: its rounding 2^-8 |y| (bf16; none in fp32) and, of its N + 1 terms, fp32 errors of at most 2^-14 y_abs (256 operations).
"""
import pytest
import torch

import mamba_selective_state_causal_b200 as ssd
import packed_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64 = torch.float64


def _pool(b, n, H, P, N, G, dtype, slots, seed):
    g = torch.Generator().manual_seed(seed)
    cch = H * P + 2 * G * N
    return dict(H=H, P=P, N=N, G=G, dtype=dtype, slots=slots, n=n, cch=cch,
                u=torch.randn(b, cch, generator=g).to(dtype), w=torch.rand(cch, 4, generator=g) - 0.5,
                bias=torch.randn(cch, generator=g) * 0.1, raw=torch.randn(b, H, generator=g) * 0.5,
                dt_bias=torch.randn(H, generator=g) * 0.3 - 3.5, A=-torch.exp(torch.rand(H, generator=g) * 2.77),
                D=torch.randn(H, generator=g), tail=torch.randn(n, 3, cch, generator=g).to(dtype),
                h=torch.randn(n, H, P, N, generator=g))


def _step(d, **kw):
    f = lambda k: d[k].to(DEV)  # noqa: E731
    return ssd.decode_slots(f("u"), f("w"), f("raw"), f("A"), f("D"), slots=torch.tensor(d["slots"], dtype=torch.int32, device=DEV),
                            H=d["H"], P=d["P"], N=d["N"], G=d["G"], conv_bias=f("bias"), dt_bias=f("dt_bias"), dt_softplus=True,
                            dt_limit=(1e-3, 1e-1), **kw)


def _ref_step(d, slots):
    H, P, N, G = (d[k] for k in "HPNG")
    hp, gn = H * P, G * N
    dt = ref.dt_used(d["raw"], d["dt_bias"], True, (1e-3, 1e-1))
    y, ya = torch.zeros(len(slots), H, P, dtype=F64), torch.zeros(len(slots), H, P, dtype=F64)
    h, tail = d["h"].to(F64).clone(), d["tail"].to(F64).clone()
    for i, k in enumerate(slots):
        if k < 0:
            continue
        v, tail[k] = ref.conv_seq(d["u"][i:i + 1].to(F64), d["tail"][k].to(F64), d["w"].to(F64), d["bias"].to(F64))
        x, B, C = v[:, :hp].view(1, H, P), v[:, hp:hp + gn].view(1, G, N), v[:, hp + gn:].view(1, G, N)
        one = lambda f, h0: ref.scan(f(x), f(B), f(C), dt[i:i + 1], d["A"], f(d["D"]), [0, 1], [0], [1], h0, h0,  # noqa: E731
                                     torch.zeros(1, H, P), G)
        yi, hi = one(lambda t: t, d["h"][k:k + 1])
        ai, _ = one(torch.abs, d["h"][k:k + 1].abs())
        y[i], h[k], ya[i] = yi[0], hi[0], ai[0]
    return y, h, tail, ya


SHAPES = [
    (1, 2, 64, 128, 1, torch.bfloat16), (5, 32, 64, 128, 1, torch.bfloat16), (3, 80, 64, 128, 2, torch.bfloat16),
    (4, 1, 16, 16, 1, torch.float32), (3, 3, 32, 64, 3, torch.float32), (2, 12, 128, 128, 4, torch.float32),
    (2, 10, 16, 32, 5, torch.bfloat16), (1, 9, 128, 16, 1, torch.bfloat16), (2, 8, 64, 128, 8, torch.bfloat16),
]


@pytest.mark.parametrize("b,H,P,N,G,dtype", SHAPES)
def test_step(b, H, P, N, G, dtype):
    slots = [2 * i for i in range(b)][::-1]
    d = _pool(b, 2 * b + 1, H, P, N, G, dtype, slots, 31)
    y, h, tail, ya = _ref_step(d, slots)
    hp, tp = d["h"].to(DEV), d["tail"].to(DEV)
    o = _step(d, tail_in=tp, h_in=hp)
    ssd.sync_status()
    assert o["h_out"] is hp and o["tail_out"] is tp
    assert ref.rel(hp, h) <= 1e-5
    assert torch.equal(tp.cpu().double(), tail)
    near = (2.0 ** -8 if dtype == torch.bfloat16 else 0.0) * y.abs() + 2.0 ** -14 * ya
    assert ((o["y"].cpu().double() - y).abs() <= near).all()
    untouched = [k for k in range(d["n"]) if k not in slots]
    assert torch.equal(hp.cpu()[untouched], d["h"][untouched])


def test_empty_rows_and_other_outputs():
    d = _pool(6, 8, 32, 64, 128, 1, torch.bfloat16, [3, -1, 0, 7, -1, 5], 32)
    y, h, tail, _ = _ref_step(d, d["slots"])
    ho, to = torch.full_like(d["h"], 9.0).to(DEV), torch.full_like(d["tail"], 9.0).to(DEV)
    o = _step(d, tail_in=d["tail"].to(DEV), h_in=d["h"].to(DEV), tail_out=to, h_out=ho,
              y=torch.full((6, 32, 64), float("nan"), dtype=torch.bfloat16, device=DEV))
    ssd.sync_status()
    live = [0, 3, 5, 7]
    assert ref.rel(ho[live], h[live]) <= 1e-5 and torch.equal(to[live].cpu().double(), tail[live])
    assert (ho[[1, 2, 4, 6]] == 9.0).all() and (to[[1, 2, 4, 6]] == 9.0).all()
    assert (o["y"][[1, 4]] == 0).all() and torch.isfinite(o["y"]).all()


def test_bad_slots_are_left_out_and_reported():
    """A slot out of range and the second row of one slot count as empty, and the status says so."""
    d = _pool(5, 4, 2, 64, 128, 1, torch.bfloat16, [1, 9, 1, -5, 2], 33)
    good = _pool(5, 4, 2, 64, 128, 1, torch.bfloat16, [1, -1, -1, -1, 2], 33)
    hp, tp = d["h"].to(DEV), d["tail"].to(DEV)
    o = _step(d, tail_in=tp, h_in=hp)
    with pytest.raises(ssd.SSDError) as e:
        ssd.sync_status()
    assert e.value.code == 10
    hg, tg = good["h"].to(DEV), good["tail"].to(DEV)
    p = _step(good, tail_in=tg, h_in=hg)
    ssd.sync_status()
    assert torch.equal(hp, hg) and torch.equal(tp, tg) and torch.equal(o["y"], p["y"])


def test_captured_and_replayed():
    """One captured step, replayed with other tokens, steps and slots in the same buffers."""
    b = 4
    d = _pool(b, 9, 32, 64, 128, 1, torch.bfloat16, [0, 1, 2, 3], 34)
    hp, tp = d["h"].to(DEV), d["tail"].to(DEV)
    buf = {k: d[k].to(DEV) for k in ("u", "w", "raw", "A", "D", "bias", "dt_bias")}
    slots = torch.tensor(d["slots"], dtype=torch.int32, device=DEV)
    y = torch.empty(b, 32, 64, dtype=torch.bfloat16, device=DEV)

    def call():
        ssd.decode_slots(buf["u"], buf["w"], buf["raw"], buf["A"], buf["D"], slots=slots, H=32, P=64, N=128, conv_bias=buf["bias"],
                         dt_bias=buf["dt_bias"], dt_softplus=True, dt_limit=(1e-3, 1e-1), tail_in=tp, h_in=hp, y=y)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    hp.copy_(d["h"])
    tp.copy_(d["tail"])
    for step, ks in enumerate(([5, 0, 8, -1], [0, 5, 3, 8])):
        e = _pool(b, 9, 32, 64, 128, 1, torch.bfloat16, ks, 40 + step)
        e.update({k: d[k] for k in ("w", "bias", "dt_bias", "A", "D")}, h=hp.cpu().clone(), tail=tp.cpu().clone())
        yr, hr, tr, ya = _ref_step(e, ks)
        buf["u"].copy_(e["u"])
        buf["raw"].copy_(e["raw"])
        slots.copy_(torch.tensor(ks, dtype=torch.int32))
        graph.replay()
        ssd.sync_status()
        assert ref.rel(hp, hr) <= 1e-5 and torch.equal(tp.cpu().double(), tr)
        assert ((y.cpu().double() - yr).abs() <= 2.0 ** -8 * yr.abs() + 2.0 ** -14 * ya).all()


def test_prompts_then_tokens():
    """Serving: prompts of a batch through the convolution and the scan into their slots (one of them in two parts), then two
    tokens of the same streams in another order; the states against the 64-bit recurrence over the whole
    sequences.  The convolution stores v in bf16 (half a step, 2^-8 of each of x and B, which a state is a sum of products
    of): 2^-8 in the 2-norm bounds it with room."""
    H, P, N, G, cch = 4, 64, 128, 1, 4 * 64 + 256
    g = torch.Generator().manual_seed(50)
    lens, slots, n = [150, 5, 40], [2, 0, 3], 4
    full = [m + 2 for m in lens]
    u = [torch.randn(m, cch, generator=g).to(torch.bfloat16) for m in full]
    dt = [torch.rand(m, H, generator=g) * 0.1 for m in full]
    w, bias = (torch.rand(cch, 4, generator=g) - 0.5).to(DEV), (torch.randn(cch, generator=g) * 0.1).to(DEV)
    A, D = -torch.exp(torch.rand(H, generator=g) * 2.77).to(DEV), torch.randn(H, generator=g).to(DEV)
    tail, h = torch.randn(n, 3, cch, generator=g).to(torch.bfloat16).to(DEV), torch.randn(n, H, P, N, generator=g).to(DEV)
    old = (tail.clone(), h.clone())
    i32 = dict(dtype=torch.int32, device=DEV)
    for part in range(2):
        spans = [(0, 70), (0, 5), (0, 40)] if part == 0 else [(70, 150)]
        who = [0, 1, 2] if part == 0 else [0]
        cu = [0]
        for a, b in spans:
            cu.append(cu[-1] + b - a)
        plan = ssd.packed_plan(torch.tensor(cu, **i32), cu[-1], slots=torch.tensor([slots[i] for i in who], **i32),
                               resume=torch.tensor([part] * len(who), **i32), n_slots=n)
        uu = torch.cat([u[i][a:b] for i, (a, b) in zip(who, spans)]).to(DEV)
        dd = torch.cat([dt[i][a:b] for i, (a, b) in zip(who, spans)]).to(DEV)
        v, _ = ssd.packed_conv_forward(uu, w, plan, bias, tail, tail)
        ssd.packed_scan_forward(v[:, :H * P], v[:, H * P:H * P + N], v[:, H * P + N:], dd, A, D, plan=plan, H=H, h_in=h, h_out=h)
    for k in range(2):
        order = [2, 0, 1]
        ssd.decode_slots(torch.stack([u[i][lens[i] + k] for i in order]).to(DEV), w, torch.stack([dt[i][lens[i] + k] for i in order]).to(DEV),
                         A, D, slots=torch.tensor([slots[i] for i in order], **i32), H=H, P=P, N=N, conv_bias=bias, tail_in=tail, h_in=h)
    ssd.sync_status()
    for i, k in enumerate(slots):
        v, last = ref.conv_seq(u[i].double(), torch.zeros(3, cch, dtype=F64), w.cpu().double(), bias.cpu().double())
        x, B, C = v[:, :H * P].view(-1, H, P), v[:, H * P:H * P + N].view(-1, 1, N), v[:, H * P + N:].view(-1, 1, N)
        _, hr = ref.scan(x, B, C, dt[i], A.cpu(), D.cpu(), [0, full[i]], [0], [0], None, torch.zeros(1, H, P, N),
                         torch.zeros(full[i], H, P), G)
        assert ref.rel(h[k], hr[0]) <= 2.0 ** -8
        assert torch.equal(tail[k].cpu().double(), last)
    assert torch.equal(h[1], old[1][1]) and torch.equal(tail[1], old[0][1])


def test_training_chain():
    """Training: gradients of a loss on the gated norm's output back through norm, scan and convolution of packed documents,
    in fp32, against automatic differentiation of the 64-bit statements.  Each stage keeps 1e-5 of its own, four in a
    row and the forward's v, y (1e-5 each) through derivatives of order one: 1e-4."""
    H, P, N, G = 2, 16, 16, 1
    hp, gn, cch = 32, 16, 64
    lens = [40, 3, 77]
    cu, total, _, _ = ref.batch(lens)
    g = torch.Generator().manual_seed(51)
    u, w, bias = torch.randn(total, cch, generator=g), torch.rand(cch, 4, generator=g) - 0.5, torch.randn(cch, generator=g) * 0.1
    dt, A, D = torch.rand(total, H, generator=g) * 0.1, -torch.exp(torch.rand(H, generator=g) * 2.0), torch.randn(H, generator=g)
    z, nw, dout = torch.randn(total, hp, generator=g), torch.randn(hp, generator=g), torch.randn(total, hp, generator=g)
    leaf = [t.double().requires_grad_() for t in (u, w, bias, dt, A, D, z, nw)]
    U, W, Bi, T, AA, DD, Z, NW = leaf
    outs = []
    for a, b in zip(cu, cu[1:]):
        v, _ = ref.conv_seq(U[a:b], torch.zeros(3, cch, dtype=F64), W, Bi)
        h = torch.zeros(H, P, N, dtype=F64)
        for t in range(b - a):
            x, B, C = v[t, :hp].view(H, P), v[t, hp:hp + gn], v[t, hp + gn:]
            h = h * torch.exp(T[a + t] * AA)[:, None, None] + (T[a + t][:, None] * x)[..., None] * B
            outs.append(((h * C).sum(-1) + DD[:, None] * x).flatten())
    y = torch.stack(outs)
    v = y * Z / (1 + torch.exp(-Z))
    loss = ((v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5)) * NW * dout.double()).sum()
    want = torch.autograd.grad(loss, leaf)
    c = [t.to(DEV) for t in (u, w, bias, dt, A, D, z, nw, dout)]
    plan = ssd.packed_plan(torch.tensor(cu, dtype=torch.int32, device=DEV), total)
    v, _ = ssd.packed_conv_forward(c[0], c[1], plan, c[2])
    parts = (v[:, :hp], v[:, hp:hp + gn], v[:, hp + gn:])
    y, _ = ssd.packed_scan_forward(*parts, c[3], c[4], c[5], plan=plan, H=H)
    ng = ssd.gated_rmsnorm_backward(c[8], y.flatten(1), c[6], c[7], eps=1e-5)
    sg = ssd.packed_scan_backward(*parts, c[3], c[4], c[5], ng["dy"], plan=plan, H=H)
    cg = ssd.packed_conv_backward(c[0], c[1], plan, sg["dx"], sg["dB"], sg["dC"], bias=c[2])
    ssd.sync_status()
    got = [cg["du"], cg["dconv_w"], cg["dconv_bias"], sg["ddt"], sg["dA"], sg["dD"], ng["dz"], ng["dweight"]]
    for k, a, b in zip("u w bias dt A D z norm".split(), got, want):
        assert ref.rel(a, b) <= 1e-4, (k, ref.rel(a, b))
