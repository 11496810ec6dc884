"""The packed operators as a program uses them: gradients whose heads are dealt out in blocks, batches of nothing but empty
sequences, refused offsets and slots, two streams at once, captured and replayed batches, a wait that runs out.

Tolerances as in test_gpu_packed_scan.py and test_gpu_packed_conv.py (relL2 1e-5 against 64 bits for fp32 outputs); dB
and dC of the tensor-core form add at most 8 heads' sums in TMEM, each addition cut off at 2^-23 of it: 160 additions
of 2^-24 on average are 1e-5 if no term had a sign, and a tenth of that with signs at random.
"""
import os
import subprocess
import sys

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
if __name__ == "__main__":
    sys.path[:0] = [HERE, os.path.dirname(HERE)]

import mamba_selective_state_causal_b200 as ssd
import packed_ref as ref
from test_gpu_packed_scan import DEV, F64, _data, _parts, _plan, _ref_in, _run

pytestmark = pytest.mark.gpu


def _grad_inputs(d, seed):
    g = torch.Generator().manual_seed(seed)
    n = len(d["slots"])
    return (torch.randn(d["total"], d["H"] * d["P"], generator=g).to(d["dtype"]),
            torch.randn(n, d["H"], d["P"], d["N"], generator=g))


def _grads(d, dy, dh, plan=None, **kw):
    x, B, C = _parts(d, d["v"].to(DEV))
    return ssd.packed_scan_backward(x, B, C, d["dt"].to(DEV), d["A"].to(DEV), d["D"].to(DEV), dy.to(DEV), plan=plan or _plan(d),
                                    H=d["H"], G=d["G"], h_in=d["h"].to(DEV), dh_out=dh.to(DEV), **kw)


@pytest.mark.parametrize("lens,H,G,resume", [
    ([130, 64], 3, 1, [1, 0]),                  # an odd number of heads, one to a block
    ([200, 10, 0, 70], 6, 6, [1, 1, 1, 0]),     # every head its own group
    ([300, 65, 700], 24, 1, [0, 1, 1]),         # blocks of two heads
    ([1500, 1, 2339], 20, 1, [1, 1, 0]),        # blocks of eight heads, the last of four
    ([900, 0, 0, 33, 800], 32, 2, [1, 1, 0, 0, 1]),
])
def test_gradient_blocks_of_heads(lens, H, G, resume):
    """(the 64-bit recurrence runs on the GPU)"""
    n = len(lens)
    d = _data(lens, H, 64, 128, G, torch.bfloat16, 51, slots=list(range(n))[::-1], resume=resume, before=1, behind=2, n_slots=n)
    dy, dh = _grad_inputs(d, 52)
    x, B, C = (t.to(DEV) for t in _ref_in(d))
    with torch.device(DEV):
        r = ref.scan_grad(x, B, C, d["dt"].to(DEV), d["A"].to(DEV), d["D"].to(DEV), d["cu"], d["slots"], resume, d["h"].to(DEV),
                          dy.to(DEV).view(-1, H, 64), dh.to(DEV), G)
    plan = _plan(d)
    o = _grads(d, dy, dh, plan)
    a, b = d["cu"][0], d["cu"][-1]
    for k in r:
        got, want = (o[k], r[k]) if k in ("dA", "dD", "dh_in") else (o[k][a:b], r[k][a:b])
        assert ref.rel(got, want) <= 1e-5, (k, ref.rel(got, want))
    p = _grads(d, dy, dh, plan)
    ssd.sync_status()
    for k in r:                                 # sums in a fixed order
        u, v = (o[k], p[k]) if k in ("dA", "dD", "dh_in") else (o[k][a:b], p[k][a:b])
        assert torch.equal(u, v), k


@pytest.mark.parametrize("dtype,P,N", [(torch.bfloat16, 64, 128), (torch.float32, 16, 16)])
@pytest.mark.parametrize("behind", [0, 5])
def test_nothing_but_empty_sequences(dtype, P, N, behind):
    """States pass through, gradients of the weights are zero, rows of no sequence stay."""
    d = _data([0, 0, 0], 2, P, N, 1, dtype, 53, slots=[2, 0, 1], resume=[1, 0, 1], behind=behind, n_slots=3)
    pool = d["h"].to(DEV)
    _run(d, h_in=pool, h_out=pool)
    want = d["h"].clone()
    want[0] = 0
    assert torch.equal(pool.cpu(), want)
    dy, dh = _grad_inputs(d, 54)
    o = _grads(d, dy, dh)
    ssd.sync_status()
    assert (o["dA"] == 0).all() and (o["dD"] == 0).all()
    assert torch.equal(o["dh_in"].cpu(), dh * torch.tensor([1.0, 0.0, 1.0])[:, None, None, None])


def _refused():
    with pytest.raises(ssd.SSDError) as e:
        ssd.sync_status()
    assert e.value.code == 10


@pytest.mark.parametrize("cu,slots,kept", [
    ([0, 40, 30, 100], [0, 1, 2], [0]),             # an offset behind the next one
    ([0, 40, 70, 999], [0, 1, 2], [0, 1]),          # behind the rows
    ([-3, 40, 70, 100], [0, 1, 2], [1, 2]),         # before them
    ([0, 40, 70, 100], [0, 7, -9], [0]),            # slots that are none: computed, not kept
    ([0, 40, 70, 100], [1, 1, 1], [0]),             # a slot named twice belongs to the first
])
@pytest.mark.parametrize("dtype,P,N", [(torch.bfloat16, 64, 128), (torch.float32, 16, 16)])
def test_refused_offsets_and_slots(cu, slots, kept, dtype, P, N):
    """What a plan refuses is reported, reads and writes nothing out of place, and leaves the other sequences as they are."""
    total = 100
    d = _data([total], 2, P, N, 1, dtype, 55, n_slots=3)
    pool = d["h"].to(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    plan = ssd.packed_plan(torch.tensor(cu, **i32), total, slots=torch.tensor(slots, **i32), resume=torch.ones(3, **i32), n_slots=3)
    y = torch.full((total, 2, P), 7.0, dtype=dtype, device=DEV)
    _run(d, plan=plan, h_in=pool, h_out=pool, y=y)
    dy, _ = _grad_inputs(d, 56)
    o = _grads(d, dy, torch.zeros(3, 2, P, N), plan)
    torch.cuda.synchronize()
    _refused()
    assert all(torch.isfinite(o[k]).all() for k in ("dA", "dD"))
    touched = {slots[i] for i in kept}
    for i in kept:
        a, b = cu[i], cu[i + 1]
        e = dict(d, cu=[0, b - a], total=b - a, slots=[slots[i]], resume=[1], v=d["v"][a:b], dt=d["dt"][a:b])
        p1 = d["h"].to(DEV)
        y1, _ = _run(e, h_in=p1, h_out=p1)
        ssd.sync_status()
        assert torch.equal(p1[slots[i]], pool[slots[i]]) and torch.equal(y1, y[a:b])
    for k in set(range(3)) - touched:
        assert torch.equal(pool[k].cpu(), d["h"][k])


@pytest.mark.parametrize("dtype,P,N", [(torch.bfloat16, 64, 128), (torch.float32, 32, 16)])
def test_two_streams_at_once(dtype, P, N):
    """Two batches in flight on two streams, each with its own workspace, get what each gets alone."""
    ds = [_data([900, 40, 128], 4, P, N, 1, dtype, 57), _data([33, 700, 64, 1], 4, P, N, 2, dtype, 58)]
    alone = []
    for d in ds:
        dy, dh = _grad_inputs(d, 59)
        plan = _plan(d)
        y, h = _run(d, plan=plan, h_in=d["h"].to(DEV), h_out=d["h"].to(DEV))
        alone.append((d, dy, dh, plan, y, h, _grads(d, dy, dh, plan)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    for _ in range(3):
        got = []
        for s, (d, dy, dh, plan, *_x) in zip(streams, alone):
            with torch.cuda.stream(s):
                got.append((*_run(d, plan=plan, h_in=d["h"].to(DEV), h_out=d["h"].to(DEV)), _grads(d, dy, dh, plan)))
        torch.cuda.synchronize()
        for (y, h, o), (d, _a, _b, _c, y0, h0, o0) in zip(got, alone):
            assert torch.equal(y, y0) and torch.equal(h, h0)
            for k in o0:
                assert torch.equal(o[k], o0[k]), k
    ssd.sync_status()


@pytest.mark.parametrize("dtype,P,N", [(torch.bfloat16, 64, 128), (torch.float32, 32, 16)])
def test_on_a_stream_that_is_behind(dtype, P, N):
    """A call on a stream of its own allocates and clears there: tensors that the current stream makes meanwhile do not
    take the place of its workspace and outputs."""
    d = _data([700, 40, 128], 4, P, N, 1, dtype, 63)
    dy, dh = _grad_inputs(d, 64)
    x, B, C = _parts(d, d["v"].to(DEV))
    dt, A, D, h0, dy, dh = (t.to(DEV) for t in (d["dt"], d["A"], d["D"], d["h"], dy, dh))
    u, w = torch.randn(d["total"], x.shape[1] + 2 * N, device=DEV).to(dtype), torch.randn(x.shape[1] + 2 * N, 4, device=DEV)
    z, nw = torch.randn_like(dy), torch.randn(4 * P, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    cu, slots, resume = torch.tensor(d["cu"], **i32), torch.tensor(d["slots"], **i32), torch.tensor(d["resume"], **i32)

    def calls(stream):
        plan = ssd.packed_plan(cu, d["total"], slots=slots, resume=resume, n_slots=d["n_slots"], stream=stream)
        v = ssd.packed_conv_forward(u, w, plan, stream=stream)[0]
        y, _ = ssd.packed_scan_forward(x, B, C, dt, A, D, plan=plan, H=4, h_in=h0, stream=stream)
        o = ssd.packed_scan_backward(x, B, C, dt, A, D, dy, plan=plan, H=4, h_in=h0, dh_out=dh, stream=stream)
        c = ssd.packed_conv_backward(u, w, plan, o["dx"], o["dB"], o["dC"], stream=stream)
        n = ssd.gated_rmsnorm_backward(dy, x.contiguous(), z, nw, stream=stream)
        return {"v": v, "y": y, **{"s" + k: t for k, t in o.items()}, **{"c" + k: t for k, t in c.items()}, **{"n" + k: t for k, t in n.items()}}

    want = calls(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
    got = calls(s)
    junk = [torch.full((1 << 22,), float("nan"), device=DEV) for _ in range(64)]
    torch.cuda.synchronize()
    ssd.sync_status()
    del junk
    for k, t in want.items():
        assert t is None or torch.equal(got[k], t), k


def test_captured_batch_replayed_with_other_offsets():
    """Plan, convolution, scan and their gradients in one graph, replayed for batches of other lengths in the same buffers."""
    H, P, N, G, total, nseq = 4, 64, 128, 1, 512, 4
    cch, g = H * P + 2 * G * N, torch.Generator().manual_seed(60)
    u = torch.randn(total, cch, generator=g).to(DEV, torch.bfloat16)
    w, bias = (torch.randn(cch, 4, generator=g) / 2).to(DEV), torch.randn(cch, generator=g).to(DEV)
    dt = (torch.rand(total, H, generator=g) * 0.1).to(DEV)
    A, D = -torch.exp(torch.rand(H, generator=g) * 2.77).to(DEV), torch.randn(H, generator=g).to(DEV)
    dy = torch.randn(total, H * P, generator=g).to(DEV, torch.bfloat16)
    tail0, h0 = torch.randn(nseq, 3, cch, generator=g).to(DEV, torch.bfloat16), torch.randn(nseq, H, P, N, generator=g).to(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    cu, slots, resume = torch.tensor([0, 100, 100, 300, 512], **i32), torch.tensor([0, 1, 2, 3], **i32), torch.ones(nseq, **i32)
    tail, h = tail0.clone(), h0.clone()
    keep = {}

    def step():
        plan = ssd.packed_plan(cu, total, slots=slots, resume=resume, n_slots=nseq)
        t_in, h_in = tail.clone(), h.clone()
        v = ssd.packed_conv_forward(u, w, plan, bias, tail_in=t_in, tail_out=tail)
        v = v[0] if isinstance(v, tuple) else v
        x, B, C = v[:, :H * P], v[:, H * P:H * P + N], v[:, H * P + N:]
        y, _ = ssd.packed_scan_forward(x, B, C, dt, A, D, plan=plan, H=H, G=G, h_in=h_in, h_out=h)
        o = ssd.packed_scan_backward(x, B, C, dt, A, D, dy, plan=plan, H=H, G=G, h_in=h_in)
        c = ssd.packed_conv_backward(u, w, plan, o["dx"].view(total, -1), o["dB"].view(total, -1), o["dC"].view(total, -1), bias=bias, tail_in=t_in)
        keep.update(y=y, **{"s_" + k: t for k, t in o.items()}, **{"c_" + k: t for k, t in c.items() if t is not None})

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graphed = dict(keep)
    for c, k, r in (([0, 100, 100, 300, 512], [0, 1, 2, 3], [1, 1, 1, 1]), ([0, 512, 512, 512, 512], [3, 1, 0, 2], [1, 0, 1, 1]),
                    ([7, 8, 200, 201, 500], [2, -1, 0, 3], [0, 1, 1, 1])):
        for t, v in ((cu, c), (slots, k), (resume, r)):
            t.copy_(torch.tensor(v, dtype=torch.int32))
        tail.copy_(tail0)
        h.copy_(h0)
        graph.replay()
        torch.cuda.synchronize()
        got, gt, gh = {n: t.clone() for n, t in graphed.items()}, tail.clone(), h.clone()
        tail.copy_(tail0)
        h.copy_(h0)
        step()
        ssd.sync_status()
        assert torch.equal(gt, tail) and torch.equal(gh, h)
        for n, t in keep.items():
            a, b = (c[0], c[-1]) if t.shape[0] == total else (0, t.shape[0])
            assert torch.equal(got[n][a:b], t[a:b]), n


@pytest.mark.parametrize("dtype,P,N", [(torch.bfloat16, 64, 128), (torch.float32, 32, 16)])
def test_rows_far_apart(dtype, P, N):
    """Rows whose offsets pass 32 bits (views of a buffer of 2.2e9 elements) give what rows side by side give."""
    d = _data([200, 31, 65], 2, P, N, 1, dtype, 67)
    total, cch, far = d["total"], 2 * P + 2 * N, 7_400_000
    assert (total - 1) * far > 1 << 31
    dy, dh = _grad_inputs(d, 68)
    wide = torch.empty(total, far, dtype=dtype, device=DEV)
    v, dyw, yw = wide[:, :cch], wide[:, 4096:4096 + 2 * P], wide[:, 8192:8192 + 2 * P].unflatten(1, (2, P))
    v.copy_(d["v"])
    dyw.copy_(dy)
    plan = _plan(d)
    dt, A, D, h0, dh = (t.to(DEV) for t in (d["dt"], d["A"], d["D"], d["h"], dh))
    got = []
    for src, g, y in ((d["v"].to(DEV), dy.to(DEV), None), (v, dyw, yw)):
        x, B, C = _parts(d, src)
        y, h = ssd.packed_scan_forward(x, B, C, dt, A, D, plan=plan, H=2, h_in=h0, h_out=h0.clone(), y=y)
        o = ssd.packed_scan_backward(x, B, C, dt, A, D, g, plan=plan, H=2, h_in=h0, dh_out=dh)
        w = torch.linspace(-0.5, 0.5, cch * 4, device=DEV).view(cch, 4)
        c = ssd.packed_conv_forward(src, w, plan)[0]
        e = ssd.packed_conv_backward(src, w, plan, o["dx"], o["dB"], o["dC"])
        got.append({"y": y, "h": h, "v": c, **{"s" + k: t for k, t in o.items()}, **{"c" + k: t for k, t in e.items()}})
    ssd.sync_status()
    for k, t in got[0].items():
        assert t is None or torch.equal(got[1][k], t), k


@pytest.mark.parametrize("dtype,P,N,H", [(torch.bfloat16, 64, 128, 4), (torch.bfloat16, 64, 128, 16), (torch.float32, 32, 16, 2)])
def test_what_may_be_left_out(dtype, P, N, H):
    """Without D, start states and the states' gradients: as with zeros.  A slot that a sequence does not resume from is not
    read, whatever it holds."""
    lens = [1100, 70]
    d = _data(lens, H, P, N, 1, dtype, 72, resume=[0, 0], n_slots=2)
    dy, dh = _grad_inputs(d, 73)
    plan = _plan(d)
    x, B, C = _parts(d, d["v"].to(DEV))
    dt, A, dy = d["dt"].to(DEV), d["A"].to(DEV), dy.to(DEV)
    none = ssd.packed_scan_backward(x, B, C, dt, A, None, dy, plan=plan, H=H)
    y0, _ = ssd.packed_scan_forward(x, B, C, dt, A, None, plan=plan, H=H)
    bad = torch.full((2, H, P, N), float("nan"), device=DEV)
    zero = ssd.packed_scan_backward(x, B, C, dt, A, torch.zeros(H, device=DEV), dy, plan=plan, H=H, h_in=bad, dh_out=torch.zeros_like(bad))
    y1, h = ssd.packed_scan_forward(x, B, C, dt, A, torch.zeros(H, device=DEV), plan=plan, H=H, h_in=bad, h_out=bad)
    ssd.sync_status()
    assert torch.equal(y0, y1) and torch.isfinite(h).all()
    for k in ("dx", "dB", "dC", "ddt", "dA"):
        assert torch.equal(none[k], zero[k]), k
    assert (zero["dh_in"] == 0).all()


@pytest.mark.parametrize("dtype,P,N,H", [(torch.bfloat16, 64, 128, 4), (torch.float32, 32, 16, 2)])
def test_batch_padded_with_empty_sequences(dtype, P, N, H):
    """Empty sequences without a slot change nothing of the others, and their states' and buffers' gradients are zero."""
    lens, cch = [100, 0, 0, 300, 0, 30, 0, 0, 0], H * P + 2 * N
    slots, resume = [2, -1, -1, 0, 3, 1, -1, -1, -1], [1, 1, 0, 1, 1, 0, 1, 1, 1]
    on = [i for i, m in enumerate(lens) if m]
    d = _data(lens, H, P, N, 1, dtype, 74, slots=slots, resume=resume, n_slots=4)
    dy, dh = _grad_inputs(d, 75)
    bare = dict(d, cu=[0, 100, 400, 430], slots=[2, 0, 1], resume=[1, 1, 0])
    g = torch.Generator().manual_seed(76)
    w, bias = (torch.rand(cch, 4, generator=g) - 0.5).to(DEV), torch.randn(cch, generator=g).to(DEV)
    tails = torch.randn(4, 3, cch, generator=g).to(DEV, dtype)
    got = []
    for e, dhe in ((d, dh), (bare, dh[on])):
        plan, n = _plan(e), len(e["slots"])
        y, h = _run(e, plan=plan, h_in=d["h"].to(DEV), h_out=d["h"].to(DEV))
        out = {"dh_in": torch.full((n, H, P, N), float("nan"), device=DEV)}
        o = _grads(e, dy, dhe, plan, out=out)
        u = d["v"].to(DEV)
        v, t = ssd.packed_conv_forward(u, w, plan, bias, tail_in=tails, tail_out=tails.clone())
        c = ssd.packed_conv_backward(u, w, plan, o["dx"], o["dB"], o["dC"], bias=bias, tail_in=tails,
                                     out={"dtail_in": torch.full((n, 3, cch), float("nan"), device=DEV)})
        got.append({"y": y, "h": h, "v": v, "t": t, **{"s" + k: x for k, x in o.items()}, **{"c" + k: x for k, x in c.items() if x is not None}})
    ssd.sync_status()
    for k, x in got[1].items():
        z = got[0][k]
        if k in ("sdh_in", "cdtail_in"):
            rest = [i for i in range(len(lens)) if i not in on and slots[i] < 0]
            assert (z[rest] == 0).all() and torch.isfinite(z).all(), k
            z = z[on]
        if k in ("y", "h", "sdA", "sdD", "cdconv_w", "cdconv_bias"):
            # (windows and partial sums are cut elsewhere)
            assert ref.rel(z.float(), x.float()) <= (1e-5 if z.dtype == torch.float32 else 2.0 ** -8), k
        else:
            assert ref.rel(z.float(), x.float()) <= 1e-5, k


def test_slots_far_into_a_large_pool():
    """States past 2^31 elements of their pool (8.8 GB): prompts, their gradients and a token give what a small pool gives."""
    H, P, N, many = 64, 64, 128, 4200
    assert (many - 1) * H * P * N > 1 << 31
    d = _data([130, 20], H, P, N, 1, torch.bfloat16, 69, slots=[0, 1], n_slots=2)
    cch, g = H * P + 2 * N, torch.Generator().manual_seed(70)
    dy, dh = _grad_inputs(d, 71)
    x, B, C = _parts(d, d["v"].to(DEV))
    dt, A, D, h0, dy, dh = (t.to(DEV) for t in (d["dt"], d["A"], d["D"], d["h"], dy, dh))
    u, w = torch.randn(2, cch, generator=g).to(DEV, torch.bfloat16), (torch.rand(cch, 4, generator=g) - 0.5).to(DEV)
    tails = torch.randn(2, 3, cch, generator=g).to(DEV, torch.bfloat16)
    i32 = dict(dtype=torch.int32, device=DEV)
    cu, got = torch.tensor(d["cu"], **i32), []
    for n, ks in ((2, [0, 1]), (many, [many - 1, many - 2])):
        slots = torch.tensor(ks, **i32)
        pool, tp = torch.empty(n, H, P, N, device=DEV), torch.empty(n, 3, cch, dtype=torch.bfloat16, device=DEV)
        pool[slots.long()], tp[slots.long()] = h0, tails
        plan = ssd.packed_plan(cu, d["total"], slots=slots, n_slots=n)
        o = ssd.packed_scan_backward(x, B, C, dt, A, D, dy, plan=plan, H=H, h_in=pool, dh_out=dh)
        y, _ = ssd.packed_scan_forward(x, B, C, dt, A, D, plan=plan, H=H, h_in=pool, h_out=pool)
        s = ssd.decode_slots(u, w, dt[:2].contiguous(), A, D, slots=slots, H=H, P=P, N=N, tail_in=tp, h_in=pool)
        got.append({"y": y, "t": s["y"], "h": pool[slots.long()], "tail": tp[slots.long()], **o})
        del pool
    ssd.sync_status()
    for k, t in got[0].items():
        assert torch.equal(got[1][k], t), k


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("total", [130, 2400, 5000, 12000])
def test_convolution_in_pieces_is_the_layers(total, dtype):
    """Whatever pieces of a chunk a thread takes (8, 4, 2 and 1 at these sizes), each sequence gets the layer's
    convolution bit for bit, and hands on its last rows."""
    cch = 2304
    lens = [total - total // 3 - 66, 1, 65, total // 3]
    g = torch.Generator().manual_seed(65)
    u = torch.randn(total, cch, generator=g).to(DEV, dtype)
    w, bias = (torch.rand(cch, 4, generator=g) - 0.5).to(DEV), torch.randn(cch, generator=g).to(DEV)
    tails = torch.randn(4, 3, cch, generator=g).to(DEV, dtype)
    i32 = dict(dtype=torch.int32, device=DEV)
    cu = [0, lens[0], lens[0] + 1, lens[0] + 66, total]
    plan = ssd.packed_plan(torch.tensor(cu, **i32), total, slots=torch.tensor([2, 0, 1, 3], **i32), resume=torch.tensor([1, 1, 0, 1], **i32), n_slots=4)
    t = tails.clone()
    v = ssd.packed_conv_forward(u, w, plan, bias, tail_in=t, tail_out=t)[0]
    ssd.sync_status()
    for i, (k, r) in enumerate(zip([2, 0, 1, 3], [1, 1, 0, 1])):
        rows = u[None, cu[i]:cu[i + 1]]
        tail = tails[k][None] if r else torch.zeros_like(tails[k])[None]
        one = ssd.conv_forward(rows, w, bias, tail_in=tail)
        one = one[0] if isinstance(one, tuple) else one
        assert torch.equal(v[cu[i]:cu[i + 1]], one[0]), i
        assert torch.equal(t[k], torch.cat((tail[0], rows[0]))[-3:]), i


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,d,group", [(700, 4096, 0), (601, 4096, 1024), (450, 5120, 0), (460, 5120, 1280), (301, 6144, 0), (310, 8192, 2048)])
def test_norm_gradient_of_wide_rows(rows, d, group, dtype):
    """Several rows per CTA at every number of threads a row can take."""
    g = torch.Generator().manual_seed(66)
    dout, y, z = (torch.randn(rows, d, generator=g).to(DEV, dtype) for _ in range(3))
    w = (1 + 0.2 * torch.randn(d, generator=g)).to(DEV)
    dy, dz, dw = ref.norm_grad(dout, y, z, w, 1e-5, group or d)
    o = ssd.gated_rmsnorm_backward(dout, y, z, w, eps=1e-5, group_size=group)
    ssd.sync_status()
    assert ref.rel(o["dweight"], dw) <= 1e-5
    for k, r in (("dy", dy), ("dz", dz)):
        # one rounding of half a step of bf16 per element, in the 2-norm below its largest 2^-8
        assert ref.rel(o[k], r) <= (1e-5 if dtype == torch.float32 else 2.0 ** -8), k


def _child(backward):
    d = _data([700, 300], 4, 64, 128, 1, torch.bfloat16, 61)
    dy, dh = _grad_inputs(d, 62)

    def call():
        if backward:
            return _grads(d, dy, dh)["dx"]
        return _run(d, h_in=d["h"].to(DEV), h_out=d["h"].to(DEV))[0]

    call()
    try:
        ssd.sync_status()
    except ssd.SSDError as e:
        assert e.code == 8, e
    else:
        raise AssertionError("the dropped unit did not time out")
    ssd.sync_status()
    a, b = call(), call()
    ssd.sync_status()
    assert torch.isfinite(a).all() and torch.equal(a, b)
    print("child ok")


@pytest.mark.parametrize("backward", [0, 1])
def test_wait_that_runs_out_is_reported(backward):
    """One CTA's products are left out in the first call of a process (its hook): every wait for them is bounded, the status
    says so, and the calls after it are right."""
    env = dict(os.environ, SSD_TEST_DROP_UNIT="0", SSD_WAIT_LIMIT_MS="200")
    r = subprocess.run([sys.executable, os.path.abspath(__file__), str(backward)], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "child ok" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


if __name__ == "__main__":
    _child(int(sys.argv[1]))
