"""The packed operators where a batch has less to do than its buffers hold, and at shapes of their own.

Tolerances as in test_gpu_packed_scan.py and test_gpu_slots.py (relL2 1e-5 against 64 bits for fp32 outputs); where two
calls have the same arithmetic, their outputs are equal.
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


@pytest.mark.parametrize("lens", [[1] * 5, [3, 0, 70], [1, 500, 2]])
@pytest.mark.parametrize("H,dtype,P,N", [(16, torch.bfloat16, 64, 128), (32, torch.bfloat16, 64, 128), (4, torch.float32, 32, 16)])
def test_gradient_of_few_rows_in_large_buffers(H, dtype, P, N, lens):
    """Rows of no sequence behind a few live ones change no bit of their gradients (a captured batch in buffers of a fixed
    size), and those are as near to 64 bits as in buffers of their own."""
    n = len(lens)
    for seed in range(4):
        got = []
        for behind in (0, 8192):
            d = _data(lens, H, P, N, 1, dtype, 80 + seed)
            g = torch.Generator().manual_seed(90 + seed)
            live = d["total"]
            dy, dh = torch.randn(live, H * P, generator=g).to(dtype), torch.randn(n, H, P, N, generator=g)
            more = lambda t: torch.cat((t, torch.full((behind, t.shape[1]), float("nan")).to(t.dtype))).to(DEV)  # noqa: E731
            x, B, C = _parts(d, more(d["v"]))
            plan = _plan(dict(d, total=live + behind))
            o = ssd.packed_scan_backward(x, B, C, more(d["dt"]), d["A"].to(DEV), d["D"].to(DEV), more(dy), plan=plan, H=H,
                                         h_in=d["h"].to(DEV), dh_out=dh.to(DEV))
            got.append({k: t if k in ("dA", "dD", "dh_in") else t[:live] for k, t in o.items()})
        ssd.sync_status()
        for k, t in got[0].items():
            assert torch.equal(got[1][k], t), k
        x, B, C = _ref_in(d)
        r = ref.scan_grad(x, B, C, d["dt"], d["A"], d["D"], d["cu"], d["slots"], d["resume"], d["h"], dy.view(-1, H, P), dh, 1)
        for k, t in got[1].items():
            assert ref.rel(t, r[k]) <= 1e-5, (k, ref.rel(t, r[k]))


@pytest.mark.parametrize("dtype,P,N,H", [(torch.bfloat16, 64, 128, 4), (torch.float32, 32, 16, 2)])
def test_start_states_left_out_are_zeros(dtype, P, N, H):
    """Without h_in and tail_in every sequence starts from zeros: as with pools of zeros, only that no sequence has a state or a
    buffer whose gradient could be asked for."""
    lens, cch = [100, 0, 2, 65], H * P + 2 * N
    d = _data(lens, H, P, N, 1, dtype, 85, resume=[1, 1, 1, 0])
    g = torch.Generator().manual_seed(86)
    dy, dh = torch.randn(d["total"], H * P, generator=g).to(DEV, dtype), torch.randn(4, H, P, N, generator=g).to(DEV)
    w, dtail = (torch.rand(cch, 4, generator=g) - 0.5).to(DEV), torch.randn(4, 3, cch, generator=g).to(DEV)
    u, plan = d["v"].to(DEV), _plan(d)
    x, B, C = _parts(d, u)
    got = []
    for h0, t0 in ((None, None), (torch.zeros_like(d["h"]).to(DEV), torch.zeros(d["n_slots"], 3, cch, device=DEV, dtype=dtype))):
        out = {"dh_in": torch.full_like(dh, float("nan"))}
        o = ssd.packed_scan_backward(x, B, C, d["dt"].to(DEV), d["A"].to(DEV), d["D"].to(DEV), dy, plan=plan, H=H, h_in=h0, dh_out=dh, out=out)
        c = ssd.packed_conv_backward(u, w, plan, o["dx"], o["dB"], o["dC"], tail_in=t0, dtail_out=dtail,
                                     out={"dtail_in": torch.full_like(dtail, float("nan"))})
        got.append({**o, **c})
    ssd.sync_status()
    for k, t in got[0].items():
        if k in ("dh_in", "dtail_in"):
            norms = got[1][k].flatten(1).norm(dim=1)
            assert (t == 0).all() and (norms[:3] > 0).all() and norms[3] == 0, k
        else:
            assert torch.equal(got[1][k], t), k


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b", [2, 12])
def test_step_of_many_groups(b, dtype):
    """A group to each of 40 heads: 10240 channels of B and C, more than the CTAs of a stream hold in registers."""
    from test_gpu_slots import _pool, _ref_step, _step
    slots = [(4 * i + 1) % (b + 3) for i in range(b)]
    d = _pool(b, b + 3, 40, 16, 128, 40, dtype, slots, 87)
    y, h, tail, ya = _ref_step(d, slots)
    hp, tp = d["h"].to(DEV), d["tail"].to(DEV)
    o = _step(d, tail_in=tp, h_in=hp)
    ssd.sync_status()
    assert ref.rel(hp, h) <= 1e-5
    assert torch.equal(tp.cpu().double(), tail)
    near = (2.0 ** -8 if dtype == torch.bfloat16 else 0.0) * y.abs() + 2.0 ** -14 * ya
    assert ((o["y"].cpu().double() - y).abs() <= near).all()


def test_convolution_of_large_sums():
    """bf16 v element by element, sums z of up to about 10 either way: z sigma(z) = h + h tanh(h), h = z / 2, by a hardware tanh
    of relative error 2^-11 is off by 2^-11 |h|, by its fp32 sums 2^-20 of their terms, and by its rounding 2^-8 of what
    is rounded."""
    cch, total = 256, 700
    g = torch.Generator().manual_seed(89)
    u, w = 6 * torch.randn(total, cch, generator=g).to(torch.bfloat16), torch.rand(cch, 4, generator=g) - 0.5
    bias = torch.randn(cch, generator=g)
    plan = ssd.packed_plan(torch.tensor([0, 3, 400, total], **I32), total)
    v, _ = ssd.packed_conv_forward(u.to(DEV), w.to(DEV), plan, bias.to(DEV))
    ssd.sync_status()
    small = 0
    for a, b in ((0, 3), (3, 400), (400, total)):
        rows = torch.cat((torch.zeros(3, cch, dtype=torch.float64), u[a:b].double()))
        terms = torch.stack([rows[k:k + b - a] * w[:, k].double() for k in range(4)] + [bias.double().expand(b - a, -1)])
        z = terms.sum(0)
        want = z / (1 + torch.exp(-z))
        near = 2.0 ** -11 * z.abs() / 2 + 2.0 ** -20 * terms.abs().sum(0)
        near = near + 2.0 ** -8 * (want.abs() + near)
        assert ((v[a:b].cpu().double() - want).abs() <= near).all()
        small += int((z < -6).sum())
    assert small > 100



def _child():
    from test_gpu_slots import _pool, _step
    H, P, N, slots, dtype = 32, 64, 128, [4, 0, 2], torch.bfloat16
    d = _pool(3, 5, H, P, N, 1, dtype, slots, 88)
    hp, tp = d["h"].to(DEV), d["tail"].to(DEV)
    _step(d, tail_in=tp, h_in=hp)
    try:
        ssd.sync_status()
    except ssd.SSDError as e:
        assert e.code == 8, e
    else:
        raise AssertionError("the dropped unit did not time out")
    h1, t1 = d["h"].to(DEV), d["tail"].to(DEV)
    _step(d, tail_in=t1, h_in=h1)
    ssd.sync_status()
    for k in (4, 2, 1, 3):                  # the other streams, and the slots of none
        assert torch.equal(hp[k], h1[k]) and torch.equal(tp[k], t1[k]), k
    # 16 CTAs to a stream: the second one of the second stream has heads 2 and 3 and channels 16 .. 31 of B and C
    old, new = d["tail"][0].to(DEV), tp[0]
    for a, b in ((2 * P, 4 * P), (H * P + 16, H * P + 32)):
        assert torch.equal(new[:, a:b], old[:, a:b])
    assert torch.equal(hp[0, 2:4], d["h"][0, 2:4].to(DEV))
    print("child ok")


def test_step_whose_copies_never_come():
    """A CTA of the slot step that gives up writes none of its states and nothing into the conv buffer; the other streams and the
    next call are right."""
    env = dict(os.environ, SSD_TEST_DROP_UNIT="17", SSD_WAIT_LIMIT_MS="200")
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "child ok" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


if __name__ == "__main__":
    _child()
