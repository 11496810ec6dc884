"""Host side of the packed calls, the slot step and the norm's gradient: argument checks, sizes and the binding's refusals
(no GPU needed: nothing here launches)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def ssd():
    import __graft_entry__
    __graft_entry__.build()
    import mamba_selective_state_causal_b200 as pkg
    return pkg


def _args(cls, base, **kw):
    a = cls()
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


PLAN = dict(nseq=3, total=500, cu_seqlens=0x1000, slots=0x2000, resume=None, n_slots=5, max_seqlen=0, plan=0x10000, plan_bytes=1 << 20)


@pytest.mark.parametrize("change,code", [
    (dict(nseq=-1), 2), (dict(total=-1), 2), (dict(total=1 << 31), 2), (dict(plan=None), 1), (dict(plan=0x10004), 3),
    (dict(plan_bytes=64), 9), (dict(cu_seqlens=None), 1), (dict(n_slots=-1), 2), (dict(max_seqlen=-5), 2),
    (dict(slots=None, n_slots=2), 2), (dict(nseq=20000, plan_bytes=1 << 24), 6),
])
def test_plan_refuses(ssd, change, code):
    assert ssd.lib().ssd_packed_plan(ctypes.byref(_args(ssd.PackedPlanArgs, PLAN, **change)), None) == code
    assert ssd.lib().ssd_last_error_string()


def test_plan_size(ssd):
    """64 bytes of header, 32 per sequence, 16 per chunk of 64 and of 128 rows (one more of each per sequence)."""
    for n, t in ((0, 0), (1, 1), (3, 500), (256, 8191), (7, 65536)):
        need = 64 + 32 * n + 16 * (t // 64 + n) + 16 * (t // 128 + n)
        assert ssd.lib().ssd_packed_plan_size(n, t) == (need + 255) // 256 * 256


CONV = dict(dtype=1, nseq=3, total=500, C_ch=384, plan=0x10000, u=0x20000, u_row_stride=384, conv_w=0x30000, conv_bias=None,
            tail_in=None, tail_out=0x40000, v=0x50000, v_row_stride=384)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), 5), (dict(C_ch=380), 2), (dict(C_ch=0), 2), (dict(nseq=-1), 2), (dict(plan=None), 1), (dict(u=None), 1),
    (dict(u_row_stride=383), 4), (dict(u_row_stride=388), 3), (dict(u=0x20008), 3), (dict(v=None), 1), (dict(v=0x20000), 2),
    (dict(conv_w=None), 1), (dict(conv_w=0x30004), 3), (dict(tail_out=0x40002), 3),
])
def test_conv_refuses(ssd, change, code):
    assert ssd.lib().ssd_packed_conv_forward(ctypes.byref(_args(ssd.PackedConvArgs, CONV, **change)), None) == code


CONVB = dict(dtype=1, nseq=3, total=500, d_inner=256, d_bc=64, plan=0x10000, u=0x20000, u_row_stride=384, conv_w=0x30000,
             conv_bias=None, tail_in=None, dx=0x40000, dB=0x50000, dC=0x60000, dtail_out=None, du=0x70000, dtail_in=None,
             dconv_w=0x80000, dconv_bias=None, workspace=0x100000, workspace_bytes=1 << 30)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=9), 5), (dict(d_inner=250), 2), (dict(d_bc=0), 2), (dict(conv_w=None), 1), (dict(dconv_w=None), 1), (dict(dx=None), 1),
    (dict(dC=0x60004), 3), (dict(workspace=None), 9), (dict(workspace_bytes=100), 9), (dict(workspace=0x100010), 3),
    (dict(u_row_stride=100), 4), (dict(plan=None), 1),
])
def test_conv_backward_refuses(ssd, change, code):
    assert ssd.lib().ssd_packed_conv_backward(ctypes.byref(_args(ssd.PackedConvBwdArgs, CONVB, **change)), None) == code


SCAN = dict(dtype=1, nseq=3, total=5000, max_seqlen=0, H=4, P=64, N=128, G=1, plan=0x10000, x=0x20000, x_row_stride=512,
            B=0x30000, B_row_stride=512, C=0x40000, C_row_stride=512, dt=0x50000, A=0x60000, D=None, h_in=None, h_out=0x70000,
            y=0x80000, y_row_stride=256, workspace=0x100000, workspace_bytes=1 << 34)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=2), 5), (dict(P=48), 2), (dict(N=256), 2), (dict(H=3, G=2), 2), (dict(G=0), 2), (dict(x=None), 1), (dict(dt=None), 1),
    (dict(A=None), 1), (dict(x_row_stride=200), 4), (dict(x=0x20008), 3), (dict(B_row_stride=511), 3), (dict(dt=0x50004), 3),
    (dict(h_out=0x70004), 3), (dict(workspace=None), 9), (dict(workspace_bytes=1), 9), (dict(y_row_stride=128), 4),
    (dict(max_seqlen=-1), 2), (dict(total=1 << 31), 2), (dict(plan=0x10001), 3),
])
def test_scan_refuses(ssd, change, code):
    assert ssd.lib().ssd_packed_scan_forward(ctypes.byref(_args(ssd.PackedScanArgs, SCAN, **change)), None) == code


def test_scan_workspace(ssd):
    """Nothing is handed on between windows when no sequence has a second chunk; else two or three states per window and head."""
    f = ssd.lib().ssd_packed_scan_workspace_size
    assert f(40, 4000, 128, 32, 64, 128, 1, 1) == 0
    assert f(40, 4000, 64, 32, 64, 128, 1, 0) == 0
    assert f(0, 0, 0, 32, 64, 128, 1, 1) == 0
    n = f(2, 65536, 0, 32, 64, 128, 1, 1)
    state = 32 * 64 * 128 * 4
    assert n >= 2 * state and (n - 1) // (2 * state) <= 148


BWD = dict(dtype=1, nseq=3, total=500, H=4, P=64, N=128, G=1, plan=0x10000, x=0x20000, x_row_stride=512, B=0x30000, B_row_stride=512,
           C=0x40000, C_row_stride=512, dt=0x50000, A=0x60000, D=None, h_in=None, dy=0x70000, dy_row_stride=256, dh_out=None,
           dx=0x80000, dB=0x90000, dC=0xa0000, ddt=0xb0000, dA=0xc0000, dD=None, dh_in=None, workspace=0x1000000, workspace_bytes=1 << 34)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=2), 5), (dict(P=48), 2), (dict(dA=None), 1), (dict(dx=None), 1), (dict(dy=None), 1), (dict(dy_row_stride=100), 4),
    (dict(dB=0x90004), 3), (dict(workspace=None), 9), (dict(workspace_bytes=4), 9), (dict(dt=None), 1), (dict(plan=None), 1),
])
def test_scan_backward_refuses(ssd, change, code):
    assert ssd.lib().ssd_packed_scan_backward(ctypes.byref(_args(ssd.PackedScanBwdArgs, BWD, **change)), None) == code


STEP = dict(dtype=1, b=4, n_slots=9, H=4, P=64, N=128, G=1, slots=0x1000, u=0x20000, u_batch_stride=512, conv_w=0x30000, conv_bias=None,
            tail_in=0x40000, tail_out=0x40000, dt=0x50000, A=0x60000, D=None, h_in=0x70000, h_out=0x70000, y=0x80000, y_batch_stride=256)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=2), 5), (dict(b=-1), 2), (dict(n_slots=-1), 2), (dict(P=8), 2), (dict(H=4, G=3), 2), (dict(slots=None), 1),
    (dict(h_in=None), 1), (dict(tail_out=None), 1), (dict(u=None), 1), (dict(u_batch_stride=500), 4), (dict(u_batch_stride=516), 3),
    (dict(h_out=0x70004), 3), (dict(y=None), 1), (dict(y_batch_stride=10), 4),
])
def test_step_refuses(ssd, change, code):
    assert ssd.lib().ssd_decode_slots(ctypes.byref(_args(ssd.DecodeSlotsArgs, STEP, **change)), None) == code


NORM = dict(dtype=1, rows=16, d=2048, group_size=0, eps=1e-5, dout=0x10000, dout_row_stride=2048, y=0x20000, y_row_stride=2048,
            z=0x30000, z_row_stride=2048, weight=0x40000, dy=0x50000, dy_row_stride=2048, dz=0x60000, dz_row_stride=2048,
            dweight=0x70000, workspace=0x100000, workspace_bytes=1 << 30)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=4), 5), (dict(d=2047), 2), (dict(d=16384), 2), (dict(group_size=100), 2), (dict(group_size=24), 2), (dict(eps=-1.0), 2),
    (dict(rows=-1), 2), (dict(y=None), 1), (dict(dout=None), 1), (dict(weight=None), 1), (dict(dweight=None), 1), (dict(z_row_stride=1024), 4),
    (dict(dz=0x60002), 3), (dict(dy_row_stride=2052), 3), (dict(weight=0x40004), 3), (dict(workspace=None), 9), (dict(workspace_bytes=8), 9),
])
def test_norm_backward_refuses(ssd, change, code):
    assert ssd.lib().ssd_gated_rmsnorm_backward(ctypes.byref(_args(ssd.GatedRmsnormBwdArgs, NORM, **change)), None) == code


def test_nothing_to_do_is_no_error(ssd):
    lib = ssd.lib()
    assert lib.ssd_packed_conv_forward(ctypes.byref(_args(ssd.PackedConvArgs, CONV, nseq=0, plan=None, u=None)), None) == 0
    assert lib.ssd_packed_scan_forward(ctypes.byref(_args(ssd.PackedScanArgs, SCAN, nseq=0, plan=None, x=None)), None) == 0
    assert lib.ssd_decode_slots(ctypes.byref(_args(ssd.DecodeSlotsArgs, STEP, b=0, slots=None)), None) == 0
    for f in ("ssd_packed_plan", "ssd_packed_conv_forward", "ssd_packed_scan_forward", "ssd_decode_slots", "ssd_gated_rmsnorm_backward",
              "ssd_packed_scan_backward", "ssd_packed_conv_backward"):
        assert getattr(lib, f)(None, None) == 1


def test_binding_refuses_host_tensors_and_wrong_shapes(ssd):
    cpu, f32 = torch.device("cpu"), torch.float32
    cu = torch.tensor([0, 3], dtype=torch.int32)
    with pytest.raises(ValueError):
        ssd.packed_plan(cu, 3)
    with pytest.raises(ValueError):
        ssd.gated_rmsnorm_backward(torch.zeros(2, 8), torch.zeros(2, 8), torch.zeros(2, 8), torch.ones(8))
    with pytest.raises(ValueError):
        ssd._rows2(torch.zeros(4, 6), 4, 8, f32, cpu, "u")
    with pytest.raises(ValueError):
        ssd._rows2(torch.zeros(4, 8), 5, 8, f32, cpu, "u")
    with pytest.raises(TypeError):
        ssd._rows2(torch.zeros(4, 8), 4, 8, torch.bfloat16, cpu, "u")
    with pytest.raises(ValueError):
        ssd._rows2(torch.zeros(8, 4).t(), 4, 8, f32, cpu, "u")
    with pytest.raises(ValueError):
        ssd._rows2(torch.zeros(4, 8), 4, 8, f32, torch.device("cuda:0"), "u")
    with pytest.raises(ValueError):
        ssd._ptr_of(torch.zeros(3), (4,), f32, cpu, "A")
    with pytest.raises(TypeError):
        ssd._ptr_of(torch.zeros(4, 2).t(), (2, 4), f32, cpu, "A")
    with pytest.raises(TypeError):
        ssd._ptr_of(torch.zeros(4, dtype=torch.float64), (4,), f32, cpu, "A")
    with pytest.raises(ValueError):
        ssd._ptr_of(torch.zeros(4), (4,), f32, torch.device("cuda:1"), "A")
    assert ssd._ptr_of(None, (4,), f32, cpu, "A") is None
    with pytest.raises(ValueError):
        ssd._head_dims(torch.zeros(4, 10), torch.zeros(4, 8), 3, 1)


def test_rows_of_a_view(ssd):
    """Column slices keep their row stride; one row takes its width, whatever stride it carries."""
    cpu, f32 = torch.device("cpu"), torch.float32
    t = torch.zeros(4, 32)
    assert ssd._rows2(t[:, 8:16], 4, 8, f32, cpu, "u") == (t.data_ptr() + 32, 32)
    assert ssd._rows2(t[:1, :8], 1, 8, f32, cpu, "u") == (t.data_ptr(), 8)
    y = torch.zeros(4, 2, 8)
    assert ssd._rows3(y, 4, 2, 8, f32, cpu, "y") == (y.data_ptr(), 16)
    wide = torch.zeros(4, 5, 8)
    assert ssd._rows3(wide[:, 1:3], 4, 2, 8, f32, cpu, "y") == (wide.data_ptr() + 32, 40)
    with pytest.raises(ValueError):
        ssd._rows3(y.transpose(1, 2), 4, 8, 2, f32, cpu, "y")


def test_binding_refuses_another_devices_stream(ssd):
    class Stream:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="stream"):
        ssd.decode_slots(torch.zeros(1, 48), None, None, None, slots=None, tail_in=None, h_in=None, H=1, P=16, N=16, stream=Stream())
