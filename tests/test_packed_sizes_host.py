"""Workspaces of the packed calls: on which device they are sized, and what the binding takes for one (no GPU needed)."""
import contextlib
import types

import pytest
import torch


@pytest.fixture(scope="module")
def ssd():
    import __graft_entry__
    __graft_entry__.build()
    import mamba_selective_state_causal_b200 as pkg
    return pkg


def test_sized_on_the_plans_device(ssd, monkeypatch):
    """The sizes go by the number of SMs: they are asked for with the plan's device current, whichever one was."""
    current = ["cuda:0"]

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], str(torch.device(d))
        yield
        current[0] = before

    asked = {}
    names = ("ssd_packed_scan_workspace_size", "ssd_packed_scan_backward_workspace_size", "ssd_gated_rmsnorm_backward_workspace_size")
    fake = types.SimpleNamespace(**{k: lambda *a, k=k: asked.setdefault(k, current[0]) and 64 for k in names})
    monkeypatch.setattr(ssd, "lib", lambda: fake)
    monkeypatch.setattr(ssd, "_bytes_on", lambda dev, n: n)
    monkeypatch.setattr(torch.cuda, "device", device)
    plan = types.SimpleNamespace(device=torch.device("cuda", 1), nseq=3, total=100, max_seqlen=0)
    assert ssd.packed_scan_workspace(plan, 4, 64, 128, torch.bfloat16) == 64
    assert ssd.packed_scan_backward_workspace(plan, 4, 64, 128) == 64
    assert ssd.gated_rmsnorm_backward_workspace(10, 64, device="cuda:1") == 64
    assert asked == dict.fromkeys(names, "cuda:1") and current == ["cuda:0"]


def test_memory_that_is_not_there_is_refused(ssd):
    """A workspace or a plan's buffer counts with the bytes that lie behind its pointer, not with its elements."""
    cpu = torch.device("cpu")
    a = types.SimpleNamespace()
    ws = torch.zeros(4096, dtype=torch.uint8)
    ssd._set_ws(a, ws, cpu)
    assert (a.workspace, a.workspace_bytes) == (ws.data_ptr(), 4096)
    ssd._set_ws(a, torch.zeros(16, 8), cpu)
    assert a.workspace_bytes == 512
    for bad in (ws[:1].expand(4096), ws[::2], ws.view(64, 64).t()):
        with pytest.raises(TypeError, match="contiguous"):
            ssd._set_ws(a, bad, cpu)
        with pytest.raises(TypeError, match="contiguous"):
            ssd._memory(bad, cpu, "buf")
    with pytest.raises(ValueError, match="workspace"):
        ssd._set_ws(a, ws, torch.device("cuda", 0))
