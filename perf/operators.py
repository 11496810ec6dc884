"""What is timed of the layer on packed sequences: the causal convolution and the selective scan over the rows of many
sequences laid end to end (prompts of different lengths, resumed or fresh, with their states in a pool of slots; packed
documents in training), one token of many streams of such a pool, and the gradient of the gated norm.

Each operator has a plain form of elementary torch operations in 32 bits (decays from sums in 64), and a definition in
64 bits that follows the recurrence token by token.
"""
import math
import random

import torch

own = False

_PKG = []


def _pkg():
    if not _PKG:
        import mamba_selective_state_causal_b200 as ssd
        _PKG.append(ssd)
    return _PKG[0]


# ------------------------------------------------------------------ cases
def _case(op, name=None, **kw):
    c = {"op": op, "dtype": "bf16", "H": 32, "P": 64, "N": 128, "G": 1}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # a serving step's prompts through the convolution, most of them fresh, some resumed
        _case("conv", "conv-prompts-64k", total=65536, nseq=48, longest=16384, resumed=0.3, cut=1),
        # packed documents of a training step, the convolution's gradient (the wider 1.3B layer)
        _case("conv_grad", "conv-grad-16k-h64", H=64, total=16384, nseq=12, longest=5000, resumed=0.0, cut=2),
        # the smallest layer of the tests in 32 bits: a few short sequences, latency
        _case("scan", "scan-f32-tiny", dtype="f32", H=2, P=16, N=16, total=331, nseq=6, longest=130, resumed=0.5, cut=3),
        # an ordinary mix of prompts, half of them the next part of a longer one
        _case("scan", "scan-prompts-12k", total=12001, nseq=24, longest=2200, resumed=0.5, cut=4),
        # many very short prompts: the states weigh as much as the tokens
        _case("scan", "scan-short-256", total=8191, nseq=256, longest=120, resumed=0.25, cut=5),
        # one long video beside short prompts: a single sequence has to be spread over the GPU
        _case("scan", "scan-long-64k", total=65536, nseq=5, longest=58000, resumed=0.4, cut=6),
        # packed documents of a training step
        _case("scan_grad", "scan-grad-16k", total=16384, nseq=9, longest=7000, resumed=0.0, cut=7),
        # the gradient in 32 bits at another head layout, several groups
        _case("scan_grad", "scan-grad-f32-2k", dtype="f32", H=8, P=32, N=64, G=2, total=2003, nseq=7, longest=900,
              resumed=0.5, cut=8),
        # one token of two streams: latency
        _case("step", "step-2", streams=2, slots=4, empty=0, cut=9),
        # one token of a large batch of streams, padded up to a fixed size
        _case("step", "step-256", streams=256, slots=272, empty=9, cut=10),
        # the gradient of the output norm at the 0.3B width
        _case("norm_grad", "norm-grad-64k", rows=65536, d=2048, group=0),
        # a small one in 32 bits, in groups
        _case("norm_grad", "norm-grad-f32-333", dtype="f32", rows=333, d=768, group=256),
    ]


def _span(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    """(dtype, H, P, N, G): mostly the backbones' head layouts in bf16, sometimes another one, in either type."""
    if rng.random() < 0.6:
        return "bf16", rng.choice((16, 24, 32, 32, 64, 80)), 64, 128, rng.choice((1, 1, 2))
    h = rng.choice((2, 3, 4, 8))
    return rng.choice(("bf16", "f32")), h, rng.choice((16, 32, 64)), rng.choice((16, 64, 128)), 1 if h != 4 else rng.choice((1, 2))


def draw(rng):
    op = rng.choice(("conv", "conv_grad", "scan", "scan", "scan", "scan_grad", "scan_grad", "step", "step", "norm_grad"))
    cut = rng.randrange(1 << 20)
    if op == "norm_grad":
        d = rng.choice((256, 768, 1024, 2048, 4096, 5120))
        return _case(op, dtype=rng.choice(("bf16", "bf16", "f32")), rows=_span(rng, 1, 24000), d=d,
                     group=rng.choice((0, 0, d // 4)))
    dtype, H, P, N, G = _heads(rng)
    if op == "step":
        b = _span(rng, 1, 200 if H <= 32 else 100)
        return _case(op, dtype=dtype, H=H, P=P, N=N, G=G, streams=b, slots=b + rng.randrange(1, 20),
                     empty=min(b - 1, rng.choice((0, 0, 1, 7))), cut=cut)
    most = {"conv": 60000, "conv_grad": 16000, "scan": 60000, "scan_grad": 14000}[op] * 32 // max(32, H)
    if P * N != 64 * 128 or dtype == "f32":
        most //= 8
    total = _span(rng, 1, most)
    nseq = min(total, _span(rng, 1, 64))
    longest = max(-(-total // nseq), min(total - nseq + 1, _span(rng, 1, total)))
    return _case(op, dtype=dtype, H=H, P=P, N=N, G=G, total=total, nseq=nseq, longest=longest,
                 resumed=rng.choice((0.0, 0.5, 1.0)), cut=cut)


def _lengths(case):
    """The sequences' lengths: one of the longest length, the others cut at random from what is left."""
    rng = random.Random(case["cut"])
    total, n, longest = case["total"], case["nseq"], min(case["longest"], case["total"] - case["nseq"] + 1)
    lens, left = [longest], total - longest
    for k in range(1, n):
        rest = n - 1 - k
        hi = min(longest, left - rest)
        lo = max(1, left - rest * longest)
        even = left / (rest + 1)
        x = left if rest == 0 else max(lo, min(hi, int(even * rng.uniform(0.2, 1.8))))
        lens.append(x)
        left -= x
    rng.shuffle(lens)
    return lens


def _flags(case, n):
    """(slot, resumed) of each sequence: slots in no order, some more than there are sequences."""
    rng = random.Random(case["cut"] + 1)
    slots = rng.sample(range(n + 3), n)
    return slots, [1 if rng.random() < case["resumed"] else 0 for _ in range(n)]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    io = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    f32 = torch.float32

    def randn(*shape, dtype=f32, scale=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=f32).mul_(scale).to(dtype)

    def rand(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device=dev, dtype=f32) * (hi - lo) + lo

    s = {"case": dict(case)}
    if case["op"] == "norm_grad":
        rows, d = case["rows"], case["d"]
        s.update(y=randn(rows, d, dtype=io), z=randn(rows, d, dtype=io, scale=1.5), dout=randn(rows, d, dtype=io),
                 weight=1.0 + randn(d, scale=0.1), dy=torch.empty(rows, d, device=dev, dtype=io),
                 dz=torch.empty(rows, d, device=dev, dtype=io), dweight=torch.empty(d, device=dev))
        if own:
            s["ws"] = _pkg().gated_rmsnorm_backward_workspace(rows, d, device=dev)
        return s
    H, P, N, G = (case[k] for k in "HPNG")
    cch = H * P + 2 * G * N
    s.update(A=-torch.exp(rand(H, hi=math.log(16.0))), D=randn(H), w=rand(cch, 4, lo=-0.5, hi=0.5), bias=randn(cch, scale=0.1))
    # the step's bias, so that softplus(raw + bias) lies about the block's range [1e-3, 1e-1]
    dt0 = torch.exp(rand(H, lo=math.log(1e-3), hi=math.log(1e-1)))
    dt_bias = dt0 + torch.log(-torch.expm1(-dt0))
    if case["op"] == "step":
        b, n = case["streams"], case["slots"]
        rng = random.Random(case["cut"])
        slots = rng.sample(range(n), b)
        for i in rng.sample(range(b), case["empty"]):
            slots[i] = -1
        s.update(u=randn(b, cch, dtype=io), dt=randn(b, H, scale=0.5), dt_bias=dt_bias,
                 slots=torch.tensor(slots, device=dev, dtype=torch.int32),
                 tail_in=randn(n, 3, cch, dtype=io), h_in=randn(n, H, P, N),
                 tail_out=torch.zeros(n, 3, cch, device=dev, dtype=io), h_out=torch.zeros(n, H, P, N, device=dev),
                 y=torch.empty(b, H, P, device=dev, dtype=io))
        return s
    lens = _lengths(case)
    n, total = len(lens), case["total"]
    slots, resumed = _flags(case, n)
    train = case["op"].endswith("grad")
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    s.update(lens=lens, longest=max(lens), cu=torch.tensor(cu, device=dev, dtype=torch.int32))
    # in training the state entering a sequence and its gradient go by the sequence, in serving by the slot
    s["slots"] = None if train else torch.tensor(slots, device=dev, dtype=torch.int32)
    s["resumed"] = torch.tensor(resumed, device=dev, dtype=torch.int32)
    m = n if train else n + 3
    if case["op"].startswith("conv"):
        s.update(u=randn(total, cch, dtype=io), tail_in=randn(m, 3, cch, dtype=io))
        if train:
            s.update(dx=randn(total, H * P), dB=randn(total, G * N), dC=randn(total, G * N),
                     dtail_out=randn(n, 3, cch), du=torch.zeros(total, cch, device=dev),
                     dtail_in=torch.zeros(n, 3, cch, device=dev), dw=torch.empty(cch, 4, device=dev),
                     dbias=torch.empty(cch, device=dev))
        else:
            s.update(tail_out=torch.zeros(m, 3, cch, device=dev, dtype=io), v=torch.zeros(total, cch, device=dev, dtype=io))
    else:
        # x, B and C are column slices of the convolution's output
        v = torch.nn.functional.silu(randn(total, cch)).to(io)
        s.update(x=v[:, :H * P], B=v[:, H * P:H * P + G * N], C=v[:, H * P + G * N:])
        if case["resumed"] > 0:
            s["h_in"] = randn(m, H, P, N)
        else:
            s["h_in"] = None
        raw = randn(total, H, scale=0.5)
        if train:
            s.update(dt=torch.nn.functional.softplus(raw + dt_bias).clamp(1e-3, 1e-1), dy=randn(total, H * P, dtype=io),
                     dh_out=randn(n, H, P, N))
            s["out"] = {"dx": torch.zeros(total, H, P, device=dev), "dB": torch.zeros(total, G, N, device=dev),
                        "dC": torch.zeros(total, G, N, device=dev), "ddt": torch.zeros(total, H, device=dev),
                        "dA": torch.empty(H, device=dev), "dD": torch.empty(H, device=dev),
                        "dh_in": torch.zeros(n, H, P, N, device=dev)}
        else:
            s.update(dt=raw, dt_bias=dt_bias, h_out=torch.zeros(m, H, P, N, device=dev),
                     y=torch.zeros(total, H, P, device=dev, dtype=io))
    if own:
        # a program makes the plan once for a batch and hands it to every layer
        ssd = _pkg()
        s["plan"] = ssd.packed_plan(s["cu"], total, slots=s["slots"], resume=s["resumed"], n_slots=m, max_seqlen=s["longest"])
        if case["op"] == "conv_grad":
            s["ws"] = ssd.packed_conv_backward_workspace(s["plan"], cch)
        elif case["op"] == "scan":
            s["ws"] = ssd.packed_scan_workspace(s["plan"], H, P, N, io)
        elif case["op"] == "scan_grad":
            s["ws"] = ssd.packed_scan_backward_workspace(s["plan"], H, P, N)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    return {"conv": _conv, "conv_grad": _conv_grad, "scan": _scan, "scan_grad": _scan_grad, "step": _step,
            "norm_grad": _norm_grad}[c["op"]](s, c)


def _rows(s):
    """Of each row: its sequence, and its position in it."""
    cu = s["cu"].long()
    t = torch.arange(s["case"]["total"], device=cu.device)
    q = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return t, q, t - cu[q]


def _source(s, n):
    """Of each sequence, the slot that its state comes from and goes to."""
    return torch.arange(n, device=s["cu"].device) if s["slots"] is None else s["slots"].long()


def _window(s):
    """u[t-3 .. t] of every row, [total, 4, C]; rows before a sequence come from its buffer, or are zero."""
    n = s["cu"].numel() - 1
    t, q, pos = _rows(s)
    tail = s["tail_in"][_source(s, n)].float() * s["resumed"].float()[:, None, None]
    k = torch.arange(4, device=t.device) - 3
    inside = (pos[:, None] + k) >= 0
    rows = s["u"].float()[(t[:, None] + k).clamp_min(0)]
    before = tail[q[:, None], (3 + pos[:, None] + k).clamp(0, 2)]
    return torch.where(inside[:, :, None], rows, before), tail, q, pos


def _conv(s, c):
    if own:
        return dict(zip(("v", "tail"), _pkg().packed_conv_forward(s["u"], s["w"], s["plan"], s["bias"], s["tail_in"], s["tail_out"], s["v"])))
    win, tail, q, pos = _window(s)
    z = (win * s["w"].t()[None]).sum(1) + s["bias"]
    cu, n = s["cu"].long(), s["cu"].numel() - 1
    back = (cu[1:] - cu[:-1])[:, None] - 3 + torch.arange(3, device=cu.device)
    last = torch.where((back >= 0)[:, :, None], s["u"].float()[(cu[:-1, None] + back).clamp_min(0)],
                       tail[torch.arange(n, device=cu.device)[:, None], (3 + back).clamp(0, 2)])
    out = s["tail_out"].clone()
    out[_source(s, n)] = last.to(out.dtype)
    return {"v": (z * torch.sigmoid(z)).to(s["u"].dtype), "tail": out}


def _conv_grad(s, c):
    if own:
        o = _pkg().packed_conv_backward(s["u"], s["w"], s["plan"], s["dx"], s["dB"], s["dC"], bias=s["bias"], tail_in=s["tail_in"],
                                        dtail_out=s["dtail_out"], workspace=s["ws"],
                                        out={"du": s["du"], "dtail_in": s["dtail_in"], "dconv_w": s["dw"], "dconv_bias": s["dbias"]})
        return {"du": o["du"], "dtail": o["dtail_in"], "dw": o["dconv_w"], "dbias": o["dconv_bias"]}
    win, tail, q, pos = _window(s)
    w = s["w"]
    z = (win * w.t()[None]).sum(1) + s["bias"]
    sg = torch.sigmoid(z)
    dz = torch.cat((s["dx"], s["dB"], s["dC"]), 1) * sg * (1 + z * (1 - sg))
    total, cu = c["total"], s["cu"].long()
    n = cu.numel() - 1
    lens = cu[1:] - cu[:-1]
    j = torch.arange(4, device=dz.device)
    t = torch.arange(total, device=dz.device)
    later = (t[:, None] + j).clamp_max(total - 1)
    du = (dz[later] * ((t[:, None] + j) < cu[q + 1][:, None])[:, :, None] * w.flip(1).t()[None]).sum(1)
    # the last three rows also feed the buffer that is handed on
    r = torch.arange(3, device=dz.device)
    back = lens[:, None] - 3 + r
    has = back >= 0
    du.index_add_(0, (cu[:-1, None] + back).clamp_min(0).flatten(), (s["dtail_out"] * has[:, :, None]).flatten(0, 1))
    # the buffer's rows before a sequence: row 3 + p at position p reaches token p + 3 - k through tap k
    p = r[:, None] - 3 + j                                   # token reached from buffer row r by the tap 3 - j
    reach = (p >= 0) & (p < lens[:, None, None])
    dtail = (dz[(cu[:-1, None, None] + p.clamp_min(0)).clamp_max(total - 1)] * reach[..., None] * w.flip(1).t()[None, None]).sum(2)
    moved = r + lens[:, None]                                # buffer row that a short sequence hands on as row r
    dtail = dtail + torch.zeros_like(dtail).scatter_add_(1, moved.clamp_max(2)[:, :, None].expand_as(dtail),
                                                         s["dtail_out"] * (moved < 3)[:, :, None])
    return {"du": du, "dtail": dtail * s["resumed"].float()[:, None, None],
            "dw": (dz[:, None] * win).sum(0).t().contiguous(), "dbias": dz.sum(0)}


_Q = 64


class _Cut:
    """The sequences cut into chunks of _Q rows, each sequence's last one padded with rows that count for nothing."""

    def __init__(self, s, c, dt):
        cu = s["cu"].long()
        dev, n, H = cu.device, cu.numel() - 1, c["H"]
        lens = cu[1:] - cu[:-1]
        per = (lens + _Q - 1) // _Q
        ends = per.cumsum(0)
        self.n, self.m = n, c["total"] // _Q + n
        k = torch.arange(self.m, device=dev)
        q = torch.searchsorted(ends, k, right=True)
        self.used = q < n
        self.seq = q.clamp_max(n - 1)
        first = (ends - per)[self.seq]
        row = cu[self.seq, None] + (k - first)[:, None] * _Q + torch.arange(_Q, device=dev)
        self.valid = (row < cu[self.seq + 1][:, None]) & self.used[:, None]
        self.row = row.clamp_max(c["total"] - 1)
        self.dt = dt[self.row] * self.valid[..., None]
        step = self.dt.double() * s["A"].double()
        self.cs = step.cumsum(1)                                              # [m, Q, H]
        lam = self.cs[:, -1]
        self.E = torch.cat((torch.zeros(1, H, device=dev, dtype=torch.float64), lam.cumsum(0)))
        self.lam, self.first = lam, first
        self.fin = ends.clamp_max(self.m)
        d = torch.arange(self.m, device=dev)
        same = (self.seq[:, None] == self.seq[None]) & self.used[:, None] & self.used[None]
        # decay from the end of chunk d to the start of chunk k, both of one sequence
        self.between = torch.where((same & (d[None] < k[:, None]))[..., None], self.E[:-1, None] - self.E[None, 1:],
                                   torch.tensor(-math.inf, device=dev, dtype=torch.float64)).exp_().float()   # [k, d, H]
        i = torch.arange(_Q, device=dev)
        low = (i[:, None] >= i[None])[None, :, :, None]
        self.inside = torch.where(low, self.cs[:, :, None] - self.cs[:, None], torch.tensor(-math.inf, device=dev, dtype=torch.float64)).exp_().float()

    def take(self, t, *shape):
        return (t.float()[self.row] * self.valid[..., None]).view(self.m, _Q, *shape)

    def put(self, t, out):
        out[self.row[self.valid]] = t.reshape(self.m, _Q, *out.shape[1:])[self.valid].to(out.dtype)
        return out


def _start(s, c, n):
    """The state that each sequence starts from."""
    if s["h_in"] is None:
        return torch.zeros(n, c["H"], c["P"], c["N"], device=s["cu"].device)
    return s["h_in"][_source(s, n)] * s["resumed"].float()[:, None, None, None]


def _each(t, c, k):
    """B or C of a head from its group's."""
    return t.repeat_interleave(c["H"] // c["G"], dim=k)


def _scan(s, c):
    if own:
        y, h = _pkg().packed_scan_forward(s["x"], s["B"], s["C"], s["dt"], s["A"], s["D"], plan=s["plan"], H=c["H"], G=c["G"],
                                          h_in=s["h_in"], h_out=s["h_out"], y=s["y"], workspace=s["ws"], dt_bias=s["dt_bias"],
                                          dt_softplus=True, dt_limit=(1e-3, 1e-1))
        return {"y": y, "h": h}
    H, P, N, G = (c[k] for k in "HPNG")
    v = s["dt"] + s["dt_bias"]
    k = _Cut(s, c, torch.where(v > 20, v, torch.log1p(torch.exp(v))).clamp(1e-3, 1e-1))
    x, B, C = k.take(s["x"], H, P), k.take(s["B"], G, N), k.take(s["C"], G, N)
    h0 = _start(s, c, k.n)
    S = torch.einsum("mqhp,mqhn->mhpn", x * (k.dt * (k.lam[:, None] - k.cs).exp().float())[..., None], _each(B, c, 2))
    enter = torch.einsum("kdh,dhpn->khpn", k.between, S)
    enter += h0[k.seq] * (k.E[:-1] - k.E[k.first]).exp().float()[..., None, None]
    M = _each(torch.einsum("mign,mjgn->mijg", C, B), c, 3) * k.inside * k.dt[:, None]
    y = torch.einsum("mijh,mjhp->mihp", M, x)
    y += torch.einsum("mihn,mhpn->mihp", _each(C, c, 2), enter) * k.cs.exp().float()[..., None]
    y += x * s["D"][:, None]
    last = (k.fin - 1).clamp_min(0)
    h = enter[last] * k.lam[last].exp().float()[..., None, None] + S[last]
    out = s["h_out"].clone()
    out[_source(s, k.n)] = h
    return {"y": k.put(y, s["y"].clone()), "h": out}


def _scan_grad(s, c):
    if own:
        o = _pkg().packed_scan_backward(s["x"], s["B"], s["C"], s["dt"], s["A"], s["D"], s["dy"], plan=s["plan"], H=c["H"], G=c["G"],
                                        h_in=s["h_in"], dh_out=s["dh_out"], out=s["out"], workspace=s["ws"])
        return {k: o[k] for k in ("dx", "dB", "dC", "ddt", "dA", "dD", "dh_in")}
    H, P, N, G = (c[k] for k in "HPNG")
    k = _Cut(s, c, s["dt"])
    x, B, C, dy = k.take(s["x"], H, P), k.take(s["B"], G, N), k.take(s["C"], G, N), k.take(s["dy"], H, P)
    Bh, Ch = _each(B, c, 2), _each(C, c, 2)
    h0 = _start(s, c, k.n)
    up = (k.lam[:, None] - k.cs).exp().float()                                # from a token to its chunk's end
    down = k.cs.exp().float()                                                 # from its chunk's start to a token
    S = torch.einsum("mqhp,mqhn->mhpn", x * (k.dt * up)[..., None], Bh)
    R = torch.einsum("mqhp,mqhn->mhpn", dy * down[..., None], Ch)
    from0 = (k.E[:-1] - k.E[k.first]).exp().float()[..., None, None]
    enter = torch.einsum("kdh,dhpn->khpn", k.between, S) + h0[k.seq] * from0
    stop = k.fin[k.seq]
    leave = torch.einsum("kdh,khpn->dhpn", k.between, R)
    leave += s["dh_out"][k.seq] * ((k.E[stop] - k.E[1:]) * k.used[:, None]).exp().float()[..., None, None]
    CB = _each(torch.einsum("mign,mjgn->mijg", C, B), c, 3)
    YX = torch.einsum("mihp,mjhp->mijh", dy, x) * k.inside
    Bl = torch.einsum("mjhn,mhpn->mjhp", Bh, leave) * up[..., None]           # what later chunks want of x_j
    dxr = torch.einsum("mijh,mihp->mjhp", CB * k.inside, dy) + Bl
    dBr = torch.einsum("mijh,mihn->mjhn", YX, Ch) + torch.einsum("mjhp,mhpn->mjhn", x, leave) * up[..., None]
    hy = torch.einsum("mihp,mhpn->mihn", dy, enter) * down[..., None]
    dCh = hy + torch.einsum("mijh,mjhn->mihn", YX * k.dt[:, None], Bh)
    # dLoss/d(dt_t A): every path from a token before t (or the entering state) to one at or after t
    al, be = (hy * Ch).sum(-1), (x * Bl).sum(-1) * k.dt
    across = (YX * CB * k.dt[:, None]).flip(1).cumsum(1).flip(1)                                      # sum over rows at or after t
    i = torch.arange(_Q, device=x.device)
    dl = (across * (i[None] < i[:, None])[None, :, :, None]).sum(2)
    dl = dl + al.flip(1).cumsum(1).flip(1) + (be.cumsum(1) - be)
    dl = dl + ((enter * leave).sum((-1, -2)) * k.lam.exp().float())[:, None]
    ddt = dl * s["A"] + (Bh * dBr).sum(-1)
    tot = s["dt"].shape[0]
    dx = k.put(dxr * k.dt[..., None] + dy * s["D"][:, None], x.new_zeros(tot, H, P))
    dB = k.put((dBr * k.dt[..., None]).view(k.m, _Q, G, H // G, N).sum(3), x.new_zeros(tot, G, N))
    dC = k.put(dCh.view(k.m, _Q, G, H // G, N).sum(3), x.new_zeros(tot, G, N))
    begin = torch.cat((k.fin.new_zeros(1), k.fin[:-1]))
    dh = R[begin] + leave[begin] * k.lam[begin].exp().float()[..., None, None]
    return {"dx": dx, "dB": dB, "dC": dC, "ddt": k.put(ddt, x.new_zeros(tot, H)),
            "dA": (k.dt * dl).sum((0, 1)), "dD": (x * dy).sum((0, 1, 3)),
            "dh_in": dh * s["resumed"].float()[:, None, None, None]}


def _step(s, c):
    H, P, N, G = (c[k] for k in "HPNG")
    if own:
        o = _pkg().decode_slots(s["u"], s["w"], s["dt"], s["A"], s["D"], slots=s["slots"], H=H, P=P, N=N, G=G, conv_bias=s["bias"],
                                tail_in=s["tail_in"], tail_out=s["tail_out"], h_in=s["h_in"], h_out=s["h_out"], y=s["y"],
                                dt_bias=s["dt_bias"], dt_softplus=True, dt_limit=(1e-3, 1e-1))
        return {"y": o["y"], "h": o["h_out"], "tail": o["tail_out"]}
    k = s["slots"].long()
    live = k >= 0
    at = k.clamp_min(0)
    b = k.numel()
    win = torch.cat((s["tail_in"][at], s["u"][:, None]), 1)
    z = (win.float() * s["w"].t()[None]).sum(1) + s["bias"]
    v = z * torch.sigmoid(z)
    x, B, C = v[:, :H * P].view(b, H, P), v[:, H * P:H * P + G * N].view(b, G, N), v[:, H * P + G * N:].view(b, G, N)
    r = s["dt"] + s["dt_bias"]
    dt = torch.where(r > 20, r, torch.log1p(torch.exp(r))).clamp(1e-3, 1e-1)
    h = s["h_in"][at] * torch.exp(dt * s["A"])[..., None, None] + (x * dt[..., None])[..., None] * _each(B, c, 1)[:, :, None]
    y = (h * _each(C, c, 1)[:, :, None]).sum(-1) + x * s["D"][:, None]
    h_out, tail = s["h_out"].clone(), s["tail_out"].clone()
    h_out[at[live]] = h[live]
    tail[at[live]] = win[live, 1:]
    return {"y": (y * live[:, None, None]).to(s["u"].dtype), "h": h_out, "tail": tail}


def _norm_grad(s, c):
    if own:
        o = _pkg().gated_rmsnorm_backward(s["dout"], s["y"], s["z"], s["weight"], eps=1e-5, group_size=c["group"],
                                          out={"dy": s["dy"], "dz": s["dz"], "dweight": s["dweight"]}, workspace=s["ws"])
        return {"dy": o["dy"], "dz": o["dz"], "dweight": o["dweight"]}
    rows, d = c["rows"], c["d"]
    n = c["group"] or d
    y, z, do = s["y"].float(), s["z"].float(), s["dout"].float()
    sg = torch.sigmoid(z)
    v = y * z * sg
    vg = v.view(rows, d // n, n)
    r = torch.rsqrt((vg * vg).mean(-1, keepdim=True) + 1e-5)
    g = (do * s["weight"]).view(rows, d // n, n)
    dv = (r * (g - vg * r * r * (g * vg).mean(-1, keepdim=True))).view(rows, d)
    return {"dy": (dv * z * sg).to(s["y"].dtype), "dz": (dv * y * sg * (1 + z * (1 - sg))).to(s["y"].dtype),
            "dweight": (do * (vg * r).view(rows, d)).sum(0)}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "norm_grad":
        rows, d = case["rows"], case["d"]
        return {"bytes": 5 * rows * d * e + 8 * d, "flops": 30 * rows * d}
    H, P, N, G = (case[k] for k in "HPNG")
    cch, state = H * P + 2 * G * N, 4 * H * P * N
    if op == "step":
        b = case["streams"] - case["empty"]
        return {"bytes": b * (2 * state + 7 * cch * e + 4 * H + e * H * P) + 20 * cch, "flops": b * (5 * H * P * N + 12 * cch)}
    T, n = case["total"], case["nseq"]
    resumed = sum(_flags(case, n)[1])
    if op == "conv":
        return {"bytes": 2 * T * cch * e + (n + resumed) * 3 * cch * e + 20 * cch, "flops": 12 * T * cch}
    if op == "conv_grad":
        return {"bytes": T * cch * (e + 8) + n * 24 * cch + resumed * 3 * cch * e + 40 * cch, "flops": 30 * T * cch}
    row = (H * P + 2 * G * N) * e + 4 * H
    if op == "scan":
        return {"bytes": T * (row + H * P * e) + (n + resumed) * state, "flops": 5 * T * H * P * N}
    return {"bytes": T * (row + H * P * e + 4 * (H * P + 2 * G * N + H)) + (2 * n + resumed) * state, "flops": 14 * T * H * P * N}


# ------------------------------------------------------------------ the definitions in 64 bits, token by token
def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _conv_exact, "conv_grad": _conv_grad_exact, "scan": _scan_exact, "scan_grad": _scan_grad_exact,
            "step": _step_exact, "norm_grad": _norm_grad_exact}[case["op"]](s, case)


def _pieces(s):
    """(sequence, its slot, its first row, its end) in turn."""
    a = 0
    for i, m in enumerate(s["lens"]):
        yield i, (i if s["slots"] is None else int(s["slots"][i])), a, a + m
        a += m


def _conv_of(u, tail, w, bias):
    full = torch.cat((tail, u))
    m = u.shape[0]
    z = bias + full[:m] * w[:, 0] + full[1:m + 1] * w[:, 1] + full[2:m + 2] * w[:, 2] + full[3:] * w[:, 3]
    return z / (1 + torch.exp(-z)), full[m:]


def _conv_exact(s, c):
    v, out = torch.zeros_like(s["u"], dtype=torch.float64), s["tail_out"].double()
    for i, k, a, b in _pieces(s):
        tail = s["tail_in"][k].double() * int(s["resumed"][i])
        v[a:b], out[k] = _conv_of(s["u"][a:b].double(), tail, s["w"].double(), s["bias"].double())
    return {"v": v, "tail": out}


def _conv_grad_exact(s, c):
    w, bias = s["w"].double().requires_grad_(), s["bias"].double().requires_grad_()
    du, dt = torch.zeros_like(s["u"], dtype=torch.float64), torch.zeros_like(s["dtail_out"], dtype=torch.float64)
    dv = torch.cat((s["dx"], s["dB"], s["dC"]), 1)
    dw, db = torch.zeros_like(w), torch.zeros_like(bias)
    for i, k, a, b in _pieces(s):
        u, tail = s["u"][a:b].double().requires_grad_(), s["tail_in"][k].double().requires_grad_()
        v, last = _conv_of(u, tail * int(s["resumed"][i]), w, bias)
        g = torch.autograd.grad((v * dv[a:b]).sum() + (last * s["dtail_out"][i]).sum(), (u, tail, w, bias))
        du[a:b], dt[i] = g[0], g[1]
        dw, db = dw + g[2], db + g[3]
    return {"du": du, "dtail": dt, "dw": dw.detach(), "dbias": db.detach()}


def _softplus64(raw, bias):
    v = raw.double() + bias.double()
    return torch.log1p(torch.exp(v)).clamp(1e-3, 1e-1)


def _scan_exact(s, c):
    H, P, N, G = (c[k] for k in "HPNG")
    dt = _softplus64(s["dt"], s["dt_bias"])
    a, n, dev = torch.exp(dt * s["A"].double()), len(s["lens"]), dt.device
    y, out = torch.zeros(c["total"], H, P, device=dev, dtype=torch.float64), s["h_out"].double()
    order = sorted(_pieces(s), key=lambda p: p[2] - p[3])                     # the longest first: the others drop out behind
    h = torch.stack([(s["h_in"][k].double() * int(s["resumed"][i])) if s["h_in"] is not None else torch.zeros(H, P, N, device=dev, dtype=torch.float64)
                     for i, k, _, _ in order])
    starts = torch.tensor([p[2] for p in order], device=dev)
    lens = [p[3] - p[2] for p in order]
    live = n
    x, B, C, D = s["x"], s["B"], s["C"], s["D"].double()
    for t in range(lens[0]):
        while lens[live - 1] <= t:
            live -= 1
        r = starts[:live] + t
        xt = x[r].double().view(live, H, P)
        Bt, Ct = (_each(z[r].double().view(live, G, N), c, 1) for z in (B, C))
        hh = h[:live]
        hh.mul_(a[r][..., None, None]).add_((xt * dt[r][..., None])[..., None] * Bt[:, :, None])
        y[r] = torch.matmul(hh, Ct[..., None])[..., 0] + xt * D[:, None]
    for j, (i, k, _, _) in enumerate(order):
        out[k] = h[j]
    return {"y": y, "h": out}


def _scan_grad_exact(s, c):
    H, P, N, G = (c[k] for k in "HPNG")
    dev, f = s["dt"].device, torch.float64
    T, dt, A, D = c["total"], s["dt"].double(), s["A"].double(), s["D"].double()
    a = torch.exp(dt * A)
    x, dy = s["x"].double().view(T, H, P), s["dy"].double().view(T, H, P)
    B, C = (_each(z.double().view(T, G, N), c, 1) for z in (s["B"], s["C"]))
    o = {"dx": torch.zeros(T, H, P, device=dev, dtype=f), "dB": torch.zeros(T, H, N, device=dev, dtype=f),
         "dC": torch.zeros(T, H, N, device=dev, dtype=f), "ddt": torch.zeros(T, H, device=dev, dtype=f)}
    dA, dh = torch.zeros(H, device=dev, dtype=f), torch.zeros(len(s["lens"]), H, P, N, device=dev, dtype=f)
    cell = 256
    for i, k, lo, hi in _pieces(s):
        h = torch.zeros(H, P, N, device=dev, dtype=f)
        if s["h_in"] is not None:
            h = s["h_in"][k].double() * int(s["resumed"][i])
        marks = []
        for t in range(lo, hi):                                               # the states, kept every `cell` tokens
            if (t - lo) % cell == 0:
                marks.append(h)
            h = h * a[t][:, None, None] + (x[t] * dt[t][:, None])[..., None] * B[t][:, None]
        g = s["dh_out"][i].double()
        for m in range(len(marks) - 1, -1, -1):
            b0 = lo + m * cell
            b1 = min(hi, b0 + cell)
            hs = torch.empty(b1 - b0 + 1, H, P, N, device=dev, dtype=f)       # the cell's states, rebuilt
            hs[0] = marks[m]
            for t in range(b0, b1):
                hs[t - b0 + 1] = hs[t - b0] * a[t][:, None, None] + (x[t] * dt[t][:, None])[..., None] * B[t][:, None]
            gs = torch.empty(b1 - b0, H, P, N, device=dev, dtype=f)           # dLoss/dh_t
            for t in range(b1 - 1, b0 - 1, -1):
                g = g + dy[t][..., None] * C[t][:, None]
                gs[t - b0] = g
                g = g * a[t][:, None, None]
            w = slice(b0, b1)
            gB = torch.einsum("thpn,thn->thp", gs, B[w])
            o["dx"][w] = D[:, None] * dy[w] + dt[w][..., None] * gB
            o["dB"][w] = dt[w][..., None] * torch.einsum("thpn,thp->thn", gs, x[w])
            o["dC"][w] = torch.einsum("thpn,thp->thn", hs[1:], dy[w])
            dl = (gs * hs[:-1]).sum((-1, -2)) * a[w]
            o["ddt"][w] = A * dl + (gB * x[w]).sum(-1)
            dA += (dt[w] * dl).sum(0)
        dh[i] = g * int(s["resumed"][i])
    for k in ("dB", "dC"):
        o[k] = o[k].view(T, G, H // G, N).sum(2)
    return {**o, "dA": dA, "dD": (x * dy).sum((0, 2)), "dh_in": dh}


def _step_exact(s, c):
    H, P, N, G = (c[k] for k in "HPNG")
    y = torch.zeros(s["y"].shape, device=s["y"].device, dtype=torch.float64)
    h_out, tail = s["h_out"].double(), s["tail_out"].double()
    w, bias, A, D = (s[k].double() for k in ("w", "bias", "A", "D"))
    for i, k in enumerate(s["slots"].tolist()):
        if k < 0:
            continue
        v, tail[k] = _conv_of(s["u"][i:i + 1].double(), s["tail_in"][k].double(), w, bias)
        x, B, C = v[0, :H * P].view(H, P), v[0, H * P:H * P + G * N].view(G, N), v[0, H * P + G * N:].view(G, N)
        dt = _softplus64(s["dt"][i], s["dt_bias"])
        h = s["h_in"][k].double() * torch.exp(dt * A)[:, None, None]
        h = h + (dt[:, None] * x)[..., None] * _each(B, c, 0)[:, None]
        y[i] = (h * _each(C, c, 0)[:, None]).sum(-1) + D[:, None] * x
        h_out[k] = h
    return {"y": y, "h": h_out, "tail": tail}


def _norm_grad_exact(s, c):
    n, parts, dw = c["group"] or c["d"], [], 0.0
    for y, z, do in zip(*(s[k].split(4096) for k in ("y", "z", "dout"))):     # row by row the same, in blocks for memory
        y, z, w = y.double().requires_grad_(), z.double().requires_grad_(), s["weight"].double().requires_grad_()
        v = y * z / (1 + torch.exp(-z))
        g = v.view(y.shape[0], -1, n)
        out = (g / torch.sqrt(g.pow(2).mean(-1, keepdim=True) + 1e-5)).view_as(v) * w
        gy, gz, gw = torch.autograd.grad((out * do.double()).sum(), (y, z, w))
        parts.append((gy, gz))
        dw = dw + gw
    return {"dy": torch.cat([p[0] for p in parts]), "dz": torch.cat([p[1] for p in parts]), "dweight": dw}
