"""Plain 64-bit statements of the packed operators, sequence by sequence and token by token, and batches for their tests."""
import torch

F64 = torch.float64


def batch(lens, n_slots=None, slots=None, resume=None, before=0, behind=0):
    """(cu, total, slots, resume) as lists: sequences laid end to end after `before` rows, with `behind` rows after them."""
    cu = [before]
    for m in lens:
        cu.append(cu[-1] + m)
    n = len(lens)
    return cu, cu[-1] + behind, slots if slots is not None else list(range(n)), resume if resume is not None else [1] * n


def conv_seq(u, tail, w, bias):
    """(v, last three rows) of one sequence u [m, C] after the rows tail [3, C]."""
    full = torch.cat((tail, u))
    m = u.shape[0]
    z = bias + sum(full[k:k + m] * w[:, k] for k in range(4))
    return z / (1 + torch.exp(-z)), full[m:]


def conv(u, w, bias, cu, slots, resume, tail_in, tail_out, v):
    """v (rows of no sequence as given) and tail_out (slots of no sequence as given), in 64 bits."""
    u, w, bias, tin = u.to(F64), w.to(F64), bias.to(F64), tail_in.to(F64)
    v, tout = v.to(F64).clone(), tail_out.to(F64).clone()
    for i, k in enumerate(slots):
        a, b = cu[i], cu[i + 1]
        tail = tin[k] if k >= 0 and resume[i] else torch.zeros(3, u.shape[1], dtype=F64)
        v[a:b], last = conv_seq(u[a:b], tail, w, bias)
        if k >= 0:
            tout[k] = last
    return v, tout


def conv_grad(u, w, bias, cu, slots, resume, tail_in, dv, dtail_out):
    """Gradients (du, dtail by sequence, dw, dbias) by automatic differentiation of conv_seq."""
    w, bias = w.to(F64).requires_grad_(), bias.to(F64).requires_grad_()
    du, dtail = torch.zeros(u.shape, dtype=F64), torch.zeros(dtail_out.shape, dtype=F64)
    dw, db = torch.zeros(w.shape, dtype=F64), torch.zeros(bias.shape, dtype=F64)
    for i, k in enumerate(slots):
        a, b = cu[i], cu[i + 1]
        on = k >= 0 and resume[i]
        x = u[a:b].to(F64).requires_grad_()
        tail = (tail_in[k].to(F64) if on else torch.zeros(3, u.shape[1], dtype=F64)).requires_grad_()
        v, last = conv_seq(x, tail, w, bias)
        g = torch.autograd.grad((v * dv[a:b].to(F64)).sum() + (last * dtail_out[i].to(F64)).sum(), (x, tail, w, bias),
                                allow_unused=True)
        du[a:b] = g[0]
        if on:
            dtail[i] = g[1]
        dw += g[2]
        db += g[3]
    return du, dtail, dw, db


def heads_of(t, H, G):
    return t.repeat_interleave(H // G, dim=-2)


def scan(x, B, C, dt, A, D, cu, slots, resume, h_in, h_out, y, G):
    """y [total, H, P] and h_out in 64 bits; x [total, H, P], B, C [total, G, N], dt as the scan uses it."""
    x, B, C, dt, A, D = (t.to(F64) for t in (x, B, C, dt, A, D))
    H = x.shape[1]
    y, out = y.to(F64).clone(), h_out.to(F64).clone()
    for i, k in enumerate(slots):
        h = torch.zeros(out.shape[1:], dtype=F64)
        if k >= 0 and resume[i] and h_in is not None:
            h = h_in[k].to(F64)
        for t in range(cu[i], cu[i + 1]):
            Bt, Ct = heads_of(B[t], H, G), heads_of(C[t], H, G)
            h = h * torch.exp(dt[t] * A)[:, None, None] + (dt[t][:, None] * x[t])[..., None] * Bt[:, None]
            y[t] = (h * Ct[:, None]).sum(-1) + D[:, None] * x[t]
        if k >= 0:
            out[k] = h
    return y, out


def scan_grad(x, B, C, dt, A, D, cu, slots, resume, h_in, dy, dh_out, G):
    """Gradients by the reverse recurrence: dict dx, dB, dC, ddt, dA, dD, dh_in (by sequence)."""
    x, B, C, dt, A, D, dy = (t.to(F64) for t in (x, B, C, dt, A, D, dy))
    T, H, P = x.shape
    N = B.shape[2]
    o = {"dx": torch.zeros(T, H, P, dtype=F64), "dB": torch.zeros(T, H, N, dtype=F64), "dC": torch.zeros(T, H, N, dtype=F64),
         "ddt": torch.zeros(T, H, dtype=F64), "dA": torch.zeros(H, dtype=F64), "dD": torch.zeros(H, dtype=F64),
         "dh_in": torch.zeros(len(slots), H, P, N, dtype=F64)}
    for i, k in enumerate(slots):
        on = k >= 0 and resume[i] and h_in is not None
        h = h_in[k].to(F64) if on else torch.zeros(H, P, N, dtype=F64)
        states = [h]
        for t in range(cu[i], cu[i + 1]):
            h = h * torch.exp(dt[t] * A)[:, None, None] + (dt[t][:, None] * x[t])[..., None] * heads_of(B[t], H, G)[:, None]
            states.append(h)
        g = dh_out[i].to(F64) if dh_out is not None else torch.zeros(H, P, N, dtype=F64)
        for t in range(cu[i + 1] - 1, cu[i] - 1, -1):
            Bt, Ct, a = heads_of(B[t], H, G), heads_of(C[t], H, G), torch.exp(dt[t] * A)
            h, hp = states[t - cu[i] + 1], states[t - cu[i]]
            g = g + dy[t][..., None] * Ct[:, None]
            gB = (g * Bt[:, None]).sum(-1)
            o["dx"][t] = D[:, None] * dy[t] + dt[t][:, None] * gB
            o["dB"][t] = dt[t][:, None] * (g * x[t][..., None]).sum(1)
            o["dC"][t] = (h * dy[t][..., None]).sum(1)
            dl = (g * hp).sum((-1, -2)) * a
            o["ddt"][t] = A * dl + (gB * x[t]).sum(-1)
            o["dA"] += dt[t] * dl
            o["dD"] += (dy[t] * x[t]).sum(-1)
            g = g * a[:, None, None]
        if on:
            o["dh_in"][i] = g
    for k in ("dB", "dC"):
        o[k] = o[k].view(T, G, H // G, N).sum(2)
    return o


def dt_used(raw, bias=None, softplus=False, limit=None):
    v = raw.to(F64) + (bias.to(F64) if bias is not None else 0)
    if softplus:
        v = torch.log1p(torch.exp(v))
    return v.clamp(*limit) if limit is not None else v


def norm_grad(dout, y, z, w, eps, group):
    """(dy, dz, dw) of the gated norm by its formula, in 64 bits."""
    dout, y, z, w = (t.to(F64) for t in (dout, y, z, w))
    rows, d = y.shape
    sg = 1 / (1 + torch.exp(-z))
    v = (y * z * sg).view(rows, d // group, group)
    g = (dout * w).view_as(v)
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    dv = (r * (g - v * r * r * (g * v).mean(-1, keepdim=True))).view(rows, d)
    return dv * z * sg, dv * y * sg * (1 + z * (1 - sg)), (dout * (v * r).view(rows, d)).sum(0)


def rel(got, ref):
    got, ref = got.detach().to("cpu", F64), ref.to("cpu", F64)
    if not torch.isfinite(got).all():
        return float("inf")
    return float((got - ref).norm() / ref.norm().clamp_min(1e-300))
