"""Plain 64-bit references of the operators around the recurrence, for their tests: sequence by sequence and
token by token, on the CPU. The scan's also runs on the inputs' absolute values, which bounds what roundings
of its terms can add up to."""
from __future__ import annotations

import torch

F64 = torch.float64


def half_step(dtype) -> float:
    """Largest relative error of rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def spans(lengths):
    at, out = 0, []
    for n in lengths:
        out.append((at, at + n))
        at += n
    return out


def worst(got, want, tol) -> float:
    """max of |got - want| / tol over the elements (0 / 0 counts 0); NaN and infinities in got count as inf."""
    got, want, tol = got.detach().cpu().to(F64), want.to(F64), tol.to(F64)
    d = (got - want).abs()
    d = torch.where(torch.isfinite(got), d, torch.full_like(d, float("inf")))
    r = torch.where(d == 0, torch.zeros_like(d), d / tol)
    return float(r.max()) if r.numel() else 0.0


# ---------------------------------------------------------------- convolution

def conv(x, w, bias, silu, lengths, init):
    """x [R, C] -> dict(out, pre, pre_abs [R, C], final [N, W - 1, C]), all fp64."""
    x, w = x.to(F64), w.to(F64)
    C, W = w.shape
    out, pre_all, mag, final = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x), []
    for i, (a, b) in enumerate(spans(lengths)):
        e = torch.cat([init[i].to(F64) if init is not None else torch.zeros(W - 1, C, dtype=F64), x[a:b]])
        for t in range(b - a):
            pre_all[a + t] = (e[t:t + W] * w.t()).sum(0) + (bias.to(F64) if bias is not None else 0)
            mag[a + t] = (e[t:t + W] * w.t()).abs().sum(0) + (bias.to(F64).abs() if bias is not None else 0)
        final.append(e[b - a:])
    out = pre_all * torch.sigmoid(pre_all) if silu else pre_all.clone()
    return dict(out=out, pre=pre_all, pre_abs=mag, final=torch.stack(final) if final else None)


def conv_loss(x, w, bias, silu, lengths, init, dout, dfinal):
    """The scalar whose gradients kda_conv_bwd returns, differentiable in fp64."""
    W = w.shape[1]
    total = torch.zeros((), dtype=F64)
    for i, (a, b) in enumerate(spans(lengths)):
        e = torch.cat([init[i] if init is not None else torch.zeros(W - 1, w.shape[0], dtype=F64), x[a:b]])
        if b > a:
            pre = sum(e[k:k + b - a] * w[:, k] for k in range(W))
            if bias is not None:
                pre = pre + bias
            y = pre * torch.sigmoid(pre) if silu else pre
            total = total + (y * dout[a:b]).sum()
        if dfinal is not None:
            total = total + (e[b - a:] * dfinal[i]).sum()
    return total


# ---------------------------------------------------------------- q/k

def qk(x, weight, norm, eps, pos, inv_freq, interleaved, factor):
    """x [R, H, D] fp64 -> the normed and rotated heads, differentiable."""
    z = x
    if norm != "none":
        ss = (x * x).sum(-1, keepdim=True)
        ss = (ss / x.shape[-1] if norm == "rms" else ss) + eps
        z = x * torch.where(ss > 0, ss, torch.ones_like(ss)).rsqrt()
    if weight is not None:
        z = z * weight
    if pos is None:
        return z
    rot = 2 * inv_freq.numel()
    ang = pos.to(F64)[:, None] * inv_freq.to(F64)
    c, s = factor * torch.cos(ang)[:, None], factor * torch.sin(ang)[:, None]
    a, b = (z[..., 0:rot:2], z[..., 1:rot:2]) if interleaved else (z[..., :rot // 2], z[..., rot // 2:rot])
    u, v = a * c - b * s, a * s + b * c
    y = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([y, z[..., rot:]], -1)


# ---------------------------------------------------------------- scan

def scan(x, dt, A, B, C, D, bias, softplus, lengths, h0, dout=None, dhT=None):
    """The recurrence x [R, H, P], dt [R, H], B, C [R, G, N]: dict(out, state) in fp64; with dout also the
    gradients, by the adjoint recurrence with every state kept: dlog a_t = <R_t, a_t S_(t-1)>."""
    f = lambda t: None if t is None else t.to(F64)  # noqa: E731
    x, dt, A, B, C, D, bias, h0, dout, dhT = map(f, (x, dt, A, B, C, D, bias, h0, dout, dhT))
    R, H, P = x.shape
    G, N = B.shape[1:]
    rep = H // G
    u = dt + (bias if bias is not None else 0)
    d = torch.logaddexp(u, torch.zeros_like(u)) if softplus else u
    a = torch.exp(d * A)
    Bh, Ch = B.repeat_interleave(rep, 1), C.repeat_interleave(rep, 1)
    out = torch.zeros_like(x)
    n = len(lengths)
    state = torch.zeros(n, H, N, P, dtype=F64)
    g = {}
    if dout is not None:
        g = dict(dx=torch.zeros_like(x), ddelta=torch.zeros_like(dt), dBh=torch.zeros_like(Bh), dCh=torch.zeros_like(Ch),
                 dla=torch.zeros_like(dt), dd=torch.zeros_like(dt), dh0=torch.zeros(n, H, N, P, dtype=F64))
    for i, (s, e) in enumerate(spans(lengths)):
        S = h0[i].clone() if h0 is not None else torch.zeros(H, N, P, dtype=F64)
        kept = [S]
        for t in range(s, e):
            S = a[t][:, None, None] * S + (d[t][:, None] * Bh[t])[:, :, None] * x[t][:, None, :]
            out[t] = torch.einsum("hnp,hn->hp", S, Ch[t])
            if dout is not None:
                kept.append(S)
                g["dCh"][t] = torch.einsum("hnp,hp->hn", S, dout[t])
        state[i] = S
        if dout is None:
            continue
        Rt = dhT[i].clone() if dhT is not None else torch.zeros(H, N, P, dtype=F64)
        for t in range(e - 1, s - 1, -1):
            Rt = Rt + Ch[t][:, :, None] * dout[t][:, None, :]
            bx = torch.einsum("hn,hnp->hp", Bh[t], Rt)
            g["dx"][t] = d[t][:, None] * bx
            g["dBh"][t] = d[t][:, None] * torch.einsum("hnp,hp->hn", Rt, x[t])
            g["dd"][t] = (bx * x[t]).sum(-1)
            g["dla"][t] = (Rt * kept[t - s]).sum((-1, -2)) * a[t]
            Rt = a[t][:, None, None] * Rt
        g["dh0"][i] = Rt
    if D is not None:
        out = out + D[:, None] * x
    r = dict(out=out, state=state, d=d)
    if dout is not None:
        if D is not None:
            g["dx"] = g["dx"] + D[:, None] * dout
            r["dD"] = (dout * x).sum((0, 2))
        r.update(dx=g["dx"], dh0=g["dh0"], dla=g["dla"], dd=g["dd"],
                 dB=g["dBh"].reshape(R, G, rep, N).sum(2), dC=g["dCh"].reshape(R, G, rep, N).sum(2),
                 dA=(g["dla"] * d).sum(0))
        r["ddt"] = (g["dd"] + g["dla"] * A) * (torch.sigmoid(u) if softplus else 1)
        r["ddt_bias"] = r["ddt"].sum(0)
    return r
