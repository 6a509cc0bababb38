"""Workloads of the operators around the recurrence: the short causal convolution, the norm and rotation of
queries and keys, and the selective state space scan, each with its backward pass and, where it has one, its
single-token form.

``run`` computes each operator in plain torch, in 32 bits (64 for positions' angles and for sums of log decays),
or through the library's entry points where ``own`` is true. ``exact`` gives the same outputs in 64 bits from the
operators' definitions.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
CHUNK = 64          # chunk of the plain form of the scan
LOG_DECAY_MIN = -1000.0   # a step that decays by more leaves nothing in 64 bits either


# ---------------------------------------------------------------- cases

def listed():
    return [
        # prompts of 16 requests packed back to back, one projection (32 heads x 128 channels), states kept
        dict(name="conv_prefill_packed", op="conv_fwd", seqs=16, lo=512, hi=8192, lseed=2, rows=0, C=4096, W=4,
             dtype="bf16", states=True, bias=False),
        # a training step's rows, gradient of input, taps and bias
        dict(name="conv_train_bwd", op="conv_bwd", seqs=0, lo=0, hi=0, lseed=0, rows=4, T=4096, C=4096, W=4,
             dtype="bf16", states=False, bias=True),
        # one token of 256 requests, q, k and v channels together
        dict(name="conv_decode_256", op="conv_decode", rows=256, C=12288, W=4, dtype="bf16", bias=True),
        # one token of 64 requests, grouped key heads, RMS norm with weights, half layout, far positions
        dict(name="qk_decode_64", op="qk_fwd", rows=64, T=1, Hq=32, Hk=8, D=128, rot=128, interleaved=False,
             norm="rms", weights=True, far=1 << 20),
        # a prompt's rows, the same model
        dict(name="qk_prefill", op="qk_fwd", rows=1, T=16384, Hq=32, Hk=8, D=128, rot=128, interleaved=False,
             norm="rms", weights=True, far=0),
        # the gradient through the L2 norm of the recurrence's own q and k, part of the head rotated in pairs
        dict(name="qk_train_bwd", op="qk_bwd", rows=2, T=4096, Hq=32, Hk=32, D=128, rot=64, interleaved=True,
             norm="l2", weights=True, far=0),
        # a short prompt alone, where latency counts
        dict(name="scan_prompt_short", op="scan_fwd", seqs=0, lo=0, hi=0, lseed=0, rows=1, T=200, H=32, G=1, P=64,
             N=128, states=True, state_dtype="fp32"),
        # packed ragged prompts with states carried in and out
        dict(name="scan_prefill_packed", op="scan_fwd", seqs=8, lo=129, hi=8192, lseed=5, rows=0, T=0, H=64, G=1,
             P=64, N=128, states=True, state_dtype="fp32"),
        # one long prompt
        dict(name="scan_prefill_long", op="scan_fwd", seqs=0, lo=0, hi=0, lseed=0, rows=1, T=65536, H=32, G=1, P=128,
             N=128, states=False, state_dtype="bf16"),
        # a training step's rows
        dict(name="scan_train_bwd", op="scan_bwd", seqs=0, lo=0, hi=0, lseed=0, rows=2, T=4096, H=64, G=1, P=64,
             N=128, states=False, state_dtype="fp32"),
        # packed rows with carried states, two groups, the smaller state
        dict(name="scan_packed_bwd", op="scan_bwd", seqs=5, lo=1, hi=2000, lseed=9, rows=0, T=0, H=32, G=2, P=128,
             N=64, states=True, state_dtype="fp32"),
        # one token of 256 requests
        dict(name="scan_decode_256", op="scan_decode", rows=256, H=64, G=1, P=64, N=128, state_dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_decode", "qk_fwd", "qk_bwd", "scan_fwd", "scan_bwd",
                     "scan_decode"])
    if op == "conv_decode":
        return dict(op=op, rows=_log_int(rng, 1, 512), C=8 * _log_int(rng, 16, 1536), W=rng.choice([2, 3, 4]),
                    dtype=rng.choice(["bf16", "fp32"]), bias=rng.random() < 0.5)
    if op in ("conv_fwd", "conv_bwd"):
        packed = rng.random() < 0.6
        c = dict(op=op, seqs=rng.randint(1, 16) if packed else 0, lo=rng.randint(1, 200), hi=_log_int(rng, 256, 4096),
                 lseed=rng.randrange(1 << 20), rows=0 if packed else rng.randint(1, 4),
                 T=0 if packed else _log_int(rng, 1, 4096), C=8 * _log_int(rng, 16, 512), W=rng.choice([2, 3, 4]),
                 dtype=rng.choice(["bf16", "bf16", "fp32"]), states=rng.random() < 0.5, bias=rng.random() < 0.5)
        return c
    if op in ("qk_fwd", "qk_bwd"):
        D = rng.choice([64, 128, 256])
        Hk = _log_int(rng, 1, 16)
        return dict(op=op, rows=rng.randint(1, 4), T=_log_int(rng, 1, 3000), Hq=Hk * rng.choice([1, 2, 4]), Hk=Hk,
                    D=D, rot=rng.choice([0, D // 4, D // 2, D]), interleaved=rng.random() < 0.5,
                    norm=rng.choice(["none", "l2", "rms"]), weights=rng.random() < 0.5,
                    far=rng.choice([0, 1 << 17, 1 << 20]))
    G = rng.choice([1, 2])
    H = G * _log_int(rng, 1, 24)
    P, N = rng.choice([64, 128]), rng.choice([64, 128])
    dt = rng.choice(["fp32", "bf16"])
    if op == "scan_decode":
        return dict(op=op, rows=_log_int(rng, 1, 256), H=H, G=G, P=P, N=N, state_dtype=dt)
    packed = rng.random() < 0.6
    top = 8000 if op == "scan_fwd" else 1500
    return dict(op=op, seqs=rng.randint(1, 8) if packed else 0, lo=1, hi=_log_int(rng, 64, top),
                lseed=rng.randrange(1 << 20), rows=0 if packed else rng.randint(1, 3),
                T=0 if packed else _log_int(rng, 1, top), H=H, G=G, P=P, N=N, states=rng.random() < 0.5,
                state_dtype=dt)


def _lengths(c):
    """The sequences' lengths: drawn from the case alone."""
    if not c.get("seqs"):
        return [c.get("T", 1)] * c["rows"]
    r = random.Random(c["lseed"])
    return [r.randint(c["lo"], max(c["lo"], c["hi"])) for _ in range(c["seqs"])]


_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    ru = lambda *s: torch.rand(s, generator=gen, device=DEV)  # noqa: E731
    c, op = case, case["op"]
    s = dict(case=dict(case), op=op)
    if op.startswith("conv"):
        C, W, dt = c["C"], c["W"], _DT[c["dtype"]]
        s["weight"] = (rn(C, W) / math.sqrt(W)).float()
        s["bias"] = 0.1 * rn(C) if c["bias"] else None
        if op == "conv_decode":
            s["x"] = rn(c["rows"], C).to(dt)
            s["state"] = rn(c["rows"], W - 1, C).to(dt)
            s["state_out"] = torch.empty_like(s["state"])
            return s
        L = _lengths(c)
        packed = bool(c["seqs"])
        n, shape = len(L), ((1, sum(L), C) if packed else (c["rows"], c["T"], C))
        s["x"] = rn(*shape).to(dt)
        s["cu"] = torch.tensor(np.cumsum([0] + L), dtype=torch.int32, device=DEV) if packed else None
        s["init"] = rn(n, W - 1, C).to(dt) if c["states"] else None
        if op == "conv_bwd":
            s["dout"] = rn(*shape).to(dt)
            s["dfinal"] = rn(n, W - 1, C).to(dt) if c["states"] else None
        return s
    if op.startswith("qk"):
        R, T, D = c["rows"], c["T"], c["D"]
        s["q"] = rn(R, T, c["Hq"], D).to(torch.bfloat16)
        s["k"] = rn(R, T, c["Hk"], D).to(torch.bfloat16)
        first = torch.randint(0, c["far"] + 1, (R, 1), generator=gen, device=DEV)
        s["pos"] = (first + torch.arange(T, device=DEV)).to(torch.int32)
        half = c["rot"] // 2
        s["inv_freq"] = (1e4 ** (-torch.arange(half, device=DEV).double() / max(half, 1))).float()
        w = c["weights"] and c["norm"] != "none"
        s["qw"] = 1 + 0.2 * rn(D) if w else None
        s["kw"] = 1 + 0.2 * rn(D) if w else None
        if op == "qk_bwd":
            s["dq"] = rn(R, T, c["Hq"], D).to(torch.bfloat16)
            s["dk"] = rn(R, T, c["Hk"], D).to(torch.bfloat16)
        return s
    H, G, P, N = c["H"], c["G"], c["P"], c["N"]
    if op == "scan_decode":
        lead, n, packed = (c["rows"],), c["rows"], False
    else:
        L = _lengths(c)
        packed = bool(c["seqs"])
        lead, n = ((1, sum(L)) if packed else (c["rows"], c["T"])), len(L)
        s["cu"] = torch.tensor(np.cumsum([0] + L), dtype=torch.int32, device=DEV) if packed else None
        s["lmax"] = max(L)
    s["x"] = (0.7 * rn(*lead, H, P)).to(torch.bfloat16)
    s["B"] = (0.5 * rn(*lead, G, N)).to(torch.bfloat16)
    s["C"] = (0.5 * rn(*lead, G, N)).to(torch.bfloat16)
    s["dt"] = 0.5 * rn(*lead, H)
    step = torch.exp(math.log(1e-3) + math.log(1e2) * ru(H))           # steps of 0.001 to 0.1
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))               # the inverse of softplus
    s["A"] = -(1 + 15 * ru(H))
    s["D"] = 1 + 0.2 * rn(H)
    sd = _DT[c["state_dtype"]]
    if op == "scan_decode":
        s["state"] = (0.3 * rn(n, H, N, P)).to(sd)
        s["state_out"] = torch.empty_like(s["state"])
        return s
    s["h0"] = (0.3 * rn(n, H, N, P)).to(sd) if c["states"] else None
    if op == "scan_bwd":
        s["dout"] = rn(*lead, H, P).to(torch.bfloat16)
        s["dhT"] = 0.3 * rn(n, H, N, P) if c["states"] else None
    return s


# ---------------------------------------------------------------- plain forms

def _seqs(x, cu, n, pad):
    """Rows of every sequence side by side: (index [n, pad] into the flat rows, valid [n, pad])."""
    j = torch.arange(pad, device=x.device)
    if cu is None:
        T = x.shape[1]
        return torch.arange(n, device=x.device)[:, None] * T + j.clamp(max=max(T - 1, 0)), (j < T).expand(n, pad)
    start, end = cu[:-1].long()[:, None], cu[1:].long()[:, None]
    at = start + j
    return torch.minimum(at, (end - 1).clamp(min=0)).clamp(max=max(x.shape[1] - 1, 0)), at < end


def _sequence_of(x, cu):
    """(number of the sequence, place in it, its length) of every flat row."""
    B, T = x.shape[:2]
    row = torch.arange(B * T, device=x.device)
    if cu is None:
        return row // T, row % T, torch.full_like(row, T)
    i = torch.searchsorted(cu[1:].long(), row, right=True)
    return i, row - cu[i].long(), (cu[i + 1] - cu[i]).long()


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _conv_taps(s):
    """The inputs under each of the W taps, [rows, W, C] one at a time: e_(t-W+1+i)."""
    x, c = s["x"], s["case"]
    W, C = c["W"], c["C"]
    flat = x.reshape(-1, C).float()
    i, t, _ = _sequence_of(x, s["cu"])
    init = torch.zeros(1, W - 1, C, device=x.device) if s["init"] is None else s["init"].float()
    i = torch.zeros_like(i) if s["init"] is None else i

    def tap(k):
        back = W - 1 - k                      # how far behind the row
        old = (t < back)[:, None]
        if back == 0:
            return flat
        e = flat[(torch.arange(flat.shape[0], device=x.device) - back).clamp(min=0)]
        return torch.where(old, init[i, (W - 1 + t - back).clamp(0, W - 2)], e)
    return tap


def _conv_final(s):
    """The last W - 1 rows of every sequence, with its initial state before it."""
    x, c, cu = s["x"], s["case"], s["cu"]
    W, C = c["W"], c["C"]
    n = len(_lengths(c))
    start = (torch.arange(n, device=x.device) * x.shape[1] if cu is None else cu[:-1].long())[:, None]
    length = (torch.full((n, 1), x.shape[1], device=x.device) if cu is None
              else (cu[1:] - cu[:-1]).long()[:, None])
    at = length - (W - 1) + torch.arange(W - 1, device=x.device)           # place in the sequence
    rows = x.reshape(-1, C)[(start + at).clamp(0, max(x.shape[0] * x.shape[1] - 1, 0))]
    old = torch.zeros_like(rows)
    if s["init"] is not None:
        old = torch.gather(s["init"], 1, (at + W - 1).clamp(0, W - 2)[:, :, None].expand(-1, -1, C))
    return torch.where((at < 0)[:, :, None], old, rows)


def _plain_conv_fwd(s):
    w, tap = s["weight"], _conv_taps(s)
    pre = sum(tap(k) * w[:, k] for k in range(w.shape[1]))
    if s["bias"] is not None:
        pre = pre + s["bias"]
    out = (pre * _sigmoid(pre)).to(s["x"].dtype).reshape(s["x"].shape)
    return dict(out=out, final=_conv_final(s) if s["case"]["states"] else None)


def _plain_conv_bwd(s):
    x, w, tap, c = s["x"], s["weight"], _conv_taps(s), s["case"]
    W, C = c["W"], c["C"]
    pre = sum(tap(k) * w[:, k] for k in range(W))
    if s["bias"] is not None:
        pre = pre + s["bias"]
    g = _sigmoid(pre)
    dpre = s["dout"].reshape(-1, C).float() * (g * (1 + pre * (1 - g)))
    del pre, g
    dweight = torch.stack([(tap(k) * dpre).sum(0) for k in range(W)], 1)
    i, t, length = _sequence_of(x, s["cu"])
    dx = torch.zeros_like(dpre)
    rows = torch.arange(dpre.shape[0], device=x.device)
    for k in range(W):
        ahead = W - 1 - k
        dx += torch.where((t + ahead < length)[:, None], dpre[(rows + ahead).clamp(max=dpre.shape[0] - 1)] * w[:, k], 0)
    dinit = None
    if s["init"] is not None:
        n = s["init"].shape[0]
        start = (torch.arange(n, device=x.device) * x.shape[1] if s["cu"] is None else s["cu"][:-1].long())[:, None]
        ln = (torch.full((n, 1), x.shape[1], device=x.device) if s["cu"] is None
              else (s["cu"][1:] - s["cu"][:-1]).long()[:, None])
        j = torch.arange(W - 1, device=x.device)           # row j of the state is place j - (W - 1)
        dinit = torch.zeros(n, W - 1, C, device=x.device)
        for k in range(W):
            at = (j - k).expand(n, W - 1)                  # the output whose tap k it is under
            ok = (at >= 0) & (at < ln)
            dinit += torch.where(ok[:, :, None], dpre[(start + at).clamp(0, dpre.shape[0] - 1)] * w[:, k], 0)
    if s["dfinal"] is not None:
        df = s["dfinal"].float()
        slot = (t - length + (W - 1))
        dx += torch.where((slot >= 0)[:, None], df[i, slot.clamp(min=0)], 0)
        if dinit is not None:                              # sequences shorter than the state pass part of it on
            slot = j - ln                                  # row j of the initial state is row j - length of the final
            dinit += torch.where((slot >= 0)[:, :, None],
                                 torch.gather(df, 1, slot.clamp(min=0)[:, :, None].expand(-1, -1, C)), 0)
    return dict(dx=dx.to(x.dtype).reshape(x.shape), dweight=dweight,
                dbias=dpre.sum(0) if s["bias"] is not None else None,
                dinit=dinit.to(x.dtype) if dinit is not None else None)


def _plain_conv_decode(s):
    e = torch.cat([s["state"], s["x"][:, None]], 1)
    pre = (e.float() * s["weight"].t()).sum(1)
    if s["bias"] is not None:
        pre = pre + s["bias"]
    return dict(out=(pre * _sigmoid(pre)).to(s["x"].dtype), state=e[:, 1:])


EPS = 1e-6


def _rotate(x, pos, inv_freq, rot, interleaved, sign):
    """x [R, T, heads, D] in 32 bits; the first `rot` channels rotated by sign * pos * inv_freq."""
    if rot == 0:
        return x
    angle = pos.double()[..., None] * inv_freq.double()
    cos, sin = angle.cos().to(x.dtype)[:, :, None], (sign * angle.sin()).to(x.dtype)[:, :, None]
    y, rest = x[..., :rot], x[..., rot:]
    a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([y, rest], -1)


def _inverse_norm(x, norm):
    ss = (x * x).sum(-1, keepdim=True)
    return torch.rsqrt(ss + EPS) if norm == "l2" else torch.rsqrt(ss / x.shape[-1] + EPS)


def _plain_qk_fwd(s):
    c = s["case"]

    def one(x, w):
        z = x.float()
        if c["norm"] != "none":
            z = z * _inverse_norm(z, c["norm"])
        if w is not None:
            z = z * w
        return _rotate(z, s["pos"], s["inv_freq"], c["rot"], c["interleaved"], 1).to(x.dtype)
    return dict(q=one(s["q"], s["qw"]), k=one(s["k"], s["kw"]))


def _plain_qk_bwd(s):
    c = s["case"]

    def one(x, w, dy):
        dz = _rotate(dy.float(), s["pos"], s["inv_freq"], c["rot"], c["interleaved"], -1)
        if c["norm"] == "none":
            return dz.to(x.dtype), None
        xf = x.float()
        r = _inverse_norm(xf, c["norm"])
        xh = xf * r
        dw = (dz * xh).sum((0, 1, 2)) if w is not None else None
        dz = dz * w if w is not None else dz
        mean = (xh * dz).sum(-1, keepdim=True) / (c["D"] if c["norm"] == "rms" else 1)
        return (r * (dz - xh * mean)).to(x.dtype), dw
    dq, dqw = one(s["q"], s["qw"], s["dq"])
    dk, dkw = one(s["k"], s["kw"], s["dk"])
    return dict(dq=dq, dk=dk, dqw=dqw, dkw=dkw)


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _scan_core(s, x, dt, A, B, C, D, dt_bias, h0):
    """The chunked form over sequences laid side by side, differentiable: (y in flat rows, final states)."""
    c = s["case"]
    H, G, P, N = c["H"], c["G"], c["P"], c["N"]
    n = len(_lengths(c))
    Q = min(CHUNK, max(1, s["lmax"]))
    nc = -(-max(1, s["lmax"]) // Q)
    at, ok = _seqs(s["x"], s["cu"], n, nc * Q)
    d = _softplus(dt.reshape(-1, H)[at] + dt_bias) * ok[:, :, None]         # a step of zero changes nothing
    d = d.reshape(n, nc, Q, H)
    xs = x.reshape(-1, H, P)[at].reshape(n, nc, Q, G, H // G, P)
    Bs = B.reshape(-1, G, N)[at].reshape(n, nc, Q, G, N)
    Cs = C.reshape(-1, G, N)[at].reshape(n, nc, Q, G, N)
    cs = (d * A).double().clamp(min=LOG_DECAY_MIN).cumsum(2)                # [n, nc, Q, H]
    low = torch.ones(Q, Q, dtype=torch.bool, device=x.device).tril()
    diff = (cs[:, :, :, None] - cs[:, :, None]).float().masked_fill(~low[:, :, None], -math.inf)
    L = torch.exp(diff).reshape(n, nc, Q, Q, G, H // G)
    M = torch.einsum("zcqgk,zcsgk->zcqsg", Cs, Bs)[..., None] * L * d.reshape(n, nc, 1, Q, G, H // G)
    y = torch.einsum("zcqsgh,zcsghp->zcqghp", M, xs)
    to_end = torch.exp((cs[:, :, -1:] - cs).float()) * d
    local = torch.einsum("zcsgk,zcsghp->zcghkp", Bs, xs * to_end.reshape(n, nc, Q, G, H // G, 1))
    tot = torch.cat([torch.zeros(n, 1, H, dtype=torch.float64, device=x.device), cs[:, :, -1].cumsum(1)], 1)
    low = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=x.device).tril()
    over = (tot[:, :, None] - tot[:, None]).float().masked_fill(~low[:, :, None], -math.inf)
    over = torch.exp(over).permute(0, 3, 1, 2)                              # [n, H, to, from]
    first = torch.zeros(n, 1, H, N * P, device=x.device) if h0 is None else h0.reshape(n, 1, H, N * P)
    states = torch.cat([first, local.reshape(n, nc, H, N * P)], 1).transpose(1, 2)
    states = (over @ states).reshape(n, G, H // G, nc + 1, N, P)            # entering each chunk, and at the end
    inter = torch.einsum("zcqgk,zghckp->zcqghp", Cs, states[:, :, :, :-1])
    y = y + inter * torch.exp(cs.float()).reshape(n, nc, Q, G, H // G, 1)
    y = (y + xs * D.reshape(G, H // G, 1)).reshape(n, nc * Q, H, P)
    i, t, _ = _sequence_of(s["x"], s["cu"])
    return y[i, t].reshape(s["x"].shape), states[:, :, :, -1].reshape(n, H, N, P)


def _plain_scan_fwd(s):
    h0 = s["h0"].float() if s["h0"] is not None else None
    y, hT = _scan_core(s, s["x"].float(), s["dt"], s["A"], s["B"].float(), s["C"].float(), s["D"], s["dt_bias"], h0)
    return dict(out=y.to(s["x"].dtype), state=hT.to(_DT[s["case"]["state_dtype"]]))


def _plain_scan_bwd(s):
    names = ["x", "dt", "A", "B", "C", "D", "dt_bias"] + (["h0"] if s["h0"] is not None else [])
    leaf = {k: s[k].detach().float().requires_grad_() for k in names}
    with torch.enable_grad():
        y, hT = _scan_core(s, *(leaf[k] for k in ("x", "dt", "A", "B", "C", "D", "dt_bias")), leaf.get("h0"))
        loss = [y] + ([hT] if s["dhT"] is not None else [])
        g = torch.autograd.grad(loss, [leaf[k] for k in names],
                                [s["dout"].float()] + ([s["dhT"]] if s["dhT"] is not None else []))
    g = dict(zip(names, g))
    for k in ("x", "B", "C"):
        g[k] = g[k].to(torch.bfloat16)
    return {"d" + k: v for k, v in g.items()}


def _plain_scan_decode(s):
    c = s["case"]
    b, H, G = c["rows"], c["H"], c["G"]
    d = _softplus(s["dt"] + s["dt_bias"])
    a = torch.exp(d * s["A"])
    Bh = s["B"].float().repeat_interleave(H // G, 1)
    Ch = s["C"].float().repeat_interleave(H // G, 1)
    x = s["x"].float()
    S = s["state"].float() * a[..., None, None] + Bh[..., None] * (x * d[..., None])[:, :, None]
    y = (S * Ch[..., None]).sum(2) + x * s["D"][:, None]
    return dict(out=y.to(s["x"].dtype), state=S.to(s["state"].dtype))


# ---------------------------------------------------------------- the library's calls

def _own_conv_fwd(s):
    import kimi_delta_attention_27_b200 as kda
    out, final = kda.kda_conv_fwd(s["x"], s["weight"], bias=s["bias"], cu_seqlens=s["cu"], initial_state=s["init"],
                                  want_final_state=s["case"]["states"])
    return dict(out=out, final=final)


def _own_conv_bwd(s):
    import kimi_delta_attention_27_b200 as kda
    g = kda.kda_conv_bwd(s["x"], s["weight"], s["dout"], bias=s["bias"], cu_seqlens=s["cu"], initial_state=s["init"],
                         dfinal_state=s["dfinal"], want_dinitial_state=s["init"] is not None)
    return dict(dx=g["dx"], dweight=g["dweight"], dbias=g["dbias"], dinit=g["dinitial_state"])


def _own_conv_decode(s):
    import kimi_delta_attention_27_b200 as kda
    out, state = kda.kda_conv_decode(s["x"], s["weight"], s["state"], s["state_out"], bias=s["bias"])
    return dict(out=out, state=state)


def _own_qk_fwd(s):
    import kimi_delta_attention_27_b200 as kda
    c = s["case"]
    q, k = kda.kda_qk_fwd(s["q"], s["k"], norm=c["norm"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                          positions=s["pos"] if c["rot"] else None, inv_freq=s["inv_freq"] if c["rot"] else None,
                          interleaved=c["interleaved"])
    return dict(q=q, k=k)


def _own_qk_bwd(s):
    import kimi_delta_attention_27_b200 as kda
    c = s["case"]
    g = kda.kda_qk_bwd(s["q"], s["k"], s["dq"], s["dk"], norm=c["norm"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                       positions=s["pos"] if c["rot"] else None, inv_freq=s["inv_freq"] if c["rot"] else None,
                       interleaved=c["interleaved"])
    return dict(dq=g["dq"], dk=g["dk"], dqw=g["dq_weight"], dkw=g["dk_weight"])


def _own_scan_fwd(s):
    import kimi_delta_attention_27_b200 as kda
    out, state = kda.kda_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], dt_bias=s["dt_bias"],
                                  dt_softplus=True, cu_seqlens=s["cu"], initial_state=s["h0"],
                                  final_state_dtype=_DT[s["case"]["state_dtype"]])
    return dict(out=out, state=state)


def _own_scan_bwd(s):
    import kimi_delta_attention_27_b200 as kda
    g = kda.kda_scan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["dout"], D=s["D"], dt_bias=s["dt_bias"],
                         dt_softplus=True, cu_seqlens=s["cu"], initial_state=s["h0"], dfinal_state=s["dhT"],
                         want_dinitial_state=s["h0"] is not None)
    out = {k: g[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias")}
    if s["h0"] is not None:
        out["dh0"] = g["dh0"]
    return out


def _own_scan_decode(s):
    import kimi_delta_attention_27_b200 as kda
    out, state = kda.kda_scan_decode(s["x"], s["dt"], s["A"], s["B"], s["C"], state_in=s["state"],
                                     state_out=s["state_out"], D=s["D"], dt_bias=s["dt_bias"], dt_softplus=True)
    return dict(out=out, state=state)


_PLAIN = dict(conv_fwd=_plain_conv_fwd, conv_bwd=_plain_conv_bwd, conv_decode=_plain_conv_decode,
              qk_fwd=_plain_qk_fwd, qk_bwd=_plain_qk_bwd, scan_fwd=_plain_scan_fwd, scan_bwd=_plain_scan_bwd,
              scan_decode=_plain_scan_decode)
_OWN = dict(conv_fwd=_own_conv_fwd, conv_bwd=_own_conv_bwd, conv_decode=_own_conv_decode, qk_fwd=_own_qk_fwd,
            qk_bwd=_own_qk_bwd, scan_fwd=_own_scan_fwd, scan_bwd=_own_scan_bwd, scan_decode=_own_scan_decode)


def run(state):
    with torch.no_grad():
        if own:
            return _OWN[state["op"]](state)
        return _PLAIN[state["op"]](state)


# ---------------------------------------------------------------- work

def work(case):
    """Bytes of every input and output once; operations of the definitions (the scan's as a recurrence)."""
    c, op = case, case["op"]
    if op.startswith("conv"):
        C, W, e = c["C"], c["W"], 2 if c["dtype"] == "bf16" else 4
        if op == "conv_decode":
            return dict(bytes=c["rows"] * C * e * 2 * W + C * 4 * (W + 1), flops=c["rows"] * C * (2 * W + 4))
        L = _lengths(c)
        t, st = sum(L), len(L) * (W - 1) * C * e if c["states"] else 0
        taps = C * 4 * (W + bool(c["bias"]))
        if op == "conv_fwd":
            return dict(bytes=2 * t * C * e + 2 * st + taps, flops=t * C * (2 * W + 4))
        return dict(bytes=3 * t * C * e + 3 * st + 2 * taps, flops=t * C * (6 * W + 10))
    if op.startswith("qk"):
        heads, rows, D = c["Hq"] + c["Hk"], c["rows"] * c["T"], c["D"]
        n = rows * heads * D
        small = rows * 4 + c["rot"] * 2 + (16 * D if c["weights"] else 0)
        if op == "qk_fwd":
            return dict(bytes=4 * n + small, flops=8 * n)
        return dict(bytes=6 * n + small, flops=16 * n)
    H, G, P, N = c["H"], c["G"], c["P"], c["N"]
    sb = 4 if c["state_dtype"] == "fp32" else 2
    if op == "scan_decode":
        b = c["rows"]
        return dict(bytes=b * H * N * P * sb * 2 + b * (H * P * 4 + G * N * 4 + H * 4) + 12 * H,
                    flops=5 * b * H * N * P)
    L = _lengths(c)
    t, n = sum(L), len(L)
    st = n * H * N * P
    if op == "scan_fwd":
        return dict(bytes=t * (4 * H * P + 4 * G * N + 4 * H) + st * sb * (2 if c["states"] else 1) + 12 * H,
                    flops=5 * t * H * N * P)
    return dict(bytes=t * (6 * H * P + 8 * G * N + 8 * H) + (st * (sb + 8) if c["states"] else 0) + 24 * H,
                flops=14 * t * H * N * P)


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return dict(conv_fwd=_exact_conv, conv_bwd=_exact_conv, conv_decode=_exact_conv_decode, qk_fwd=_exact_qk,
                    qk_bwd=_exact_qk, scan_fwd=_exact_scan, scan_bwd=_exact_scan,
                    scan_decode=_exact_scan_decode)[case["op"]](s)


def _rows_of(s):
    c = s["case"]
    ends = np.cumsum([0] + _lengths(c))
    return [(int(a), int(b)) for a, b in zip(ends[:-1], ends[1:])]


def _exact_conv(s):
    """Sequence by sequence: the extended rows, and each tap as a shifted slice; gradients by shifted slices too."""
    c = s["case"]
    C, W = c["C"], c["W"]
    x = s["x"].reshape(-1, C)
    w = s["weight"].double()
    bwd = s["op"] == "conv_bwd"
    dy = s["dout"].reshape(-1, C) if bwd else None
    out = torch.empty(x.shape, dtype=torch.float64, device=DEV)
    dw, db = torch.zeros(C, W, dtype=torch.float64, device=DEV), torch.zeros(C, dtype=torch.float64, device=DEV)
    edge = []
    for i, (a, b) in enumerate(_rows_of(s)):
        n = b - a
        before = s["init"][i].double() if s["init"] is not None else torch.zeros(W - 1, C, dtype=torch.float64,
                                                                                 device=DEV)
        e = torch.cat([before, x[a:b].double()])
        pre = torch.zeros(n, C, dtype=torch.float64, device=DEV)
        for k in range(W):
            pre += e[k:k + n] * w[:, k]
        if s["bias"] is not None:
            pre += s["bias"].double()
        if not bwd:
            out[a:b] = pre * torch.sigmoid(pre)
            edge.append(e[n:])
            continue
        g = torch.sigmoid(pre)
        dpre = dy[a:b].double() * g * (1 + pre * (1 - g))
        de = torch.zeros_like(e)
        for k in range(W):
            de[k:k + n] += dpre * w[:, k]
            dw[:, k] += (dpre * e[k:k + n]).sum(0)
        db += dpre.sum(0)
        if s["dfinal"] is not None:
            de[n:] += s["dfinal"][i].double()
        out[a:b] = de[W - 1:]
        edge.append(de[:W - 1])
    shape = s["x"].shape
    if not bwd:
        return dict(out=out.reshape(shape), final=torch.stack(edge) if c["states"] else None)
    return dict(dx=out.reshape(shape), dweight=dw, dbias=db if s["bias"] is not None else None,
                dinit=torch.stack(edge) if s["init"] is not None else None)


def _exact_conv_decode(s):
    W = s["case"]["W"]
    w = s["weight"].double()
    pre = s["x"].double() * w[:, W - 1]
    for k in range(W - 1):
        pre += s["state"][:, k].double() * w[:, k]
    if s["bias"] is not None:
        pre += s["bias"].double()
    return dict(out=pre * torch.sigmoid(pre), state=torch.cat([s["state"][:, 1:], s["x"][:, None]], 1).double())


def _exact_qk(s):
    """Complex rotation of the normed heads, and the gradients by differentiating that in 64 bits."""
    c = s["case"]
    rot, D = c["rot"], c["D"]

    def turn(z):
        if rot == 0:
            return z
        a = s["pos"].double()[..., None] * s["inv_freq"].double()
        u = torch.polar(torch.ones_like(a), a)[:, :, None]
        if c["interleaved"]:
            v = torch.view_as_complex(z[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * u
            y = torch.view_as_real(v).flatten(-2)
        else:
            v = torch.complex(z[..., :rot // 2].contiguous(), z[..., rot // 2:rot].contiguous()) * u
            y = torch.cat([v.real, v.imag], -1)
        return torch.cat([y, z[..., rot:]], -1)

    def one(x, w):
        z = x
        if c["norm"] == "l2":
            z = z / (z.square().sum(-1, keepdim=True) + EPS).sqrt()
        elif c["norm"] == "rms":
            z = z / (z.square().mean(-1, keepdim=True) + EPS).sqrt()
        return turn(z if w is None else z * w)

    if s["op"] == "qk_fwd":
        return dict(q=one(s["q"].double(), s["qw"].double() if s["qw"] is not None else None),
                    k=one(s["k"].double(), s["kw"].double() if s["kw"] is not None else None))
    got = {}
    for name, wn in (("q", "qw"), ("k", "kw")):
        with torch.enable_grad():
            x = s[name].double().requires_grad_()
            w = s[wn].double().requires_grad_() if s[wn] is not None else None
            g = torch.autograd.grad(one(x, w), [x] + ([w] if w is not None else []), s["d" + name].double())
        got["d" + name] = g[0]
        got["d" + wn] = g[1] if w is not None else None
    return got


def _exact_scan(s):
    """The recurrence, one token after another, over all sequences at once; its adjoint likewise."""
    c = s["case"]
    H, G, P, N = c["H"], c["G"], c["P"], c["N"]
    spans = _rows_of(s)
    n, T = len(spans), sum(b - a for a, b in spans)
    top = max(b - a for a, b in spans)
    bwd = s["op"] == "scan_bwd"
    if top * max(30e-6, n * H * N * P * 8 * 4 / 4e12) * (3 if bwd else 1) > 15:
        return None
    start = torch.tensor([a for a, _ in spans], device=DEV)
    length = torch.tensor([b - a for a, b in spans], device=DEV)
    x, dt = s["x"].reshape(T, H, P), s["dt"].reshape(T, H).double()
    Bm, Cm = s["B"].reshape(T, G, N), s["C"].reshape(T, G, N)
    A, D = s["A"].double(), s["D"].double()
    u = dt + s["dt_bias"].double()
    d = torch.logaddexp(u, torch.zeros_like(u))
    decay = torch.exp(d * A)
    S = s["h0"].double() if s["h0"] is not None else torch.zeros(n, H, N, P, dtype=torch.float64, device=DEV)
    S = S.reshape(n, G, H // G, N, P).clone()
    live = [int((length > t).sum()) for t in range(top)]
    order = torch.argsort(length, descending=True)         # the longest first: the live ones are a slice
    S, start, length = S[order], start[order], length[order]
    dy = s["dout"].reshape(T, H, P) if bwd else None
    y = torch.empty(T, H, P, dtype=torch.float64, device=DEV)
    dC_h = torch.zeros(T, G, N, dtype=torch.float64, device=DEV) if bwd else None
    for t in range(top):
        m = live[t]
        r = start[:m] + t
        St = S[:m]
        St.mul_(decay[r].reshape(m, G, H // G, 1, 1))
        xd = (x[r].double() * d[r][..., None]).reshape(m, G, H // G, 1, P)
        St.addcmul_(Bm[r].double().reshape(m, G, 1, N, 1), xd)
        y[r] = torch.matmul(Cm[r].double().reshape(m, G, 1, 1, N), St).reshape(m, H, P)
        if bwd:
            dC_h[r] = torch.matmul(St, dy[r].double().reshape(m, G, H // G, P, 1)).sum(2).reshape(m, G, N)
    if not bwd:
        hT = torch.empty_like(S)
        hT[order] = S
        return dict(out=(y + x.double() * D[:, None]).reshape(s["x"].shape), state=hT.reshape(n, H, N, P))
    back = torch.empty_like(order)
    back[order] = torch.arange(n, device=DEV)
    R = (s["dhT"].double() if s["dhT"] is not None else torch.zeros(n, H, N, P, dtype=torch.float64, device=DEV))
    R = R.reshape(n, G, H // G, N, P)[order].clone()
    end_dot = (R * S).sum((-1, -2)).reshape(n, H)          # <dhT, S_L>: what the decay of every step scales
    dx = torch.empty(T, H, P, dtype=torch.float64, device=DEV)
    dB = torch.empty(T, G, N, dtype=torch.float64, device=DEV)
    for t in reversed(range(top)):
        m = live[t]
        r = start[:m] + t
        Rt = R[:m]
        Rt.addcmul_(Cm[r].double().reshape(m, G, 1, N, 1), dy[r].double().reshape(m, G, H // G, 1, P))
        dx[r] = torch.matmul(Bm[r].double().reshape(m, G, 1, 1, N), Rt).reshape(m, H, P)
        xd = (x[r].double() * d[r][..., None]).reshape(m, G, H // G, P, 1)
        dB[r] = torch.matmul(Rt, xd).sum(2).reshape(m, G, N)
        Rt.mul_(decay[r].reshape(m, G, H // G, 1, 1))
    dd = (dx * x.double()).sum(-1)                         # through the input term
    gam = (y * dy.double()).sum(-1) - d * dd               # with respect to the cumulated log decay
    dla = torch.empty_like(gam)
    for i, (a, b) in enumerate(spans):
        dla[a:b] = gam[a:b].flip(0).cumsum(0).flip(0) + end_dot[back[i]]
    ddt = (dd + dla * A) * torch.sigmoid(u)
    got = dict(dx=(dx * d[..., None] + D[:, None] * dy.double()).reshape(s["x"].shape), ddt=ddt.reshape(s["dt"].shape),
               dA=(dla * d).sum(0), dB=dB.reshape(s["B"].shape), dC=dC_h.reshape(s["C"].shape),
               dD=(dy.double() * x.double()).sum((0, 2)), ddt_bias=ddt.sum(0))
    if s["h0"] is not None:
        got["dh0"] = R[back].reshape(n, H, N, P)
    return got


def _exact_scan_decode(s):
    c = s["case"]
    per = c["H"] // c["G"]
    u = s["dt"].double() + s["dt_bias"].double()
    d = torch.logaddexp(u, torch.zeros_like(u))
    S = torch.empty(s["state"].shape, dtype=torch.float64, device=DEV)
    y = torch.empty(s["x"].shape, dtype=torch.float64, device=DEV)
    for h in range(c["H"]):
        k = s["B"][:, h // per].double()
        S[:, h] = (s["state"][:, h].double() * torch.exp(d[:, h] * s["A"][h].double())[:, None, None]
                   + torch.einsum("bn,bp->bnp", k * d[:, h, None], s["x"][:, h].double()))
        y[:, h] = torch.einsum("bn,bnp->bp", s["C"][:, h // per].double(), S[:, h]) + s["D"][h].double() * s["x"][:, h].double()
    return dict(out=y, state=S)
