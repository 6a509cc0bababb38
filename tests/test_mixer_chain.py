"""The operators together, as a layer runs them: projection -> convolution -> norm and rotation -> recurrence, or
projection -> convolution -> scan; prompts, gradients, single tokens, and all of it captured. Each stage is held to the
64-bit reference on what the stage before it really gave."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_27_b200 as kda
import mixer_ref as ref
from kda_testutil import OUT_TOL, STATE_TOL, rel
from test_bwd_gpu import BWD_TOL
from test_conv import out_tol
from test_scan import H16, check_bwd, check_fwd, cu_of, fp32_ops, mags

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    from kimi_delta_attention_27_b200 import build
    build.build()
    return kda.load_library()


def randn(gen, *s, scale=1.0):
    return scale * torch.randn(*s, generator=gen)


def conv_check(x, w, b, lengths, init, out, final):
    r = ref.conv(x.cpu(), w.cpu(), b.cpu(), True, lengths, init.cpu())
    assert ref.worst(out, r["out"], out_tol(r, BF, True)) <= 1 and torch.equal(final.cpu().to(ref.F64), r["final"])


# ---------------------------------------------------------------- the delta-rule layer

H, D, W = 2, 128, 4
CH = 3 * H * D


class Layer:
    """Weights and the three calls of a layer's mixer over a packed batch."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.w, self.b = randn(g, CH, W, scale=0.5).cuda(), randn(g, CH, scale=0.1).cuda()
        self.qw, self.kw = (1 + randn(g, D, scale=0.2)).cuda(), (1 + randn(g, D, scale=0.2)).cuda()
        self.freq = (1e4 ** (-torch.arange(32) / 32)).float().cuda()

    def heads(self, c, pos):
        q, k, v = (t.unflatten(-1, (H, D)) for t in c.split(H * D, -1))
        qn, kn = kda.kda_qk_fwd(q, k, "l2", self.qw, self.kw, positions=pos, inv_freq=self.freq)
        return q, k, qn, kn, v.contiguous()

    def heads_reference(self, x, w, pos):
        return ref.qk(x, w, "l2", 1e-6, pos.reshape(-1).cpu(), self.freq.cpu(), False, 1.0)


def inputs(lengths, seed):
    g = torch.Generator().manual_seed(seed)
    R, n = sum(lengths), len(lengths)
    # the projection holds other columns too
    proj = randn(g, 1, R, CH + 16).to(BF)
    pos = torch.cat([torch.arange(m) for m in lengths]).to(torch.int32)[None]
    return dict(proj=proj.cuda(), pos=pos.cuda(), g=(-0.3 * torch.rand(1, R, H, D, generator=g)).cuda(),
                beta=torch.rand(1, R, H, generator=g).cuda(), conv0=randn(g, n, W - 1, CH).to(BF).cuda(),
                h0=randn(g, n, H, D, D, scale=0.1).cuda(), dout=randn(g, 1, R, H, D).to(BF).cuda(),
                dhT=randn(g, n, H, D, D, scale=0.1).cuda(), cu=cu_of(lengths))


def head_tol(want, big):
    return H16 * want.abs() * (1 + 2.0 ** -8) + 2.0 ** -20 * big + 1e-37


def test_delta_layer_prompt_and_gradients(oracle_mod):
    lengths, L = [130, 0, 1, 67], Layer(1)
    R, i = sum(lengths), inputs(lengths, 2)
    x = i["proj"][..., 8:8 + CH]
    c, final = kda.kda_conv_fwd(x, L.w, L.b, True, i["cu"], i["conv0"], want_final_state=True)
    q, k, qn, kn, v = L.heads(c, i["pos"])
    args = (qn, kn, v, i["g"], i["beta"])
    out, hT = kda.kda_fwd(*args, cu_seqlens=i["cu"], initial_state=i["h0"], final_state_dtype=F32)
    g = kda.kda_bwd(*args, i["dout"], cu_seqlens=i["cu"], initial_state=i["h0"], dfinal_state=i["dhT"])
    gq = kda.kda_qk_bwd(q, k, g["dq"], g["dk"], "l2", L.qw, L.kw, positions=i["pos"], inv_freq=L.freq)
    dc = torch.cat([gq["dq"].flatten(2), gq["dk"].flatten(2), g["dv"].flatten(2).to(BF)], -1)
    dproj = torch.full_like(i["proj"], 3.0)
    gc = kda.kda_conv_bwd(x, L.w, dc, L.b, True, i["cu"], i["conv0"], want_dinitial_state=True, dx=dproj[..., 8:8 + CH])
    torch.cuda.synchronize()
    assert kda.device_error() == 0

    conv_check(x[0], L.w, L.b, lengths, i["conv0"], c[0], final)
    pos = i["pos"]
    for got, h, w in ((qn, q, L.qw), (kn, k, L.kw)):
        h, w = h[0].cpu().to(ref.F64), w.cpu().to(ref.F64)
        want = L.heads_reference(h, w, pos)
        assert ref.worst(got[0], want, head_tol(want, want.abs().amax(-1, keepdim=True) * 2 ** 0.5)) <= 1

    cu = i["cu"].cpu().numpy().astype(np.int64)
    cpu = [t[0].cpu().double() for t in args]
    eo, eh = oracle_mod.kda_oracle(*(t.float() for t in cpu), D ** -0.5, cu_seqlens=cu, h0=i["h0"].cpu().double())
    assert rel(out[0].float().cpu().numpy(), eo) <= OUT_TOL and rel(hT.cpu().numpy(), eh) <= STATE_TOL[F32]
    eg = oracle_mod.kda_oracle_bwd(*cpu, D ** -0.5, i["dout"][0].cpu().double(), cu_seqlens=cu,
                                   h0=i["h0"].cpu().double(), dhT=i["dhT"].cpu().double())
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert rel(g[n][0].cpu().numpy(), eg[n].reshape(g[n][0].shape)) <= BWD_TOL, n

    for n, h, w in (("q", q, L.qw), ("k", k, L.kw)):
        h, dy = h[0].cpu().to(ref.F64).requires_grad_(), g["d" + n][0].cpu().to(ref.F64)
        want, = torch.autograd.grad(L.heads_reference(h, w.cpu().to(ref.F64), pos), h, dy)
        r = (h.detach().square().sum(-1, keepdim=True) + 1e-6).rsqrt()
        big = r * dy.norm(dim=-1, keepdim=True) * float(w.abs().max())
        tol = H16 * want.abs() * (1 + 2.0 ** -8) + 2.0 ** -18 * big + 1e-37
        assert ref.worst(gq["d" + n][0], want, tol) <= 1

    leaves = [t.cpu().to(ref.F64).requires_grad_() for t in (x[0], L.w, L.b, i["conv0"])]
    loss = ref.conv_loss(*leaves[:3], True, lengths, leaves[3], dc[0].cpu().to(ref.F64), None)
    mag = [t.detach().abs().requires_grad_() for t in leaves]
    size = ref.conv_loss(*mag[:3], False, lengths, mag[3], dc[0].cpu().to(ref.F64).abs(), None)
    want, terms = torch.autograd.grad(loss, leaves), torch.autograd.grad(size, mag)
    pre = ref.conv(leaves[0].detach(), leaves[1].detach(), leaves[2].detach(), True, lengths, leaves[3].detach())["pre_abs"]
    slack = 1.1 * (2.0 ** -18 * (1 + float(pre.max())) + 2.0 ** -24 * (R + 64))
    for got, j, half in ((gc["dx"][0], 0, H16), (gc["dweight"], 1, 0), (gc["dbias"], 2, 0), (gc["dinitial_state"], 3, H16)):
        assert ref.worst(got, want[j], half * want[j].abs() + slack * terms[j] + 1e-37) <= 1
    rest = torch.ones_like(dproj, dtype=torch.bool)
    rest[0, :, 8:8 + CH] = False
    assert bool((dproj[rest] == 3).all())


def test_delta_layer_single_tokens_after_a_prompt(oracle_mod):
    """Prompts of one length, then three tokens each, in place and replayed from one graph."""
    B, T, more, L = 3, 70, 3, Layer(4)
    g = torch.Generator().manual_seed(5)
    proj = randn(g, B, T + more, CH + 16).to(BF).cuda()
    gate, beta = (-0.3 * torch.rand(B, T + more, H, D, generator=g)).cuda(), torch.rand(B, T + more, H, generator=g).cuda()
    pos = torch.arange(T + more).to(torch.int32).expand(B, -1).contiguous().cuda()
    x = proj[..., :CH]
    c, conv_state = kda.kda_conv_fwd(x[:, :T].contiguous(), L.w, L.b, want_final_state=True)
    _, _, qn, kn, v = L.heads(c, pos[:, :T].contiguous())
    cut = lambda t: t[:, :T].contiguous()  # noqa: E731
    out, S = kda.kda_fwd(qn, kn, v, cut(gate), cut(beta), final_state_dtype=F32)
    seen = [[qn, kn, v, out]]

    tok = dict(x=torch.empty(B, CH + 16, dtype=BF, device="cuda"), g=torch.empty(B, H, D, device="cuda"),
               beta=torch.empty(B, H, device="cuda"), pos=torch.empty(B, 1, dtype=torch.int32, device="cuda"))

    def step():
        c1, _ = kda.kda_conv_decode(tok["x"][:, :CH], L.w, conv_state, conv_state, bias=L.b)
        _, _, q1, k1, v1 = L.heads(c1[:, None], tok["pos"])
        o, _ = kda.kda_decode(q1[:, 0], k1[:, 0], v1[:, 0], tok["g"], tok["beta"], state_in=S, state_out=S)
        return q1, k1, v1, o[:, None]

    def load(t):
        tok["x"].copy_(proj[:, t]), tok["g"].copy_(gate[:, t]), tok["beta"].copy_(beta[:, t]), tok["pos"].copy_(pos[:, t:t + 1])

    load(T)
    seen.append([t.clone() for t in step()])                     # one by a call
    torch.cuda.synchronize()
    keep = [t.clone() for t in (conv_state, S)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    conv_state.copy_(keep[0]), S.copy_(keep[1])
    for t in range(T + 1, T + more):                             # the others by replays
        load(t)
        graph.replay()
        seen.append([r.clone() for r in res])
    torch.cuda.synchronize()
    assert kda.device_error() == 0
    q, k, v, o = (torch.cat(t, 1) for t in zip(*seen))
    eo, eh = oracle_mod.kda_oracle(*(t.cpu().float() for t in (q, k, v, gate)), beta.cpu(), D ** -0.5)
    assert rel(o.float().cpu().numpy(), eo) <= OUT_TOL and rel(S.cpu().numpy(), eh) <= STATE_TOL[F32]
    assert torch.equal(conv_state, x[:, T + more - (W - 1):])
    whole, _ = kda.kda_conv_fwd(x, L.w, L.b)
    vw = whole[..., 2 * H * D:].unflatten(-1, (H, D)).double().cpu()
    assert ref.worst(v, vw, 2 * H16 * vw.abs() + 1e-5) <= 1       # another order of the same five terms


# ---------------------------------------------------------------- the scan's layer

SH, SG, SP, SN = 4, 2, 64, 128
SC = SH * SP + 2 * SG * SN


class ScanLayer:
    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.w, self.b = randn(g, SC, W, scale=0.5).cuda(), randn(g, SC, scale=0.1).cuda()
        self.A, self.D = -(0.5 + 4 * torch.rand(SH, generator=g)).cuda(), (1 + randn(g, SH, scale=0.2)).cuda()
        self.bias = randn(g, SH, scale=0.3).cuda() - 2

    def parts(self, c):
        return (c[..., :SH * SP].unflatten(-1, (SH, SP)), c[..., SH * SP:SH * SP + SG * SN].unflatten(-1, (SG, SN)),
                c[..., SH * SP + SG * SN:].unflatten(-1, (SG, SN)))

    def dict(self, x, B, C, dt, h0, **kw):
        cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
        return dict(x=cpu(x), B=cpu(B), C=cpu(C), dt=cpu(dt), A=self.A.cpu(), D=self.D.cpu(), bias=self.bias.cpu(),
                    h0=cpu(h0), **{k: cpu(v) for k, v in kw.items()})


@pytest.mark.parametrize("lengths", [[130, 0, 1, 67], [300, 520]])
def test_scan_layer_prompt_and_gradients(lengths):
    """The scan reads the convolution's output where it lies, and its gradients go where the convolution's backward
    reads them: no copies."""
    L, R, n = ScanLayer(7), sum(lengths), len(lengths)
    g = torch.Generator().manual_seed(8)
    x = randn(g, 1, R, SC).to(BF).cuda()
    dt, conv0 = randn(g, 1, R, SH, scale=0.7).cuda(), randn(g, n, W - 1, SC).to(BF).cuda()
    h0, dhT = randn(g, n, SH, SN, SP, scale=0.3).cuda(), randn(g, n, SH, SN, SP, scale=0.3).cuda()
    dout, cu = randn(g, 1, R, SH, SP).to(BF).cuda(), cu_of(lengths)
    c, final = kda.kda_conv_fwd(x, L.w, L.b, True, cu, conv0, want_final_state=True)
    xs, B, C = L.parts(c)
    out, hT = kda.kda_scan_fwd(xs, dt, L.A, B, C, L.D, L.bias, True, cu, h0, final_state_dtype=F32)
    dc = torch.empty_like(c)
    dx, dB, dC = L.parts(dc)
    gs = kda.kda_scan_bwd(xs, dt, L.A, B, C, dout, L.D, L.bias, True, cu, h0, dhT, dx=dx, dB=dB, dC=dC)
    gc = kda.kda_conv_bwd(x, L.w, dc, L.b, True, cu, conv0, want_dinitial_state=True)
    torch.cuda.synchronize()
    assert kda.device_error() == 0
    conv_check(x[0], L.w, L.b, lengths, conv0, c[0], final)
    d = L.dict(xs[0], B[0], C[0], dt[0], h0, dout=dout[0], dhT=dhT)
    check_fwd(d, lengths, True, out, hT)
    check_bwd(d, lengths, True, gs)
    again = kda.kda_conv_bwd(x, L.w, dc.clone(), L.b, True, cu, conv0, want_dinitial_state=True)
    assert all(torch.equal(gc[k], again[k]) and bool(torch.isfinite(gc[k]).all()) for k in gc)


def test_scan_layer_single_tokens_after_a_prompt():
    B, T, more, L = 3, 300, 3, ScanLayer(9)
    g = torch.Generator().manual_seed(10)
    x, dt = randn(g, B, T + more, SC).to(BF).cuda(), randn(g, B, T + more, SH, scale=0.7).cuda()
    c, conv_state = kda.kda_conv_fwd(x[:, :T].contiguous(), L.w, L.b, want_final_state=True)
    xs, Bm, Cm = L.parts(c)
    out, S = kda.kda_scan_fwd(xs, dt[:, :T].contiguous(), L.A, Bm, Cm, L.D, L.bias, True, final_state_dtype=F32)
    seen, outs = [c], [out]
    for t in range(T, T + more):
        c1, _ = kda.kda_conv_decode(x[:, t], L.w, conv_state, conv_state, bias=L.b)
        xs, Bm, Cm = L.parts(c1)
        o, _ = kda.kda_scan_decode(xs, dt[:, t].contiguous(), L.A, Bm, Cm, S, S, D=L.D, dt_bias=L.bias, dt_softplus=True)
        seen.append(c1[:, None]), outs.append(o[:, None])
    torch.cuda.synchronize()
    assert kda.device_error() == 0
    xs, Bm, Cm = (t.flatten(0, 1) for t in L.parts(torch.cat(seen, 1)))
    d, lengths = L.dict(xs, Bm, Cm, dt.flatten(0, 1), None), [T + more] * B
    r, m = ref.scan(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["bias"], True, lengths, None), mags(d, True, lengths)
    f = fp32_ops([T]) + more * 2.0 ** -23 * (SN + 20)             # the prompt's roundings and the steps'
    tol = H16 * (1 + 2.0 ** -7) * (r["out"].abs() + m["out"]) + f * m["out"] + 1e-37
    assert ref.worst(torch.cat(outs, 1).flatten(0, 1), r["out"], tol) <= 1
    assert ref.worst(S, r["state"], f * m["state"]) <= 1
