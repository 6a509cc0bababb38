"""kda_qk_fwd and kda_qk_bwd, the per-head norm and rotation of q and k, against 64-bit references."""
import ctypes

import pytest
import torch

import kimi_delta_attention_27_b200 as kda
import mixer_ref as ref

OK, NULL_PTR, BAD_SHAPE, CUDA, ALIGN, TOO_LARGE = 0, 1, 2, 5, 7, 8
BAD_OPTION, WORKSPACE, OVERLAP, DTYPE = 14, 15, 16, 17
FAR = [(1 << 32) + (i << 32) for i in range(12)]   # aligned, never dereferenced
P = lambda a: None if a is None else ctypes.c_void_p(a)  # noqa: E731


@pytest.fixture(scope="module")
def lib():
    from kimi_delta_attention_27_b200 import build
    build.build()
    return kda.load_library()


def fwd(lib, q=FAR[0], qs=256, k=FAR[1], ks=128, rows=4, Hq=2, Hk=1, D=128, norm=1, eps=1e-6, qw=None, pos=FAR[2],
        freq=FAR[3], rot=64, factor=1.0, qo=FAR[4], qos=256, ko=FAR[5], kos=128):
    return lib.kda_qk_fwd(P(q), qs, P(k), ks, rows, Hq, Hk, D, norm, eps, P(qw), None, P(pos), P(freq), rot, 0, factor,
                          P(qo), qos, P(ko), kos, None)


def bwd(lib, q=FAR[0], k=FAR[1], dqo=FAR[6], dko=FAR[7], dt=1, dq=FAR[4], dk=FAR[5], qw=FAR[8], ws=FAR[9], size=1 << 20):
    return lib.kda_qk_bwd(P(q), 256, P(k), 128, 4, 2, 1, 128, 1, 0.0, None, None, P(FAR[2]), P(FAR[3]), 64, 0, 1.0,
                          P(dqo), 256, P(dko), 128, dt, P(dq), 256, P(dk), 128, P(qw), None, P(ws), size, None)


def test_qk_refusals(lib):
    assert fwd(lib, norm=3) == BAD_OPTION and fwd(lib, norm=-1) == BAD_OPTION
    assert fwd(lib, eps=-1e-6) == BAD_OPTION and fwd(lib, eps=float("nan")) == BAD_OPTION
    assert fwd(lib, factor=float("inf")) == BAD_OPTION
    for D in (32, 96, 512, 0):
        assert fwd(lib, D=D) == BAD_SHAPE
    assert fwd(lib, rot=144) == BAD_SHAPE and fwd(lib, rot=8) == BAD_SHAPE and fwd(lib, rot=-16) == BAD_SHAPE
    assert fwd(lib, Hq=0) == BAD_SHAPE and fwd(lib, Hk=-1) == BAD_SHAPE and fwd(lib, rows=-1) == BAD_SHAPE
    assert fwd(lib, q=None) == NULL_PTR and fwd(lib, k=None) == NULL_PTR and fwd(lib, qo=None) == NULL_PTR
    assert fwd(lib, pos=None) == NULL_PTR and fwd(lib, freq=None) == NULL_PTR
    assert fwd(lib, q=FAR[0] + 8) == ALIGN and fwd(lib, qs=260) == ALIGN and fwd(lib, qw=FAR[8] + 2) == ALIGN
    assert fwd(lib, qs=128) == BAD_SHAPE
    assert fwd(lib, rows=1 << 40) == TOO_LARGE
    assert fwd(lib, rows=0, q=None, k=None, qo=None, ko=None, pos=None, freq=None) == OK
    assert bwd(lib, dt=0) == DTYPE and bwd(lib, dqo=None) == NULL_PTR and bwd(lib, dk=None) == NULL_PTR
    need = lib.kda_qk_bwd_workspace(4, 2, 1, 128)
    assert need > 0 and bwd(lib, size=need - 1) == WORKSPACE and bwd(lib, ws=None) == NULL_PTR
    assert lib.kda_qk_bwd_workspace(4, 2, 1, 96) == 0 and lib.kda_qk_bwd_workspace(4, 0, 1, 128) == 0


def test_qk_overlaps(lib):
    assert fwd(lib, qo=FAR[0], qos=512) == OVERLAP          # the same buffer, other rows
    assert fwd(lib, qo=FAR[0] + 16) == OVERLAP
    assert fwd(lib, ko=FAR[0]) == OVERLAP and fwd(lib, ko=FAR[4]) == OVERLAP and fwd(lib, qo=FAR[2]) == OVERLAP
    assert bwd(lib, dq=FAR[6]) == OVERLAP and bwd(lib, ws=FAR[0]) == OVERLAP
    if not torch.cuda.is_available():
        assert fwd(lib, qo=FAR[0], ko=FAR[1]) == CUDA       # in place
        assert fwd(lib, qs=512, ks=512, k=FAR[0] + 512, qo=FAR[0], ko=FAR[0] + 512, qos=512, kos=512) == CUDA
        assert bwd(lib) == CUDA and bwd(lib, qw=None, ws=None) == CUDA
        assert fwd(lib, rot=0, pos=None, freq=None) == CUDA and fwd(lib, Hk=0, k=None, ko=None) == CUDA


def test_qk_binding_refusals():
    q = torch.zeros(1, 3, 2, 128, dtype=torch.bfloat16)
    pos, freq = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(32)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_qk_fwd(q, q)
    with pytest.raises(ValueError, match="norm"):
        kda.kda_qk_fwd(q, q, norm="layer")
    with pytest.raises(ValueError, match="come together"):
        kda.kda_qk_fwd(q, q, positions=pos)
    with pytest.raises(ValueError, match="positions"):
        kda.kda_qk_fwd(q, q, positions=pos.long(), inv_freq=freq)
    with pytest.raises(ValueError, match="q_weight"):
        kda.kda_qk_fwd(q, q, q_weight=torch.zeros(64))
    with pytest.raises(ValueError, match="q must be"):
        kda.kda_qk_fwd(q.float(), q)
    with pytest.raises(ValueError, match="k_weight"):
        kda.kda_qk_bwd(q, None, q, None, k_weight=torch.zeros(128))


# ---------------------------------------------------------------- GPU

CASES = [
    # T, Hq, Hk, D, rot, interleaved, norm, weights, eps, first position, factor
    (1, 1, 1, 128, 128, False, "rms", True, 1e-6, 0, 1.0),
    (37, 4, 2, 128, 64, True, "l2", False, 0.0, (1 << 20) - 3, 1.0),
    (5, 3, 1, 64, 16, False, "l2", True, 1e-6, 131072, 1.0),
    (200, 8, 8, 256, 256, True, "rms", True, 1e-5, 5, 1.25),
    (64, 7, 0, 128, 0, False, "l2", False, 1e-6, 0, 1.0),
    (130, 5, 3, 64, 64, False, "none", False, 0.0, -70, 0.7),
    (3, 40, 9, 256, 112, False, "none", True, 0.0, 2 ** 31 - 4, 1.0),
    (19, 32, 32, 128, 48, True, "rms", False, 0.0, 1000, 1.0),
]


def make(T, Hq, Hk, D, rot, first, weights, seed, B=2):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(q=rn(B, T, Hq, D).bfloat16(), k=rn(B, T, Hk, D).bfloat16() if Hk else None)
    d["q"][0, 0, 0] = 0                                # a head of zeros
    d["pos"] = (first + torch.arange(T)).clamp(max=2 ** 31 - 1).expand(B, T).to(torch.int32).contiguous() if rot else None
    d["freq"] = (1e4 ** (-torch.arange(rot // 2) / max(1, rot // 2))).float() if rot else None
    d["qw"] = 1 + 0.3 * rn(D) if weights else None
    d["kw"] = 1 + 0.3 * rn(D) if weights and Hk else None
    return d


def dev(t):
    return None if t is None else t.cuda()


def reference(x, w, d, norm, eps, inter, factor):
    B, T, H, D = x.shape
    pos = None if d["pos"] is None else d["pos"].reshape(-1)
    y = ref.qk(x.reshape(B * T, H, D), w, norm, eps, pos, d["freq"], inter, factor)
    return y.reshape(x.shape)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES)
def test_qk_fwd(lib, case):
    T, Hq, Hk, D, rot, inter, norm, weights, eps, first, factor = case
    d = make(T, Hq, Hk, D, rot, first, weights, seed=T)
    q, k = kda.kda_qk_fwd(dev(d["q"]), dev(d["k"]), norm, dev(d["qw"]), dev(d["kw"]), eps, dev(d["pos"]), dev(d["freq"]),
                          inter, factor)
    for got, x, w in ((q, d["q"], d["qw"]), (k, d["k"], d["kw"])):
        if x is None:
            assert got is None
            continue
        x64, w64 = x.to(ref.F64), None if w is None else w.to(ref.F64)
        want = reference(x64, w64, d, norm, eps, inter, factor)
        # the rounding of the result, and in fp32 the sum of D squares, the root, two products and the rotation: 2^-20
        # of the head's largest channel (the partner may be the larger of a pair)
        big = reference(x64, w64, dict(d, pos=None), norm, eps, inter, factor).abs().amax(-1, keepdim=True)
        tol = ref.half_step(torch.bfloat16) * want.abs() * (1 + 2.0 ** -8) + 2.0 ** -20 * big * max(1, factor) + 1e-37
        assert ref.worst(got, want, tol) <= 1


@pytest.mark.gpu
def test_qk_l2_is_the_forward_flags_norm(lib):
    """kda_qk_fwd's L2 norm and kda_fwd's own (KDA_FLAG_L2NORM_QK) feed the same recurrence."""
    from kimi_delta_attention_27_b200.inputs import make_inputs
    inp = make_inputs({"B": 1, "T": 200, "H": 2, "lengths": None, "g_mu": 3.0, "init": None, "final": "fp32", "seed": 5},
                      device="cuda")
    q, k = (3 * inp["q"].float()).bfloat16(), (0.5 * inp["k"].float()).bfloat16()
    a, sa = kda.kda_fwd(q, k, inp["v"], inp["g"], inp["beta"], l2norm_qk=True, final_state_dtype=torch.float32)
    qn, kn = kda.kda_qk_fwd(q, k, norm="l2", eps=0.0)
    b, sb = kda.kda_fwd(qn, kn, inp["v"], inp["g"], inp["beta"], final_state_dtype=torch.float32)
    # one bf16 rounding of q and k apart, and kda_fwd's own bars
    assert float((a.float() - b.float()).abs().max() / b.float().abs().max()) <= 2e-2
    assert float((sa - sb).abs().max() / sb.abs().max()) <= 1e-2


@pytest.mark.gpu
def test_qk_in_place_and_slices_of_one_projection(lib):
    d = make(33, 4, 2, 128, 64, 10, True, seed=3)
    args = ("rms", dev(d["qw"]), dev(d["kw"]), 1e-6, dev(d["pos"]), dev(d["freq"]))
    q, k = kda.kda_qk_fwd(dev(d["q"]), dev(d["k"]), *args)
    proj = torch.full((2, 33, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")   # q, k and something else side by side
    proj[:, :, :4], proj[:, :, 4:6] = dev(d["q"]), dev(d["k"])
    a, b = kda.kda_qk_fwd(proj[:, :, :4], proj[:, :, 4:6], *args, q_out=proj[:, :, :4], k_out=proj[:, :, 4:6])
    assert torch.equal(a, q) and torch.equal(b, k) and bool((proj[:, :, 6:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_qk_bwd(lib, case, fp32):
    T, Hq, Hk, D, rot, inter, norm, weights, eps, first, factor = case
    d = make(T, Hq, Hk, D, rot, first, weights, seed=T + 1)
    g = torch.Generator().manual_seed(T + 2)
    dy = {n: torch.randn(d[n].shape, generator=g) for n in ("q", "k") if d[n] is not None}
    dy = {n: v if fp32 else v.bfloat16() for n, v in dy.items()}
    got = kda.kda_qk_bwd(dev(d["q"]), dev(d["k"]), dev(dy["q"]), dev(dy.get("k")), norm, dev(d["qw"]), dev(d["kw"]), eps,
                         dev(d["pos"]), dev(d["freq"]), inter, factor)
    for n in dy:
        x = d[n].to(ref.F64).requires_grad_()
        w = None if d[n + "w"] is None else d[n + "w"].to(ref.F64).requires_grad_()
        y = reference(x, w, d, norm, eps, inter, factor)
        grads = torch.autograd.grad(y, [x] + ([w] if w is not None else []), dy[n].to(ref.F64))
        dx = grads[0]
        if norm != "none" and eps == 0 and n == "q":
            dx = dx.clone()
            dx[0, 0, 0] = 0                            # a vector of zeros stays zero, and passes nothing on
        # r |w dz| bounds every term of a head's dx; 2^-18 for some 30 fp32 operations and sums of 256
        x64 = d[n].to(ref.F64)
        ss = (x64 * x64).sum(-1, keepdim=True)
        r = 1 if norm == "none" else ((ss / D if norm == "rms" else ss) + eps).clamp(min=1e-30).rsqrt()
        big = r * (dy[n].to(ref.F64).norm(dim=-1, keepdim=True) * max(1, factor) *
                   (1 if w is None else float(w.detach().abs().max())))
        tol = ref.half_step(torch.bfloat16) * dx.abs() * (1 + 2.0 ** -8) + 2.0 ** -18 * big + 1e-37
        ok = torch.ones_like(dx, dtype=torch.bool)
        if norm != "none" and eps == 0 and n == "q":
            assert bool((got["dq"][0, 0, 0] == 0).all())
            ok[0, 0, 0] = False
        assert ref.worst(got["d" + n].cpu()[ok], dx[ok], tol[ok]) <= 1
        if w is None:
            assert got[f"d{n}_weight"] is None
        else:
            xh = (x64 * r).abs()
            rows = dy[n].to(ref.F64).norm(dim=-1, keepdim=True) * max(1, factor)
            mag = (xh * rows).sum((0, 1, 2))
            assert ref.worst(got[f"d{n}_weight"], grads[1], 2.0 ** -20 * mag + 1e-37) <= 1


@pytest.mark.gpu
def test_qk_bwd_takes_kda_bwds_gradients_and_repeats(lib):
    """The fp32 dq, dk of kda_bwd through the norm: against the differences of the whole chain's loss."""
    from kimi_delta_attention_27_b200.inputs import make_inputs
    inp = make_inputs({"B": 1, "T": 70, "H": 2, "lengths": None, "g_mu": 3.0, "init": None, "final": "fp32", "seed": 8},
                      device="cuda")
    q, k = torch.randn_like(inp["q"].float()).bfloat16(), torch.randn_like(inp["k"].float()).bfloat16()
    w = torch.rand(128, device="cuda") + 0.5
    qn, kn = kda.kda_qk_fwd(q, k, norm="l2", q_weight=w)
    dout = torch.randn_like(inp["v"].float()).bfloat16()
    g = kda.kda_bwd(qn, kn, inp["v"], inp["g"], inp["beta"], dout, want_dinitial_state=False)
    a = kda.kda_qk_bwd(q, k, g["dq"], g["dk"], norm="l2", q_weight=w)
    b = kda.kda_qk_bwd(q, k, g["dq"], g["dk"], norm="l2", q_weight=w)
    assert all(torch.equal(a[n], b[n]) for n in ("dq", "dk", "dq_weight")) and a["dk_weight"] is None

    def loss(step):
        qn, kn = kda.kda_qk_fwd(q, k, norm="l2", q_weight=w + step)
        out, _ = kda.kda_fwd(qn, kn, inp["v"], inp["g"], inp["beta"])
        return float((out.double() * dout.double()).sum()), float((out.double() * dout.double()).abs().sum())

    way = torch.randn(128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * 0.25
    (hi, mag), (lo, _) = loss(way), loss(-way)
    # out is linear in q, so the difference is exact but for roundings: kda_fwd's operands are bf16 (2^-8 each, of
    # terms that add up to `mag` at most; they average out over more than 10^4 of them)
    assert abs((hi - lo) / 2 - float((a["dq_weight"] * way).sum())) <= 2.0 ** -8 * mag


@pytest.mark.gpu
def test_qk_calls_at_once_and_captured(lib):
    """Both directions in flight on two streams, and replayed from a graph."""
    sets = []
    for s in (1, 2):
        d = make(400, 6, 2, 128, 64, 5 * s, True, seed=s)
        g = torch.Generator().manual_seed(s)
        d.update(dyq=torch.randn(d["q"].shape, generator=g), dyk=torch.randn(d["k"].shape, generator=g))
        sets.append({k: dev(v) for k, v in d.items()})

    def run(d):
        opt = ("rms", d["qw"], d["kw"], 1e-6, d["pos"], d["freq"])
        q, k = kda.kda_qk_fwd(d["q"], d["k"], *opt)
        return dict(kda.kda_qk_bwd(d["q"], d["k"], d["dyq"], d["dyk"], *opt), q=q, k=k)

    want = [run(d) for d in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for d, s in zip(sets, streams):
            with torch.cuda.stream(s):
                got.append(run(d))
        torch.cuda.synchronize()
        assert all(torch.equal(w[k], g[k]) for w, g in zip(want, got) for k in w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = run(sets[0])
    for k, v in sets[1].items():
        sets[0][k].copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(want[1][k], res[k]) for k in res) and kda.device_error() == 0
