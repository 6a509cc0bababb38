"""kda_scan_fwd, kda_scan_bwd, kda_scan_decode against the 64-bit recurrence, and their refusals."""
import ctypes

import pytest
import torch

import kimi_delta_attention_27_b200 as kda
import mixer_ref as ref

OK, NULL_PTR, BAD_SHAPE, VARLEN, STATE_DTYPE, CUDA, ALIGN, TOO_LARGE, STATE_OVERLAP = 0, 1, 2, 3, 4, 5, 7, 8, 11
BAD_OPTION, WORKSPACE, OVERLAP = 14, 15, 16
FAR = [(1 << 36) + (i << 36) for i in range(24)]   # aligned, never dereferenced
P = lambda a: None if a is None else ctypes.c_void_p(a)  # noqa: E731
H16 = ref.half_step(torch.bfloat16)


@pytest.fixture(scope="module")
def lib():
    from kimi_delta_attention_27_b200 import build
    build.build()
    return kda.load_library()


def fwd(lib, x=FAR[0], xs=256, dt=FAR[1], A=FAR[2], B=FAR[3], bs=128, C=FAR[4], cs=128, flags=1, cu=None, n=0, batch=2,
        T=100, H=4, G=1, hd=64, sd=128, h0=None, h0t=0, hT=None, hTt=0, out=FAR[5], os=256, ws=FAR[6], size=1 << 34):
    return lib.kda_scan_fwd(P(x), xs, P(dt), P(A), P(B), bs, P(C), cs, None, None, flags, P(cu), n, batch, T, H, G, hd,
                            sd, P(h0), h0t, P(hT), hTt, P(out), os, P(ws), size, None)


def bwd(lib, T=100, H=4, G=1, dout=FAR[7], dx=FAR[8], ddt=FAR[9], dA=FAR[10], dB=FAR[11], dC=FAR[12], ws=FAR[6],
        size=1 << 34, dcs=128, dh0=None):
    return lib.kda_scan_bwd(P(FAR[0]), 256, P(FAR[1]), P(FAR[2]), P(FAR[3]), 128, P(FAR[4]), 128, None, None, 1, None, 0,
                            2, T, H, G, 64, 128, None, 0, P(dout), 256, None, P(dx), 256, P(ddt), P(dA), P(dB), 128,
                            P(dC), dcs, None, None, P(dh0), P(ws), size, None)


def dec(lib, batch=3, H=4, G=1, hd=64, sd=128, sin=FAR[5], sout=FAR[6], st=2, out=FAR[7], flags=0):
    return lib.kda_scan_decode(P(FAR[0]), 256, P(FAR[1]), P(FAR[2]), P(FAR[3]), 128, P(FAR[4]), 128, None, None, flags,
                               batch, H, G, hd, sd, P(sin), P(sout), st, P(out), None)


def test_scan_refusals(lib):
    assert fwd(lib, flags=2) == BAD_OPTION and dec(lib, flags=4) == BAD_OPTION
    for hd, sd in ((32, 128), (64, 96), (256, 64), (64, 256)):
        assert fwd(lib, hd=hd, sd=sd) == BAD_SHAPE and dec(lib, hd=hd, sd=sd) == BAD_SHAPE
    assert fwd(lib, H=0) == BAD_SHAPE and fwd(lib, G=0) == BAD_SHAPE and fwd(lib, G=3) == BAD_SHAPE
    assert fwd(lib, T=-1) == BAD_SHAPE and fwd(lib, batch=-1) == BAD_SHAPE and dec(lib, batch=-1) == BAD_SHAPE
    assert fwd(lib, cu=FAR[13], n=1, batch=2) == VARLEN
    assert fwd(lib, h0=FAR[13], h0t=0) == STATE_DTYPE and fwd(lib, hT=FAR[13], hTt=3) == STATE_DTYPE
    assert fwd(lib, h0=FAR[13], h0t=1, hT=FAR[14], hTt=2) == STATE_DTYPE and dec(lib, st=0) == STATE_DTYPE
    for name in ("x", "dt", "A", "B", "C", "out"):
        assert fwd(lib, **{name: None}) == NULL_PTR
    for name in ("dout", "dx", "ddt", "dA", "dB", "dC", "ws"):
        assert bwd(lib, **{name: None}) == NULL_PTR
    assert fwd(lib, x=FAR[0] + 8) == ALIGN and fwd(lib, bs=132) == ALIGN and fwd(lib, dt=FAR[1] + 2) == ALIGN
    assert fwd(lib, xs=128) == BAD_SHAPE and bwd(lib, dcs=64) == BAD_SHAPE
    assert fwd(lib, T=1 << 40) == TOO_LARGE and fwd(lib, T=1 << 30, H=1 << 10, xs=1 << 16) == TOO_LARGE
    need = kda.scan_workspace_bytes(200000, 2, 4, 64, 128)
    assert need > 0 and fwd(lib, T=100000, size=need - 1) == WORKSPACE and fwd(lib, T=100000, ws=None) == NULL_PTR
    assert fwd(lib, T=100000, ws=FAR[6] + 16) == ALIGN
    assert kda.scan_workspace_bytes(200, 2, 4, 64, 128) == 0          # nothing is cut
    need = lib.kda_scan_bwd_workspace(200, 2, 4, 1, 64, 128)
    assert need > 0 and bwd(lib, size=need - 1) == WORKSPACE
    assert lib.kda_scan_bwd_workspace(200, 2, 4, 3, 64, 128) == 0 and lib.kda_scan_fwd_workspace(200, 2, 4, 96, 128) == 0
    assert fwd(lib, batch=0, x=None, dt=None, A=None, B=None, C=None, out=None, ws=None) == OK
    assert dec(lib, batch=0, sin=None, sout=None, out=None) == OK


def test_scan_overlaps(lib):
    state = 2 * 4 * 128 * 64 * 4
    assert fwd(lib, out=FAR[0]) == OVERLAP and fwd(lib, out=FAR[3] - 16) == OVERLAP
    assert fwd(lib, h0=FAR[13], h0t=2, hT=FAR[13] + 16, hTt=2) == STATE_OVERLAP
    assert fwd(lib, h0=FAR[13], h0t=2, out=FAR[13]) == OVERLAP
    assert bwd(lib, dB=FAR[3]) == OVERLAP and bwd(lib, dB=FAR[12]) == OVERLAP and bwd(lib, ws=FAR[0]) == OVERLAP
    assert bwd(lib, dh0=FAR[6]) == OVERLAP
    assert dec(lib, sout=FAR[5] + 64) == STATE_OVERLAP and dec(lib, out=FAR[5]) == OVERLAP
    if not torch.cuda.is_available():
        assert fwd(lib, h0=FAR[13], h0t=2, hT=FAR[13], hTt=2) == CUDA            # in place
        assert fwd(lib, h0=FAR[13], h0t=2, hT=FAR[13] + state, hTt=2) == CUDA    # right behind
        assert dec(lib, sout=FAR[5]) == CUDA and bwd(lib) == CUDA
        # x, B, C as columns of one projection, the output in other columns of it
        assert fwd(lib, x=FAR[0], B=FAR[0] + 512, C=FAR[0] + 768, out=FAR[0] + 1024, xs=768, bs=768, cs=768, os=768) == CUDA


def test_scan_binding_refusals():
    x, dt, A = torch.zeros(1, 5, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 5, 2), torch.zeros(2)
    B = torch.zeros(1, 5, 1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_scan_fwd(x, dt, A, B, B)
    with pytest.raises(ValueError, match="C must have shape"):
        kda.kda_scan_fwd(x, dt, A, B, B[:, :4])
    with pytest.raises(ValueError, match="dt must be"):
        kda.kda_scan_fwd(x, dt.bfloat16(), A, B, B)
    with pytest.raises(ValueError, match="A must have shape"):
        kda.kda_scan_fwd(x, dt, torch.zeros(3), B, B)
    with pytest.raises(ValueError, match="initial_state must have shape"):
        kda.kda_scan_fwd(x, dt, A, B, B, initial_state=torch.zeros(1, 2, 64, 128))
    with pytest.raises(ValueError, match="dfinal_state must be"):
        kda.kda_scan_bwd(x, dt, A, B, B, x, dfinal_state=torch.zeros(1, 2, 128, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="same dtype"):
        kda.kda_scan_decode(x[:, 0], dt[:, 0], A, B[:, 0], B[:, 0], torch.zeros(1, 2, 128, 64),
                            torch.zeros(1, 2, 128, 64, dtype=torch.bfloat16))


# ---------------------------------------------------------------- GPU

LENGTHS = {
    "one": [1], "tile": [64], "past_tile": [65], "ragged": [63, 0, 1, 130, 2, 0, 64, 37], "long": [520], "empty": [0, 0],
    "none_then_some": [0, 300],
}
SHAPES = [(2, 1, 64, 128), (4, 2, 128, 64), (3, 3, 64, 64), (6, 2, 128, 128)]   # H, G, P, N


def make(lengths, H, G, P, N, seed, state=torch.float32, sharp=False):
    g = torch.Generator().manual_seed(seed)
    R, n = sum(lengths), len(lengths)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    bf = torch.bfloat16
    d = dict(x=(0.7 * rn(R, H, P)).to(bf), B=(0.5 * rn(R, G, N)).to(bf), C=(0.5 * rn(R, G, N)).to(bf),
             dt=0.7 * rn(R, H) - (0 if sharp else 2), A=-(0.5 + 8 * torch.rand(H, generator=g)), D=1 + 0.2 * rn(H),
             bias=0.3 * rn(H), h0=None if state is None else (0.3 * rn(n, H, N, P)).to(state),
             dout=rn(R, H, P).to(bf), dhT=0.3 * rn(n, H, N, P))
    return d


def cu_of(lengths):
    return torch.tensor([0] + [b for _, b in ref.spans(lengths)], dtype=torch.int32, device="cuda")


def dev(t):
    return None if t is None else t.cuda()


def call_fwd(d, lengths, softplus=True, **kw):
    return kda.kda_scan_fwd(dev(d["x"])[None], dev(d["dt"])[None], dev(d["A"]), dev(d["B"])[None], dev(d["C"])[None],
                            dev(d["D"]), dev(d["bias"]), softplus, cu_of(lengths), dev(d["h0"]), **kw)


def call_bwd(d, lengths, softplus=True, **kw):
    return kda.kda_scan_bwd(dev(d["x"])[None], dev(d["dt"])[None], dev(d["A"]), dev(d["B"])[None], dev(d["C"])[None],
                            dev(d["dout"])[None], dev(d["D"]), dev(d["bias"]), softplus, cu_of(lengths), dev(d["h0"]),
                            dev(d["dhT"]), **kw)


def mags(d, softplus, lengths, grads=False):
    """The recurrence on absolute values (with the same decays): what the terms of each result add up to."""
    ab = lambda n: None if d[n] is None else d[n].double().abs()  # noqa: E731
    return ref.scan(ab("x"), d["dt"], d["A"], ab("B"), ab("C"), ab("D"), d["bias"], softplus, lengths, ab("h0"),
                    ab("dout") if grads else None, ab("dhT") if grads else None)


def fp32_ops(lengths):
    """Roundings of 2^-23 on the way of one value: per tile of 64 tokens a decay and twelve accumulations, and 100 for
    the gates (exponentials of 2^-22), the splits (2^-24) and sums within a tile."""
    return 2.0 ** -23 * (13 * (max(lengths, default=0) // 64 + 2) + 100)


def check_fwd(d, lengths, softplus, out, state):
    r, m = (ref.scan(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["bias"], softplus, lengths, d["h0"]),
            mags(d, softplus, lengths))
    f = fp32_ops(lengths)
    # y is rounded once; before that, one factor of each of its terms is (L . (C B^T) d, or the state's copy)
    tol = H16 * (1 + 2.0 ** -7) * (r["out"].abs() + m["out"]) + f * m["out"] + 1e-37
    assert ref.worst(out[0], r["out"], tol) <= 1
    tol = ref.half_step(state.dtype) * r["state"].abs() + (f + 2.0 ** -15 * (state.dtype != torch.float32)) * m["state"]
    assert ref.worst(state, r["state"], tol + 1e-37) <= 1


@pytest.mark.gpu
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16, None])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("name", list(LENGTHS))
def test_scan_fwd(lib, name, shape, state):
    lengths = LENGTHS[name]
    d = make(lengths, *shape, seed=len(name), state=state, sharp=name == "long")
    softplus = shape[0] != 3
    if not softplus:
        d["dt"] = d["dt"].abs() * 0.2
        d["bias"] = None
    out, hT = call_fwd(d, lengths, softplus, final_state_dtype=state or torch.float32)
    torch.cuda.synchronize()
    assert kda.device_error() == 0
    check_fwd(d, lengths, softplus, out, hT)


@pytest.mark.gpu
def test_scan_fwd_cut_into_pieces(lib):
    """Few heads and a long row: cut into pieces (the workspace is not empty), with ragged neighbours."""
    lengths = [3000, 1, 0, 1500, 64]
    assert kda.scan_workspace_bytes(sum(lengths), len(lengths), 2, 64, 64) > 0
    d = make(lengths, 2, 1, 64, 64, seed=3)
    out, hT = call_fwd(d, lengths, final_state_dtype=torch.float32)
    check_fwd(d, lengths, True, out, hT)
    # in place, and with a workspace of the caller's on another stream
    s = torch.cuda.Stream()
    h = dev(d["h0"]).clone()
    ws = torch.full((kda.scan_workspace_bytes(sum(lengths), len(lengths), 2, 64, 64),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    o2, h2 = kda.kda_scan_fwd(dev(d["x"])[None], dev(d["dt"])[None], dev(d["A"]), dev(d["B"])[None], dev(d["C"])[None],
                              dev(d["D"]), dev(d["bias"]), True, cu_of(lengths), h, final_state=h, workspace=ws,
                              stream=s.cuda_stream)
    s.synchronize()
    assert h2 is h and torch.equal(o2, out) and torch.equal(h, hT)


@pytest.mark.gpu
def test_scan_fixed_rows_and_split_calls(lib):
    """Rows of one batch equal packed ones; two calls that pass the state on equal one, to fp32 roundings."""
    H, G, Pd, N = 4, 2, 64, 128
    d = make([100, 100, 100], H, G, Pd, N, seed=6)
    a, sa = call_fwd(d, [100] * 3, final_state_dtype=torch.float32)
    v = lambda n, *s: dev(d[n]).view(3, 100, *s)  # noqa: E731
    args = lambda lo, hi: (v("x", H, Pd)[:, lo:hi].contiguous(), v("dt", H)[:, lo:hi].contiguous(), dev(d["A"]),  # noqa: E731
                           v("B", G, N)[:, lo:hi].contiguous(), v("C", G, N)[:, lo:hi].contiguous(), dev(d["D"]),
                           dev(d["bias"]), True)
    b, sb = kda.kda_scan_fwd(*args(0, 100), initial_state=dev(d["h0"]), final_state_dtype=torch.float32)
    assert ref.worst(b.view(1, 300, H, Pd), a.double().cpu(), 4 * H16 * mags(d, True, [100] * 3)["out"][None]) <= 1
    assert torch.allclose(sa, sb, rtol=1e-4, atol=1e-5)
    _, s1 = kda.kda_scan_fwd(*args(0, 64), initial_state=dev(d["h0"]), final_state_dtype=torch.float32)
    _, s2 = kda.kda_scan_fwd(*args(64, 100), initial_state=s1, final_state=s1)
    assert s2 is s1 and torch.allclose(s1, sb, rtol=1e-4, atol=1e-5)


@pytest.mark.gpu
def test_scan_slices_of_one_projection_and_padding(lib):
    """x, B, C as columns of one tensor (no copies), a packed batch that ends before its rows do; the rows behind hold
    NaN, are not read into anything and not written."""
    lengths, (H, G, Pd, N) = [70, 5, 129], SHAPES[0]
    d = make(lengths, H, G, Pd, N, seed=7)
    R, pad = sum(lengths), 50
    cols = H * Pd + 2 * G * N
    proj = torch.full((1, R + pad, cols), float("nan"), dtype=torch.bfloat16, device="cuda")
    proj[0, :R] = torch.cat([d["x"].flatten(1), d["B"].flatten(1), d["C"].flatten(1)], 1).cuda()
    dt = torch.full((1, R + pad, H), float("nan"), device="cuda")
    dt[0, :R] = dev(d["dt"])
    x = proj[..., :H * Pd].unflatten(-1, (H, Pd))
    B = proj[..., H * Pd:H * Pd + G * N].unflatten(-1, (G, N))
    C = proj[..., H * Pd + G * N:].unflatten(-1, (G, N))
    out = torch.full((1, R + pad, H, Pd), 7.0, dtype=torch.bfloat16, device="cuda")
    rest = (dev(d["D"]), dev(d["bias"]), True, cu_of(lengths), dev(d["h0"]))
    want, wT = call_fwd(d, lengths, final_state_dtype=torch.float32)
    _, hT = kda.kda_scan_fwd(x, dt, dev(d["A"]), B, C, *rest, out=out, final_state_dtype=torch.float32)
    assert torch.equal(out[:, :R], want) and torch.equal(hT, wT) and bool((out[:, R:] == 7).all())
    dproj = torch.full_like(proj, 7.0)
    dout = torch.full_like(out, float("nan"))
    dout[0, :R] = dev(d["dout"])
    g = kda.kda_scan_bwd(x, dt, dev(d["A"]), B, C, dout, *rest, dfinal_state=dev(d["dhT"]),
                         dx=dproj[..., :H * Pd].unflatten(-1, (H, Pd)),
                         dB=dproj[..., H * Pd:H * Pd + G * N].unflatten(-1, (G, N)),
                         dC=dproj[..., H * Pd + G * N:].unflatten(-1, (G, N)))
    w = call_bwd(d, lengths)
    assert bool((dproj[:, R:] == 7).all()) and torch.equal(g["ddt"][:, :R], w["ddt"])
    flat = torch.cat([w["dx"].flatten(2), w["dB"].flatten(2), w["dC"].flatten(2)], -1)
    # B's and C's gradients are shared out over CTAs by the number of rows: another order of an fp32 sum
    assert float((dproj[:, :R].float() - flat.float()).abs().max() / flat.float().abs().max()) <= 2 * H16
    for k in ("dA", "dD", "ddt_bias", "dh0"):
        assert torch.allclose(g[k], w[k], rtol=1e-5, atol=1e-5), k
    assert kda.device_error() == 0


def check_bwd(d, lengths, softplus, g):
    r = ref.scan(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["bias"], softplus, lengths, d["h0"], d["dout"], d["dhT"])
    m = mags(d, softplus, lengths, grads=True)
    f = fp32_ops(lengths)
    # bf16 results: their own rounding and one of a factor of each term
    for k in ("dx", "dB", "dC"):
        tol = H16 * (1 + 2.0 ** -7) * (r[k].abs() + m[k]) + f * m[k] + 1e-37
        assert ref.worst(g[k][0], r[k], tol) <= 1, k
    assert ref.worst(g["dh0"], r["dh0"], f * m["dh0"] + 1e-37) <= 1
    # the steps' gradients: dd + A dlog a; dlog a takes prefix and suffix sums over a tile, whose terms add up to the
    # tile's sum of d dd and of dlog a
    R, H = d["dt"].shape
    tile = torch.zeros(R, H, dtype=ref.F64)
    for a, b in ref.spans(lengths):
        for t0 in range(a // 64 * 64, b, 64):
            lo, hi = max(a, t0), min(b, t0 + 64)
            if hi > lo:
                tile[lo:hi] = (m["d"] * m["dd"])[lo:hi].sum(0) + m["dla"][lo:hi].amax(0)
    sig = 1 if not softplus else torch.sigmoid(d["dt"].double() + (d["bias"].double() if d["bias"] is not None else 0))
    tol = f * (m["dd"] + (m["dla"] + tile) * d["A"].double().abs()) * sig + 1e-37
    assert ref.worst(g["ddt"][0], r["ddt"], tol) <= 1
    if d["bias"] is not None:
        assert ref.worst(g["ddt_bias"], r["ddt_bias"], tol.sum(0)) <= 1
    assert ref.worst(g["dA"], r["dA"], f * (m["d"] * (m["dla"] + tile)).sum(0) + 1e-37) <= 1
    if d["D"] is not None:
        assert ref.worst(g["dD"], r["dD"], f * m["dD"] + 1e-37) <= 1


@pytest.mark.gpu
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16, None])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("name", list(LENGTHS))
def test_scan_bwd(lib, name, shape, state):
    lengths = LENGTHS[name]
    d = make(lengths, *shape, seed=len(name) + 50, state=state, sharp=name == "long")
    softplus = shape[0] != 3
    if not softplus:
        d["dt"] = d["dt"].abs() * 0.2
        d["bias"] = d["D"] = None
    g = call_bwd(d, lengths, softplus)
    torch.cuda.synchronize()
    assert kda.device_error() == 0
    check_bwd(d, lengths, softplus, g)


@pytest.mark.gpu
def test_scan_bwd_cut_into_pieces_and_repeats(lib):
    lengths = [1500, 1, 0, 700]
    assert kda.scan_workspace_bytes(sum(lengths), len(lengths), 2, 64, 64) > 0
    d = make(lengths, 2, 1, 64, 64, seed=13)
    g, h = call_bwd(d, lengths), call_bwd(d, lengths)
    check_bwd(d, lengths, True, g)
    assert all(torch.equal(g[k], h[k]) for k in g)


@pytest.mark.gpu
def test_scan_bwd_matches_differences(lib):
    """Directional derivatives of the forward's final state (fp32) by central differences in dt, A and the bias."""
    lengths, shape = [50, 3, 90], (2, 1, 64, 64)
    d = make(lengths, *shape, seed=31)
    d["dout"] = torch.zeros_like(d["dout"])
    g = call_bwd(d, lengths)
    gen = torch.Generator().manual_seed(32)
    way = {k: torch.randn(d[k].shape, generator=gen) for k in ("dt", "A", "bias")}

    def loss(s):
        e = dict(d, **{k: d[k] + s * v for k, v in way.items()})
        _, hT = call_fwd(e, lengths, final_state_dtype=torch.float32)
        return float((hT.cpu().double() * d["dhT"].double()).sum())

    h = 2e-3
    by_diff = (loss(h) - loss(-h)) / (2 * h)
    by_grad = sum(float((g[k].cpu().double().reshape(v.shape) * v.double()).sum())
                  for k, v in (("ddt", way["dt"]), ("dA", way["A"]), ("ddt_bias", way["bias"])))
    size = sum(float(g[k].double().norm()) for k in ("ddt", "dA", "ddt_bias"))
    assert abs(by_diff - by_grad) <= 2e-3 * (abs(by_grad) + size)


@pytest.mark.gpu
def test_scan_steps_that_forget_everything(lib):
    """Steps whose decay is 0 in any precision, in the middle of a tile: what is behind them starts afresh, with no
    loss of precision; and steps of zero, which change nothing."""
    lengths = [150]
    d = make(lengths, 2, 1, 64, 128, seed=17)
    d["bias"], d["D"] = None, None
    d["dt"] = d["dt"].abs() * 0.1
    d["dt"][70], d["dt"][100] = 1e30, 0
    d["x"][70] = 0                                   # d B x^T would be 10^30
    d["dt"][20, 0] = 500.0
    d["x"][20] *= 1e-3
    out, hT = call_fwd(d, lengths, False, final_state_dtype=torch.float32)
    check_fwd(d, lengths, False, out, hT)


@pytest.mark.gpu
def test_scan_infinities_stay_in_their_sequence(lib):
    lengths = [70, 64, 30]
    d = make(lengths, 2, 1, 64, 64, seed=18)
    want, wT = call_fwd(d, lengths, final_state_dtype=torch.float32)
    d["x"][75, 0, 3], d["B"][80, 0, 5], d["C"][90, 0, 1] = float("inf"), float("nan"), float("-inf")
    out, hT = call_fwd(d, lengths, final_state_dtype=torch.float32)
    for a, b, i in ((0, 70, 0), (134, 164, 2)):
        assert torch.equal(out[:, a:b], want[:, a:b]) and torch.equal(hT[i], wT[i])
    assert not bool(torch.isfinite(hT[1]).all())
    # head 1 has an infinity in B alone, from token 80 on
    assert torch.equal(out[:, 70:80, 1], want[:, 70:80, 1])


@pytest.mark.gpu
@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES)
def test_scan_decode(lib, shape, state):
    H, G, Pd, N = shape
    Bn = 5
    d = make([1] * Bn, H, G, Pd, N, seed=H, state=state)
    r, m = ref.scan(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["bias"], True, [1] * Bn, d["h0"]), mags(d, True, [1] * Bn)
    args = (dev(d["x"]), dev(d["dt"]), dev(d["A"]), dev(d["B"]), dev(d["C"]))
    kw = dict(D=dev(d["D"]), dt_bias=dev(d["bias"]), dt_softplus=True)
    S = dev(d["h0"])
    out, s1 = kda.kda_scan_decode(*args, S, state_dtype=state, **kw)
    S2 = S.clone()
    out2, s2 = kda.kda_scan_decode(*args, S2, S2, **kw)
    assert s2 is S2 and torch.equal(out, out2) and torch.equal(s1, s2) and torch.equal(S, dev(d["h0"]))
    f = 2.0 ** -23 * (N + 20)                        # a sum of N terms, the gates
    assert ref.worst(out, r["out"], H16 * r["out"].abs() * (1 + 2.0 ** -8) + f * m["out"]) <= 1
    assert ref.worst(s1, r["state"], ref.half_step(state) * r["state"].abs() + f * m["state"]) <= 1
    zero, _ = kda.kda_scan_decode(*args, torch.zeros_like(S), **kw)
    none, sn = kda.kda_scan_decode(*args, **kw)
    assert sn is None and torch.equal(zero, none)


@pytest.mark.gpu
def test_scan_decode_continues_a_prompt(lib):
    Bn, T, (H, G, Pd, N) = 3, 66, SHAPES[0]
    d = make([T + 3] * Bn, H, G, Pd, N, seed=41)
    v = lambda n, *s: dev(d[n]).view(Bn, T + 3, *s)  # noqa: E731
    x, dt, B, C = v("x", H, Pd), v("dt", H), v("B", G, N), v("C", G, N)
    kw = dict(D=dev(d["D"]), dt_bias=dev(d["bias"]), dt_softplus=True)
    S = kda.kda_scan_fwd(x[:, :T].contiguous(), dt[:, :T].contiguous(), dev(d["A"]), B[:, :T].contiguous(),
                         C[:, :T].contiguous(), initial_state=dev(d["h0"]), final_state_dtype=torch.float32, **kw)[1]
    r, m = ref.scan(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["bias"], True, [T + 3] * Bn, d["h0"]), mags(d, True, [T + 3] * Bn)
    for t in range(T, T + 3):
        o, _ = kda.kda_scan_decode(x[:, t], dt[:, t].contiguous(), dev(d["A"]), B[:, t], C[:, t], S, S, **kw)
        want, mag = r["out"].view(Bn, T + 3, H, Pd)[:, t], m["out"].view(Bn, T + 3, H, Pd)[:, t]
        assert ref.worst(o, want, H16 * 1.01 * want.abs() + (fp32_ops([T]) + 2.0 ** -23 * (N + 20)) * mag) <= 1
    assert ref.worst(S, r["state"], (fp32_ops([T]) + 2.0 ** -18) * m["state"]) <= 1


@pytest.mark.gpu
def test_scan_bad_offsets_are_reported(lib):
    d = make([100, 120], 2, 1, 64, 64, seed=3)
    args = (dev(d["x"])[None], dev(d["dt"])[None], dev(d["A"]), dev(d["B"])[None], dev(d["C"])[None])
    for bad in ([0, 230, 220], [0, 100, 221], [1, 100, 220], [0, -7, 220]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        kda.kda_scan_fwd(*args, cu_seqlens=cu, final_state_dtype=torch.float32)
        assert kda.device_error() == 12
        kda.kda_scan_bwd(*args, dev(d["dout"])[None], cu_seqlens=cu)
        assert kda.device_error() == 12
    assert kda.device_error() == 0


@pytest.mark.gpu
def test_scan_graph_replays_with_new_inputs(lib):
    """A captured forward and backward, replayed on new inputs, against eager calls; two graphs with their own
    workspaces, replayed one after the other on different streams."""
    lengths, shape = [900, 40], (2, 1, 64, 64)
    ds = [make(lengths, *shape, seed=60 + i) for i in range(2)]
    bufs = [{k: dev(v).clone() for k, v in ds[0].items()} for _ in range(2)]
    cu = cu_of(lengths)

    def step(b):
        out, hT = kda.kda_scan_fwd(b["x"][None], b["dt"][None], b["A"], b["B"][None], b["C"][None], b["D"], b["bias"], True,
                                   cu, b["h0"], final_state_dtype=torch.float32)
        g = kda.kda_scan_bwd(b["x"][None], b["dt"][None], b["A"], b["B"][None], b["C"][None], b["dout"][None], b["D"],
                             b["bias"], True, cu, b["h0"], b["dhT"])
        return [out, hT] + [g[k] for k in sorted(g)]

    eager = []
    for d in ds:
        eager.append([t.clone() for t in step({k: dev(v) for k, v in d.items()})])
    graphs, outs = [], []
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(b))
        graphs.append(g)
    for b, d in zip(bufs, ds):
        for k, v in d.items():
            b[k].copy_(dev(v))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, want in zip(outs, eager):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert kda.device_error() == 0
