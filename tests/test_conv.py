"""kda_conv_fwd, kda_conv_bwd, kda_conv_decode against 64-bit references, and their refusals."""
import ctypes

import pytest
import torch

import kimi_delta_attention_27_b200 as kda
import mixer_ref as ref

OK, NULL_PTR, BAD_SHAPE, VARLEN, CUDA, ALIGN, TOO_LARGE, STATE_OVERLAP = 0, 1, 2, 3, 5, 7, 8, 11
BAD_OPTION, WORKSPACE, OVERLAP, DTYPE = 14, 15, 16, 17
BF16, FP32 = 1, 2
FAKE = 1 << 32                     # aligned, never dereferenced
FAR = [FAKE + (i << 32) for i in range(12)]
P = lambda a: None if a is None else ctypes.c_void_p(a)  # noqa: E731


@pytest.fixture(scope="module")
def lib():
    from kimi_delta_attention_27_b200 import build
    build.build()
    return kda.load_library()


def fwd(lib, x=FAR[0], dtype=BF16, xs=64, w=FAR[1], bias=None, flags=1, cu=None, n=0, batch=2, T=10, C=64, W=4,
        init=None, final=None, out=FAR[2], os=64):
    return lib.kda_conv_fwd(P(x), dtype, xs, P(w), P(bias), flags, P(cu), n, batch, T, C, W, P(init), P(final), P(out),
                            os, None)


def bwd(lib, x=FAR[0], dtype=BF16, xs=64, w=FAR[1], T=10, C=64, W=4, dout=FAR[3], ddt=BF16, dx=FAR[4], dw=FAR[5],
        ws=FAR[6], size=1 << 20, init=None, dinit=None):
    return lib.kda_conv_bwd(P(x), dtype, xs, P(w), None, 1, None, 0, 1, T, C, W, P(init), P(dout), ddt, 64, None, P(dx),
                            64, P(dw), None, P(dinit), P(ws), size, None)


def dec(lib, x=FAR[0], xs=64, C=64, W=4, batch=3, sin=FAR[1], sout=FAR[2], out=FAR[3]):
    return lib.kda_conv_decode(P(x), BF16, xs, P(FAR[4]), None, 1, batch, C, W, P(sin), P(sout), P(out), 64, None)


def no_device(status):
    """A call that validation lets through: it stops at the device query (or is not checked where there is one)."""
    assert status == CUDA


def test_conv_fwd_refusals(lib):
    assert fwd(lib, flags=2) == BAD_OPTION
    assert fwd(lib, C=60) == BAD_SHAPE and fwd(lib, C=0) == BAD_SHAPE
    assert fwd(lib, W=1) == BAD_SHAPE and fwd(lib, W=5) == BAD_SHAPE
    assert fwd(lib, T=-1) == BAD_SHAPE and fwd(lib, batch=-1) == BAD_SHAPE
    assert fwd(lib, dtype=0) == DTYPE and fwd(lib, dtype=3) == DTYPE
    assert fwd(lib, cu=FAR[7], n=2, batch=2) == VARLEN
    assert fwd(lib, x=None) == NULL_PTR and fwd(lib, w=None) == NULL_PTR and fwd(lib, out=None) == NULL_PTR
    assert fwd(lib, x=FAR[0] + 8) == ALIGN and fwd(lib, bias=FAR[7] + 2) == ALIGN and fwd(lib, init=FAR[7] + 4) == ALIGN
    assert fwd(lib, xs=68) == ALIGN            # rows of 136 bytes: not on 16
    assert fwd(lib, xs=56) == BAD_SHAPE and fwd(lib, os=0) == BAD_SHAPE
    assert fwd(lib, T=1 << 40) == TOO_LARGE
    assert kda.status_string(OVERLAP).startswith("KDA_ERR_OVERLAP")
    assert kda.status_string(DTYPE).startswith("KDA_ERR_DTYPE")


def test_conv_overlaps(lib):
    assert fwd(lib, out=FAR[0]) == OVERLAP                      # in place: neighbours' rows are still needed
    assert fwd(lib, out=FAR[0] + 128 * 19) == OVERLAP           # the last row only
    assert fwd(lib, init=FAR[3], final=FAR[3]) == OVERLAP
    assert fwd(lib, out=FAR[3], final=FAR[3] + 128 * 5) == OVERLAP
    assert fwd(lib, out=FAR[0] + 64, xs=128, os=128) == OVERLAP     # interleaved columns that meet
    assert bwd(lib, dx=FAR[3]) == OVERLAP and bwd(lib, ws=FAR[0]) == OVERLAP
    assert dec(lib, sout=FAR[1] + 16) == STATE_OVERLAP
    assert dec(lib, out=FAR[1] + 128) == OVERLAP and dec(lib, out=FAR[2]) == OVERLAP
    if not torch.cuda.is_available():
        no_device(fwd(lib, out=FAR[0] + 128, xs=128, os=128))       # columns 64.. of the same rows
        no_device(fwd(lib, out=FAR[0] - 128, xs=128, os=128))
        no_device(fwd(lib, out=FAR[0] + 128 * 20))                  # right behind
        no_device(dec(lib, sout=FAR[1]))                            # states in place
        no_device(fwd(lib))
        no_device(bwd(lib))


def test_conv_bwd_and_decode_refusals(lib):
    assert bwd(lib, ddt=0) == DTYPE and bwd(lib, dtype=FP32, ddt=BF16) == DTYPE
    assert bwd(lib, dout=None) == NULL_PTR and bwd(lib, dx=None) == NULL_PTR and bwd(lib, ws=None) == NULL_PTR
    need = lib.kda_conv_bwd_workspace(10, 64, 4)
    assert need > 0 and bwd(lib, size=need - 1) == WORKSPACE
    assert bwd(lib, ws=FAR[6] + 128) == ALIGN
    assert lib.kda_conv_bwd_workspace(-1, 64, 4) == 0 and lib.kda_conv_bwd_workspace(10, 63, 4) == 0
    assert lib.kda_conv_bwd_workspace(10, 64, 5) == 0
    assert dec(lib, batch=-1) == BAD_SHAPE and dec(lib, xs=32) == BAD_SHAPE and dec(lib, x=None) == NULL_PTR
    assert dec(lib, batch=0, x=None, sin=None, sout=None, out=None) == OK
    assert fwd(lib, batch=0, x=None, w=None, out=None) == OK


def test_conv_binding_refusals():
    x, w = torch.zeros(1, 5, 16, dtype=torch.bfloat16), torch.zeros(16, 4)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_conv_fwd(x, w)
    with pytest.raises(ValueError, match="weight"):
        kda.kda_conv_fwd(x, torch.zeros(15, 4))
    with pytest.raises(ValueError, match="initial_state"):
        kda.kda_conv_fwd(x, w, initial_state=torch.zeros(1, 2, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="initial_state"):
        kda.kda_conv_fwd(x, w, initial_state=torch.zeros(1, 3, 16))
    with pytest.raises(ValueError, match="contiguous within a row"):
        kda.kda_conv_fwd(torch.zeros(1, 5, 32, dtype=torch.bfloat16)[..., ::2], w)
    with pytest.raises(ValueError, match="evenly spaced"):
        kda.kda_conv_fwd(torch.zeros(2, 6, 16, dtype=torch.bfloat16)[:, :5], w)
    with pytest.raises(ValueError, match="overlap"):
        kda.kda_conv_fwd(torch.zeros(1, 1, 16, dtype=torch.bfloat16).expand(1, 5, 16), w)
    with pytest.raises(ValueError, match="cu_seqlens"):
        kda.kda_conv_fwd(x, w, cu_seqlens=torch.zeros(0, dtype=torch.int32))
    with pytest.raises(ValueError, match="dout"):
        kda.kda_conv_bwd(x.float(), w, x)


# ---------------------------------------------------------------- GPU

LENGTHS = {
    "one": [1], "short": [2], "state_long": [3], "ragged": [5, 0, 1, 2, 70, 3, 0, 129], "long": [700], "empty": [0, 0],
}


def make(lengths, C, W, dtype, seed, bias=True, init=True):
    g = torch.Generator().manual_seed(seed)
    R, N = sum(lengths), len(lengths)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=rn(R, C).to(dtype), w=rn(C, W), b=rn(C) if bias else None,
                init=rn(N, W - 1, C).to(dtype) if init else None, dout=rn(R, C).to(dtype),
                dfinal=rn(N, W - 1, C).to(dtype))


def cu_of(lengths):
    return torch.tensor([0] + [b for _, b in ref.spans(lengths)], dtype=torch.int32, device="cuda")


def dev(t):
    return None if t is None else t.cuda()


def out_tol(r, dtype, silu):
    """One rounding of the result; in fp32, W + 1 roundings of pre, and a sigmoid whose exponential and
    division are good to 2^-21 and whose argument adds |pre| 2^-23; SiLU's slope is below 1.1."""
    fp = 8 * 2.0 ** -24 * r["pre_abs"] * 1.1
    if silu:
        fp = fp + r["out"].abs() * (2.0 ** -20 + r["pre"].abs() * 2.0 ** -22)
    return ref.half_step(dtype) * (r["out"].abs() + fp) + fp + 1e-37


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("name", list(LENGTHS))
def test_conv_fwd(lib, name, W, dtype):
    lengths, silu, C = LENGTHS[name], W != 3, 8 * (33 if name == "ragged" else 5)
    d = make(lengths, C, W, dtype, seed=W, bias=W != 2, init=name != "long")
    r = ref.conv(d["x"], d["w"], d["b"], silu, lengths, d["init"])
    out, final = kda.kda_conv_fwd(dev(d["x"])[None], dev(d["w"]), dev(d["b"]), silu, cu_of(lengths), dev(d["init"]),
                                  want_final_state=True)
    torch.cuda.synchronize()
    assert kda.device_error() == 0
    assert ref.worst(out[0], r["out"], out_tol(r, dtype, silu)) <= 1
    assert torch.equal(final.cpu().to(ref.F64), r["final"])


@pytest.mark.gpu
def test_conv_fixed_rows_equal_packed_ones(lib):
    d = make([50, 50, 50], 264, 4, torch.bfloat16, seed=5)
    a, fa = kda.kda_conv_fwd(dev(d["x"])[None], dev(d["w"]), dev(d["b"]), True, cu_of([50] * 3), dev(d["init"]),
                             want_final_state=True)
    b, fb = kda.kda_conv_fwd(dev(d["x"]).view(3, 50, 264), dev(d["w"]), dev(d["b"]), True, None, dev(d["init"]),
                             want_final_state=True)
    assert torch.equal(a.view(-1), b.view(-1)) and torch.equal(fa, fb)


@pytest.mark.gpu
def test_conv_strided_rows_and_padding(lib):
    """x and out as column slices of wider tensors; a packed batch that ends before its rows do: those behind keep
    what they held, and whatever x holds there is not read into anything."""
    lengths, C = [40, 7, 90], 72
    d = make(lengths, C, 4, torch.bfloat16, seed=6)
    R = sum(lengths)
    wide = torch.full((1, R + 30, 3 * C + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[0, :R, C:2 * C] = dev(d["x"])
    outw = torch.full((1, R + 30, 2 * C), 7.0, dtype=torch.bfloat16, device="cuda")
    x, out = wide[..., C:2 * C], outw[..., C:]
    _, final = kda.kda_conv_fwd(x, dev(d["w"]), dev(d["b"]), True, cu_of(lengths), dev(d["init"]), out=out,
                                want_final_state=True)
    want, wf = kda.kda_conv_fwd(dev(d["x"])[None], dev(d["w"]), dev(d["b"]), True, cu_of(lengths), dev(d["init"]),
                                want_final_state=True)
    assert torch.equal(out[:, :R], want) and torch.equal(final, wf)
    assert bool((out[:, R:] == 7).all()) and bool((outw[..., :C] == 7).all())
    dw = torch.full_like(wide, float("nan"))
    dw[0, :R, C:2 * C] = dev(d["dout"])
    dxw = torch.full_like(outw, 7.0)
    g = kda.kda_conv_bwd(x, dev(d["w"]), dw[..., C:2 * C], dev(d["b"]), True, cu_of(lengths), dev(d["init"]),
                         dev(d["dfinal"]), True, dx=dxw[..., C:])
    h = kda.kda_conv_bwd(dev(d["x"])[None], dev(d["w"]), dev(d["dout"])[None], dev(d["b"]), True, cu_of(lengths),
                         dev(d["init"]), dev(d["dfinal"]), True)
    assert torch.equal(g["dx"][:, :R], h["dx"]) and bool((dxw[:, R:] == 7).all()) and bool((dxw[..., :C] == 7).all())
    assert torch.equal(g["dinitial_state"], h["dinitial_state"])
    assert torch.allclose(g["dweight"], h["dweight"], rtol=1e-4, atol=1e-4) and bool(torch.isfinite(g["dweight"]).all())
    assert kda.device_error() == 0


def conv_grads(d, silu, lengths):
    leaves = {k: d[k].to(ref.F64).requires_grad_() for k in ("x", "w", "b", "init") if d[k] is not None}
    loss = ref.conv_loss(leaves["x"], leaves["w"], leaves.get("b"), silu, lengths, leaves.get("init"),
                         d["dout"].to(ref.F64), d["dfinal"].to(ref.F64))
    got = torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)
    return {k: torch.zeros_like(v) if g is None else g for (k, v), g in zip(leaves.items(), got)}


def grad_mags(d, silu, lengths):
    """What the terms of each gradient add up to in absolute value (|act'| <= 1.1)."""
    ab = {k: (v.to(ref.F64).abs() if v is not None else None) for k, v in d.items()}
    return {k: 1.1 * v for k, v in conv_grads(ab, False, lengths).items()}


def pre_slack(d, lengths):
    """Relative error of dpre: the sigmoid's 2^-20 and |pre| 2^-22 of its argument, twice, and the rounding of pre."""
    r = ref.conv(d["x"], d["w"], d["b"], True, lengths, d["init"])
    return float(2.0 ** -18 * (1 + r["pre_abs"].max())) if r["pre_abs"].numel() else 2.0 ** -18


@pytest.mark.gpu
@pytest.mark.parametrize("types", ["bf16", "bf16_fp32", "fp32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("name", list(LENGTHS))
def test_conv_bwd(lib, name, W, types):
    lengths, silu, C = LENGTHS[name], W != 2, 8 * (33 if name == "ragged" else 5)
    dtype = torch.float32 if types == "fp32" else torch.bfloat16
    d = make(lengths, C, W, dtype, seed=W + 10, bias=W != 3, init=name != "long")
    if types == "bf16_fp32":
        d["dout"] = d["dout"].float() * 1.001
    want, mag = conv_grads(d, silu, lengths), grad_mags(d, silu, lengths)
    g = kda.kda_conv_bwd(dev(d["x"])[None], dev(d["w"]), dev(d["dout"])[None], dev(d["b"]), silu, cu_of(lengths),
                         dev(d["init"]), dev(d["dfinal"]), d["init"] is not None)
    torch.cuda.synchronize()
    assert kda.device_error() == 0
    slack = pre_slack(d, lengths)
    tol = lambda k, hs: hs * want[k].abs() + slack * mag[k] + 1e-37  # noqa: E731
    # sums over R tokens in fp32, at most R / 8 of them one behind the other
    sums = 2.0 ** -24 * (sum(lengths) + 64)
    assert ref.worst(g["dx"][0], want["x"], tol("x", ref.half_step(dtype))) <= 1
    assert ref.worst(g["dweight"], want["w"], tol("w", 0) + sums * mag["w"]) <= 1
    if d["b"] is not None:
        assert ref.worst(g["dbias"], want["b"], tol("b", 0) + sums * mag["b"]) <= 1
    if d["init"] is not None:
        assert ref.worst(g["dinitial_state"], want["init"], tol("init", ref.half_step(dtype))) <= 1


@pytest.mark.gpu
def test_conv_bwd_matches_differences(lib):
    """fp32: the directional derivative of the forward by central differences."""
    lengths, C, W = [9, 2, 30], 16, 4
    d = make(lengths, C, W, torch.float32, seed=21)
    g = kda.kda_conv_bwd(dev(d["x"])[None], dev(d["w"]), dev(d["dout"])[None], dev(d["b"]), True, cu_of(lengths),
                         dev(d["init"]), dev(d["dfinal"]), True)
    gen = torch.Generator().manual_seed(22)
    way = {k: torch.randn(d[k].shape, generator=gen) for k in ("x", "w", "b", "init")}

    def loss(s):
        out, final = kda.kda_conv_fwd(dev(d["x"] + s * way["x"])[None], dev(d["w"] + s * way["w"]),
                                      dev(d["b"] + s * way["b"]), True, cu_of(lengths), dev(d["init"] + s * way["init"]),
                                      want_final_state=True)
        return float((out[0].cpu().double() * d["dout"].double()).sum() + (final.cpu().double() * d["dfinal"].double()).sum())

    h = 1e-2
    by_diff = (loss(h) - loss(-h)) / (2 * h)
    by_grad = sum(float((g[k].cpu().double().reshape(v.shape) * v.double()).sum())
                  for k, v in (("dx", way["x"]), ("dweight", way["w"]), ("dbias", way["b"]), ("dinitial_state", way["init"])))
    # third derivatives: h^2 / 6 of the loss's scale (about 600 terms of size 1 to 10)
    assert abs(by_diff - by_grad) <= 1e-2 * (abs(by_grad) + 60)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_decode_continues_a_prompt(lib, W, dtype):
    """A prompt, then single tokens in place, give what one call over all tokens gives, bit for bit."""
    B, T, C = 3, 11, 40
    g = torch.Generator().manual_seed(W)
    x = torch.randn(B, T + 4, C, generator=g).to(dtype).cuda()
    w, b = torch.randn(C, W, generator=g).cuda(), torch.randn(C, generator=g).cuda()
    whole, final = kda.kda_conv_fwd(x, w, b, want_final_state=True)
    out, state = kda.kda_conv_fwd(x[:, :T].contiguous(), w, b, want_final_state=True)
    assert torch.equal(out, whole[:, :T])
    for t in range(T, T + 4):
        y, s2 = kda.kda_conv_decode(x[:, t], w, state, state, bias=b)
        assert s2 is state
        tol = ref.half_step(dtype) * 2 * whole[:, t].double().abs().cpu() + 1e-5
        assert ref.worst(y, whole[:, t].double().cpu(), tol) <= 1   # another order of the same W + 1 terms
    assert torch.equal(state, final)
    y0, s0 = kda.kda_conv_decode(x[:, 0], w, None, torch.empty_like(state), bias=b)
    assert torch.equal(s0[:, -1], x[:, 0]) and bool((s0[:, :-1] == 0).all())
    assert ref.worst(y0, whole[:, 0].double().cpu(), ref.half_step(dtype) * 2 * whole[:, 0].double().abs().cpu() + 1e-5) <= 1


@pytest.mark.gpu
def test_conv_bad_offsets_are_reported(lib):
    d = make([20, 30], 64, 4, torch.bfloat16, seed=3)
    x, w = dev(d["x"])[None], dev(d["w"])
    for bad in ([0, 60, 50], [0, 30, 51], [1, 20, 50], [-5, 20, 50]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        kda.kda_conv_fwd(x, w, cu_seqlens=cu, want_final_state=True)
        assert kda.device_error() == 12
        kda.kda_conv_bwd(x, w, dev(d["dout"])[None], cu_seqlens=cu)
        assert kda.device_error() == 12
    assert kda.device_error() == 0


@pytest.mark.gpu
def test_conv_many_sequences(lib):
    """More sequences than one probe of the search covers, many of them empty."""
    g = torch.Generator().manual_seed(9)
    lengths = [int(v) for v in torch.randint(0, 4, (1500,), generator=g)]
    d = make(lengths, 16, 4, torch.bfloat16, seed=4)
    r = ref.conv(d["x"], d["w"], d["b"], True, lengths, d["init"])
    out, final = kda.kda_conv_fwd(dev(d["x"])[None], dev(d["w"]), dev(d["b"]), True, cu_of(lengths), dev(d["init"]),
                                  want_final_state=True)
    assert ref.worst(out[0], r["out"], out_tol(r, torch.bfloat16, True)) <= 1
    assert torch.equal(final.cpu().to(ref.F64), r["final"])
    assert kda.device_error() == 0


@pytest.mark.gpu
def test_conv_bwd_repeats(lib):
    d = make([3000, 1, 2500], 256, 4, torch.bfloat16, seed=8)
    a, b = (kda.kda_conv_bwd(dev(d["x"])[None], dev(d["w"]), dev(d["dout"])[None], dev(d["b"]), cu_seqlens=cu_of([3000, 1, 2500]))
            for _ in range(2))
    assert all(torch.equal(a[k], b[k]) for k in ("dx", "dweight", "dbias"))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("batch,C", [(1, 8), (3, 8), (2, 304128), (1187, 1024), (1186, 1032)])
def test_conv_decode_batches(lib, batch, C, dtype):
    """Small batches, and ones large enough for four requests per thread, whole and with a rest; rows of x and out
    strided."""
    g = torch.Generator().manual_seed(batch)
    W = 4
    x = torch.randn(batch, C + 8, generator=g).to(dtype).cuda()[:, :C]
    w, b = torch.randn(C, W, generator=g).cuda(), torch.randn(C, generator=g).cuda()
    state = torch.randn(batch, W - 1, C, generator=g).to(dtype).cuda()
    out = torch.full((batch + 1, C + 16), 7.0, dtype=dtype, device="cuda")
    new = torch.empty_like(state)
    kda.kda_conv_decode(x, w, state, new, bias=b, out=out[:batch, 8:8 + C])
    e = torch.cat([state, x[:, None]], 1).double()
    pre = (e * w.t().double()).sum(1) + b.double()
    mag = (e.abs() * w.t().double().abs()).sum(1) + b.double().abs()
    r = dict(out=(pre * pre.sigmoid()).cpu(), pre=pre.cpu(), pre_abs=mag.cpu())
    assert ref.worst(out[:batch, 8:8 + C], r["out"], out_tol(r, dtype, True)) <= 1
    assert torch.equal(new, e[:, 1:].to(dtype))
    assert bool((out[batch] == 7).all()) and bool((out[:, :8] == 7).all()) and bool((out[:, 8 + C:] == 7).all())
    inplace = state.clone()
    kda.kda_conv_decode(x, w, inplace, inplace, bias=b)
    assert torch.equal(inplace, new) and kda.device_error() == 0


@pytest.mark.gpu
def test_conv_calls_at_once_and_captured(lib):
    """Gradients (which need scratch memory) in flight on two streams, and replayed from a graph."""
    lengths = [900, 3, 410]
    sets = [{k: dev(v) for k, v in make(lengths, 512, 4, torch.bfloat16, seed=s).items()} for s in (1, 2)]
    cu = cu_of(lengths)

    def run(d):
        return kda.kda_conv_bwd(d["x"][None], d["w"], d["dout"][None], d["b"], True, cu, d["init"], d["dfinal"], True)

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
    for d, w in ((sets[1], want[1]), (sets[1], want[1])):
        for k in ("x", "w", "b", "init", "dout", "dfinal"):
            sets[0][k].copy_(d[k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(w[k], res[k]) for k in w)
    assert kda.device_error() == 0
