"""What the operators around the recurrence do with arguments that are malformed, empty, not finite, or at an end of their
range: refused, reported, or passed on, and never an access out of bounds."""
import ctypes

import pytest
import torch

import kimi_delta_attention_27_b200 as kda
import mixer_ref as ref

BF = torch.bfloat16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from kimi_delta_attention_27_b200 import build
    build.build()
    return kda.load_library()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [[7, 20, 50], [50, 20, 50], [2 ** 31 - 1, 2 ** 31 - 1, 50], [50, 50, 50]])
def test_conv_table_that_does_not_begin_at_zero_reads_no_other_state(lib, bad):
    """Rows before cu[0] belong to no sequence. They are taken as the first one's, whose initial state has W - 1 rows and
    no more: what lies around the states (NaN here) is not read into anything."""
    W, C, rows, guard = 4, 64, 50, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1, rows, C, generator=g, device="cuda").to(BF)
    w = torch.randn(C, W, generator=g, device="cuda")
    dy = torch.randn(1, rows, C, generator=g, device="cuda").to(BF)
    around = torch.full((2 * guard + 2 * (W - 1), C), NAN, dtype=BF, device="cuda")
    init = around[guard:guard + 2 * (W - 1)].view(2, W - 1, C)
    init.normal_(generator=g)
    cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
    out, final = torch.zeros_like(x), torch.zeros_like(init)
    kda.kda_conv_fwd(x, w, cu_seqlens=cu, initial_state=init, out=out, final_state=final)
    assert kda.device_error() == 12 and bool(torch.isfinite(out).all()) and bool(torch.isfinite(final).all())
    dx = torch.zeros_like(x)
    r = kda.kda_conv_bwd(x, w, dy, cu_seqlens=cu, initial_state=init, dfinal_state=init, want_dinitial_state=True, dx=dx)
    assert kda.device_error() == 12
    assert all(bool(torch.isfinite(r[k]).all()) for k in ("dx", "dweight", "dinitial_state"))


@pytest.mark.gpu
@pytest.mark.parametrize("rot", [0, 64])
def test_qk_bwd_of_no_rows_reads_nothing(lib, rot):
    """Positions, frequencies, q and k may be NULL where there are no rows; the weights' gradients are zeros."""
    D = 128
    P = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731
    dqw, dkw = torch.full((D,), 7.0, device="cuda"), torch.full((D,), 7.0, device="cuda")
    ws = torch.zeros(lib.kda_qk_bwd_workspace(0, 4, 2, D), dtype=torch.uint8, device="cuda")
    st = lib.kda_qk_bwd(None, 0, None, 0, 0, 4, 2, D, 1, 1e-6, None, None, None, None, rot, 0, 1.0, None, 0, None, 0, 1, None, 0,
                        None, 0, P(dqw), P(dkw), P(ws), ws.numel(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert st == 0 and bool((dqw == 0).all()) and bool((dkw == 0).all()) and kda.device_error() == 0
    # and through the binding, with rows of no tokens
    q = torch.zeros(2, 0, 4, D, dtype=BF, device="cuda")
    w, f = torch.ones(D, device="cuda"), torch.ones(rot // 2, device="cuda")
    pos = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    r = kda.kda_qk_bwd(q, q, q, q, q_weight=w, k_weight=w, positions=pos, inv_freq=f)
    assert r["dq"].shape == q.shape and bool((r["dq_weight"] == 0).all()) and bool((r["dk_weight"] == 0).all())


def test_sizes_whose_product_passes_64_bits_are_refused(lib):
    """batch * seq_len = 2^64 rows are not 0 rows; workspaces of sizes that a call refuses are 0."""
    TOO_LARGE, far = 8, [ctypes.c_void_p((i + 1) << 36) for i in range(12)]   # aligned, never dereferenced
    big = (1 << 24, 1 << 40)
    assert lib.kda_conv_fwd(far[0], 1, 64, far[1], None, 1, None, 0, *big, 64, 4, None, far[3], far[2], 64, None) == TOO_LARGE
    assert lib.kda_conv_bwd(far[0], 1, 64, far[1], None, 1, None, 0, *big, 64, 4, None, far[3], 1, 64, None, far[4], 64,
                            far[5], None, None, far[6], 1 << 30, None) == TOO_LARGE
    assert lib.kda_scan_fwd(far[0], 256, far[1], far[2], far[3], 128, far[4], 128, None, None, 1, None, 0, *big, 4, 1, 64,
                            128, None, 0, far[7], 2, far[5], 256, far[6], 1 << 34, None) == TOO_LARGE
    assert lib.kda_scan_bwd(far[0], 256, far[1], far[2], far[3], 128, far[4], 128, None, None, 1, None, 0, *big, 4, 1, 64,
                            128, None, 0, far[5], 256, None, far[6], 256, far[7], far[8], far[9], 128, far[10], 128, None,
                            None, None, far[11], 1 << 34, None) == TOO_LARGE
    most = (1 << 63) - 1
    assert lib.kda_conv_bwd_workspace(most, 64, 4) == 0 and lib.kda_qk_bwd_workspace(most, 1, 0, 128) == 0
    assert lib.kda_scan_fwd_workspace(1 << 32, 1, 1, 64, 64) == 0
    assert lib.kda_scan_bwd_workspace(0, (1 << 31) - 1, 1 << 20, 1, 128, 128) == 0


def terms_of_steps_of_both_signs(d, softplus, lengths, grads=False):
    """What the terms of each result add up to: the recurrence on absolute values, with x given the sign of its step so
    that d x is positive (no D, no bias)."""
    ab = lambda n: None if d[n] is None else d[n].double().abs()  # noqa: E731
    x = ab("x") * d["dt"].double().sign()[..., None]
    m = ref.scan(x, d["dt"], d["A"], ab("B"), ab("C"), None, None, False, lengths, ab("h0"), ab("dout") if grads else None,
                 ab("dhT") if grads else None)
    return {k: v.abs() for k, v in m.items()}


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,N", [([600], 128), ([90, 41], 128), ([300, 70], 64)])
def test_scan_steps_below_zero_among_steep_ones(lib, monkeypatch, lengths, N):
    """Every third step is below zero (its decay is up to e^0.8), in blocks whose decay is far below 2^-60."""
    import test_scan as base
    monkeypatch.setattr(base, "mags", terms_of_steps_of_both_signs)
    d = base.make(lengths, 4, 2, 64, N, seed=N)
    d["bias"] = d["D"] = None
    d["dt"] = 0.2 + d["dt"].abs()
    d["dt"][1::3] *= -0.04
    d["A"] = -(1 + 7 * torch.arange(4) / 3)
    out, hT = base.call_fwd(d, lengths, False, final_state_dtype=torch.float32)
    base.check_fwd(d, lengths, False, out, hT)
    base.check_bwd(d, lengths, False, base.call_bwd(d, lengths, False))
    assert kda.device_error() == 0


# lengths, H, G, state size: the tcgen05 kernel whole and in pieces, the warp-level one whole and in pieces
SCANS = {"tc": ([300, 290, 310] * 4, 32, 4, 128), "tc_pieces": ([900, 700], 4, 2, 128), "warp": ([70, 64, 1], 4, 2, 128),
         "small_state": ([130, 5], 4, 2, 64), "small_state_pieces": ([2000, 90], 4, 2, 64)}


def lost(got, want):
    """Values that are not finite in the reference and are in the result."""
    return int((torch.isfinite(got.detach().cpu()) & ~torch.isfinite(want)).sum())


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(SCANS))
def test_scan_nan_rate_of_one_head(lib, name):
    """A NaN in one head's A: NaN in all that the 64-bit recurrence makes NaN of; the other heads bit for bit as without."""
    import test_scan as base
    lengths, H, G, N = SCANS[name]
    assert (kda.scan_workspace_bytes(sum(lengths), len(lengths), H, 64, N) > 0) == name.endswith("pieces")
    d = base.make(lengths, H, G, 64, N, seed=3)
    e = dict(d, A=d["A"].clone())
    bad, rest = 1, [h for h in range(H) if h != 1]
    e["A"][bad] = NAN
    r = ref.scan(e["x"], e["dt"], e["A"], e["B"], e["C"], e["D"], e["bias"], True, lengths, e["h0"], e["dout"], e["dhT"])
    for dtype in (torch.float32, None):
        f = dict(e, h0=e["h0"] if dtype else None)
        out, hT = base.call_fwd(f, lengths, final_state_dtype=dtype)
        want, wT = base.call_fwd(dict(f, A=d["A"]), lengths, final_state_dtype=dtype)
        assert lost(out[0], r["out"]) == 0 and torch.equal(out[:, :, rest], want[:, :, rest])
        assert dtype is None or (lost(hT, r["state"]) == 0 and torch.equal(hT[:, rest], wT[:, rest]))
    got, want = base.call_bwd(e, lengths), base.call_bwd(d, lengths)
    for k in ("dx", "dB", "dC", "ddt", "dA", "ddt_bias", "dh0"):
        g = got[k][0] if k in ("dx", "dB", "dC", "ddt") else got[k]
        assert lost(g, r[k]) == 0 and not bool(torch.isfinite(g).all()), k
    for k, at in (("dx", 2), ("ddt", 2), ("dA", 0), ("ddt_bias", 0), ("dh0", 1)):
        pick = torch.tensor(rest, device="cuda")
        assert torch.equal(got[k].index_select(at, pick), want[k].index_select(at, pick)), k
    for k in ("dB", "dC"):
        assert torch.equal(got[k][:, :, 1:], want[k][:, :, 1:]), k
    assert torch.equal(got["dD"], want["dD"]) and kda.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(SCANS))
def test_scan_nan_step_of_one_token(lib, name):
    """A NaN in one token's dt reaches every later output of its head and sequence, no earlier one, and no other sequence."""
    import test_scan as base
    lengths, H, G, N = SCANS[name]
    d = base.make(lengths, H, G, 64, N, seed=4)
    want, _ = base.call_fwd(d, lengths, final_state_dtype=torch.float32)
    t, h = 33, 2
    d["dt"][t, h] = NAN
    r = ref.scan(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["bias"], True, lengths, d["h0"], d["dout"], d["dhT"])
    out, hT = base.call_fwd(d, lengths, final_state_dtype=torch.float32)
    assert torch.equal(torch.isnan(out[0]).cpu(), torch.isnan(r["out"]))
    assert torch.equal(torch.isnan(hT).cpu(), torch.isnan(r["state"]))
    assert torch.equal(out[0, lengths[0]:], want[0, lengths[0]:])
    got = base.call_bwd(d, lengths)
    for k in ("dx", "dB", "dC", "ddt", "dA", "ddt_bias", "dh0"):
        g = got[k][0] if k in ("dx", "dB", "dC", "ddt") else got[k]
        assert lost(g, r[k]) == 0, k
    assert bool(torch.isfinite(got["dx"][0, lengths[0]:]).all()) and bool(torch.isfinite(got["dh0"][1:]).all())
    assert kda.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(SCANS))
def test_scan_rate_of_minus_infinity_forgets_everything(lib, name):
    """The same as a rate of -1e30, in partly filled tiles too."""
    import test_scan as base
    lengths, H, G, N = SCANS[name]
    d = base.make(lengths, H, G, 64, N, seed=5)
    res = []
    for a in (-1e30, -INF):
        d["A"][1] = a
        res.append(base.call_fwd(d, lengths, final_state_dtype=torch.float32))
    assert bool(torch.isfinite(res[0][0]).all()) and bool(torch.isfinite(res[0][1]).all())
    assert all(torch.equal(a, b) for a, b in zip(*res)) and kda.device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("state", [torch.float32, BF])
@pytest.mark.parametrize("N", [64, 128])
def test_scan_decode_nan_rate_and_step(lib, N, state):
    import test_scan as base
    d = base.make([1] * 5, 4, 2, 64, N, seed=N, state=state)
    kw = dict(D=base.dev(d["D"]), dt_bias=base.dev(d["bias"]), dt_softplus=True)

    def call(d):
        S = base.dev(d["h0"]).clone()
        return kda.kda_scan_decode(*(base.dev(d[k]) for k in ("x", "dt", "A", "B", "C")), S, S, **kw)

    want, wS = call(d)
    e = dict(d, A=d["A"].clone(), dt=d["dt"].clone())
    e["A"][1], e["dt"][3, 2] = NAN, NAN
    r = ref.scan(e["x"], e["dt"], e["A"], e["B"], e["C"], e["D"], e["bias"], True, [1] * 5, e["h0"])
    out, S = call(e)
    assert torch.equal(torch.isnan(out).cpu(), torch.isnan(r["out"])) and torch.equal(torch.isnan(S).cpu(), torch.isnan(r["state"]))
    assert torch.equal(out[:, [0, 3]], want[:, [0, 3]]) and torch.equal(S[:, [0, 3]], wS[:, [0, 3]])


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,norm", [(128, 64, "l2"), (64, 64, "none"), (256, 112, "rms")])
def test_qk_frequencies_that_are_not_finite(lib, D, rot, norm, interleaved):
    """NaN in their pairs, as the 64-bit form has it (and through the norm in a head's whole gradient); the other pairs bit
    for bit as without."""
    T, H = 21, 3
    g = torch.Generator().manual_seed(D)
    q, dy = torch.randn(1, T, H, D, generator=g).to(BF), torch.randn(1, T, H, D, generator=g).to(BF)
    pos = torch.arange(T, dtype=torch.int32)[None]
    f = torch.rand(rot // 2, generator=g)
    bad = f.clone()
    bad[0], bad[5], bad[rot // 2 - 1] = NAN, INF, -INF
    x = q[0].to(ref.F64).requires_grad_()
    y = ref.qk(x, None, norm, 1e-6, pos[0], bad, interleaved, 1.0)
    dx, = torch.autograd.grad(y, x, dy[0].to(ref.F64))
    opt = dict(norm=norm, positions=pos.cuda(), interleaved=interleaved)
    got, _ = kda.kda_qk_fwd(q.cuda(), inv_freq=bad.cuda(), **opt)
    clean, _ = kda.kda_qk_fwd(q.cuda(), inv_freq=f.cuda(), **opt)
    nan = torch.isnan(y)
    assert torch.equal(torch.isnan(got[0]).cpu(), nan) and bool(nan.any()) and torch.equal(got[0].cpu()[~nan], clean[0].cpu()[~nan])
    got = kda.kda_qk_bwd(q.cuda(), None, dy.cuda(), None, inv_freq=bad.cuda(), **opt)["dq"][0].cpu()
    clean = kda.kda_qk_bwd(q.cuda(), None, dy.cuda(), None, inv_freq=f.cuda(), **opt)["dq"][0].cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(dx)) and torch.equal(got[~torch.isnan(dx)], clean[~torch.isnan(dx)])


@pytest.mark.gpu
def test_what_a_call_allocates_belongs_to_the_stream_it_is_given(lib, monkeypatch):
    """Outputs and workspaces too, and for the default stream's handle, which is 0, while another stream is current: else
    their memory could be given out again while the kernels on the default stream still use it."""
    seen = []
    for name in ("empty", "empty_like"):
        real = getattr(torch, name)

        def noted(*a, real=real, **k):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return real(*a, **k)
        monkeypatch.setattr(torch, name, noted)
    x, w = torch.ones(1, 9, 16, dtype=BF, device="cuda"), torch.ones(16, 4, device="cuda")
    q = torch.ones(1, 9, 2, 64, dtype=BF, device="cuda")
    dt, A, B = torch.ones(1, 9, 2, device="cuda"), -torch.ones(2, device="cuda"), torch.ones(1, 9, 1, 64, dtype=BF, device="cuda")
    calls = (lambda s: kda.kda_conv_fwd(x, w, want_final_state=True, stream=s), lambda s: kda.kda_conv_bwd(x, w, x, stream=s),
             lambda s: kda.kda_conv_decode(x[0], w, stream=s), lambda s: kda.kda_qk_fwd(q, q, stream=s),
             lambda s: kda.kda_qk_bwd(q, None, q, None, q_weight=torch.ones(64, device="cuda"), stream=s),
             lambda s: kda.kda_scan_fwd(q, dt, A, B, B, final_state_dtype=torch.float32, stream=s),
             lambda s: kda.kda_scan_bwd(q, dt, A, B, B, q, stream=s),
             lambda s: kda.kda_scan_decode(q[0], dt[0], A, B[0], B[0], state_dtype=torch.float32, stream=s))
    side, third = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for given, want in ((None, side.cuda_stream), (0, 0), (third.cuda_stream, third.cuda_stream)):
        for call in calls:
            with torch.cuda.stream(side):
                seen.clear()
                call(given)
                assert seen and set(seen) == {want}, (given, seen)
                assert torch.cuda.current_stream() == side
        torch.cuda.synchronize()
    assert kda.device_error() == 0


@pytest.mark.gpu
def test_what_the_recurrence_allocates_belongs_to_the_stream_it_is_given(lib, monkeypatch):
    """The same of kda_fwd, kda_fwd_segmented, kda_bwd and kda_decode."""
    from kimi_delta_attention_27_b200.inputs import make_inputs
    inp = make_inputs({"B": 1, "T": 128, "H": 1, "lengths": None, "g_mu": 3.0, "init": None, "final": "fp32", "seed": 8},
                      device="cuda")
    args = [inp[k] for k in ("q", "k", "v", "g", "beta")]
    one = [t[:, 0].contiguous() for t in args]
    seen, real = [], torch.empty

    def noted(*a, **k):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return real(*a, **k)
    monkeypatch.setattr(torch, "empty", noted)
    f32 = torch.float32
    calls = (lambda s: kda.kda_fwd(*args, final_state_dtype=f32, stream=s), lambda s: kda.kda_bwd(*args, inp["v"], stream=s),
             lambda s: kda.kda_fwd_segmented(*args, segment_len=64, final_state_dtype=f32, stream=s),
             lambda s: kda.kda_decode(*one, state_dtype=f32, stream=s))
    side, third = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    want = [c(None) for c in calls]
    torch.cuda.synchronize()
    for given, handle in ((None, side.cuda_stream), (0, 0), (third.cuda_stream, third.cuda_stream)):
        for call, w in zip(calls, want):
            with torch.cuda.stream(side):
                seen.clear()
                got = call(given)
                assert seen and set(seen) == {handle}, (given, seen)
            torch.cuda.synchronize()
            pairs = zip(w.values(), got.values()) if isinstance(w, dict) else zip(w, got)
            assert all(a is b or torch.allclose(a.float(), b.float(), rtol=1e-3, atol=1e-3) for a, b in pairs)
    assert kda.device_error() == 0


def test_scan_cuts_no_sequence_that_makes_no_two_pieces(lib):
    """Several short sequences are not worth a cut: no state run, no join, no workspace. Equal rows ask for no more than
    packed ones of the same number and length, whose need is what the query returns."""
    need = kda.scan_workspace_bytes
    for n, tokens in ((2, 200), (4, 200), (8, 128), (1, 400), (3, 250)):
        for H, N in ((8, 64), (8, 128), (32, 64), (32, 128)):
            assert need(n * tokens, n, H, 64, N) == 0 and need(n * tokens, n, H // 2, 128, N) == 0, (n, tokens, H, N)
    for N in (64, 128):
        assert need(65536, 1, 32, 128, N) > 0 and need(2 * 4096, 2, 8, 64, N) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("n,tokens,H,N", [(2, 200, 4, 128), (4, 129, 3, 64), (2, 640, 2, 128), (2, 1100, 2, 64), (1, 1030, 2, 128)])
def test_scan_rows_below_and_above_the_cut(lib, n, tokens, H, N, packed):
    """Equal rows, as a batch and packed, in one workspace of the size that the query gives, to its last byte."""
    import test_scan as base
    lengths = [tokens] * n
    d = base.make(lengths, H, 1, 64, N, seed=tokens)
    rows = (1, n * tokens) if packed else (n, tokens)
    v = lambda k: base.dev(d[k]).view(*rows, *d[k].shape[1:])  # noqa: E731
    kw = dict(D=base.dev(d["D"]), dt_bias=base.dev(d["bias"]), dt_softplus=True, initial_state=base.dev(d["h0"]),
              cu_seqlens=base.cu_of(lengths) if packed else None)
    args = (v("x"), v("dt"), base.dev(d["A"]), v("B"), v("C"))
    sizes = (kda.scan_workspace_bytes(n * tokens, n, H, 64, N), lib.kda_scan_bwd_workspace(n * tokens, n, H, 1, 64, N))
    spaces = [torch.full((s + 1024,), 165, dtype=torch.uint8, device="cuda") for s in sizes]
    out, hT = kda.kda_scan_fwd(*args, final_state_dtype=torch.float32, workspace=spaces[0][:sizes[0]], **kw)
    base.check_fwd(d, lengths, True, out.view(1, n * tokens, H, 64), hT)
    g = kda.kda_scan_bwd(*args, v("dout"), dfinal_state=base.dev(d["dhT"]), workspace=spaces[1][:sizes[1]], **kw)
    g = {k: t.view(1, n * tokens, *t.shape[2:]) if k in ("dx", "dB", "dC", "ddt") else t for k, t in g.items()}
    base.check_bwd(d, lengths, True, g)
    assert all(bool((w[s:] == 165).all()) for w, s in zip(spaces, sizes)) and kda.device_error() == 0


# lengths, H, G, P; runs of 64 columns per group: 3, 2, 1, 4. Longest (twice the mean) 1024 tokens or more: the states of
# the gradients in pieces
CUT_BWD = {
    "odd_runs": ([1500, 129, 1, 0, 1100], 6, 2, 64),
    "two_runs_of_one_head": ([0, 257, 0, 2100], 1, 1, 128),
    "one_run": ([127, 128, 2000], 2, 2, 64),
    "four_runs": ([985, 783], 2, 1, 128),
}


@pytest.mark.gpu
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("name", list(CUT_BWD))
def test_scan_bwd_of_long_sequences_in_pieces(lib, name, N):
    import test_scan as base
    lengths, H, G, P = CUT_BWD[name]
    d = base.make(lengths, H, G, P, N, seed=len(name), state=None if name == "one_run" else torch.float32, sharp=name == "one_run")
    softplus = name != "four_runs"
    if not softplus:
        d["dt"], d["D"], d["bias"] = d["dt"].abs() * 0.2, None, None
    g, again = base.call_bwd(d, lengths, softplus), base.call_bwd(d, lengths, softplus)
    assert kda.device_error() == 0 and all(g[k] is None or torch.equal(g[k], again[k]) for k in g)
    base.check_bwd(d, lengths, softplus, g)


def test_conv_weight_of_many_channels_is_seen_whole(lib):
    """2^30 channels x 4 taps are 16 GiB of weights: an output in the midst of them is refused."""
    at = lambda i: ctypes.c_void_p(i << 40)  # noqa: E731
    out = ctypes.c_void_p((5 << 40) + (1 << 33))
    assert lib.kda_conv_decode(at(1), 1, 1 << 30, at(5), None, 1, 3, 1 << 30, 4, at(2), at(3), out, 1 << 30, None) == 16


def test_outputs_over_the_offsets_are_refused(lib):
    """cu_seqlens is an input like the others: a kernel that wrote over it would look its sequences up in its own results."""
    OVERLAP, n, f = 16, 5, [ctypes.c_void_p((i + 1) << 36) for i in range(16)]   # aligned, never dereferenced
    cu, last = f[15], ctypes.c_void_p((16 << 36) + 16)                           # the last of six offsets at + 20
    conv = lambda **o: lib.kda_conv_fwd(f[0], 1, 64, f[1], None, 1, cu, n, 1, 100, 64, 4, None, o.get("final", f[3]),  # noqa: E731
                                        o.get("out", f[2]), 64, None)
    assert conv(out=last) == OVERLAP and conv(final=last) == OVERLAP
    conv = lambda **o: lib.kda_conv_bwd(f[0], 1, 64, f[1], None, 1, cu, n, 1, 100, 64, 4, None, f[3], 1, 64, None,  # noqa: E731
                                        o.get("dx", f[4]), 64, o.get("dw", f[5]), None, None, o.get("ws", f[6]), 1 << 30, None)
    assert conv(dx=last) == OVERLAP and conv(dw=last) == OVERLAP
    scan = lambda **o: lib.kda_scan_fwd(f[0], 256, f[1], f[2], f[3], 128, f[4], 128, None, None, 1, cu, n, 1, 100, 4, 1, 64,  # noqa: E731
                                        128, None, 0, o.get("hT", f[7]), 2, o.get("out", f[5]), 256, f[6], 1 << 34, None)
    assert scan(out=last) == OVERLAP and scan(hT=last) == OVERLAP
    scan = lambda **o: lib.kda_scan_bwd(f[0], 256, f[1], f[2], f[3], 128, f[4], 128, None, None, 1, cu, n, 1, 100, 4, 1, 64,  # noqa: E731
                                        128, None, 0, f[5], 256, None, f[6], 256, o.get("ddt", f[7]), f[8], f[9], 128, f[10],
                                        128, None, None, None, o.get("ws", f[11]), 1 << 34, None)
    assert scan(ddt=last) == OVERLAP and scan(ws=cu) == OVERLAP
    if not torch.cuda.is_available():
        assert conv() == 5 and scan() == 5              # let through, as far as the device query


@pytest.mark.gpu
@pytest.mark.parametrize("N", [64, 128])
@pytest.mark.parametrize("lengths", [[140], [290, 11]])
def test_scan_steps_below_zero_that_let_the_state_grow(lib, monkeypatch, lengths, N):
    """By up to 2^57 over 128 tokens, and by as much down again in other stretches."""
    import test_scan as base
    monkeypatch.setattr(base, "mags", terms_of_steps_of_both_signs)
    d = base.make(lengths, 3, 1, 64, N, seed=N + 1)
    d["bias"] = d["D"] = None
    t = torch.arange(sum(lengths))[:, None]
    d["A"] = -torch.tensor([1.0, 0.5, 2.0])
    d["dt"] = torch.where(t // 130 % 2 == 0, -0.31, 0.31) * (0.9 + 0.1 * torch.rand(sum(lengths), 3)) / d["A"].abs()
    out, hT = base.call_fwd(d, lengths, False, final_state_dtype=torch.float32)
    base.check_fwd(d, lengths, False, out, hT)
    base.check_bwd(d, lengths, False, base.call_bwd(d, lengths, False))
    assert kda.device_error() == 0
