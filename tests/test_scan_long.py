"""The scan at state size 128 over sequences of more than 256 tokens on average (tiles of 128 tokens, two runs of 64
columns per CTA), in pieces and whole, and its calls on other streams, at once and captured."""
import pytest
import torch

import kimi_delta_attention_27_b200 as kda
import mixer_ref as ref
import test_scan as base
from test_scan import call_bwd, call_fwd, check_bwd, check_fwd, cu_of, dev, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    from kimi_delta_attention_27_b200 import build
    build.build()
    return kda.load_library()


def workspace(lengths, H, P):
    return kda.scan_workspace_bytes(sum(lengths), len(lengths), H, P, 128)


# lengths, H, G, P; runs of 64 columns per group: 3, 2, 1, 4
CUT = {
    "odd_runs": ([700, 129, 1, 0, 600], 6, 2, 64),
    "two_runs_of_one_head": ([0, 257, 0, 900], 1, 1, 128),
    "one_run": ([127, 128, 1000], 2, 2, 64),
    "four_runs": ([385, 383], 2, 1, 128),
}


@pytest.mark.parametrize("state", [torch.float32, torch.bfloat16, None])
@pytest.mark.parametrize("name", list(CUT))
def test_long_fwd_in_pieces(lib, name, state):
    lengths, H, G, P = CUT[name]
    assert sum(lengths) > 256 * len(lengths) and workspace(lengths, H, P) > 0
    d = make(lengths, H, G, P, 128, seed=len(name), state=state, sharp=name == "one_run")
    softplus = name != "four_runs"
    if not softplus:
        d["dt"], d["D"] = d["dt"].abs() * 0.2, None
    out, hT = call_fwd(d, lengths, softplus, final_state_dtype=state or torch.float32)
    torch.cuda.synchronize()
    assert kda.device_error() == 0
    check_fwd(d, lengths, softplus, out, hT)
    none, _ = call_fwd(d, lengths, softplus)          # no final state: fewer parts for the state, y from the same copies
    m = base.mags(d, softplus, lengths)
    # each is within H16 (1 + 2^-7) (|y| + its terms) of the exact one, and |y| is at most its terms
    assert ref.worst(none[0], out[0].double().cpu(), 4 * base.H16 * 1.01 * m["out"] + 1e-37) <= 1


@pytest.mark.parametrize("state", [torch.float32, None])
@pytest.mark.parametrize("name", list(CUT))
def test_long_bwd_in_pieces(lib, name, state):
    lengths, H, G, P = CUT[name]
    assert lib.kda_scan_bwd_workspace(sum(lengths), len(lengths), H, G, P, 128) > 0
    d = make(lengths, H, G, P, 128, seed=len(name) + 9, state=state, sharp=name == "one_run")
    softplus = name != "four_runs"
    if not softplus:
        d["dt"], d["D"], d["bias"] = d["dt"].abs() * 0.2, None, None
    g, again = call_bwd(d, lengths, softplus), call_bwd(d, lengths, softplus)
    assert kda.device_error() == 0 and all(g[k] is None or torch.equal(g[k], again[k]) for k in g)
    check_bwd(d, lengths, softplus, g)


@pytest.mark.parametrize("n", [20, 66])
def test_long_whole_sequences(lib, n):
    """Enough sequences that none is cut: up to 64 go longest first, more in their order."""
    H = 20 if n == 20 else 5
    g = torch.Generator().manual_seed(n)
    lengths = [int(v) for v in torch.randint(0, 600, (n,), generator=g)]
    lengths[3] = max(0, 258 * n - sum(lengths[:3] + lengths[4:]))
    assert sum(lengths) > 256 * n and workspace(lengths, H, 64) == 0
    d = make(lengths, H, 1, 64, 128, seed=n)
    out, hT = call_fwd(d, lengths, final_state_dtype=torch.float32)
    assert kda.device_error() == 0
    check_fwd(d, lengths, True, out, hT)


def test_short_sequences_beyond_the_ordered_ones(lib):
    g = torch.Generator().manual_seed(5)
    lengths = [int(v) for v in torch.randint(0, 90, (75,), generator=g)]
    d = make(lengths, 8, 2, 64, 64, seed=5)
    out, hT = call_fwd(d, lengths, final_state_dtype=torch.float32)
    check_fwd(d, lengths, True, out, hT)
    check_bwd(d, lengths, True, call_bwd(d, lengths))


@pytest.mark.parametrize("P", [64, 128])
def test_long_blocks_that_decay_steeply(lib, P):
    """Decays by far more than 2^60 within a block of 32 tokens, by 0 in one step, and none at all for a while."""
    lengths = [512, 300]
    d = make(lengths, 2, 1, P, 128, seed=61)
    d["bias"] = d["D"] = None
    d["dt"] = d["dt"].abs() * 0.1
    d["dt"][64:96, 0] = 2.0                          # one block of the first head
    d["x"][64:96] *= 0.1
    d["dt"][200] = 1e30                              # forgets all
    d["x"][200] = 0
    d["dt"][256:400] = 0
    d["dt"][511] = 40.0                              # a tile's last token
    d["x"][511] *= 1e-2
    d["dt"][512] = 40.0                              # a sequence's first
    d["x"][512] *= 1e-2
    out, hT = call_fwd(d, lengths, False, final_state_dtype=torch.float32)
    assert kda.device_error() == 0
    check_fwd(d, lengths, False, out, hT)


def test_long_padding_and_neighbours(lib):
    """Rows behind the last sequence hold NaN and stay unwritten; a NaN stays in its sequence, and reaches at most the
    127 tokens before it."""
    lengths, H, G, P = [300, 333, 401], 3, 1, 64
    d = make(lengths, H, G, P, 128, seed=71)
    want, wT = call_fwd(d, lengths, final_state_dtype=torch.float32)
    R, pad = sum(lengths), 90
    wide = lambda t, v: torch.cat([dev(t), torch.full((pad,) + t.shape[1:], v, dtype=t.dtype, device="cuda")])[None]  # noqa: E731
    nan = float("nan")
    out = torch.full((1, R + pad, H, P), 7.0, dtype=torch.bfloat16, device="cuda")
    args = (wide(d["x"], nan), wide(d["dt"], nan), dev(d["A"]), wide(d["B"], nan), wide(d["C"], nan), dev(d["D"]),
            dev(d["bias"]), True, cu_of(lengths), dev(d["h0"]))
    _, hT = kda.kda_scan_fwd(*args, out=out, final_state_dtype=torch.float32)
    # the pieces lie on a grid whose width the number of rows gives, so other pieces are added up
    check_fwd(d, lengths, True, out[:, :R], hT)
    assert bool((out[:, R:] == 7).all())
    dout = torch.full_like(out, nan)
    dout[0, :R] = dev(d["dout"])
    g = kda.kda_scan_bwd(*args[:5], dout, *args[5:], dfinal_state=dev(d["dhT"]))
    check_bwd(d, lengths, True, {k: v[:, :R] if k in ("dx", "dB", "dC", "ddt") else v for k, v in g.items()})
    d["B"][300 + 200, 0, 5], d["x"][300 + 201, 0, 1], d["C"][300 + 200, 0, 7] = nan, float("inf"), nan
    got, gT = call_fwd(d, lengths, final_state_dtype=torch.float32)
    for i, (a, b) in enumerate(ref.spans(lengths)):
        if i != 1:
            assert torch.equal(got[:, a:b], want[:, a:b]) and torch.equal(gT[i], wT[i])
    assert torch.equal(got[:, 300:300 + 200 - 127], want[:, 300:300 + 200 - 127]) and bool(gT[1].isnan().any())
    assert kda.device_error() == 0


def everything(d, lengths, **kw):
    out, hT = call_fwd(d, lengths, final_state_dtype=torch.float32)
    return dict(call_bwd(d, lengths), out=out, hT=hT)


def test_long_calls_at_once_and_another_stream(lib):
    """Two calls in flight on two streams, each with its own scratch memory, equal the same calls one by one."""
    lengths = [900, 70, 400]
    sets = [make(lengths, 4, 2, 64, 128, seed=s) for s in (1, 2)]
    want = [everything(d, lengths) for d in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    ready = [{k: dev(v) if torch.is_tensor(v) else v for k, v in d.items()} for d in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for d, s in zip(ready, streams):
            with torch.cuda.stream(s):
                got.append(everything(d, lengths))
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert all(torch.equal(w[k], g[k]) for k in w)
    assert kda.device_error() == 0


def test_long_calls_captured(lib):
    """Forward, gradients and a single token captured in one graph, twice over, with one workspace for both graphs:
    replayed in turn they equal the calls."""
    lengths, (H, G, P, N) = [500, 300], (4, 1, 64, 128)
    d = {k: dev(v) if torch.is_tensor(v) else v for k, v in make(lengths, H, G, P, N, seed=8).items()}
    cu = cu_of(lengths)
    need = max(kda.scan_workspace_bytes(800, 2, H, P, N), lib.kda_scan_bwd_workspace(800, 2, H, G, P, N))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    S = torch.zeros(2, H, N, P, device="cuda")

    def step():
        a = (d["x"][None], d["dt"][None], d["A"], d["B"][None], d["C"][None])
        out, hT = kda.kda_scan_fwd(*a, d["D"], d["bias"], True, cu, d["h0"], final_state=S, workspace=ws)
        g = kda.kda_scan_bwd(*a, d["dout"][None], d["D"], d["bias"], True, cu, d["h0"], d["dhT"], workspace=ws)
        tok, _ = kda.kda_scan_decode(d["x"][:2], d["dt"][:2], d["A"], d["B"][:2], d["C"][:2], S, S, D=d["D"],
                                     dt_bias=d["bias"], dt_softplus=True)
        return dict(g, out=out, S=S, tok=tok)

    want = {k: v.clone() for k, v in step().items()}
    torch.cuda.synchronize()
    graphs, results = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append(step())
        graphs.append(g)
    for _ in range(2):
        for g, r in zip(graphs, results):
            ws.fill_(255)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(want[k], r[k]) for k in want)
    assert kda.device_error() == 0
