"""Calls at the ends of what the operators around the recurrence allow: nothing to do, offsets past 32 bits, values that
are not finite, malformed tables at a state size of 128."""
import pytest
import torch

import kimi_delta_attention_27_b200 as kda
import mixer_ref as ref
from test_scan import call_bwd, call_fwd, check_bwd, check_fwd, make

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    from kimi_delta_attention_27_b200 import build
    build.build()
    yield kda.load_library()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("N", [64, 128])
def test_rows_of_no_tokens_pass_their_states_on(N):
    x, dt, A = torch.zeros(3, 0, 2, 64, dtype=BF, device="cuda"), torch.zeros(3, 0, 2, device="cuda"), -torch.ones(2, device="cuda")
    B = torch.zeros(3, 0, 1, N, dtype=BF, device="cuda")
    h0, dh = torch.randn(3, 2, N, 64, device="cuda"), torch.randn(3, 2, N, 64, device="cuda")
    out, hT = kda.kda_scan_fwd(x, dt, A, B, B, initial_state=h0, final_state_dtype=torch.float32)
    assert out.shape == x.shape and torch.equal(hT, h0)
    g = kda.kda_scan_bwd(x, dt, A, B, B, x, D=A, initial_state=h0, dfinal_state=dh)
    assert torch.equal(g["dh0"], dh) and bool((g["dA"] == 0).all()) and bool((g["dD"] == 0).all())
    c = torch.zeros(3, 0, 16, dtype=BF, device="cuda")
    w, s0 = torch.randn(16, 4, device="cuda"), torch.randn(3, 3, 16, device="cuda").to(BF)
    out, s1 = kda.kda_conv_fwd(c, w, initial_state=s0, want_final_state=True)
    assert torch.equal(s1, s0)
    g = kda.kda_conv_bwd(c, w, c, initial_state=s0, dfinal_state=s0, want_dinitial_state=True)
    assert torch.equal(g["dinitial_state"], s0) and bool((g["dweight"] == 0).all())
    q, _ = kda.kda_qk_fwd(torch.zeros(2, 0, 4, 128, dtype=BF, device="cuda"))
    assert q.shape == (2, 0, 4, 128)
    none = torch.zeros(0, 1, N, dtype=BF, device="cuda")
    o, _ = kda.kda_scan_decode(torch.zeros(0, 2, 64, dtype=BF, device="cuda"), torch.zeros(0, 2, device="cuda"), A, none, none)
    assert o.shape == (0, 2, 64)
    assert kda.device_error() == 0


def far(rows, width):
    """rows x width bf16, uninitialised but for what the caller writes, its last rows past 2^32 bytes."""
    assert rows * width > 1 << 31
    return torch.zeros(rows, width, dtype=BF, device="cuda")


def test_conv_and_qk_past_32_bits():
    rows, C, last = 524300, 4104, 37
    x = far(rows, C)
    x[-last:] = torch.randn(last, C, device="cuda").to(BF)
    w, b = torch.randn(C, 4, device="cuda"), torch.randn(C, device="cuda")
    cu = torch.tensor([0, rows - last, rows], dtype=torch.int32, device="cuda")
    out, fin = kda.kda_conv_fwd(x[None], w, b, cu_seqlens=cu, want_final_state=True)
    want, wf = kda.kda_conv_fwd(x[None, -last:].contiguous(), w, b, want_final_state=True)
    assert torch.equal(out[0, -last:], want[0]) and torch.equal(fin[1], wf[0])
    del out
    dy = torch.zeros_like(x)
    dy[-last:] = torch.randn(last, C, device="cuda").to(BF)
    g = kda.kda_conv_bwd(x[None], w, dy[None], b, cu_seqlens=cu)
    h = kda.kda_conv_bwd(x[None, -last:].contiguous(), w, dy[None, -last:].contiguous(), b)
    assert torch.equal(g["dx"][0, -last:], h["dx"][0])
    assert torch.allclose(g["dbias"], h["dbias"], rtol=1e-4, atol=1e-4)
    del g, dy
    q = x[:, :4096].unflatten(1, (32, 128))[None]
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")[None]
    f = torch.rand(64, device="cuda")
    qo, _ = kda.kda_qk_fwd(q, positions=pos, inv_freq=f)
    tail = q[:, -last:].contiguous()
    assert torch.equal(qo[:, -last:], kda.kda_qk_fwd(tail, positions=pos[:, -last:].contiguous(), inv_freq=f)[0])
    gq = kda.kda_qk_bwd(q, None, qo, None, positions=pos, inv_freq=f)
    gt = kda.kda_qk_bwd(tail, None, qo[:, -last:].contiguous(), None, positions=pos[:, -last:].contiguous(), inv_freq=f)
    assert torch.equal(gq["dq"][:, -last:], gt["dq"]) and kda.device_error() == 0


@pytest.mark.parametrize("N", [64, 128])
def test_scan_past_32_bits(N):
    lengths = [66000, 200]
    rows, H, P, last = sum(lengths), 256, 128, lengths[-1]
    x = far(rows, H * P).view(1, rows, H, P)
    g = torch.Generator(device="cuda").manual_seed(N)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x[:, -last:] = rn(1, last, H, P).to(BF)
    B, C = rn(1, rows, 1, N).to(BF), rn(1, rows, 1, N).to(BF)
    dt, A = 0.1 * rn(1, rows, H).abs(), -rn(H).abs()
    cu = torch.tensor([0, lengths[0], rows], dtype=torch.int32, device="cuda")
    out, hT = kda.kda_scan_fwd(x, dt, A, B, C, cu_seqlens=cu, final_state_dtype=torch.float32)
    tail = [t[:, -last:].contiguous() for t in (x, dt, B, C)]
    want, wT = kda.kda_scan_fwd(tail[0], tail[1], A, tail[2], tail[3], final_state_dtype=torch.float32)
    # the tiles of the two calls begin at other tokens: sums in another order, one rounding of y apart
    assert float((out[:, -last:].float() - want.float()).abs().max() / want.float().abs().max()) <= 2.0 ** -6
    assert float((hT[1] - wT[0]).abs().max() / wT.abs().max()) <= 1e-4
    assert bool((out[:, :-last] == 0).all()) and bool((hT[0] == 0).all())
    dy = out
    dy[:, -last:] = rn(1, last, H, P).to(BF)
    gr = kda.kda_scan_bwd(x, dt, A, B, C, dy, cu_seqlens=cu, want_dinitial_state=False)
    gt = kda.kda_scan_bwd(tail[0], tail[1], A, tail[2], tail[3], dy[:, -last:].contiguous(), want_dinitial_state=False)
    for k in ("dx", "dB", "dC", "ddt"):
        a, b = gr[k][:, -last:].float(), gt[k].float()
        assert float((a - b).abs().max() / b.abs().max()) <= 2.0 ** -6, k
        assert bool((gr[k][:, :-last] == 0).all()), k
    assert float((gr["dA"] - gt["dA"]).abs().max() / gt["dA"].abs().max()) <= 1e-4
    assert kda.device_error() == 0


def test_scan_decode_past_32_bits():
    batch, H, P, N = 300, 64, 128, 128
    big = torch.zeros(8 * batch, H, N, P, dtype=BF, device="cuda")          # 2.5e9 elements
    g = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    n = 8 * batch
    x, dt, A = rn(n, H, P).to(BF), 0.1 * rn(n, H).abs(), -rn(H).abs()
    B, C = rn(n, 1, N).to(BF), rn(n, 1, N).to(BF)
    big[-batch:] = rn(1, 1, N, P).to(BF)
    S = big[-batch:].clone()
    out, _ = kda.kda_scan_decode(x, dt, A, B, C, big, big)
    want, _ = kda.kda_scan_decode(x[-batch:], dt[-batch:], A, B[-batch:], C[-batch:], S, S)
    assert torch.equal(out[-batch:], want) and torch.equal(big[-batch:], S) and kda.device_error() == 0


@pytest.mark.parametrize("N", [64, 128])
def test_gradients_of_a_sequence_with_infinities_leave_its_neighbours_alone(N):
    lengths, shape = [150, 290, 101], (3, 1, 64, N)
    d = make(lengths, *shape, seed=N)
    want = call_bwd(d, lengths)
    for name, at in (("x", (200, 1, 3)), ("B", (230, 0, 5)), ("C", (240, 0, 1)), ("dout", (399, 2, 7)), ("dt", (300, 0))):
        d[name][at] = float("nan") if name in ("B", "dt") else float("inf")
    got = call_bwd(d, lengths)
    for i, (a, b) in enumerate(ref.spans(lengths)):
        if i != 1:
            for k in ("dx", "dB", "dC", "ddt"):
                assert torch.equal(got[k][:, a:b], want[k][:, a:b]), k
            assert torch.equal(got["dh0"][i], want["dh0"][i])
    assert not bool(torch.isfinite(got["dh0"][1]).all()) and kda.device_error() == 0


def test_bad_offsets_at_a_state_size_of_128():
    d = make([400, 420], 2, 1, 64, 128, seed=3)
    args = [t.cuda()[None] for t in (d["x"], d["dt"], d["B"], d["C"], d["dout"])]
    for bad in ([0, 900, 820], [0, 400, 821], [1, 400, 820], [0, -7, 820], [0, 820, 100]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        kda.kda_scan_fwd(args[0], args[1], d["A"].cuda(), args[2], args[3], cu_seqlens=cu, final_state_dtype=torch.float32)
        assert kda.device_error() == 12
        kda.kda_scan_bwd(args[0], args[1], d["A"].cuda(), args[2], args[3], args[4], cu_seqlens=cu)
        assert kda.device_error() == 12
    assert kda.device_error() == 0


def test_one_head_of_many_groups_and_many_heads_of_one():
    for H, G, N in ((5, 5, 128), (70, 1, 64), (33, 1, 128)):
        lengths = [131, 5]
        d = make(lengths, H, G, 64, N, seed=H)
        out, hT = call_fwd(d, lengths, final_state_dtype=torch.float32)
        check_fwd(d, lengths, True, out, hT)
        check_bwd(d, lengths, True, call_bwd(d, lengths))
