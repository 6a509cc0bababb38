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
