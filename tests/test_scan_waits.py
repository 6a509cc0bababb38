"""The bounded waits of the scan's three tcgen05 kernels, with no GPU fault: in the test-only build (``-DKDA_TEST_HOOKS``:
100 ms wait limit) the gates of one tile or head are made but not signalled, so that the waits for them run out. The error
word reports it, the kernel winds down, and the next call on the same device is correct."""
import ctypes
import subprocess

import pytest
import torch

import kimi_delta_attention_27_b200 as kda
import test_scan as base
from kimi_delta_attention_27_b200 import build

OK, TIMEOUT = 0, 9
HOOKS = ("kda_test_set_scan_tc_stall", "kda_test_set_scan_tc_state_stall", "kda_test_set_scan_tc_bwd_stall")


def exported(path):
    return subprocess.run(["nm", "-D", "--defined-only", path], check=True, capture_output=True, text=True).stdout


def test_only_the_test_library_has_the_hooks():
    build.build()
    product, hooks = exported(kda.LIB_PATH), exported(build.build_test_hooks())
    assert all(h in hooks and h not in product for h in HOOKS) and " T kda_scan_fwd" in hooks


# kernel's hook, what is stalled, direction, lengths, heads, state size
# (pieces of cut sequences have two tiles)
CASES = {
    "outputs_first_tile": (HOOKS[0], 0, "fwd", [400] * 3, 4, 128),
    "outputs_later_tile": (HOOKS[0], 1, "fwd", [700] * 3, 3, 128),
    "states_first_tile": (HOOKS[1], 0, "fwd", [2000], 1, 64),
    "states_later_tile": (HOOKS[1], 1, "fwd", [2000], 2, 128),
    "states_both_directions": (HOOKS[1], 1, "bwd", [300], 3, 64),
    "gradients_first_head": (HOOKS[2], 0, "bwd", [300], 4, 128),
    "gradients_later_head": (HOOKS[2], 1, "bwd", [148 * 128], 2, 64),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_scan_wait_that_runs_out_is_reported_and_the_device_keeps_working(name, monkeypatch):
    hook, at, way, lengths, H, N = CASES[name]
    lib = kda.load_library(path=build.build_test_hooks())
    d = base.make(lengths, H, 1, 64, N, seed=5)
    run = (lambda: base.call_fwd(d, lengths, final_state_dtype=torch.float32)) if way == "fwd" else \
        (lambda: tuple(base.call_bwd(d, lengths).values()))  # noqa: E731
    want = run()                                        # the product library's
    torch.cuda.synchronize()
    set_stall = getattr(lib, hook)
    set_stall.restype, set_stall.argtypes = ctypes.c_int, [ctypes.c_int]
    monkeypatch.setattr(kda, "_lib", lib)
    assert kda.device_error() == OK and set_stall(at) == 0
    try:
        run()                                           # enqueued; the failure is on the device
        assert kda.device_error() == TIMEOUT and kda.device_error() == OK
    finally:
        set_stall(-1)
    got = run()
    assert kda.device_error() == OK and all(torch.equal(a, b) for a, b in zip(got, want))
    monkeypatch.undo()
    assert all(torch.equal(a, b) for a, b in zip(run(), want)) and kda.device_error() == OK
