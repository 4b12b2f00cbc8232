"""Bounded waits of the window attention's tensor-core kernels: one that runs out ends the
kernel with SS_ERR_TIMEOUT, and the context and the next call are as before."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import selective_state_space_ss_b200 as ss  # noqa: E402


def operands(L, d):
    gen = torch.Generator(device="cuda").manual_seed(4)
    return tuple(torch.randn(1, L, n, d, device="cuda", generator=gen).bfloat16() for n in (4, 2, 2, 4))


@pytest.fixture(autouse=True)
def hooks_cleared():
    yield
    ss.ss_debug_inject(ss.SS_DEBUG_CLEAR)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("L,tile", [(100, 0), (700, 2), (700, 5)])
@pytest.mark.parametrize("kind", ["fwd", "bwd"])
@pytest.mark.parametrize("ragged", [False, True])
def test_a_tile_never_loaded_times_out(kind, L, tile, d, ragged):
    q, k, v, do = operands(L, d)
    lengths = torch.tensor([L - 9], dtype=torch.int32, device="cuda") if ragged else None
    o, lse = ss.ss_winattn_fwd(q, k, v, 200, sinks=3, lengths=lengths)

    def run():
        if kind == "fwd":
            return ss.ss_winattn_fwd(q, k, v, 200, sinks=3, lengths=lengths)
        return tuple(ss.ss_winattn_bwd(q, k, v, o, lse, do, 200, sinks=3, lengths=lengths).values())

    want = run()
    assert ss.ss_last_device_error() == ss.SS_OK
    ss.ss_debug_inject(ss.SS_DEBUG_WINATTN_SKIP_LOAD, tile)
    run()
    assert ss.ss_last_device_error() == ss.SS_ERR_TIMEOUT
    assert ss.ss_last_device_error() == ss.SS_OK  # read once
    assert all(torch.equal(x, y) for x, y in zip(run(), want))
    assert ss.ss_last_device_error() == ss.SS_OK


def test_cleared_settings_do_nothing():
    q, k, v, _ = operands(300, 64)
    want = ss.ss_winattn_fwd(q, k, v, 100)
    ss.ss_debug_inject(ss.SS_DEBUG_WINATTN_SKIP_LOAD, 1)
    ss.ss_debug_inject(ss.SS_DEBUG_CLEAR)
    assert all(torch.equal(x, y) for x, y in zip(ss.ss_winattn_fwd(q, k, v, 100), want))
    assert ss.ss_last_device_error() == ss.SS_OK
