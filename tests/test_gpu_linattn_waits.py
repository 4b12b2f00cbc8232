"""Bounded waits of the linear attention: one that runs out ends the kernel with
SS_ERR_TIMEOUT, and the context and the next call are as before."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import selective_state_space_ss_b200 as ss  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def operands(batch, L, heads, dk, dv, dtype):
    gen = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen).to(dtype)  # noqa: E731
    q, k, v = r(batch, L, heads, dk), r(batch, L, heads, dk), r(batch, L, heads, dv)
    return (q, k, v, -r(batch, L, heads).abs() * 0.1), r(batch, L, heads, dv)


def run(kind, ops, do):
    return ss.ss_linattn_fwd(*ops) if kind == "fwd" else tuple(ss.ss_linattn_bwd(*ops, do).values())


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b) if x is not None)


@pytest.fixture(autouse=True)
def hooks_cleared():
    yield
    ss.ss_debug_inject(ss.SS_DEBUG_CLEAR)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["fwd", "bwd"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_a_state_never_handed_on_times_out(dtype, kind, dk, dv):
    ops, do = operands(3, 200, 60, dk, dv, dtype)  # more heads than SMs
    want = run(kind, ops, do)
    assert ss.ss_last_device_error() == ss.SS_OK
    ss.ss_debug_inject(ss.SS_DEBUG_LINATTN_SPIN_LIMIT, 2000)
    ss.ss_debug_inject(ss.SS_DEBUG_LINATTN_SKIP_PUBLISH, 5)
    run(kind, ops, do)
    assert ss.ss_last_device_error() == ss.SS_ERR_TIMEOUT
    assert ss.ss_last_device_error() == ss.SS_OK  # read once
    assert same(run(kind, ops, do), want)
    assert ss.ss_last_device_error() == ss.SS_OK


@pytest.mark.parametrize("dtype,kind,dk,dv,L,chunk", [
    (BF16, "fwd", 64, 64, 60, 0), (BF16, "fwd", 128, 128, 2000, 0), (BF16, "bwd", 128, 64, 700, 2),
    (F32, "fwd", 128, 128, 700, 2), (F32, "bwd", 64, 64, 60, 0)])
def test_a_tile_never_loaded_times_out(dtype, kind, dk, dv, L, chunk):
    ops, do = operands(1, L, 4, dk, dv, dtype)
    want = run(kind, ops, do)
    assert ss.ss_last_device_error() == ss.SS_OK
    ss.ss_debug_inject(ss.SS_DEBUG_LINATTN_SKIP_LOAD, chunk)
    run(kind, ops, do)
    assert ss.ss_last_device_error() == ss.SS_ERR_TIMEOUT
    assert same(run(kind, ops, do), want)
    assert ss.ss_last_device_error() == ss.SS_OK


def test_cleared_settings_do_nothing():
    ops, do = operands(1, 300, 2, 64, 64, BF16)
    want = run("fwd", ops, do)
    ss.ss_debug_inject(ss.SS_DEBUG_LINATTN_SKIP_LOAD, 1)
    ss.ss_debug_inject(ss.SS_DEBUG_CLEAR)
    assert same(run("fwd", ops, do), want)
    assert ss.ss_last_device_error() == ss.SS_OK
