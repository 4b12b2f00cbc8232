"""Calls as a program makes them: captured and replayed where the sequence or the heads are
cut, the first call of a process inside a capture, states advanced in place, two captured
graphs at once, and a training step and a decoding loop in one graph each."""
import ctypes
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import selective_state_space_ss_b200 as ss  # noqa: E402
from selective_state_space_ss_b200 import _native as N  # noqa: E402
from tests.test_gpu_linattn import BF16, F32, bwd, check_fwd, fwd, make  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
both = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
CUTS = {"whole": (2, 150, 2, 2), "segments": (1, 1500, 2, 1), "workers": (2, 200, 80, 80)}
cuts = pytest.mark.parametrize("cut", list(CUTS))


def same(a, b):
    return all((x is None and y is None) or torch.equal(x, y) for x, y in zip(a, b))


@both
@cuts
def test_captured_and_replayed(dtype, cut):
    x, r = make(*CUTS[cut], 64, 64, dtype)
    do, dlast = r(*x["v"].shape).to(dtype), torch.zeros_like(x["s0"])
    both_ways = lambda: (*fwd(x), *bwd(x, do, dlast).values())  # noqa: E731
    both_ways()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both_ways()
    for seed in (7, 8):
        y, r2 = make(*CUTS[cut], 64, 64, dtype, seed=seed)
        for n in x:
            x[n].copy_(y[n])
        do.copy_(r2(*do.shape))
        dlast.copy_(r2(*dlast.shape))
        graph.replay()
        graph.replay()
        assert same(out, both_ways())
        assert ss.ss_last_device_error() == ss.SS_OK


@cuts
def test_two_graphs_at_once(cut):
    """Each captured call has the workspace of its own capture."""
    xs = [make(*CUTS[cut], 64, 64, BF16, seed=s)[0] for s in (1, 2)]
    want, graphs, outs = [fwd(x) for x in xs], [], []
    torch.cuda.synchronize()
    for x in xs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(fwd(x))
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(4):
        for o in outs:
            o[0].zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(outs, want))
    assert ss.ss_last_device_error() == ss.SS_OK


@both
@cuts
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_states_in_place(dtype, cut, dk, dv):
    """last_state_out over initial_state, and through the C ABI dinitial_state over dlast_state."""
    x, r = make(*CUTS[cut], dk, dv, dtype)
    want_o, want = fwd(x)
    check_fwd(x, want_o, want)
    state = x["s0"].clone()
    o, last = fwd({**x, "s0": state}, last_state_out=state)
    assert last is state and torch.equal(o, want_o) and torch.equal(state, want)

    do, buf = r(*x["v"].shape).to(dtype), r(*x["s0"].shape)
    grads = bwd(x, do, buf)
    lib = N.load_library()
    device, ops, sizes = N._linattn_operands("bwd", x["q"], x["k"], x["v"], x["g"])
    ops.append(N._heads4("do", do, device, dtype, do.shape))
    outs = [torch.empty_like(grads[n]) for n in ("dq", "dk", "dv", "dlog_decay")]
    ws = torch.empty(ss.ss_linattn_bwd_workspace_bytes(*sizes), dtype=torch.uint8, device="cuda")
    st = lib.ss_linattn_bwd(*[ctypes.byref(t) for t in ops], 1.0, x["s0"].data_ptr(), buf.data_ptr(), None,
                            *[t.data_ptr() for t in outs], buf.data_ptr(), *sizes, ws.data_ptr(), ws.numel(),
                            torch.cuda.current_stream().cuda_stream)
    assert st == ss.SS_OK and torch.equal(buf, grads["dinitial_state"])
    assert same(outs, [grads[n] for n in ("dq", "dk", "dv", "dlog_decay")])


@both
def test_a_decoding_loop_in_one_graph(dtype):
    """Sixteen tokens by slots, the states parked and woken in between, in one graph."""
    x, r = make(3, 16, 4, 2, 64, 48, dtype, state=False)
    pool, before = r(5, 4, 64, 48), None
    slots = torch.tensor([4, 0, -1], dtype=torch.int32, device="cuda")
    codes, scales = torch.zeros(2, 4, 64, 48, dtype=torch.int8, device="cuda"), torch.zeros(2, 4, 64, device="cuda")
    here = torch.tensor([1], dtype=torch.int32, device="cuda")
    start = pool.clone()

    def loop():
        out = []
        for t in range(16):
            out.append(ss.ss_linattn_step(pool, *[x[n][:, t] for n in ("q", "k", "v", "g")], slots=slots))
            if t == 7:
                ss.ss_state_store8(pool[4:5], codes, scales, slots=here)
                pool[4:5] = ss.ss_state_load8(codes, scales, slots=here)
        return out

    want = loop()
    after = pool.clone()
    pool.copy_(start)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = loop()
    pool.copy_(start)
    graph.replay()
    assert same(got, want) and torch.equal(pool, after) and not got[0][2].any()


def test_the_first_call_of_a_process_in_a_capture():
    """Nothing of the library ran before: tensor maps, attributes and modules are set up while capturing."""
    code = """
import torch, sys
sys.path.insert(0, ".")
import selective_state_space_ss_b200 as ss
torch.manual_seed(0)
q, k, v, do = (torch.randn(1, 1500, 2, 64, device="cuda").bfloat16() for _ in range(4))
g = -torch.rand(1, 1500, 2, device="cuda").bfloat16()
state = torch.randn(1, 2, 64, 64, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
def all_of_it():
    o, last = ss.ss_linattn_fwd(q, k, v, g)
    grads = ss.ss_linattn_bwd(q, k, v, g, do)
    s = state.clone()
    o1 = ss.ss_linattn_step(s, q[:, 0], k[:, 0], v[:, 0], g[:, 0])
    return [o, last, o1, s, *(t for t in grads.values() if t is not None)]
with torch.cuda.graph(graph):
    got = all_of_it()
graph.replay()
want = all_of_it()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert ss.ss_last_device_error() == ss.SS_OK
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
