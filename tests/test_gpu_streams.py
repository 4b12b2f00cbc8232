"""`stream=` of the Python calls: what a call allocates, fills and launches is in that stream's
order, whatever the current stream still has to do, and the allocator gives its workspace to
nobody else meanwhile."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import selective_state_space_ss_b200 as ss  # noqa: E402

LONG = 30_000_000  # cycles, 15 to 25 ms: longer than any of the calls


def linattn(heads=2, L=300, batch=2):
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    q, k, v, do = (r(batch, L, heads, 64).bfloat16() for _ in range(4))
    return (q, k, v, (-0.1 * r(batch, L, heads).abs()).bfloat16()), do, r(batch, heads, 64, 64)


def scan(batch=2, dim=64, L=40000, N=16):
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    return r(batch, dim, L), r(batch, dim, L), -r(dim, N).abs(), r(batch, N, L), r(batch, N, L)


def tensors(out):
    out = out.values() if isinstance(out, dict) else out if isinstance(out, tuple) else (out,)
    return [x for x in out if x is not None]


def calls():
    """name -> a call that takes `stream`; each allocates its outputs, a workspace or both, and changes no input."""
    ops, do, state = linattn()
    lengths = torch.tensor([300, 77], dtype=torch.int32, device="cuda")
    wide, wide_do, _ = linattn(heads=90)
    long, long_do, _ = linattn(heads=1, L=3000, batch=1)
    token, slots = [x[:, 0] for x in ops], torch.tensor([1, -1], dtype=torch.int32, device="cuda")
    codes, scales = torch.zeros(2, 2, 64, 64, dtype=torch.int8, device="cuda"), torch.zeros(2, 2, 64, device="cuda")
    ss.ss_state_store8(state, codes, scales)
    u, delta, A, B, C = scan()
    small = scan(L=200)
    dy = torch.randn_like(small[0])
    return {
        "fwd_lengths": lambda **k: ss.ss_linattn_fwd(*ops, lengths=lengths, **k),
        "fwd_segments": lambda **k: ss.ss_linattn_fwd(*long, **k),
        "fwd_workers": lambda **k: ss.ss_linattn_fwd(*wide, **k),
        "bwd_lengths": lambda **k: ss.ss_linattn_bwd(*ops, do, lengths=lengths, **k),
        "bwd_segments": lambda **k: ss.ss_linattn_bwd(*long, long_do, **k),
        "bwd_workers": lambda **k: ss.ss_linattn_bwd(*wide, wide_do, **k),
        "step_slots": lambda **k: ss.ss_linattn_step(state.clone() if not k else steady, *token, slots=slots, **k),
        "load8": lambda **k: ss.ss_state_load8(codes, scales, **k),
        "scan": lambda **k: ss.ss_scan_fwd(u, delta, A, B, C, **k),
        "scan_bwd": lambda **k: ss.ss_scan_bwd(*small, dy, **k),
    }


steady = None  # the states of step_slots, advanced in place


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", ["fwd_lengths", "fwd_segments", "fwd_workers", "bwd_lengths", "bwd_segments", "bwd_workers",
                                  "step_slots", "load8", "scan", "scan_bwd"])
def test_the_current_stream_busy(name, raw):
    """The current stream is kept busy ahead of the call: a fill that waited there would come after the kernel."""
    global steady
    call = calls()[name]
    want = tensors(call())
    steady = linattn()[2]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    got = tensors(call(stream=side.cuda_stream if raw else side))
    side.synchronize()
    torch.cuda.synchronize()
    assert ss.ss_last_device_error() == ss.SS_OK
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["fwd_segments", "fwd_workers", "bwd_lengths", "bwd_segments", "bwd_workers", "scan", "scan_bwd"])
def test_the_workspace_is_not_given_away(name):
    """The given stream is kept busy ahead of the call, and the current one allocates and fills meanwhile."""
    call = calls()[name]
    want = tensors(call())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
    got = tensors(call(stream=side))
    junk = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in [1 << k for k in range(10, 28)] * 2]
    torch.cuda.synchronize()
    assert ss.ss_last_device_error() == ss.SS_OK and len(junk) == 36
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_an_output_freed_while_the_current_stream_reads_it():
    """Dropped by the caller with a read of it still queued: the given stream's next call does not write over it."""
    ops, _, _ = linattn()
    lengths = torch.tensor([300, 77], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    want = ss.ss_linattn_fwd(*ops, lengths=lengths)[0].clone()
    side.wait_stream(torch.cuda.current_stream())
    o, last = ss.ss_linattn_fwd(*ops, lengths=lengths, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(LONG)
    copy = torch.empty_like(o)
    copy.copy_(o)
    del o, last
    for _ in range(4):
        ss.ss_linattn_fwd(ops[2], ops[0], ops[1], ops[3], lengths=lengths, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


@pytest.mark.parametrize("name", ["linattn", "scan"])
def test_an_operand_dropped_right_after_the_call(name):
    """A temporary of the caller, with the given stream still busy: the current stream's next tensors do not take its place."""
    ops = linattn(L=1000)[0] if name == "linattn" else scan(L=2000)
    fn = ss.ss_linattn_fwd if name == "linattn" else ss.ss_scan_fwd
    want = tensors(fn(*ops))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    temporary = [x.clone() for x in ops]
    sizes = [x.numel() * x.element_size() for x in ops]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LONG)
    got = tensors(fn(*temporary, stream=side))
    del temporary
    junk = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes * 2]
    torch.cuda.synchronize()
    assert len(junk) and ss.ss_last_device_error() == ss.SS_OK
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_branch_of_a_captured_graph():
    """Inside a capture, on a stream that was forked from the captured one and joins it again."""
    ops, do, _ = linattn(heads=90)
    lengths = torch.tensor([300, 77], dtype=torch.int32, device="cuda")
    want = [*tensors(ss.ss_linattn_fwd(*ops, lengths=lengths)), *tensors(ss.ss_linattn_bwd(*ops, do, lengths=lengths))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        got = tensors(ss.ss_linattn_fwd(*ops, lengths=lengths, stream=side))
        got += tensors(ss.ss_linattn_bwd(*[x.clone() for x in ops], do, lengths=lengths))
        main.wait_stream(side)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert ss.ss_last_device_error() == ss.SS_OK and len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_refusals():
    ops, _, _ = linattn()
    with pytest.raises(ValueError):
        ss.ss_linattn_fwd(*[x.cpu() for x in ops], stream=torch.cuda.Stream())
    with pytest.raises((ValueError, TypeError)):
        ss.ss_linattn_fwd(*ops, stream="side")
