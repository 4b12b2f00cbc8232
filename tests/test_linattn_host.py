"""The linear attention's and the state pool's entry points without a GPU: every
bad argument is refused on the host, before any CUDA call.  Pointers are fake
addresses that are never followed."""
import ctypes

import pytest

from selective_state_space_ss_b200 import _native as N
from selective_state_space_ss_b200 import build as B

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    B.build()
    return N.load_library()


def _h(addr):
    return N.SSHeads(addr, 64, 64, 64)


BASE = dict(q=0x10000, k=0x20000, v=0x30000, g=0x40000, do=0x50000, s0=None, dl=None, lengths=None, o=0x60000,
            last=None, dq=0x70000, dk_=0x80000, dv_=0x90000, dg=0xa0000, ds0=None, batch=2, L=100, heads=4, hq=2,
            dk=64, dv=64, dt=N.SS_BF16, ws=0x1000000, wsb=1 << 40)


def _sizes(a):
    return a["batch"], a["L"], a["heads"], a["hq"], a["dk"], a["dv"], a["dt"]


def _fwd(lib, **over):
    a = {**BASE, **over}
    ops = [None if a[n] is None else _h(a[n]) for n in ("q", "k", "v", "g")]
    return lib.ss_linattn_fwd(*ops, 1.0, a["s0"], a["lengths"], a["o"], a["last"], *_sizes(a), a["ws"], a["wsb"], None)


def _bwd(lib, **over):
    a = {**BASE, **over}
    ops = [None if a[n] is None else _h(a[n]) for n in ("q", "k", "v", "g", "do")]
    return lib.ss_linattn_bwd(*ops, 1.0, a["s0"], a["dl"], a["lengths"], a["dq"], a["dk_"], a["dv_"], a["dg"],
                              a["ds0"], *_sizes(a), a["ws"], a["wsb"], None)


def _step(lib, **over):
    a = {**BASE, "state": 0xb0000, "pool": 2, "slots": None, **over}
    ops = [None if a[n] is None else _h(a[n]) for n in ("q", "k", "v", "g")]
    return lib.ss_linattn_step(*ops, 1.0, a["state"], a["pool"], a["slots"], a["o"], a["batch"], a["heads"], a["hq"],
                               a["dk"], a["dv"], a["dt"], None)


BAD_SIZES = [(dict(batch=0), N.SS_ERR_INVALID_ARG), (dict(heads=0), N.SS_ERR_INVALID_ARG),
             (dict(hq=3), N.SS_ERR_INVALID_ARG), (dict(hq=0), N.SS_ERR_INVALID_ARG),
             (dict(heads=2, hq=4), N.SS_ERR_INVALID_ARG), (dict(dk=0), N.SS_ERR_INVALID_ARG),
             (dict(dv=-1), N.SS_ERR_INVALID_ARG), (dict(dk=129), N.SS_ERR_UNSUPPORTED),
             (dict(dv=256), N.SS_ERR_UNSUPPORTED), (dict(dt=2), N.SS_ERR_UNSUPPORTED),
             (dict(batch=1 << 24), N.SS_ERR_INVALID_ARG), (dict(batch=1 << 40), N.SS_ERR_INVALID_ARG)]


@pytest.mark.parametrize("over,status", BAD_SIZES + [(dict(L=0), N.SS_ERR_INVALID_ARG),
                                                     (dict(L=1 << 31), N.SS_ERR_INVALID_ARG)])
@pytest.mark.parametrize("call", [_fwd, _bwd], ids=["fwd", "bwd"])
def test_sizes_and_types(lib, call, over, status):
    assert call(lib, **over) == status


@pytest.mark.parametrize("over,status", BAD_SIZES + [
    (dict(state=None), N.SS_ERR_INVALID_ARG), (dict(state=0xb0002), N.SS_ERR_INVALID_ARG),
    (dict(pool=1), N.SS_ERR_INVALID_ARG), (dict(pool=0, slots=0xc0000), N.SS_ERR_INVALID_ARG),
    (dict(slots=0xc0002), N.SS_ERR_INVALID_ARG), (dict(batch=65536, pool=65536), N.SS_ERR_INVALID_ARG),
    (dict(o=None), N.SS_ERR_INVALID_ARG), (dict(k=None), N.SS_ERR_INVALID_ARG)])
def test_step_refusals(lib, over, status):
    assert _step(lib, **over) == status


@pytest.mark.parametrize("over", [{n: None} for n in ("q", "k", "v", "g", "o")] + [
    dict(q=0x10001), dict(g=0x40002, dt=N.SS_F32), dict(o=0x60002, dt=N.SS_F32), dict(s0=0x1002), dict(last=0x1001),
    dict(lengths=0x1002), dict(o=0x60001)])
def test_fwd_pointers(lib, over):
    assert _fwd(lib, **over) == N.SS_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [{n: None} for n in ("q", "k", "v", "g", "do", "dq", "dk_", "dv_", "dg", "ws")] + [
    dict(do=0x50001), dict(dq=0x70002, dt=N.SS_F32), dict(dl=0x1002), dict(ds0=0x1002), dict(ws=0x1000010),
    dict(wsb=16), dict(lengths=0x1001)])
def test_bwd_pointers(lib, over):
    assert _bwd(lib, **over) == N.SS_ERR_INVALID_ARG


def test_a_null_tensor_struct_data_is_refused(lib):
    assert _fwd(lib, q=0) == N.SS_ERR_INVALID_ARG


def test_segments_need_their_workspace(lib):
    sizes = (1, 1 << 20, 1, 1, 64, 64, N.SS_BF16)
    need = lib.ss_linattn_workspace_bytes(*sizes)
    assert need > 0  # one head, a million tokens: cut into segments
    over = dict(batch=1, L=1 << 20, heads=1, hq=1)
    assert _fwd(lib, **over, ws=None) == N.SS_ERR_INVALID_ARG
    assert _fwd(lib, **over, wsb=need - 1) == N.SS_ERR_INVALID_ARG
    assert _fwd(lib, **over, ws=0x1000080) == N.SS_ERR_INVALID_ARG


@pytest.mark.parametrize("over,_", BAD_SIZES)
def test_workspace_queries_reject_what_the_calls_do(lib, over, _):
    a = {**BASE, **over}
    bad = ctypes.c_size_t(-1).value
    assert lib.ss_linattn_workspace_bytes(*_sizes(a)) == bad
    assert lib.ss_linattn_bwd_workspace_bytes(*_sizes(a)) == bad


def test_workspace_queries(lib):
    assert lib.ss_linattn_workspace_bytes(2, 64, 16, 16, 64, 64, N.SS_BF16) == 0  # a chunk each: nothing to cut
    small = lib.ss_linattn_bwd_workspace_bytes(2, 100, 4, 4, 64, 64, N.SS_BF16)
    shared = lib.ss_linattn_bwd_workspace_bytes(2, 100, 4, 2, 64, 64, N.SS_BF16)
    assert 0 < small < shared  # shared queries and keys add their heads' partial gradients
    with pytest.raises(N.SSError) as e:
        N.ss_linattn_workspace_bytes(1, 1, 1, 1, 129, 64, N.SS_BF16)
    assert e.value.status == N.SS_ERR_UNSUPPORTED


POOL = dict(state=0x10000, codes=0x20000, scales=0x30000, pool=4, slots=None, batch=2, rows=10, width=16)


@pytest.mark.parametrize("over,status", [({n: None}, N.SS_ERR_INVALID_ARG) for n in ("state", "codes", "scales")] + [
    (dict(state=0x10002), N.SS_ERR_INVALID_ARG), (dict(scales=0x30002), N.SS_ERR_INVALID_ARG),
    (dict(slots=0x40002), N.SS_ERR_INVALID_ARG), (dict(batch=0), N.SS_ERR_INVALID_ARG),
    (dict(rows=0), N.SS_ERR_INVALID_ARG), (dict(width=0), N.SS_ERR_INVALID_ARG),
    (dict(width=1025), N.SS_ERR_UNSUPPORTED), (dict(pool=0, slots=0x40000), N.SS_ERR_INVALID_ARG),
    (dict(batch=5), N.SS_ERR_INVALID_ARG), (dict(batch=65536, pool=1 << 20), N.SS_ERR_INVALID_ARG),
    (dict(rows=1 << 31), N.SS_ERR_INVALID_ARG), (dict(rows=1 << 28, width=64), N.SS_ERR_INVALID_ARG)])
def test_pool_refusals(lib, over, status):
    a = {**POOL, **over}
    assert lib.ss_state_store8(a["state"], a["codes"], a["scales"], a["pool"], a["slots"], a["batch"], a["rows"],
                               a["width"], None) == status
    assert lib.ss_state_load8(a["codes"], a["scales"], a["pool"], a["slots"], a["state"], a["batch"], a["rows"],
                              a["width"], None) == status


def test_the_binding_runs_on_cuda_tensors_only(lib):
    x = torch.zeros(1, 4, 2, 8)
    g = torch.zeros(1, 4, 2)
    state = torch.zeros(1, 2, 8, 8)
    codes, scales = torch.zeros(1, 2, 8, 8, dtype=torch.int8), torch.zeros(1, 2, 8)
    for call in (lambda: N.ss_linattn_fwd(x, x, x, g), lambda: N.ss_linattn_bwd(x, x, x, g, x),
                 lambda: N.ss_linattn_step(state, x[:, 0], x[:, 0], x[:, 0], g[:, 0]),
                 lambda: N.ss_state_store8(state, codes, scales), lambda: N.ss_state_load8(codes, scales)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_a_call_runs_with_its_stream_current(monkeypatch):
    """The `stream` of a call is the current one while it allocates, fills and launches (shown with stand-ins)."""
    import contextlib

    import selective_state_space_ss_b200 as ss

    log, now = [], ["main"]

    class Stream:
        def __init__(self, name):
            self.cuda_stream, self.device = name, "gpu"

    @contextlib.contextmanager
    def entered(s):
        old, now[0] = now[0], s.cuda_stream
        yield
        now[0] = old

    class T(torch.Tensor):
        is_cuda, device = True, type("D", (), {"index": 0, "__eq__": lambda a, b: b == "gpu" or a is b, "__hash__": None})()

        def record_stream(self, s):
            log.append(("used on", s.cuda_stream))

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", entered)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: Stream(now[0]))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: now[0], raising=False)
    make = lambda: torch.zeros(1).as_subclass(T)  # noqa: E731

    @N._on_its_stream
    def f(x, out=None, stream=None):
        assert stream is None
        log.append(("runs on", now[0]))
        return (make() if out is None else out, None)

    given = make()
    f(make())
    f(make(), stream=Stream("side"))
    f(make(), given, Stream("side"))
    f(make(), stream=Stream("main"))
    side = ("used on", "side")
    assert log == [("runs on", "main"), ("runs on", "side"), side, ("used on", "main"), ("runs on", "side"), side, side,
                   ("runs on", "main")]
    for name in dir(ss):  # every public call that takes one
        fn = getattr(ss, name)
        if callable(fn) and name.startswith("ss_") and name != "ss_last_device_error" and "stream" in getattr(fn, "__code__", f.__code__).co_varnames:
            assert hasattr(fn, "__wrapped__"), name


def test_the_waits_hooks_are_known(lib):
    for what in (N.SS_DEBUG_LINATTN_SPIN_LIMIT, N.SS_DEBUG_LINATTN_SKIP_PUBLISH, N.SS_DEBUG_LINATTN_SKIP_LOAD):
        assert lib.ss_debug_inject(what, 3) == N.SS_OK
    assert lib.ss_debug_inject(N.SS_DEBUG_CLEAR, 0) == N.SS_OK
    assert lib.ss_debug_inject(N.SS_DEBUG_LINATTN_SKIP_LOAD + 1, 0) == N.SS_ERR_INVALID_ARG


def test_a_backward_of_too_many_chunks_has_no_workspace(lib):
    """As for every size that the call rejects; the forward has one."""
    sizes = (1, 2**31 - 1025, 65536, 1, 8, 8, N.SS_BF16)
    none = ctypes.c_size_t(-1).value
    assert lib.ss_linattn_bwd_workspace_bytes(*sizes) == none
    assert lib.ss_linattn_workspace_bytes(*sizes) != none
    assert lib.ss_linattn_bwd_workspace_bytes(1, 2**31 - 1025, 8, 1, 8, 8, N.SS_BF16) != none
