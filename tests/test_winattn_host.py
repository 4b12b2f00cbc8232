"""The window attention's, the cache's and the rotation's entry points without a GPU: every
bad argument is refused on the host, before any CUDA call.  Pointers are fake addresses
that are never followed."""
import ctypes
import math

import pytest

from selective_state_space_ss_b200 import _native as N
from selective_state_space_ss_b200 import build as B

torch = pytest.importorskip("torch")

BAD, NO = N.SS_ERR_INVALID_ARG, N.SS_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    B.build()
    return N.load_library()


BASE = dict(q=0x10000, k=0x20000, v=0x30000, o=0x40000, do=0x50000, lse=0x60000, lengths=None, dq=0x70000, dk=0x80000,
            dv=0x90000, window=16, sinks=2, scale=0.125, batch=2, L=100, heads=4, hk=2, d=64, dt=N.SS_BF16, ws=0x1000000,
            wsb=1 << 40, kp=0xa0000, vp=0xb0000, pages=10, page=16, table=0xc0000, per=4, starts=0xd0000, counts=None,
            inv=0xe0000, half=32, qo=0xf0000, ko=None, inter=0, inverse=0)


def _h(addr):
    return None if addr is None else N.SSHeads(addr, 64, 64, 64)


def _sizes(a):
    return a["batch"], a["L"], a["heads"], a["hk"], a["d"], a["dt"]


def _fwd(lib, **over):
    a = {**BASE, **over}
    return lib.ss_winattn_fwd(_h(a["q"]), _h(a["k"]), _h(a["v"]), a["window"], a["sinks"], a["scale"], a["lengths"], a["o"],
                              a["lse"], *_sizes(a), None)


def _bwd(lib, **over):
    a = {**BASE, **over}
    return lib.ss_winattn_bwd(_h(a["q"]), _h(a["k"]), _h(a["v"]), _h(a["o"]), a["lse"], _h(a["do"]), a["window"], a["sinks"],
                              a["scale"], a["lengths"], a["dq"], a["dk"], a["dv"], *_sizes(a), a["ws"], a["wsb"], None)


def _cache(a):
    return N.SSPages(_h(a["kp"]) or N.SSHeads(), _h(a["vp"]) or N.SSHeads(), a["pages"], a["page"], a["table"], a["per"])


def _step(lib, **over):
    a = {**BASE, "lengths": 0x110000, "L": 1, **over}
    return lib.ss_winattn_step(_h(a["q"]), _cache(a), a["lengths"], a["window"], a["sinks"], a["scale"], a["o"], *_sizes(a),
                               None)


def _append(lib, **over):
    a = {**BASE, **over}
    return lib.ss_kv_append(_h(a["k"]), _h(a["v"]), _h(a["q"]), _cache(a), a["starts"], a["counts"],
                            N.SSRotation(a["inv"], a["half"], a["inter"]), a["qo"], a["ko"], *_sizes(a), None)


def _rotate(lib, **over):
    a = {**BASE, "ko": 0x120000, **over}
    return lib.ss_rotate(_h(a["q"]), _h(a["k"]), a["starts"], a["counts"], N.SSRotation(a["inv"], a["half"], a["inter"]),
                         a["inverse"], a["qo"], a["ko"], *_sizes(a), None)


ALL = [_fwd, _bwd, _step, _append, _rotate]
SIZES = [(dict(batch=0), BAD), (dict(L=0), BAD), (dict(heads=0), BAD), (dict(hk=0), BAD), (dict(hk=3), BAD),
         (dict(heads=2, hk=4), BAD), (dict(d=0), BAD), (dict(dt=2), NO), (dict(batch=1 << 24), BAD), (dict(batch=1 << 40), BAD),
         (dict(L=1 << 31), BAD), (dict(L=(1 << 31) - 1024), BAD), (dict(heads=65537, hk=1), BAD),
         (dict(L=1 << 30, heads=8), BAD)]


@pytest.mark.parametrize("over,status", SIZES)
@pytest.mark.parametrize("call", ALL)
def test_sizes_and_types(lib, call, over, status):
    assert call(lib, **over) == status


@pytest.mark.parametrize("call,d", [(_fwd, 129), (_bwd, 129), (_step, 129), (_append, 1025), (_rotate, 1025)])
def test_widths(lib, call, d):
    assert call(lib, d=d) == NO


@pytest.mark.parametrize("over", [dict(window=0), dict(window=-3), dict(sinks=-1), dict(scale=0.0), dict(scale=-1.0),
                                  dict(scale=math.inf), dict(scale=math.nan), dict(q=None), dict(q=0), dict(q=0x10001),
                                  dict(q=0x10002, dt=N.SS_F32), dict(o=None), dict(o=0x40001)])
@pytest.mark.parametrize("call", [_fwd, _bwd, _step])
def test_masks_and_scales(lib, call, over):
    assert call(lib, **over) == BAD


@pytest.mark.parametrize("over", [dict(k=None), dict(v=None), dict(v=0x30001), dict(lse=0x60002), dict(lengths=0x1002)])
@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_prompt_pointers(lib, call, over):
    assert call(lib, **over) == BAD


@pytest.mark.parametrize("over", [{n: None} for n in ("do", "lse", "dq", "dk", "dv", "ws")] + [
    dict(do=0x50001), dict(dq=0x70001), dict(dk=0x80002, dt=N.SS_F32), dict(ws=0x1000010), dict(wsb=16)])
def test_bwd_pointers(lib, over):
    assert _bwd(lib, **over) == BAD


PAGES = [dict(kp=None), dict(vp=None), dict(vp=0xb0001), dict(pages=0), dict(pages=1 << 31), dict(page=0), dict(per=0),
         dict(table=None), dict(table=0xc0002), dict(page=1 << 20, per=1 << 11)]


@pytest.mark.parametrize("over", PAGES + [dict(lengths=None), dict(lengths=0x1002), dict(batch=65536, heads=1, hk=1),
                                          dict(L=1 << 18, heads=4, hk=2)])
def test_step_refusals(lib, over):
    assert _step(lib, **over) == BAD


@pytest.mark.parametrize("over", PAGES + [
    dict(starts=None), dict(starts=0xd0001), dict(counts=0x1002), dict(k=None), dict(v=None), dict(qo=None), dict(q=None),
    dict(qo=0xf0001), dict(ko=0x120001), dict(half=33), dict(half=-1), dict(inv=None), dict(inv=0xe0002), dict(q=0x10001)])
def test_append_refusals(lib, over):
    assert _append(lib, **over) == BAD


@pytest.mark.parametrize("over", [dict(q=None), dict(qo=None), dict(ko=None), dict(k=None), dict(half=33), dict(half=-1),
                                  dict(inv=None), dict(starts=0xd0001), dict(counts=0x1001)])
def test_rotate_refusals(lib, over):
    assert _rotate(lib, **over) == BAD


def test_null_structures(lib):
    a = BASE
    assert lib.ss_winattn_step(_h(a["q"]), None, 0x110000, 16, 2, 1.0, a["o"], *_sizes(a), None) == BAD
    rot = N.SSRotation(a["inv"], 32, 0)
    assert lib.ss_kv_append(_h(a["k"]), _h(a["v"]), None, None, a["starts"], None, rot, None, None, *_sizes(a), None) == BAD
    assert lib.ss_kv_append(_h(a["k"]), _h(a["v"]), None, _cache(a), a["starts"], None, None, None, None, *_sizes(a), None) == BAD
    assert lib.ss_rotate(_h(a["q"]), None, None, None, None, 0, a["qo"], None, *_sizes(a), None) == BAD


@pytest.mark.parametrize("over", [o for o, _ in SIZES] + [dict(d=129), dict(window=0), dict(sinks=-1)])
def test_the_workspace_query_rejects_what_the_call_does(lib, over):
    a = {**BASE, **over}
    assert lib.ss_winattn_bwd_workspace_bytes(*_sizes(a)[:5], a["window"], a["sinks"], a["dt"]) == ctypes.c_size_t(-1).value


def test_workspace_queries(lib):
    need = lambda L, window, sinks: N.ss_winattn_bwd_workspace_bytes(2, L, 4, 2, 64, window, sinks, N.SS_BF16)  # noqa: E731
    assert need(100, 16, 0) == need(100, 16, 3) >= 2 * 4 * 100 * 4  # a number for every query's row
    assert need(20000, 128, 4) > need(20000, 128, 0)  # the sinks' gradients come in pieces
    assert need(20000, 128, 20000) == need(20000, 20000, 0) == need(20000, 1 << 40, 1 << 40)  # all the same mask
    # many sinks: a bounded number of pieces
    assert need(20000, 16, 10000) < 2 * 4 * 20000 * 4 + 5 * 2 * 2 * 2 * 10240 * 64 * 4
    assert _bwd(lib, L=20000, wsb=need(20000, 16, 2) - 1) == BAD
    with pytest.raises(N.SSError) as e:
        N.ss_winattn_bwd_workspace_bytes(1, 1, 1, 1, 129, 1, 0, N.SS_BF16)
    assert e.value.status == NO


def test_the_binding_runs_on_cuda_tensors_only(lib):
    x, lse, n = torch.zeros(1, 4, 2, 8), torch.zeros(1, 2, 4), torch.zeros(1, dtype=torch.int32)
    pages, table, f = torch.zeros(3, 4, 2, 8), torch.zeros(1, 1, dtype=torch.int32), torch.ones(4)
    for call in (lambda: N.ss_winattn_fwd(x, x, x, 4), lambda: N.ss_winattn_bwd(x, x, x, x, lse, x, 4),
                 lambda: N.ss_winattn_step(x, pages, pages, table, n, 4), lambda: N.ss_rotate(x, f),
                 lambda: N.ss_kv_append(x, x, pages, pages, table, n)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_the_waits_hook_is_known(lib):
    assert lib.ss_debug_inject(N.SS_DEBUG_WINATTN_SKIP_LOAD, 3) == N.SS_OK
    assert lib.ss_debug_inject(N.SS_DEBUG_CLEAR, 0) == N.SS_OK
    assert lib.ss_debug_inject(N.SS_DEBUG_WINATTN_SKIP_LOAD + 1, 0) == BAD
