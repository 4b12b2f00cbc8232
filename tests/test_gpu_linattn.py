"""ss_linattn_fwd / _bwd / _step on the GPU against the recurrence in 64 bits.

What a result may be off by is counted, element by element, from M, the same sums
over magnitudes (every product of absolute values, decays as they are):

  products    what the kernel forms itself (scores times decays, weighted keys, the
              state) enters a product as bf16 planes, of 16 bits for bf16 inputs and
              24 for fp32: each a relative error of 2^-16 or 2^-24 of a term.  At
              most three stand in a row (weighted key, state, or score and decay):
              4 u M, u = 2^-16 or, with the dropped products of planes, 4 * 2^-24
  sums        fp32 on the tensor core, each addition 2^-23: at most dk / 16 or 4
              steps times six plane products, twice, and one for each chunk passed
              and the 16 terms inside a step: (6 * (dk / 16 + 4) + 32 + chunks) 2^-23 M
  decays      exponents of magnitude up to |G| are fp32 numbers and ex2 is good to
              2^-22: 2^-22 + 2^-24 |G| ln 2 of a term, below 2^-20 while |G| < 20;
              a term with a larger |G| is e^-20 of its size and its error with it
  the end     one rounding to the output's type: 2^-8 of the value in bf16
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import selective_state_space_ss_b200 as ss  # noqa: E402
from tests import linattn_plain as P  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def slack(dtype, d, L):
    u = 2.0 ** -16 if dtype == BF16 else 4 * 2.0 ** -24
    return 4 * u + (6 * (d / 16 + 4) + 32 + L / 64) * 2.0 ** -23 + 2.0 ** -20


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check(name, got, ref, by, dtype, d, L):
    got = got.double()
    assert torch.isfinite(got).all(), name
    bound = (1 + half_step(dtype)) * slack(*(d if isinstance(d, tuple) else (dtype, d)), L) * by + half_step(dtype) * ref.abs()
    over = (got - ref).abs() - bound - 1e-37
    assert (over <= 0).all(), f"{name}: {float(over.max()):.3g} over a bound of {float(bound.max()):.3g}"


def make(batch, L, heads, qk_heads, dk, dv, dtype, state=True, seed=0, strided=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    x = {}
    if strided:  # slices of one projection's output, at an odd offset
        wide = r(batch, L, 2 * qk_heads * dk + heads * dv + 1).to(dtype)[..., 1:]
        a, b = qk_heads * dk, 2 * qk_heads * dk
        x["q"], x["k"] = wide[..., :a].unflatten(-1, (qk_heads, dk)), wide[..., a:b].unflatten(-1, (qk_heads, dk))
        x["v"] = wide[..., b:].unflatten(-1, (heads, dv))
    else:
        x["q"], x["k"] = r(batch, L, qk_heads, dk).to(dtype), r(batch, L, qk_heads, dk).to(dtype)
        x["v"] = r(batch, L, heads, dv).to(dtype)
    x["g"] = (-0.3 * r(batch, L, heads).abs() * torch.rand(heads, device="cuda", generator=gen)).to(dtype)
    x["s0"] = r(batch, heads, dk, dv) if state else None
    return x, r


def fwd(x, **kw):
    return ss.ss_linattn_fwd(x["q"], x["k"], x["v"], x["g"], initial_state=x["s0"], **kw)


def check_fwd(x, o, last, scale=1.0, lengths=None):
    dtype, L, dk = x["q"].dtype, x["g"].shape[1], x["q"].shape[3]
    ro, rl = P.forward(x["q"], x["k"], x["v"], x["g"], scale, x["s0"], lengths)
    mag = [None if t is None else t.double().abs() for t in (x["q"], x["k"], x["v"], x["s0"])]
    mo, ml = P.forward(mag[0], mag[1], mag[2], x["g"], abs(scale), mag[3], lengths)
    check("o", o, ro, mo, dtype, dk, L)
    check("last_state", last, rl, ml, F32, (dtype, dk), L)


DIMS = [(64, 64), (128, 64), (64, 128), (128, 128), (16, 16), (37, 21), (1, 1), (100, 65), (8, 120)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("L", [1, 63, 64, 65, 203])
def test_fwd(dtype, dk, dv, L):
    x, _ = make(2, L, 4, 2, dk, dv, dtype, state=L != 64)
    o, last = fwd(x, scale=dk ** -0.5)
    assert ss.ss_last_device_error() == ss.SS_OK
    assert o.dtype == dtype and last.dtype == F32
    check_fwd(x, o, last, scale=dk ** -0.5)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("qk_heads,heads", [(1, 1), (1, 6), (3, 6), (6, 6)])
def test_fwd_strided_shared_heads(dtype, qk_heads, heads):
    x, _ = make(2, 130, heads, qk_heads, 40, 24, dtype, strided=True)
    check_fwd(x, *fwd(x))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_fwd_segments(dtype):
    """One head and many chunks: the sequence is cut and joined."""
    sizes = (1, 2600, 1, 1, 64, 32)
    x, _ = make(*sizes, dtype)
    assert ss.ss_linattn_workspace_bytes(*sizes, ss.SS_BF16 if dtype == BF16 else ss.SS_F32) > 0
    check_fwd(x, *fwd(x))
    lengths = torch.tensor([1111], dtype=torch.int32, device="cuda")  # later segments are empty
    check_fwd(x, *fwd(x, lengths=lengths), lengths=lengths)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("ragged", [False, True])
def test_more_heads_than_sms(dtype, ragged):
    """180 heads: every SM takes an equal range of all chunks, heads are cut between two."""
    x, r = make(3, 200, 60, 20, 32, 48, dtype)
    assert ss.ss_linattn_workspace_bytes(3, 200, 60, 20, 32, 48, ss.SS_BF16 if dtype == BF16 else ss.SS_F32) > 0
    lengths = torch.tensor([200, 64, 131], dtype=torch.int32, device="cuda") if ragged else None
    o, last = fwd(x, lengths=lengths)
    assert ss.ss_last_device_error() == ss.SS_OK
    check_fwd(x, o, last, lengths=lengths)
    do, dlast = r(3, 200, 60, 48).to(dtype), r(3, 60, 32, 48)
    got = bwd(x, do, dlast, lengths=lengths)
    assert ss.ss_last_device_error() == ss.SS_OK
    check_bwd(x, do, dlast, got, 1.0, lengths)


def test_offsets_beyond_32_bits():
    """Tokens 8.4 million elements apart: the last ones lie beyond 2^31 elements."""
    step, L = 8_400_000, 300
    base = torch.empty(step * L, dtype=BF16, device="cuda")
    x, r = make(1, L, 2, 2, 64, 64, BF16)
    at = 0
    for n in ("q", "k", "v"):
        view = base[at:].as_strided((1, L, 2, 64), (0, step, 64, 1))
        view.copy_(x[n])
        x[n], at = view, at + 128
    far = base[at:].as_strided((1, L, 2), (0, step, 1))
    far.copy_(x["g"])
    x["g"] = far
    o, last = fwd(x)
    check_fwd(x, o, last)
    do = base[at + 8:].as_strided((1, L, 2, 64), (0, step, 64, 1))
    do.copy_(r(1, L, 2, 64))
    check_bwd(x, do, None, bwd(x, do), 1.0)


def test_two_calls_at_once():
    """Two streams, each with more heads than SMs, on workspaces of their own."""
    xs = [make(2, 400, 90, 90, 64, 64, BF16, seed=s)[0] for s in (1, 2)]
    want = [fwd(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(4):
        got = []
        for x, st in zip(xs, streams):
            with torch.cuda.stream(st):
                got.append(fwd(x))
        torch.cuda.synchronize()
        for (o, last), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(last, wl)
    assert ss.ss_last_device_error() == ss.SS_OK


def test_a_nan_stays_in_its_head_and_row():
    x, _ = make(2, 200, 4, 2, 64, 64, BF16)
    clean, last_clean = fwd(x)
    for n, h in (("v", 1), ("k", 1), ("q", 1)):
        bad = {m: t if t is None else t.clone() for m, t in x.items()}
        bad[n][1, 70, h] = float("nan")
        heads = [1] if n == "v" else [2, 3]  # heads 2 and 3 read shared head 1
        o, last = fwd(bad)
        others = [h2 for h2 in range(4) if h2 not in heads]
        assert torch.equal(o[0], clean[0]) and torch.equal(last[0], last_clean[0])
        assert torch.equal(o[1][:, others], clean[1][:, others]) and torch.equal(last[1, others], last_clean[1, others])
        assert torch.equal(o[1, :64], clean[1, :64])  # the chunk before
        assert o[1, 70][heads].isnan().all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_fwd_lengths_and_rows_behind(dtype):
    x, _ = make(6, 150, 2, 1, 64, 64, dtype)
    lengths = torch.tensor([0, 1, 64, 150, 900, -3], dtype=torch.int32, device="cuda")
    real = lengths.clamp(0, 150)
    for n in ("q", "k", "v", "g"):  # nothing behind a row's end is read
        for b, e in enumerate(real.tolist()):
            x[n][b, e:] = float("nan")
    o_out = torch.full((6, 150, 2, 64), 7.0, dtype=dtype, device="cuda")
    o, last = fwd(x, lengths=lengths, o_out=o_out)
    assert o is o_out
    for b, e in enumerate(real.tolist()):
        assert (o[b, e:] == 7).all()
        o[b, e:] = 0
        for n in ("q", "k", "v", "g"):
            x[n][b, e:] = 0
    check_fwd(x, o, last, lengths=real)
    assert torch.equal(last[0], x["s0"][0]) and torch.equal(last[5], x["s0"][5])
    o2, _ = fwd(x, lengths=lengths)
    assert torch.equal(o2, o)  # allocated here: zero behind the end


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", ["none", "reset", "deep", "grow", "mixed"])
def test_fwd_extreme_decays(dtype, kind):
    x, _ = make(1, 140, 2, 2, 32, 32, dtype)
    g = x["g"]
    if kind == "none":
        g.zero_()
    elif kind == "reset":
        g[0, [0, 5, 63, 64, 100]] = -float("inf")
    elif kind == "deep":
        g.fill_(-60.0)
    elif kind == "grow":
        g.fill_(0.03125)
    else:  # a reset-like token among slow ones: differences of large sums
        g.fill_(-0.0078125)
        g[0, 20] = -3e4
        g[0, 90] = -torch.finfo(dtype).max
    o, last = fwd(x)
    check_fwd(x, o, last)


def test_fwd_state_in_place_and_pieces():
    x, _ = make(2, 200, 4, 4, 64, 64, F32)
    whole_o, whole = fwd(x)
    state = x["s0"].clone()
    parts = []
    for a, b in ((0, 77), (77, 78), (78, 200)):
        piece = {n: (state if n == "s0" else t[:, a:b]) for n, t in x.items()}
        o, last = fwd(piece, last_state_out=state)
        assert last is state
        parts.append(o)
    check_fwd(x, torch.cat(parts, 1), state)
    check_fwd(x, whole_o, whole)


def test_fwd_broadcast_decay_and_no_state():
    x, _ = make(3, 90, 4, 4, 64, 64, BF16, state=False)
    x["g"] = torch.tensor([-0.01, -0.1, -1.0, 0.0], device="cuda").to(BF16).expand(3, 90, 4)
    o, last = fwd(x)
    check_fwd(x, o, last)
    o2, none = fwd(x, return_last_state=False)
    assert none is None and torch.equal(o2, o)


def check_bwd(x, do, dlast, got, scale, lengths=None):
    dtype, L, dk, dv = x["q"].dtype, x["g"].shape[1], x["q"].shape[3], x["v"].shape[3]
    ref = P.backward(x["q"], x["k"], x["v"], x["g"], do, scale, x["s0"], dlast, lengths)
    ab = lambda t: None if t is None else t.double().abs()  # noqa: E731
    mag = P.backward(ab(x["q"]), ab(x["k"]), ab(x["v"]), x["g"], ab(do), abs(scale), ab(x["s0"]), ab(dlast), lengths)
    share = x["v"].shape[2] // x["q"].shape[2]
    for n, d in (("dq", dv), ("dk", dv), ("dv", dk)):
        check(n, got[n], ref[n], mag[n] * (1 + share * 2.0 ** -23), dtype, d, L)
    if x["s0"] is not None:
        check("dinitial_state", got["dinitial_state"], ref["dinitial_state"], mag["dinitial_state"], F32, (dtype, dk), L)
    else:
        assert got["dinitial_state"] is None
    # the decay's gradient is a difference of sums from t to the next anchor and the
    # product of two states there, itself of the size of the gradient's own magnitude
    heads = x["v"].shape[2]
    rows = (P._heads(x["q"], heads).abs() * mag["dq_h"] + P._heads(x["k"], heads).abs() * mag["dk_h"]).sum(-1)
    behind = rows.flip(1).cumsum(1).flip(1)
    by = behind + mag["dlog_decay"].amax(1, keepdim=True)
    check("dlog_decay", got["dlog_decay"], ref["dlog_decay"], by, dtype, max(dk, dv) + 128, L)


def bwd(x, do, dlast=None, **kw):
    return ss.ss_linattn_bwd(x["q"], x["k"], x["v"], x["g"], do, initial_state=x["s0"], dlast_state=dlast, **kw)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("L", [1, 64, 131])
def test_bwd(dtype, dk, dv, L):
    x, r = make(2, L, 4, 2, dk, dv, dtype, state=L != 64)
    do = r(2, L, 4, dv).to(dtype)
    dlast = r(2, 4, dk, dv) if L == 131 else None
    got = bwd(x, do, dlast, scale=dk ** -0.5)
    assert ss.ss_last_device_error() == ss.SS_OK
    check_bwd(x, do, dlast, got, dk ** -0.5)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("qk_heads,heads", [(1, 1), (1, 5), (2, 4), (4, 4)])
def test_bwd_strided_shared_heads(dtype, qk_heads, heads):
    x, r = make(2, 100, heads, qk_heads, 40, 24, dtype, strided=True)
    do = r(2, 100, heads, 25).to(dtype)[..., 1:]
    got = bwd(x, do, r(2, heads, 40, 24) * 0)
    check_bwd(x, do, None, got, 1.0)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_bwd_segments_and_anchors(dtype):
    sizes = (1, 2600, 1, 1, 32, 64)
    x, r = make(*sizes, dtype)
    do, dlast = r(1, 2600, 1, 64).to(dtype), r(1, 1, 32, 64)
    got = bwd(x, do, dlast)
    check_bwd(x, do, dlast, got, 1.0)
    again = bwd(x, do, dlast)
    for n in got:
        assert torch.equal(got[n], again[n]), n  # sums in a fixed order


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_bwd_lengths(dtype):
    x, r = make(5, 150, 4, 2, 64, 64, dtype)
    lengths = torch.tensor([0, 1, 64, 150, 99], dtype=torch.int32, device="cuda")
    do, dlast = r(5, 150, 4, 64).to(dtype), r(5, 4, 64, 64)
    clean = {n: t.clone() for n, t in x.items()}
    dirty = do.clone()
    for b, e in enumerate(lengths.tolist()):
        for n in ("q", "k", "v", "g"):
            x[n][b, e:] = float("nan")
            clean[n][b, e:] = 0
        dirty[b, e:] = float("nan")
        do[b, e:] = 0
    got = bwd(x, dirty, dlast, lengths=lengths)
    check_bwd(clean, do, dlast, got, 1.0, lengths)
    assert torch.equal(got["dinitial_state"][0], dlast[0])


@pytest.mark.parametrize("kind", ["none", "reset", "deep"])
def test_bwd_extreme_decays(kind):
    x, r = make(1, 140, 2, 2, 32, 32, F32)
    if kind == "none":
        x["g"].zero_()
    elif kind == "reset":
        x["g"][0, [0, 5, 63, 64, 100]] = -float("inf")
    else:
        x["g"].fill_(-60.0)
    do = r(1, 140, 2, 32)
    got = bwd(x, do, None)
    check_bwd(x, do, None, got, 1.0)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_bwd_first_decay_acts_on_nothing(dtype):
    """Without an initial state the first token's decay has no effect: its gradient is zero, not rounding."""
    x, r = make(3, 70, 2, 2, 64, 64, dtype, state=False)
    do = r(3, 70, 2, 64).to(dtype)
    lengths = torch.tensor([70, 1, 66], dtype=torch.int32, device="cuda")
    got = bwd(x, do, r(3, 2, 64, 64), lengths=lengths)
    assert not got["dlog_decay"][:, 0].any() and got["dlog_decay"][0, 1:].all()
    one = {n: t if t is None else t[:, :1] for n, t in x.items()}
    assert not bwd(one, do[:, :1])["dlog_decay"].any()


def test_bwd_initial_gradient_in_the_last_states_buffer():
    """Through the C ABI: dinitial_state may overwrite dlast_state."""
    import ctypes

    from selective_state_space_ss_b200 import _native as N

    x, r = make(2, 70, 2, 2, 64, 64, F32)
    do, dlast = r(2, 70, 2, 64), r(2, 2, 64, 64)
    want = bwd(x, do, dlast)
    lib = N.load_library()
    device, ops, sizes = N._linattn_operands("bwd", x["q"], x["k"], x["v"], x["g"])
    ops.append(N._heads4("do", do, device, F32, (2, 70, 2, 64)))
    outs = [torch.empty_like(want[n]) for n in ("dq", "dk", "dv", "dlog_decay")]
    ws = torch.empty(ss.ss_linattn_bwd_workspace_bytes(*sizes), dtype=torch.uint8, device="cuda")
    buf = dlast.clone()
    st = lib.ss_linattn_bwd(*[ctypes.byref(o) for o in ops], 1.0, x["s0"].data_ptr(), buf.data_ptr(), None,
                            *[o.data_ptr() for o in outs], buf.data_ptr(), *sizes, ws.data_ptr(), ws.numel(),
                            torch.cuda.current_stream().cuda_stream)
    assert st == ss.SS_OK
    assert torch.equal(buf, want["dinitial_state"])
    for n, o in zip(("dq", "dk", "dv", "dlog_decay"), outs):
        assert torch.equal(o, want[n])


# ---- single tokens

def check_step(x, state, before, o, scale=1.0):
    one = {n: t[:, None] for n, t in x.items()}
    ro, rl = P.forward(**one, scale=scale, s0=before)
    mo, ml = P.forward(one["q"].double().abs(), one["k"].double().abs(), one["v"].double().abs(), one["g"], scale,
                       before.double().abs())
    dk = x["q"].shape[2]
    # fp32 throughout: a product and a sum each for the state, dk sums for the output
    for name, got, ref, by, dtype, n in (("state", state, rl, ml, F32, 4), ("o", o, ro[:, 0], mo[:, 0], x["q"].dtype, dk + 8)):
        bound = n * 2.0 ** -24 * by + (1.001 * half_step(dtype) * ref.abs() if dtype == BF16 else 0)
        assert ((got.double() - ref).abs() <= bound + 1e-37).all(), name


def make_step(batch, heads, qk_heads, dk, dv, dtype, seed=0, strided=False):
    x, r = make(batch, 1, heads, qk_heads, dk, dv, dtype, state=False, seed=seed, strided=strided)
    return {n: t[:, 0] for n, t in x.items() if t is not None}, r


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("batch,strided", [(1, False), (5, True)])
def test_step(dtype, dk, dv, batch, strided):
    x, r = make_step(batch, 6, 2, dk, dv, dtype, strided=strided)
    before = r(batch, 6, dk, dv)
    state = before.clone()
    o = ss.ss_linattn_step(state, x["q"], x["k"], x["v"], x["g"], scale=0.5)
    check_step(x, state, before, o, 0.5)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_step_slots_padding_and_doubles(dtype):
    x, r = make_step(6, 2, 1, 64, 64, dtype)
    pool = r(9, 2, 64, 64)
    before = pool.clone()
    slots = torch.tensor([4, -1, 7, 9, 4, 0], dtype=torch.int32, device="cuda")
    o_out = torch.full((6, 2, 64), 7.0, dtype=dtype, device="cuda")
    o = ss.ss_linattn_step(pool, x["q"], x["k"], x["v"], x["g"], slots=slots, o_out=o_out)
    taken = [0, 2, 5]
    at = slots[taken].long()
    check_step({n: t[taken] for n, t in x.items()}, pool[at], before[at], o[taken])
    assert (o[[1, 3, 4]] == 7).all()
    rest = [i for i in range(9) if i not in at.tolist()]
    assert torch.equal(pool[rest], before[rest])
    fresh = ss.ss_linattn_step(before, x["q"], x["k"], x["v"], x["g"], slots=slots)
    assert not fresh[[1, 3, 4]].any() and torch.equal(fresh[taken], o[taken])


def test_step_reset_and_long_offsets():
    """A decay of minus infinity leaves only the token; a state beyond 2^31 elements."""
    x, r = make_step(2, 32, 32, 128, 128, BF16)
    x["g"][0] = -float("inf")
    slots_n = 4200  # 4200 * 32 * 128 * 128 elements > 2^31
    pool = torch.empty(slots_n, 32, 128, 128, device="cuda")
    slots = torch.tensor([slots_n - 1, 3], dtype=torch.int32, device="cuda")
    pool[slots.long()] = r(2, 32, 128, 128)
    before = pool[slots.long()].clone()
    o = ss.ss_linattn_step(pool, x["q"], x["k"], x["v"], x["g"], slots=slots)
    check_step(x, pool[slots.long()], before, o)


# ---- streams, graphs, a run of all

def test_other_stream_and_graph_replay():
    x, r = make(2, 300, 2, 2, 64, 64, BF16)
    do = r(2, 300, 2, 64).to(BF16)
    want, wl = fwd(x)
    wg = bwd(x, do)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o, last = torch.zeros_like(want), torch.zeros_like(wl)
    side.wait_stream(torch.cuda.current_stream())
    fwd(x, o_out=o, last_state_out=last, stream=side)
    side.synchronize()
    assert torch.equal(o, want) and torch.equal(last, wl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, gl = fwd(x)
        gg = bwd(x, do)
    for seed in (5, 6):
        y, r2 = make(2, 300, 2, 2, 64, 64, BF16, seed=seed)
        for n in x:
            x[n].copy_(y[n])
        do.copy_(r2(2, 300, 2, 64).to(BF16))
        graph.replay()
        eo, el = fwd(x)
        eg = bwd(x, do)
        assert torch.equal(go, eo) and torch.equal(gl, el)
        for n in eg:
            assert torch.equal(gg[n], eg[n]), n
    assert wg.keys() == eg.keys()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_prompt_pool_prompt_steps(dtype):
    """A dialogue: a prompt, its states parked in 8 bits, woken, another prompt, single tokens."""
    x, r = make(3, 150, 4, 2, 64, 48, dtype, state=False)
    first = {n: None if t is None else t[:, :100] for n, t in x.items()}
    o, state = fwd(first)
    check_fwd(first, o, state)
    codes = torch.zeros(5, 4, 64, 48, dtype=torch.int8, device="cuda")
    scales = torch.zeros(5, 4, 64, device="cuda")
    slots = torch.tensor([2, 0, 4], dtype=torch.int32, device="cuda")
    ss.ss_state_store8(state, codes, scales, slots=slots)
    woken = ss.ss_state_load8(codes, scales, slots=slots)
    assert ((woken - state).abs() <= 0.5001 * scales[slots.long()][..., None]).all()
    second = {**{n: t[:, 100:140] for n, t in x.items() if n != "s0"}, "s0": woken}
    o, state = fwd(second, lengths=torch.full((3,), 40, dtype=torch.int32, device="cuda"))
    check_fwd(second, o, state)
    for t in range(140, 150):
        token = {n: x[n][:, t] for n in ("q", "k", "v", "g")}
        before = state.clone()
        check_step(token, state, before, ss.ss_linattn_step(state, *token.values()))
        assert not torch.equal(state, before)


def test_refusals_on_the_device():
    x, r = make(2, 10, 4, 2, 16, 16, BF16)
    call = lambda **over: fwd({**x, **{k: v for k, v in over.items() if k in x}},  # noqa: E731
                              **{k: v for k, v in over.items() if k not in x})
    for over in (dict(k=x["k"].float()), dict(q=x["q"].half()), dict(v=x["v"][:, :9]), dict(g=x["g"].float()),
                 dict(g=x["g"][..., :2]), dict(s0=x["s0"].to(BF16)), dict(s0=x["s0"][:1]), dict(k=x["k"].cpu()),
                 dict(q=x["q"].transpose(2, 3).contiguous().transpose(2, 3)),
                 dict(lengths=torch.tensor([1, 2], device="cuda")), dict(lengths=torch.tensor([1], dtype=torch.int32, device="cuda")),
                 dict(o_out=torch.empty(2, 10, 4, 16, device="cuda")),
                 dict(last_state_out=torch.empty(2, 4, 16, 16, device="cuda").transpose(2, 3))):
        with pytest.raises(ValueError):
            call(**over)
    with pytest.raises(ss.SSError):  # heads not a multiple of the shared ones
        fwd({**x, "q": torch.zeros(2, 10, 3, 16, dtype=BF16, device="cuda"), "k": torch.zeros(2, 10, 3, 16, dtype=BF16, device="cuda")})
    wide = torch.zeros(2, 10, 2, 129, dtype=BF16, device="cuda")
    with pytest.raises(ss.SSError) as e:
        ss.ss_linattn_fwd(wide, wide, x["v"], x["g"])
    assert e.value.status == ss.SS_ERR_UNSUPPORTED
    empty = torch.zeros(2, 0, 2, 16, dtype=BF16, device="cuda")
    with pytest.raises(ss.SSError):
        ss.ss_linattn_fwd(empty, empty, empty, empty[..., 0])
