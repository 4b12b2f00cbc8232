"""ss_state_store8 / ss_state_load8 against their definition: scale = max |x| * (1/127)
in fp32, code the integer nearest to the exact quotient x / scale (ties to even),
value = code * scale.  All of it is exact in 64 bits, so results are compared bit by
bit: a quotient of two fp32 numbers that is not a tie is at least 2^-26 away from
one relative to itself, and fp64 resolves 2^-53."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import selective_state_space_ss_b200 as ss  # noqa: E402

TINY = torch.finfo(torch.float32).tiny


def plain_store(state):
    top = state.abs().amax(-1)
    scale = top * torch.tensor(1.0, device=state.device).div(torch.tensor(127.0, device=state.device))
    scale = torch.where(scale < TINY, torch.zeros_like(scale), scale)
    scale = torch.where(torch.isfinite(state).all(-1), scale, torch.full_like(scale, float("nan")))
    by = torch.where(scale > 0, scale, torch.ones_like(scale)).double()
    codes = torch.where((scale > 0)[..., None], torch.round(state.double() / by[..., None]), 0)
    return codes.to(torch.int8), scale


def same(a, b):
    return torch.equal(a.nan_to_num(nan=1e30), b.nan_to_num(nan=1e30)) and torch.equal(a.isnan(), b.isnan())


def roundtrip(state, pad=0):
    shape = state.shape
    codes = torch.full((shape[0] + 2, *shape[1:]), 55, dtype=torch.int8, device="cuda")
    scales = torch.full((shape[0] + 2, *shape[1:-1]), 9.0, device="cuda")
    ss.ss_state_store8(state, codes, scales, slots=torch.arange(shape[0], dtype=torch.int32, device="cuda") + 1)
    want_codes, want_scales = plain_store(state)
    assert torch.equal(codes[1:-1], want_codes)
    assert same(scales[1:-1], want_scales)
    for end in (0, -1):  # the other slots as they were
        assert (codes[end] == 55).all() and (scales[end] == 9).all()
    back = ss.ss_state_load8(codes, scales, slots=torch.arange(shape[0], dtype=torch.int32, device="cuda") + 1)
    assert same(back, want_codes.float() * want_scales[..., None])
    return codes, scales


@pytest.mark.parametrize("width", [1, 2, 3, 4, 5, 12, 16, 20, 31, 32, 33, 48, 64, 100, 127, 128, 129, 132, 256, 257,
                                   300, 512, 516, 1000, 1023, 1024])
@pytest.mark.parametrize("rows", [1, 37])
def test_widths(width, rows):
    gen = torch.Generator(device="cuda").manual_seed(width)
    state = torch.randn(3, rows, width, device="cuda", generator=gen) * torch.exp(4 * torch.randn(3, rows, 1, device="cuda", generator=gen))
    roundtrip(state)


def test_borders_of_two_codes():
    """Rows whose quotients are ties, or one last place off one."""
    steps = torch.arange(-127, 128, device="cuda", dtype=torch.float32)
    rows = []
    for scale in (1.0, 0.3, 7e-5, 1e30):
        top = torch.tensor(127.0 * scale, device="cuda")
        s = top * torch.tensor(1.0, device="cuda").div(torch.tensor(127.0, device="cuda"))
        half = (steps[:-1] + 0.5) * s
        for x in (half, torch.nextafter(half, half * 2), torch.nextafter(half, half * 0)):
            rows.append(torch.cat([x, top[None]])[-128:])
            rows.append(torch.cat([top[None], x])[:128])
    roundtrip(torch.stack(rows)[None])


def test_zero_tiny_and_non_finite_rows():
    state = torch.randn(2, 8, 64, device="cuda")
    state[0, 0] = 0
    state[0, 1] *= 1e-40
    state[0, 2, 5] = float("nan")
    state[0, 3, 6] = float("inf")
    state[0, 4, 7] = -float("inf")
    state[0, 5] = TINY * 127 * 1.001
    state[0, 6] = torch.finfo(torch.float32).max
    state[0, 7] = TINY * 126
    codes, scales = roundtrip(state)
    back = ss.ss_state_load8(codes, scales, slots=torch.tensor([1], dtype=torch.int32, device="cuda"))
    assert not back[0, [0, 1, 7]].any() and back[0, 2:5].isnan().all() and torch.isfinite(back[0, 5:7]).all()


def test_slots():
    state = torch.randn(5, 6, 32, device="cuda")
    codes, scales = torch.zeros(4, 6, 32, dtype=torch.int8, device="cuda"), torch.zeros(4, 6, device="cuda")
    slots = torch.tensor([2, -1, 0, 2, 4], dtype=torch.int32, device="cuda")
    ss.ss_state_store8(state, codes, scales, slots=slots)
    want, ws = plain_store(state)
    assert torch.equal(codes[2], want[3]) and torch.equal(scales[2], ws[3])  # the last one of two
    assert torch.equal(codes[0], want[2]) and not codes[[1, 3]].any() and not scales[[1, 3]].any()
    at = torch.tensor([2, 2, -1, 0, 4, 1000], dtype=torch.int32, device="cuda")
    out = torch.full((6, 6, 32), 3.0, device="cuda")
    back = ss.ss_state_load8(codes, scales, slots=at, state_out=out)
    assert back is out and torch.equal(back[0], back[1]) and not back[[2, 4, 5]].any()
    assert torch.equal(back[0], want[3].float() * ws[3][:, None])
    everything = ss.ss_state_load8(codes, scales)
    assert everything.shape == (4, 6, 32) and torch.equal(everything[2], back[0])
    ss.ss_state_store8(state[:4], codes, scales)
    assert torch.equal(codes, want[:4])


def test_unaligned_views():
    base = torch.randn(2 * 7 * 64 + 1, device="cuda")
    state = base[1:].view(2, 7, 64)
    raw = torch.zeros(2 * 7 * 64 + 1, dtype=torch.int8, device="cuda")
    codes, scales = raw[1:].view(2, 7, 64), torch.zeros(2, 7, device="cuda")
    ss.ss_state_store8(state, codes, scales)
    want, ws = plain_store(state)
    assert torch.equal(codes, want) and torch.equal(scales, ws)
    out = torch.zeros(2 * 7 * 64 + 1, device="cuda")[1:].view(2, 7, 64)
    assert torch.equal(ss.ss_state_load8(codes, scales, state_out=out), want.float() * ws[..., None])


def test_scan_states_through_the_pool():
    """The selective scan's last state, parked, woken, and carried on from."""
    import oracle
    from selective_state_space_ss_b200 import inputs as I
    from tests.helpers import TOL, rel_err, to_device

    w = I.Workload("pool", 2, 96, 200, 16, "f32")
    x = I.make_inputs(w, seed=3)
    xd = to_device(x)
    args = lambda a, b: [xd[n][..., a:b].contiguous() if n in ("u", "delta", "B", "C") else xd[n]  # noqa: E731
                         for n in ("u", "delta", "A", "B", "C")]
    kw = lambda a, b: dict(D=xd["D"], z=xd["z"][..., a:b].contiguous(), delta_bias=xd["delta_bias"])  # noqa: E731
    _, state = ss.ss_scan_fwd(*args(0, 120), **kw(0, 120))
    codes, scales = roundtrip(state)
    woken = ss.ss_state_load8(codes, scales, slots=torch.tensor([1, 2], dtype=torch.int32, device="cuda"))
    assert ((woken - state).abs() <= 0.5001 * scales[1:3][..., None]).all()
    y, last = ss.ss_scan_fwd_from_state(woken, *args(120, 200), **kw(120, 200))
    h = woken.cpu().numpy().astype("float64")
    cut = {n: v[..., 120:].copy() if n in ("u", "delta", "B", "C", "z") else v for n, v in x.items()}
    yo, ho = oracle.scan_fwd(cut["u"], cut["delta"], cut["A"], cut["B"], cut["C"], cut["D"], cut["z"],
                             cut["delta_bias"], h0=h)
    assert rel_err(y.cpu().numpy(), yo) <= TOL["f32"] and rel_err(last.cpu().numpy(), ho) <= TOL["f32"]


def test_refusals():
    state = torch.zeros(2, 3, 16, device="cuda")
    codes, scales = torch.zeros(4, 3, 16, dtype=torch.int8, device="cuda"), torch.zeros(4, 3, device="cuda")
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    for s, c, sc, sl in ((state.half(), codes, scales, slots), (state, codes.float(), scales, slots),
                         (state, codes, scales[:3], slots), (state, codes, scales, slots.long()),
                         (state[:1], codes, scales, slots), (state.transpose(0, 1), codes, scales, slots),
                         (state, codes, scales.double(), slots), (state, codes, scales, slots[None]),
                         (state, codes[:, :, :8], scales, slots)):
        with pytest.raises(ValueError):
            ss.ss_state_store8(s, c, sc, slots=sl)
    with pytest.raises(ss.SSError):
        ss.ss_state_store8(torch.zeros(6, 3, 16, device="cuda"), codes, scales)  # six sequences, four slots
    with pytest.raises(ss.SSError) as e:
        ss.ss_state_load8(torch.zeros(1, 1, 1025, dtype=torch.int8, device="cuda"), torch.zeros(1, 1, device="cuda"))
    assert e.value.status == ss.SS_ERR_UNSUPPORTED
