"""ss_winattn_fwd and ss_winattn_bwd on the GPU against 64 bits; tests/winattn_plain.py has
the reference and what a result may be off by."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import selective_state_space_ss_b200 as ss  # noqa: E402
from tests import winattn_plain as P  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


def make(batch, L, heads, kv_heads, d, dtype, seed=0, strided=False, odd=0):
    """q, k, v, do; strided: slices of one projection's output, `odd` elements from a 16-byte border."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    if strided:
        a, b = heads * d, kv_heads * d
        wide = r(batch, L, a + 2 * b + 8 + odd).to(dtype)[..., odd:]
        q, k, v = wide[..., :a].unflatten(-1, (heads, d)), wide[..., a:a + b].unflatten(-1, (kv_heads, d)), \
            wide[..., a + b:a + 2 * b].unflatten(-1, (kv_heads, d))
        do = r(batch, heads, L, d).to(dtype).transpose(1, 2)
        return q, k, v, do
    return tuple(r(batch, L, n, d).to(dtype) for n in (heads, kv_heads, kv_heads, heads))


def both(q, k, v, do, window, sinks, lengths=None, scale=None):
    """Forward and backward checked against 64 bits."""
    ref = P.attention(q, k, v, window, sinks, scale, lengths, do)
    o, lse = ss.ss_winattn_fwd(q, k, v, window, sinks=sinks, scale=scale, lengths=lengths)
    assert o.dtype == q.dtype and lse.dtype == F32
    g = ss.ss_winattn_bwd(q, k, v, o, lse, do, window, sinks=sinks, scale=scale, lengths=lengths)
    assert ss.ss_last_device_error() == ss.SS_OK
    for name, x in {"o": o, "lse": lse, **g}.items():
        P.check(name, x, *ref[name])
    return o, lse, g


@TYPES
@pytest.mark.parametrize("L", [1, 2, 63, 64, 65, 127, 128, 129, 257, 400])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths_of_tiles(dtype, L, d):
    both(*make(2, L, 4, 2, d, dtype), 100, 3)


@TYPES
@pytest.mark.parametrize("d", [1, 7, 8, 16, 37, 40, 72, 100, 120, 127])
def test_widths(dtype, d):
    both(*make(1, 150, 2, 1, d, dtype), 60, 2)


@TYPES
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (5, 200), (63, 1), (64, 0), (65, 64), (127, 0), (128, 1),
                                          (129, 130), (256, 0), (300, 4), (599, 0), (600, 0), (601, 7), (1 << 40, 0),
                                          (10, 1 << 40), (10, 600), (10, 599)])
def test_masks(dtype, window, sinks):
    both(*make(1, 600, 2, 2, 64, dtype), window, sinks)


@TYPES
@pytest.mark.parametrize("kv_heads,heads", [(1, 1), (1, 6), (3, 6), (2, 16), (5, 5)])
@pytest.mark.parametrize("odd", [0, 1])
def test_strided_shared_heads(dtype, kv_heads, heads, odd):
    both(*make(2, 140, heads, kv_heads, 40, dtype, strided=True, odd=odd), 50, 4)


@TYPES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks,L", [(3, 5, 2500), (40, 1, 2700), (64, 130, 2300), (1, 64, 1500), (100, 700, 2100)])
def test_sinks_of_a_long_row(dtype, d, window, sinks, L):
    """The sinks' gradients come in pieces."""
    sizes = (1, L, 2, 1, d, window)
    dt = ss.SS_BF16 if dtype == BF16 else ss.SS_F32
    assert ss.ss_winattn_bwd_workspace_bytes(*sizes, sinks, dt) > ss.ss_winattn_bwd_workspace_bytes(*sizes, 0, dt)
    both(*make(1, L, 2, 1, d, dtype), window, sinks)


@TYPES
@pytest.mark.parametrize("d", [64, 100, 128])
@pytest.mark.parametrize("window,sinks", [(30, 3), (1000, 0), (3, 140)])
def test_rows_behind_a_length_are_neither_read_nor_written(dtype, d, window, sinks):
    L = 400
    q, k, v, do = make(6, L, 4, 2, d, dtype)
    ends = [400, 0, 1, 128, 130, 251]
    lengths = torch.tensor([1000, -5, *ends[2:]], dtype=torch.int32, device="cuda")
    ref = P.attention(q, k, v, window, sinks, lengths=ends, do=do)
    for b, n in enumerate(ends):
        for x in (q, k, v, do):
            x[b, n:] = float("nan") if b % 2 else float("inf")
    o, lse = torch.full_like(q, 7.0), torch.full((6, 4, L), 9.0, device="cuda")
    ss.ss_winattn_fwd(q, k, v, window, sinks=sinks, lengths=lengths, o_out=o, lse_out=lse)
    for b, n in enumerate(ends):
        assert (o[b, n:] == 7).all() and (lse[b, :, n:] == 9).all()
        o[b, n:], lse[b, :, n:] = float("nan"), float("nan")
    g = ss.ss_winattn_bwd(q, k, v, o, lse, do, window, sinks=sinks, lengths=lengths)
    assert ss.ss_last_device_error() == ss.SS_OK
    for b, n in enumerate(ends):
        o[b, n:], lse[b, :, n:] = 0, 0
        for x in g.values():
            assert (x[b, n:] == 0).all()  # as they were allocated
    for name, x in {"o": o, "lse": lse, **g}.items():
        P.check(name, x, *ref[name])
    fresh = ss.ss_winattn_fwd(q, k, v, window, sinks=sinks, lengths=lengths)
    assert torch.equal(fresh[0], o) and torch.equal(fresh[1], lse)


@TYPES
def test_large_scores(dtype):
    """Logits of some hundreds, rising over the row and falling: maxima that move, and rows that one token takes."""
    q, k, v, do = make(1, 500, 2, 2, 64, dtype)
    slope = torch.linspace(-6, 6, 500, device="cuda")[None, :, None, None]
    q = (q * 0.3 + 4).to(dtype)
    both(q, (k * 0.3 + slope).to(dtype), v, do, 200, 4)
    both(q, (k * 0.3 - slope).to(dtype), v, do, 200, 4)
    both(q, torch.zeros_like(k), v, do, 200, 4)  # all alike


@TYPES
@pytest.mark.parametrize("scale", [1e-3, 1.0])
def test_scales(dtype, scale):
    both(*make(1, 200, 2, 2, 64, dtype), 90, 0, scale=scale)


@TYPES
def test_broadcast_and_reversed_operands(dtype):
    """Strides of zero and below: keys that all heads share without copies, a row read backwards."""
    q, k, v, do = make(2, 150, 4, 1, 64, dtype)
    wide = k.expand(2, 150, 4, 64), v.expand(2, 150, 4, 64)
    assert wide[0].stride(2) == 0 or k.shape[2] == 1
    both(q, *wide, do, 70, 2)
    one = do[:, :1].expand(2, 150, 4, 64)  # one gradient for all tokens
    both(q, *wide, one, 70, 2)


@TYPES
@pytest.mark.parametrize("d", [64, 128])
def test_the_same_bits_every_time(dtype, d):
    q, k, v, do = make(2, 1500, 4, 2, d, dtype)
    first = None
    for _ in range(3):
        o, lse = ss.ss_winattn_fwd(q, k, v, 40, sinks=4)
        g = ss.ss_winattn_bwd(q, k, v, o, lse, do, 40, sinks=4)
        got = [o, lse, *g.values()]
        assert first is None or all(torch.equal(x, y) for x, y in zip(got, first))
        first = got


@TYPES
def test_many_heads(dtype):
    q, k, v, do = make(3, 130, 60, 20, 32, dtype)
    both(q, k, v, do, 64, 1)


def test_a_workspace_of_the_callers_and_without_lse():
    q, k, v, do = make(1, 300, 2, 2, 64, BF16)
    o, none = ss.ss_winattn_fwd(q, k, v, 100, return_lse=False)
    assert none is None
    o2, lse = ss.ss_winattn_fwd(q, k, v, 100)
    assert torch.equal(o, o2)
    need = ss.ss_winattn_bwd_workspace_bytes(1, 300, 2, 2, 64, 100, 0, ss.SS_BF16)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    g = ss.ss_winattn_bwd(q, k, v, o, lse, do, 100, workspace=ws)
    want = ss.ss_winattn_bwd(q, k, v, o, lse, do, 100)
    assert all(torch.equal(g[n], want[n]) for n in g)
    with pytest.raises(ss.SSError):
        ss.ss_winattn_bwd(q, k, v, o, lse, do, 100, workspace=ws[:need - 256])


@TYPES
def test_the_end_of_a_strided_operand(dtype):
    """The last row ends where its memory ends: nothing behind it is read (the checked build looks)."""
    q, k, v, do = make(1, 77, 2, 2, 64, dtype)
    whole = torch.randn(1, 77, 2, 66, device="cuda").to(dtype)
    both(whole[..., 2:], k, v, do, 30, 0)


def test_refusals():
    q, k, v, do = make(1, 20, 4, 2, 64, BF16)
    o, lse = ss.ss_winattn_fwd(q, k, v, 5)
    for bad in (lambda: ss.ss_winattn_fwd(q, k.float(), v, 5), lambda: ss.ss_winattn_fwd(q, k[:, :19], v, 5),
                lambda: ss.ss_winattn_fwd(q, k, v[..., :32], 5), lambda: ss.ss_winattn_fwd(q.half(), k.half(), v.half(), 5),
                lambda: ss.ss_winattn_fwd(q.transpose(2, 3).contiguous().transpose(2, 3), k, v, 5),
                lambda: ss.ss_winattn_fwd(q[0], k, v, 5), lambda: ss.ss_winattn_fwd(q, k, v, -1),
                lambda: ss.ss_winattn_fwd(q, k, v, 5, lengths=torch.ones(1, device="cuda")),
                lambda: ss.ss_winattn_fwd(q, k, v, 5, o_out=o.float()),
                lambda: ss.ss_winattn_fwd(q, k, v, 5, lse_out=lse[:, :3]),
                lambda: ss.ss_winattn_bwd(q, k, v, o, None, do, 5), lambda: ss.ss_winattn_bwd(q, k, v, o, lse, do[:, :3], 5)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ss.ss_winattn_fwd(q, k, v, 0), lambda: ss.ss_winattn_fwd(q, k, v, 5, scale=0.0),
                lambda: ss.ss_winattn_fwd(q[:, :, :3], k, v, 5), lambda: ss.ss_winattn_bwd(q, k, v, o, lse, do, 0)):
        with pytest.raises(ss.SSError):
            bad()


def test_offsets_beyond_32_bits():
    """More than 2^31 queries' values: the end of the row against 64 bits."""
    L, heads, kv, d, window = 1 << 17, 130, 2, 128, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, do = (torch.randn(1, L, heads, d, device="cuda", generator=gen, dtype=BF16) for _ in range(2))
    k, v = (torch.randn(1, L, kv, d, device="cuda", generator=gen, dtype=BF16) for _ in range(2))
    assert q.numel() > 1 << 31
    o, lse = ss.ss_winattn_fwd(q, k, v, window)
    g = ss.ss_winattn_bwd(q, k, v, o, lse, do, window)
    assert ss.ss_last_device_error() == ss.SS_OK
    end = slice(L - 256, L)
    ref = P.attention(q[:, end], k[:, end], v[:, end], window, do=do[:, end])
    for name, x in {"o": o, **g}.items():  # from the first token on whose window lies in the piece
        P.check(name, x[:, end][:, window:], *(y[:, window:] for y in ref[name]))
    P.check("lse", lse[..., end][..., window:], *(y[..., window:] for y in ref["lse"]))
