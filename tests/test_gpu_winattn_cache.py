"""ss_winattn_step, ss_kv_append and ss_rotate on the GPU against 64 bits, and a run of all of
them together (tests/winattn_plain.py has the references and the bounds)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import selective_state_space_ss_b200 as ss  # noqa: E402
from tests import winattn_plain as P  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
TYPES = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


def rand(gen, *s):
    return torch.randn(*s, device="cuda", generator=gen)


def cache(batch, lengths, tokens, heads, kv_heads, d, page, dtype, seed=0, per=None, order="page", junk=float("nan")):
    """q, pools whose unused places hold `junk`, the table and the lengths; order: of a page's axes in memory."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    per = per or max(1, -(-max(lengths) // page))
    pages = batch * per + 2
    shape = (pages, page, kv_heads, d) if order == "page" else (pages, kv_heads, page, d)
    pools = [rand(gen, *shape).to(dtype) for _ in range(2)]
    if order == "head":
        pools = [x.transpose(1, 2) for x in pools]
    table = torch.randperm(pages, device="cuda", generator=gen)[:batch * per].int().view(batch, per)
    live = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lengths):
        for t in range(n):
            live[table[b, t // page], t % page] = True
    for x in pools:
        x[~live] = junk
    q = rand(gen, batch, tokens, heads, d).to(dtype)
    return q, *pools, table, torch.tensor(lengths, dtype=torch.int32, device="cuda")


def run(q, k, v, table, lengths, window, sinks=0, **kw):
    o = ss.ss_winattn_step(q, k, v, table, lengths, window, sinks=sinks, **kw)
    assert ss.ss_last_device_error() == ss.SS_OK
    P.check("o", o, *P.step(q, k, v, table, lengths, window, sinks, **kw))
    return o


@TYPES
@pytest.mark.parametrize("d", [64, 128, 1, 7, 16, 40, 72, 100])
@pytest.mark.parametrize("share", [1, 5])
def test_widths_and_lengths(dtype, d, share):
    lengths = [1, 2, 15, 16, 17, 63, 64, 65, 300]
    run(*cache(9, lengths, 1, 2 * share, 2, d, 16, dtype), 50, 3)


@TYPES
@pytest.mark.parametrize("page", [1, 3, 16, 64, 100, 256])
@pytest.mark.parametrize("order", ["page", "head"])
def test_pages(dtype, page, order):
    run(*cache(3, [200, 77, 256], 1, 6, 2, 64, page, dtype, order=order), 120, 4)


@TYPES
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 5), (63, 0), (64, 0), (65, 1), (700, 0), (699, 3), (1 << 40, 0),
                                          (3, 1 << 40), (100, 600), (10, 650)])
def test_masks(dtype, window, sinks):
    run(*cache(2, [700, 650], 1, 4, 2, 64, 32, dtype), window, sinks)


@TYPES
@pytest.mark.parametrize("tokens", [2, 3, 8, 40])
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 2), (1000, 0)])
@pytest.mark.parametrize("d", [64, 128])
def test_several_tokens(dtype, tokens, window, sinks, d):
    """They see one another as in the prompt; rows with fewer tokens than that have zeros in the missing places."""
    q, *rest = cache(4, [tokens, 130, max(1, tokens - 2), 0], tokens, 6, 2, d, 16, dtype, per=9)
    o = run(q, *rest, window, sinks)
    assert (o[3] == 0).all() and (o[2, :tokens - max(1, tokens - 2)] == 0).all()


@TYPES
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (16, 1), (17, 1), (48, 1), (40, 8)])
def test_groups(dtype, heads, kv_heads):
    run(*cache(2, [150, 90], 1, heads, kv_heads, 64, 16, dtype), 100, 2)


@TYPES
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths,window", [([5000], 1 << 40), ([4097, 1], 4000), ([3000, 2999, 64], 1 << 40)])
def test_long_rows_cut_between_blocks(dtype, d, lengths, window):
    run(*cache(len(lengths), lengths, 1, 4, 2, d, 64, dtype), window, 4)


@TYPES
def test_lengths_out_of_range_and_pages_that_are_none(dtype):
    q, k, v, table, lengths = cache(5, [64, 64, 64, 64, 64], 1, 4, 2, 64, 16, dtype, per=4)
    lengths[0], lengths[1] = 1000, -3  # as 64 and 0
    table[2, 1] = -1
    table[3, 2] = 1 << 30
    table[4] = -7
    o = run(q, k, v, table, torch.tensor([64, 0, 64, 64, 64], dtype=torch.int32, device="cuda"), 1 << 40)
    got = ss.ss_winattn_step(q, k, v, table, lengths, 1 << 40)
    assert torch.equal(got, o) and (o[1] == 0).all() and (o[4] == 0).all() and (o[2] != 0).any()


@TYPES
def test_entries_that_no_visible_token_lies_in_are_not_followed(dtype):
    """Pages that the window has left behind are given back, theirs hold anything."""
    q, k, v, table, lengths = cache(1, [200], 1, 4, 2, 64, 16, dtype)
    want = run(q, k, v, table, lengths, 40, 2)
    table[0, 1:10] = torch.tensor([-1, 1 << 30, -(1 << 31), 0, 0, 0, -5, 7, (1 << 31) - 1], device="cuda")
    k[table[0, 0].item(), 2:] = float("inf")
    v[table[0, 0].item(), 2:] = float("nan")
    assert torch.equal(ss.ss_winattn_step(q, k, v, table, lengths, 40, sinks=2), want)


@TYPES
def test_strided_queries_and_shared_pages(dtype):
    """Queries out of one projection's output; two rows that share their first page; rows at odd addresses."""
    q, k, v, table, lengths = cache(2, [40, 50], 1, 6, 2, 64, 16, dtype)
    k[torch.isnan(k)], v[torch.isnan(v)] = 0.5, 0.5
    table[1, 0] = table[0, 0]
    wide = torch.randn(2, 1, 6 * 64 + 9, device="cuda").to(dtype)
    run(wide[..., 9:].unflatten(-1, (6, 64)), k, v, table, lengths, 30, 20)
    pool = torch.randn(2, k.numel() + 1, device="cuda").to(dtype)
    run(q, pool[0, 1:].view(k.shape), pool[1, 1:].view(k.shape), table, lengths, 30, 20)


def test_a_cache_beyond_32_bits():
    """Offsets of more than 2^31 elements, in the pages read and in those written."""
    page, kv, d = 64, 2, 128
    pages = (1 << 31) // (page * kv * d) + 70
    k = torch.zeros(pages, page, kv, d, dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    gen = torch.Generator(device="cuda").manual_seed(0)
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    nk, nv = rand(gen, 1, 150, kv, d).bfloat16(), rand(gen, 1, 150, kv, d).bfloat16()
    starts = torch.tensor([20], dtype=torch.int32, device="cuda")
    ss.ss_kv_append(nk, nv, k, v, table, starts)
    assert torch.equal(v[pages - 1, 20:], nv[0, :44]) and torch.equal(k[0], nk[0, 44:108]) and torch.equal(v[pages - 2, :42], nv[0, 108:])
    q = rand(gen, 1, 1, 4, d).bfloat16()
    run(q, k, v, table, torch.tensor([170], dtype=torch.int32, device="cuda"), 1000)


# ---- the rotation and the cache's appending


def freqs(half):
    return 10000.0 ** (-torch.arange(half, device="cuda") / max(half, 1))


@TYPES
@pytest.mark.parametrize("d,half", [(64, 32), (128, 64), (128, 32), (64, 0), (2, 1), (1, 0), (37, 18), (37, 5), (72, 36), (100, 24),
                                    (256, 128), (1000, 500)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotate(dtype, d, half, inter, inverse):
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k = rand(gen, 2, 33, 3, d).to(dtype), rand(gen, 2, 33, 1, d).to(dtype)
    starts = torch.tensor([0, 1_000_000_007], dtype=torch.int32, device="cuda")
    inv = freqs(half) if half else None
    for s, n in ((None, [0, 0]), (starts, starts.tolist())):
        got = ss.ss_rotate(q, inv, k=k, starts=s, interleaved=inter, inverse=inverse)
        assert ss.ss_last_device_error() == ss.SS_OK
        for name, x, y in zip("qk", got, (q, k)):
            P.check(name, x, *P.rotate(y, n, inv, inter, inverse))
            assert torch.equal(x[..., 2 * half:], y[..., 2 * half:])
    alone, none = ss.ss_rotate(q, inv, starts=starts, interleaved=inter, inverse=inverse)
    assert none is None and torch.equal(alone, got[0])


@TYPES
def test_rotate_strided_in_place_and_counts(dtype):
    gen = torch.Generator(device="cuda").manual_seed(2)
    inv, counts = freqs(20), torch.tensor([5, -1, 100, 11], dtype=torch.int32, device="cuda")
    for odd in (0, 1):
        wide = rand(gen, 4, 12, 6 * 64 + odd).to(dtype)[..., odd:]
        q, k = wide[..., :256].unflatten(-1, (4, 64)), wide[..., 256:].unflatten(-1, (2, 64))
        with pytest.raises(ss.SSError):
            ss.ss_rotate(q[:, :, :3], inv, k=k)  # heads are a multiple of the keys'
        got = ss.ss_rotate(q, inv, k=k)
        for name, x, y in zip("qk", got, (q, k)):
            P.check(name, x, *P.rotate(y, [0] * 4, inv))
        part = ss.ss_rotate(q, inv, k=k, counts=counts)
        for x, y in zip(part, got):
            for b, n in enumerate([5, 0, 12, 11]):
                assert torch.equal(x[b, :n], y[b, :n]) and (x[b, n:] == 0).all()
        mine = q.contiguous(), k.contiguous()
        kept = [x.clone() for x in mine]
        ss.ss_rotate(mine[0], inv, k=mine[1], counts=counts, q_out=mine[0], k_out=mine[1])
        for x, y, z in zip(mine, got, kept):
            for b, n in enumerate([5, 0, 12, 11]):
                assert torch.equal(x[b, :n], y[b, :n]) and torch.equal(x[b, n:], z[b, n:])


@TYPES
@pytest.mark.parametrize("d,half,inter", [(64, 32, False), (128, 32, True), (37, 18, False), (37, 9, True), (40, 0, False)])
@pytest.mark.parametrize("page", [1, 16, 50])
@pytest.mark.parametrize("order", ["page", "head"])
def test_append(dtype, d, half, inter, page, order):
    gen = torch.Generator(device="cuda").manual_seed(3)
    batch, T, kv, heads, room = 5, 37, 2, 6, 150
    per = -(-room // page)
    shape = (batch * per + 1, page, kv, d) if order == "page" else (batch * per + 1, kv, page, d)
    pools = [torch.full(shape, 3.0, device="cuda", dtype=dtype) for _ in range(2)]
    if order == "head":
        pools = [x.transpose(1, 2) for x in pools]
    table = torch.randperm(batch * per, device="cuda", generator=gen).int().view(batch, per)
    starts = torch.tensor([0, 99, per * page - 10, -4, 20], dtype=torch.int32, device="cuda")
    counts = torch.tensor([37, 200, 37, 37, 9], dtype=torch.int32, device="cuda")
    if page < 50:
        table[1, 110 // page] = -1  # no page
    k, v, q = rand(gen, batch, T, kv, d).to(dtype), rand(gen, batch, T, kv, d).to(dtype), rand(gen, batch, T, heads, d).to(dtype)
    inv = freqs(half) if half else None
    got_q, got_k = ss.ss_kv_append(k, v, *pools, table, starts, inv_freq=inv, q=q, counts=counts, interleaved=inter, return_k=True)
    assert ss.ss_last_device_error() == ss.SS_OK
    want = [torch.full(shape if order == "page" else (shape[0], page, kv, d), 3.0, device="cuda", dtype=dtype) for _ in range(2)]
    for b, (s, n) in enumerate(zip(starts.tolist(), [37, 37, 37, 37, 9])):
        for name, x, y in (("q", got_q, q), ("k", got_k, k)):
            P.check(name, x[b:b + 1, :n], *P.rotate(y[b:b + 1, :n], [s], inv, inter))
            assert (x[b, n:] == 0).all()
        for t in range(n):
            at = s + t
            if s >= 0 and at < per * page and table[b, at // page] >= 0:
                want[0][table[b, at // page], at % page] = got_k[b, t]
                want[1][table[b, at // page], at % page] = v[b, t]
    assert torch.equal(pools[0], want[0]) and torch.equal(pools[1], want[1])
    assert (table < batch * per).all() and (pools[0][-1] == 3).all()


@TYPES
def test_append_without_queries_and_in_place(dtype):
    gen = torch.Generator(device="cuda").manual_seed(4)
    pools = [torch.zeros(4, 16, 2, 64, device="cuda", dtype=dtype) for _ in range(2)]
    table, starts = torch.arange(4, device="cuda").int().view(1, 4), torch.tensor([7], dtype=torch.int32, device="cuda")
    k, v, q = (rand(gen, 1, 5, n, 64).to(dtype) for n in (2, 2, 4))
    want = ss.ss_rotate(q, freqs(32), k=k, starts=starts)
    assert ss.ss_kv_append(k, v, *pools, table, starts, inv_freq=freqs(32)) == (None, None)
    assert torch.equal(pools[0].flatten(0, 1)[7:12], want[1][0]) and torch.equal(pools[1].flatten(0, 1)[7:12], v[0])
    got = ss.ss_kv_append(k, v, *pools, table, starts, inv_freq=freqs(32), q=q, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k and torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_refusals():
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v, table, lengths = cache(2, [20, 30], 1, 4, 2, 64, 16, BF16)
    new = rand(gen, 2, 1, 2, 64).bfloat16()
    for bad in (lambda: ss.ss_winattn_step(q, k, v[:1], table, lengths, 5), lambda: ss.ss_winattn_step(q, k.float(), v, table, lengths, 5),
                lambda: ss.ss_winattn_step(q, k, v, table.long(), lengths, 5), lambda: ss.ss_winattn_step(q, k, v, table[:1], lengths, 5),
                lambda: ss.ss_winattn_step(q, k, v, table, None, 5), lambda: ss.ss_winattn_step(q, k, v, table.T.contiguous().T, lengths, 5),
                lambda: ss.ss_winattn_step(q[..., :32], k, v, table, lengths, 5),
                lambda: ss.ss_kv_append(new, new, k, v, table, None), lambda: ss.ss_kv_append(new, new.float(), k, v, table, lengths),
                lambda: ss.ss_kv_append(new, new, k, v, table, lengths, q_out=q), lambda: ss.ss_rotate(q, freqs(4).double()),
                lambda: ss.ss_kv_append(new[..., :8], new[..., :8], k, v, table, lengths), lambda: ss.ss_rotate(q, freqs(4), k_out=q)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ss.ss_winattn_step(q, k, v, table, lengths, 0), lambda: ss.ss_winattn_step(q[:, :, :3], k, v, table, lengths, 5),
                lambda: ss.ss_rotate(q, freqs(33)), lambda: ss.ss_kv_append(new, new, k, v, table, lengths, inv_freq=freqs(40))):
        with pytest.raises(ss.SSError):
            bad()


# ---- all of them together


@TYPES
@pytest.mark.parametrize("d", [64, 128])
def test_a_dialogue(dtype, d):
    """A prompt appended and attended over, then tokens one at a time and three at once, through the cache: every output is
    that of one long prompt whose rotated keys the cache holds."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    batch, heads, kv, page, window, sinks, inv = 2, 6, 2, 16, 50, 3, freqs(d // 2)
    prompt, total = [70, 41], 80
    q, k, v = rand(gen, batch, total, heads, d).to(dtype), rand(gen, batch, total, kv, d).to(dtype), rand(gen, batch, total, kv, d).to(dtype)
    pools = [torch.full((12, page, kv, d), float("nan"), device="cuda", dtype=dtype) for _ in range(2)]
    table = torch.randperm(12, device="cuda", generator=gen)[:10].int().view(2, 5)
    held = torch.zeros(2, dtype=torch.int32, device="cuda")
    lengths = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    qr, kr = ss.ss_kv_append(k[:, :70], v[:, :70], *pools, table, held, inv_freq=inv, q=q[:, :70], counts=lengths, return_k=True)
    o, _ = ss.ss_winattn_fwd(qr, kr, v[:, :70], window, sinks=sinks, lengths=lengths)
    rq, rk = ss.ss_rotate(q, inv, k=k)
    ref, by = P.attention(rq, rk, v, window, sinks)["o"]
    for b, n in enumerate(prompt):
        P.check("prompt", o[b, :n], ref[b, :n], by[b, :n])
    held = lengths.clone()
    for new in (1, 1, 3, 1):
        at = held[:, None].long() + torch.arange(new, device="cuda")
        rows = torch.arange(batch, device="cuda")[:, None], at
        qr, _ = ss.ss_kv_append(k[rows], v[rows], *pools, table, held, inv_freq=inv, q=q[rows])
        assert torch.equal(qr, rq[rows])
        held = held + new
        o = ss.ss_winattn_step(qr, *pools, table, held, window, sinks=sinks)
        P.check("step", o, ref[rows], by[rows] + ref[rows].abs() * 2.0 ** -20)
    assert ss.ss_last_device_error() == ss.SS_OK


@TYPES
def test_a_training_step_through_the_rotation(dtype):
    """Gradients of the queries and keys before the rotation: turned back from those behind it."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    q, k, v, do = (rand(gen, 1, 90, n, 32).to(dtype) for n in (4, 2, 2, 4))
    inv = freqs(16)
    rq, rk = ss.ss_rotate(q, inv, k=k)
    o, lse = ss.ss_winattn_fwd(rq, rk, v, 40, sinks=2)
    g = ss.ss_winattn_bwd(rq, rk, v, o, lse, do, 40, sinks=2)
    dq, dk = ss.ss_rotate(g["dq"], inv, k=g["dk"], inverse=True)
    leaves = [x.double().requires_grad_() for x in (q, k, v)]
    turned = [P.rotate(x, [0], inv) for x in leaves[:2]]  # differentiable
    share = torch.arange(4, device="cuda") // 2
    s = torch.einsum("blhd,bmhd->bhlm", _turn(leaves[0], inv), _turn(leaves[1], inv)[:, :, share]) * 32 ** -0.5
    p = torch.softmax(s.masked_fill(~P.mask(90, 40, 2, "cuda"), -float("inf")), -1)
    want = torch.autograd.grad(torch.einsum("bhlm,bmhd->blhd", p, leaves[2][:, :, share]), leaves, do.double())
    assert len(turned) == 2
    for name, x, y in (("dq", dq, want[0]), ("dk", dk, want[1]), ("dv", g["dv"], want[2])):
        # the rotated operands are rounded once, the gradients twice: relative to the norm, some half steps of the type
        assert float((x.double() - y).norm() / y.norm()) < (2.0 ** -7 if dtype == BF16 else 2.0 ** -18), name


def _turn(x, inv):
    half = inv.shape[0]
    a = torch.arange(x.shape[1], device=x.device).double()[:, None] * inv.double()
    c, s = a.cos()[:, None], a.sin()[:, None]
    u, w = x[..., :half], x[..., half:]
    return torch.cat([u * c - w * s, u * s + w * c], -1)


# ---- graphs, streams


@TYPES
def test_captured_and_replayed(dtype):
    """Decoding steps as a graph: lengths and tokens change between replays."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    batch, heads, kv, d, page, inv = 3, 4, 2, 64, 16, freqs(32)
    k, v, q = (rand(gen, batch, 30, n, d).to(dtype) for n in (kv, kv, heads))
    table = torch.arange(batch * 3, device="cuda").int().view(batch, 3)
    make = lambda: [torch.zeros(batch * 3, page, kv, d, device="cuda", dtype=dtype) for _ in range(2)]  # noqa: E731
    pools, held = make(), torch.zeros(batch, dtype=torch.int32, device="cuda")
    want = []
    for t in range(30):
        qr, _ = ss.ss_kv_append(k[:, t:t + 1], v[:, t:t + 1], *pools, table, held + t, inv_freq=inv, q=q[:, t:t + 1])
        want.append(ss.ss_winattn_step(qr, *pools, table, held + t + 1, 12, sinks=2))
    pools = make()
    sk, sv, sq = (x[:, :1].clone() for x in (k, v, q))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        qr, _ = ss.ss_kv_append(sk, sv, *pools, table, held, inv_freq=inv, q=sq)
        held += 1
        o = ss.ss_winattn_step(qr, *pools, table, held, 12, sinks=2)
    held.zero_()
    for t in range(30):
        for x, y in zip((sk, sv, sq), (k, v, q)):
            x.copy_(y[:, t:t + 1])
        graph.replay()
        assert torch.equal(o, want[t]), t
    assert ss.ss_last_device_error() == ss.SS_OK


@pytest.mark.parametrize("d", [64, 128])
def test_training_captured_on_two_streams(d):
    """Forward and backward of two calls at once in one graph, each with a workspace of its own."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    sets = [tuple(rand(gen, 1, 1100, n, d).bfloat16() for n in (4, 2, 2, 4)) for _ in range(2)]

    def step(q, k, v, do, **kw):
        o, lse = ss.ss_winattn_fwd(q, k, v, 30, sinks=3, **kw)
        return [o, lse, *ss.ss_winattn_bwd(q, k, v, o, lse, do, 30, sinks=3, **kw).values()]

    want = [step(*x) for x in sets]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        other = step(*sets[1], stream=side)
        mine = step(*sets[0])
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(mine + other, want[0] + want[1]))
    assert ss.ss_last_device_error() == ss.SS_OK


def test_a_stream_of_the_callers_with_the_current_one_busy():
    gen = torch.Generator(device="cuda").manual_seed(10)
    q, k, v, do = (rand(gen, 2, 700, n, 64).bfloat16() for n in (4, 2, 2, 4))
    lengths = torch.tensor([700, 123], dtype=torch.int32, device="cuda")
    cached, inv = cache(2, [300, 200], 1, 4, 2, 64, 16, BF16), freqs(32)  # made before the current stream is busy
    o, lse = ss.ss_winattn_fwd(q, k, v, 50, lengths=lengths)
    calls = [lambda **s: ss.ss_winattn_fwd(q, k, v, 50, lengths=lengths, **s),
             lambda **s: tuple(ss.ss_winattn_bwd(q, k, v, o, lse, do, 20, sinks=2, lengths=lengths, **s).values()),
             lambda **s: (ss.ss_winattn_step(*cached, 100, **s),),
             lambda **s: ss.ss_rotate(q, inv, k=k, counts=lengths, **s)]
    side = torch.cuda.Stream()
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        torch.cuda._sleep(30_000_000)
        got = call(stream=side)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    torch.cuda.synchronize()
    assert ss.ss_last_device_error() == ss.SS_OK
