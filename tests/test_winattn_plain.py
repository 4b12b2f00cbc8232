"""The 64-bit reference of the window attention against the definition token by token and
against differences, and its bounds against planted mistakes.  CPU only."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests import winattn_plain as P  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def make(batch=2, L=9, heads=4, kv_heads=2, d=5, dtype=F32, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen).to(dtype)  # noqa: E731
    return r(batch, L, heads, d), r(batch, L, kv_heads, d), r(batch, L, kv_heads, d), r(batch, L, heads, d)


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 0), (3, 2), (1, 9), (100, 0), (4, 100)])
def test_forward_is_the_definition(window, sinks):
    q, k, v, _ = make()
    lengths = torch.tensor([9, 4])
    out = P.attention(q, k, v, window, sinks, 0.3, lengths)
    for b, n in enumerate([9, 4]):
        for h in range(4):
            for t in range(9):
                o, lse = [0.0] * 5, 0.0
                if t < n:
                    js = [j for j in range(t + 1) if t - j < window or j < sinks]
                    w = [math.exp(0.3 * sum(float(q[b, t, h, c]) * float(k[b, j, h // 2, c]) for c in range(5))) for j in js]
                    o = [sum(x * float(v[b, j, h // 2, c]) for x, j in zip(w, js)) / sum(w) for c in range(5)]
                    lse = math.log(sum(w))
                assert out["lse"][0][b, h, t] == pytest.approx(lse, abs=1e-12)
                assert out["o"][0][b, t, h].tolist() == pytest.approx(o, abs=1e-12)


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (100, 0)])
def test_gradients_are_the_differences(window, sinks):
    q, k, v, do = (x.double() for x in make(batch=1, L=6))
    out = P.attention(q, k, v, window, sinks, do=do)
    loss = lambda *x: float((P.attention(*x, window, sinks)["o"][0] * do).sum())  # noqa: E731
    for i, name in enumerate(("dq", "dk", "dv")):
        x = (q, k, v)[i]
        for at in [(0, 0, 0, 0), (0, 3, 1, 2), (0, 5, 0, 4), (0, 2, 1, 1)]:
            both = []
            for step in (1e-5, -1e-5):
                y = [t.clone() for t in (q, k, v)]
                y[i][at] += step
                both.append(loss(*y))
            assert float(out[name][0][at]) == pytest.approx((both[0] - both[1]) / 2e-5, abs=1e-8), (name, at, x.shape)


def test_a_cache_is_the_prompt_at_its_end():
    q, k, v, _ = make(batch=2, L=11)
    table = torch.tensor([[3, 0, 5, -1], [1, 4, 2, 9]])
    pools = [torch.full((6, 4, 2, 5), math.nan) for _ in range(2)]
    for b in range(2):
        for t in range(11):
            for pool, x in zip(pools, (k, v)):
                pool[table[b, t // 4], t % 4] = x[b, t]
    want = P.attention(q, k, v, 5, 2, lengths=[11, 7])["o"][0]
    got, _ = P.step(torch.stack([q[0, 8:11], q[1, 4:7]]), *pools, table, [11, 7], 5, 2)
    torch.testing.assert_close(got, torch.stack([want[0, 8:11], want[1, 4:7]]))


def test_a_rotation_keeps_lengths_and_turns_back():
    x = torch.randn(2, 7, 3, 10, dtype=torch.float64)
    f = torch.tensor([1.0, 0.1, 0.01, 0.5])
    for inter in (False, True):
        y, _ = P.rotate(x, [0, 100], f, inter)
        torch.testing.assert_close(y.norm(dim=-1), x.norm(dim=-1))
        torch.testing.assert_close(P.rotate(y, [0, 100], f, inter, inverse=True)[0], x)
        assert torch.equal(y[..., 8:], x[..., 8:])
        one = y[1, 2, 0, 0], y[1, 2, 0, 1 if inter else 4]
        a, (p, q) = 102.0, (x[1, 2, 0, 0], x[1, 2, 0, 1 if inter else 4])
        assert float(one[0]) == pytest.approx(float(p * math.cos(a) - q * math.sin(a)))
        assert float(one[1]) == pytest.approx(float(p * math.sin(a) + q * math.cos(a)))


def emulated(q, k, v, do, window, sinks, mistake=""):
    """The kernels' arithmetic in torch, fp32 with bf16 operands, and a planted mistake."""
    L, d = q.shape[1], q.shape[3]
    share = q.shape[2] // k.shape[2]
    Q, K, V, G = (x.float().transpose(1, 2) for x in (q, k.repeat_interleave(share, 2), v.repeat_interleave(share, 2), do))
    seen = P.mask(L, window + (mistake == "window"), sinks - (mistake == "sinks"), q.device)
    if mistake == "future":
        seen = seen | torch.eye(L, dtype=torch.bool).roll(1, 1) & (torch.arange(L) < L - 1)[:, None]
    s = (Q @ K.mT) * d ** -0.5
    if mistake == "scale":
        s = s * (1 + 2.0 ** -6)
    s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1)
    r = lambda x: x.to(q.dtype).float()  # noqa: E731
    p = torch.exp(s - lse[..., None])
    o = r(r(p) @ V)
    if mistake == "row" and L > 3:
        o[:, :, 3] = o[:, :, 2]
    delta = (G * o).sum(-1, keepdim=True) * (0.9 if mistake == "delta" else 1)
    ds = p * (G @ V.mT - delta)
    back = lambda x, n: r(x.unflatten(1, (-1, n)).sum(2)).transpose(1, 2)  # noqa: E731
    return {"o": o.transpose(1, 2).to(q.dtype), "dq": (r(ds) @ K * d ** -0.5).transpose(1, 2).to(q.dtype),
            "dk": back(r(ds).mT @ Q * d ** -0.5, share).to(q.dtype), "dv": back(r(p).mT @ G, share).to(q.dtype)}


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_the_bounds_hold_for_the_arithmetic_and_not_for_mistakes(dtype):
    q, k, v, do = make(1, 70, 4, 2, 24, dtype)
    ref = P.attention(q, k, v, 20, 3, do=do)
    for name, x in emulated(q, k, v, do, 20, 3).items():
        P.check(name, x, *ref[name])
    for mistake, names in (("window", "o dq dk dv"), ("sinks", "o dq dk dv"), ("future", "o dq dk dv"), ("row", "o"),
                           ("delta", "dq dk")) + ((("scale", "o dq dk"),) if dtype == F32 else ()):
        bad = emulated(q, k, v, do, 20, 3, mistake)
        for name in names.split():
            with pytest.raises(AssertionError):
                P.check(name, bad[name], *ref[name])
