"""The 64-bit linear attention that the GPU tests compare with, held to what the
definition fixes: brute-force sums, and central differences for the gradients."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests import linattn_plain as P  # noqa: E402


def _inputs(batch=2, L=5, heads=4, qk_heads=2, dk=3, dv=2, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    return dict(q=r(batch, L, qk_heads, dk), k=r(batch, L, qk_heads, dk), v=r(batch, L, heads, dv),
                g=-r(batch, L, heads).abs(), s0=r(batch, heads, dk, dv)), r


def test_forward_is_the_unrolled_sum():
    x, _ = _inputs()
    o, last = P.forward(**x, scale=0.7)
    b, h, L = 1, 3, 5
    g, share = x["g"][b, :, h], 2
    for t in range(L):
        want = torch.zeros(2, dtype=torch.float64)
        q = x["q"][b, t, h // share]
        for j in range(t + 1):
            want += math.exp(g[j + 1:t + 1].sum()) * (q @ x["k"][b, j, h // share]) * x["v"][b, j, h]
        want += math.exp(g[:t + 1].sum()) * (q @ x["s0"][b, h])
        assert torch.allclose(o[b, t, h], 0.7 * want, rtol=1e-12, atol=1e-12)
    assert torch.allclose(P.forward(**{**x, "q": x["q"][:, :, :, :]})[1], last)


def test_lengths_stop_a_row():
    x, _ = _inputs()
    lengths = torch.tensor([3, 0])
    o, last = P.forward(**x, lengths=lengths)
    cut = {n: (t if n == "s0" else t[:, :3]) for n, t in x.items()}
    o3, last3 = P.forward(**cut)
    assert torch.equal(o[0, :3], o3[0]) and torch.equal(last[0], last3[0])
    assert torch.equal(last[1], x["s0"][1]) and not o[1].any() and not o[0, 3:].any()


@pytest.mark.parametrize("lengths", [None, [4, 2]])
def test_gradients_are_differences(lengths):
    x, r = _inputs(seed=3)
    lengths = None if lengths is None else torch.tensor(lengths)
    do, dlast = r(2, 5, 4, 2), r(2, 4, 3, 2)
    grads = P.backward(x["q"], x["k"], x["v"], x["g"], do, 0.7, x["s0"], dlast, lengths)

    def loss(y):
        o, last = P.forward(**y, scale=0.7, lengths=lengths)
        live = P._live(y["g"], lengths)[..., None, None]
        return float((o * do * live).sum() + (last * dlast).sum())

    for name, of in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dlog_decay"), ("s0", "dinitial_state")):
        along = torch.randn(x[name].shape, dtype=torch.float64, generator=torch.Generator().manual_seed(9))
        eps = 1e-5
        up, down = ({**x, name: x[name] + s * eps * along} for s in (1, -1))
        diff = (loss(up) - loss(down)) / (2 * eps)
        got = float((grads[of] * along).sum())
        # central differences: eps^2 times third derivatives of order one to a hundred
        assert abs(diff - got) <= 1e-7 * max(1.0, abs(got)), name


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("decay", [0.05, 2.0])
def test_the_decay_gradients_bound_rejects_mistakes(dtype, decay):
    """A flow through one border of 64 tokens left out, a wrong sign, a zero, a bf16 sum: none passes."""
    gen = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    L, d = 400, 16
    q, k, v, do = (r(1, L, 1, d).to(dtype) for _ in range(4))
    g, s0 = (-decay * r(1, L, 1).abs()).to(dtype), r(1, 1, d, d)
    ref, slack = P.decay_grad_bound(q, k, v, g, do, 0.25, s0)
    assert P.decay_grad_wrong(ref.to(dtype), ref, slack, dtype) == 0
    assert P.decay_grad_wrong(0 * ref, ref, slack, dtype) > 0.9 * L
    assert P.decay_grad_wrong(-ref, ref, slack, dtype) > 0.9 * L
    lost = ref.clone()
    lost[:, 128:192] -= P.backward(q, k, v, g, do, 0.25, s0)["dlog_decay"][:, 192:193]  # the flow at one border
    assert P.decay_grad_wrong(lost.to(dtype), ref, slack, dtype) > 32
    if dtype == torch.float32:
        assert P.decay_grad_wrong(ref.bfloat16(), ref, slack, dtype) > 0.5 * L


def test_what_bounds_the_state_of_bf16_prompts():
    """Keys weighted by their decay and kept as bf16 planes: two leave the state more than 2^-20 off, three do not."""
    gen = torch.Generator().manual_seed(1)
    L, d = 64, 64
    k, v = (torch.randn(L, d, generator=gen).bfloat16().double() for _ in range(2))
    w = torch.exp(torch.cumsum(-0.1 * torch.rand(L, generator=gen).double(), 0)).flip(0)
    ref = (k * w[:, None]).mT @ v
    off = []
    for planes in (2, 3):
        kept, rest = torch.zeros_like(k), k * w[:, None]
        for _ in range(planes):
            p = rest.bfloat16().double()
            kept, rest = kept + p, rest - p
        off.append(float((kept.mT @ v - ref).norm() / ref.norm()))
    assert off[0] > 2.0 ** -20 > 16 * off[1]
