"""Decays so slow that the state passes hundreds of chunks, whose roundings must not add up."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import selective_state_space_ss_b200 as ss  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def last_state(k, v, g):
    """In 64 bits, chunk by chunk."""
    s = torch.zeros(*g.shape[::2], k.shape[3], v.shape[3], dtype=torch.float64, device="cuda")
    for c in range(0, g.shape[1], 64):
        total = g[:, c:c + 64].double().cumsum(1)
        w = (total[:, -1:] - total).exp()
        s = s * total[:, -1].exp()[..., None, None]
        s = s + torch.einsum("bjhk,bjh,bjhv->bhkv", k[:, c:c + 64].double(), w, v[:, c:c + 64].double())
    return s


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads,L", [(2, 65536), (2, 65000), (160, 16384)], ids=["segments", "odd", "workers"])
@pytest.mark.parametrize("decay", [1e-3, 1e-4, 1e-5, 1e-6, 0.0])
def test_equal_slow_decays(dtype, heads, L, decay):
    """The state within 2^-20: 2^-24 for the factors it has passed, whose roundings are made up
    for, 2^-22 for a token's own weight, and the fp32 sums: a rounding of at most 2^-24 of the
    state a chunk, 2^-20 over 256 chunks if they all had one sign at that size, and a quarter
    of it as they have."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn(1, L, heads, 16, device="cuda", generator=gen).to(dtype) for _ in range(3))
    g = torch.full((1, L, heads), -decay, device="cuda").to(dtype)
    _, last = ss.ss_linattn_fwd(q, k, v, g)
    assert ss.ss_last_device_error() == ss.SS_OK
    want = last_state(k, v, g)
    assert float((last.double() - want).norm() / want.norm()) <= 2.0 ** -20


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_equal_slow_decays_backward(dtype):
    """The initial state's gradient passes the same factors the other way."""
    heads, L, decay = 160, 16384, 1e-6
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, k, v, do = (torch.randn(1, L, heads, 16, device="cuda", generator=gen).to(dtype) for _ in range(4))
    g = torch.full((1, L, heads), -decay, device="cuda").to(dtype)
    s0 = torch.zeros(1, heads, 16, 16, device="cuda")
    got = ss.ss_linattn_bwd(q, k, v, g, do, initial_state=s0)["dinitial_state"]
    # R before the first token: the last state of (q, do) run backwards, its first token's decay at the end
    want = last_state(q.flip(1), do.flip(1), g) * float(g[0, 0, 0].double().exp())
    assert float((got.double() - want).norm() / want.norm()) <= 2.0 ** -20
