"""The log decays' gradient of ss_linattn_bwd, element by element, at decays from hardly any
to nearly all, against the definition in 64 bits (tests/linattn_plain.py has the bound)."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import selective_state_space_ss_b200 as ss  # noqa: E402
from tests import linattn_plain as P  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
both = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])


def make(batch, L, heads, qk_heads, dk, dv, dtype, decay, state=True, seed=3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    x = {"q": r(batch, L, qk_heads, dk).to(dtype), "k": r(batch, L, qk_heads, dk).to(dtype),
         "v": r(batch, L, heads, dv).to(dtype), "g": (-decay * torch.exp(0.5 * r(batch, L, heads) - 0.125)).to(dtype),
         "do": r(batch, L, heads, dv).to(dtype)}
    x["s0"], x["dlast"] = (r(batch, heads, dk, dv), r(batch, heads, dk, dv)) if state else (None, None)
    return x


def grad(x, scale=1.0, lengths=None):
    got = ss.ss_linattn_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], scale=scale, initial_state=x["s0"],
                            dlast_state=x["dlast"], lengths=lengths)
    assert ss.ss_last_device_error() == ss.SS_OK
    return got["dlog_decay"]


def check(x, got, scale=1.0, lengths=None):
    dtype = x["q"].dtype
    ref, slack = P.decay_grad_bound(*(x[n] for n in ("q", "k", "v", "g", "do")), scale, x["s0"], x["dlast"], lengths)
    assert P.decay_grad_wrong(got, ref, slack, dtype) == 0
    # over all: roundings of 2^-24 or so, at most sixteen in a row, and the output's own
    size = max(float(ref.norm()), float(slack.norm()) / 8 * (2.0 ** 14 if dtype == BF16 else 2.0 ** 19))  # as random signs give it
    off = float((got.double() - ref).norm()) / size if size else float(got.double().norm())
    assert off <= (2.0 ** -8 if dtype == BF16 else 2.0 ** -20), off


@both
@pytest.mark.parametrize("decay", [0.003, 0.1, 1.6, 6.0, 10.0, 40.0])
@pytest.mark.parametrize("dk,dv,L", [(64, 64, 330), (128, 128, 200), (64, 128, 131), (37, 21, 150)])
def test_decays_of_every_size(dtype, decay, dk, dv, L):
    x = make(2, L, 4, 2, dk, dv, dtype, decay)
    check(x, grad(x, dk ** -0.5), dk ** -0.5)


@both
@pytest.mark.parametrize("L", [1, 2, 16, 17, 63, 64, 65, 129])
@pytest.mark.parametrize("state", [False, True])
def test_lengths_of_a_chunk(dtype, L, state):
    x = make(1, L, 3, 1, 24, 40, dtype, 0.3, state)
    check(x, grad(x))


@both
@pytest.mark.parametrize("sizes", [(1, 2600, 1, 1, 32, 64), (1, 1700, 2, 1, 128, 128), (1, 1500, 1, 1, 100, 65),
                                   (3, 200, 60, 20, 32, 48), (2, 150, 80, 80, 128, 64)])
@pytest.mark.parametrize("ragged", [False, True])
def test_long_and_many(dtype, sizes, ragged):
    """Sequences cut into segments, and more heads than SMs."""
    x = make(*sizes, dtype, 0.05)
    batch, L = sizes[:2]
    lengths = torch.tensor([L - 70, 0, 65][:batch], dtype=torch.int32, device="cuda") if ragged else None
    got = grad(x, lengths=lengths)
    check(x, got, lengths=lengths)
    if ragged:
        assert not got[0, L - 70:].any() and (batch == 1 or not got[1].any())


@both
def test_a_reset_has_no_gradient_and_its_neighbours_theirs(dtype):
    x = make(2, 200, 2, 2, 64, 64, dtype, 0.2)
    at = [0, 5, 63, 64, 65, 130, 199]
    x["g"][:, at] = -math.inf
    got = grad(x)
    assert not got[:, at].any()
    check(x, got)


@both
def test_strided_rows_and_a_token_that_forgets(dtype):
    """Plain loads (odd offsets), and single strong decays among weak ones."""
    x = make(1, 190, 4, 2, 40, 24, dtype, 0.02)
    x["g"][0, [20, 100, 101]] = -25.0
    for n in ("q", "k", "v", "do"):
        b, L, h, d = x[n].shape
        wide = torch.zeros(b, L, h * d + 1, dtype=dtype, device="cuda")
        wide[..., 1:] = x[n].flatten(2)
        x[n] = wide[..., 1:].unflatten(-1, (h, d))
    check(x, grad(x))
