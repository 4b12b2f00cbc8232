"""Heads of every width class cut into segments, and cut between CTAs where there are more
heads than SMs, forward and backward; and the fp32 state of bf16 prompts held to fp32."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import selective_state_space_ss_b200 as ss  # noqa: E402
from tests import linattn_plain as P  # noqa: E402
from tests.test_gpu_linattn import BF16, F32, bwd, check_bwd, check_fwd, fwd, make  # noqa: E402

both = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
wide = pytest.mark.parametrize("dk,dv", [(128, 128), (128, 64), (64, 128), (100, 65)])


def check_all(x, r, lengths):
    batch, L, heads, dv = x["v"].shape
    dk, dtype = x["q"].shape[3], x["v"].dtype
    o, last = fwd(x, lengths=lengths)
    assert ss.ss_last_device_error() == ss.SS_OK
    check_fwd(x, o, last, lengths=lengths)
    do, dlast = r(batch, L, heads, dv).to(dtype), r(batch, heads, dk, dv)
    got = bwd(x, do, dlast, lengths=lengths)
    assert ss.ss_last_device_error() == ss.SS_OK
    check_bwd(x, do, dlast, got, 1.0, lengths)
    ref, slack = P.decay_grad_bound(x["q"], x["k"], x["v"], x["g"], do, 1.0, x["s0"], dlast, lengths)
    assert P.decay_grad_wrong(got["dlog_decay"], ref, slack, dtype) == 0
    again = bwd(x, do, dlast, lengths=lengths)
    for n in got:
        assert torch.equal(got[n], again[n]), n


@both
@wide
@pytest.mark.parametrize("ragged", [False, True])
def test_segments(dtype, dk, dv, ragged):
    x, r = make(2, 1400, 2, 1, dk, dv, dtype)
    code = ss.SS_BF16 if dtype == BF16 else ss.SS_F32
    assert ss.ss_linattn_workspace_bytes(2, 1400, 2, 1, dk, dv, code) > 0  # it is cut
    check_all(x, r, torch.tensor([0, 777], dtype=torch.int32, device="cuda") if ragged else None)


@both
@wide
@pytest.mark.parametrize("ragged", [False, True])
def test_more_heads_than_sms(dtype, dk, dv, ragged):
    """156 or 170 heads: each SM takes an equal range of all chunks, most heads are cut between two."""
    batch, heads = (3, 52) if dv != 65 else (5, 34)
    x, r = make(batch, 330, heads, 2, dk, dv, dtype)
    lengths = torch.tensor([65, 330, 0, 0, 200][:batch], dtype=torch.int32, device="cuda") if ragged else None
    check_all(x, r, lengths)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (37, 100)])
@pytest.mark.parametrize("cut", ["whole", "segments", "workers"])
def test_the_state_of_bf16_prompts_is_good_to_fp32(dk, dv, cut):
    """Within 2^-20: an exponential good to 2^-22 for the token and one for the chunk or two
    that these decays leave, and roundings of 2^-24.  (Keys weighted to 16 bits are 2.5e-6
    off: tests/test_linattn_plain.py.)"""
    batch, L, heads = {"whole": (2, 200, 2), "segments": (1, 1400, 2), "workers": (2, 200, 90)}[cut]
    x, r = make(batch, L, heads, 1, dk, dv, BF16)
    x["g"] = (-0.02 - 0.1 * r(batch, L, heads).abs()).to(BF16)
    _, last = fwd(x)
    _, ref = P.forward(x["q"], x["k"], x["v"], x["g"], 1.0, x["s0"])
    assert float((last.double() - ref).norm() / ref.norm()) <= 2.0 ** -20
    do = r(batch, L, heads, dv).to(BF16)
    got = bwd(x, do)["dinitial_state"]
    ref = P.backward(x["q"], x["k"], x["v"], x["g"], do, 1.0, x["s0"])["dinitial_state"]
    assert float((got.double() - ref).norm() / ref.norm()) <= 2.0 ** -20
