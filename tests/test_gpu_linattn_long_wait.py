"""A CTA that has nothing to do before its part of a long head waits for another's state for
milliseconds, and gets it."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import selective_state_space_ss_b200 as ss  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_rows_of_no_tokens_behind_a_long_one(dtype):
    """192 heads: of the CTA that ends the long row's last head the rest is in empty rows, so
    it waits from its start until the one before it is 40 to 50% through that head."""
    L, heads = (300_000, 64) if dtype == torch.bfloat16 else (100_000, 64)
    gen = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    q, k = r(1, L, 1, 8).to(dtype).expand(3, L, 1, 8), r(1, L, 1, 8).to(dtype).expand(3, L, 1, 8)
    v = r(1, L, heads, 8).to(dtype).expand(3, L, heads, 8)
    g = (-0.05 * r(1, L, heads).abs()).to(dtype).expand(3, L, heads)
    lengths = torch.tensor([L, 0, 0], dtype=torch.int32, device="cuda")
    o, last = ss.ss_linattn_fwd(q, k, v, g, lengths=lengths)
    assert ss.ss_last_device_error() == ss.SS_OK
    want_o, want = ss.ss_linattn_fwd(q[:1], k[:1], v[:1], g[:1])  # cut into segments, no CTA waits for another
    assert ss.ss_last_device_error() == ss.SS_OK
    assert not last[1:].any() and not o[1:].any()
    assert float((last[0] - want[0]).norm() / want[0].norm()) < 1e-5
    step = torch.finfo(dtype).eps
    assert float((o[0] - want_o[0]).norm() / want_o[0].norm()) < max(step / 2, 1e-5)
