"""Linear attention with a decay per head, token by token in 64 bits, and its
gradients; and the same recurrence over magnitudes, from which the tests take how
much rounding a result may carry."""
from __future__ import annotations

import torch


def _heads(x, heads):
    return x.double().repeat_interleave(heads // x.shape[2], dim=2)


def _live(g, lengths):
    batch, L, _ = g.shape
    if lengths is None:
        return torch.ones(batch, L, dtype=torch.bool, device=g.device)
    return torch.arange(L, device=g.device) < lengths.to(g.device)[:, None]


def states(q, k, v, g, s0, lengths):
    """S before the first token and after each: [L + 1][batch, heads, dk, dv]."""
    heads = v.shape[2]
    live = _live(g, lengths)
    k, v, a = _heads(k, heads), v.double(), g.double().exp()
    s = torch.zeros(*a.shape[::2], k.shape[3], v.shape[3], dtype=torch.float64, device=v.device) if s0 is None else s0.double()
    out = [s]
    for t in range(g.shape[1]):
        new = s * a[:, t, :, None, None] + k[:, t, :, :, None] * v[:, t, :, None, :]
        s = torch.where(live[:, t, None, None, None], new, s)
        out.append(s)
    return out


def forward(q, k, v, g, scale=1.0, s0=None, lengths=None):
    """(o, last state); o is zero behind a row's length."""
    ss = states(q, k, v, g, s0, lengths)
    qh = _heads(q, v.shape[2])
    o = torch.stack([torch.einsum("bhk,bhkv->bhv", qh[:, t], ss[t + 1]) for t in range(g.shape[1])], 1) * scale
    return torch.where(_live(g, lengths)[..., None, None], o, torch.zeros_like(o)), ss[-1]


def backward(q, k, v, g, do, scale=1.0, s0=None, dlast=None, lengths=None):
    """Gradients by their formulas; dq_h and dk_h are those of each head before sharing heads are summed."""
    heads, qk_heads = v.shape[2], q.shape[2]
    live = _live(g, lengths)
    ss = states(q, k, v, g, s0, lengths)
    qh, kh, vd, a = _heads(q, heads), _heads(k, heads), v.double(), g.double().exp()
    r = torch.zeros_like(ss[0]) if dlast is None else dlast.double()
    dq, dk, dv, dg = [], [], [], []
    for t in reversed(range(g.shape[1])):
        m = live[:, t, None, None]
        d = do[:, t].double() * scale
        with_t = r + qh[:, t, :, :, None] * d[..., None, :]
        dq.append(torch.where(m, torch.einsum("bhkv,bhv->bhk", ss[t + 1], d), 0))
        dk.append(torch.where(m, torch.einsum("bhkv,bhv->bhk", with_t, vd[:, t]), 0))
        dv.append(torch.where(m, torch.einsum("bhkv,bhk->bhv", with_t, kh[:, t]), 0))
        back = with_t * a[:, t, :, None, None]
        dg.append(torch.where(m[..., 0], (back * ss[t]).sum((-1, -2)), 0))
        r = torch.where(m[..., None], back, r)
    dq, dk, dv, dg = (torch.stack(x[::-1], 1) for x in (dq, dk, dv, dg))
    share = (qk_heads, heads // qk_heads)
    return {"dq": dq.unflatten(2, share).sum(3), "dk": dk.unflatten(2, share).sum(3), "dv": dv, "dlog_decay": dg,
            "dinitial_state": r, "dq_h": dq, "dk_h": dk}


def decay_grad_bound(q, k, v, g, do, scale=1.0, s0=None, dlast=None, lengths=None):
    """(dlog_decay in 64 bits, what it may be off by before it is rounded).

    dg_t is a plain sum of products q do k v e^{sum of g}, without a difference that
    cancels.  A product is formed of a few rounded factors: the score or the state (planes
    of 16 bits for bf16 inputs, 24 for fp32) twice 2^-16 or 2^-24, an exponential good to
    2^-22 twice, and fp32 multiplications; in all below u = 2^-14 (bf16) or 2^-19 (fp32)
    with the fp32 sums' share.  Inputs of random signs have roundings of random signs, so
    the sum is off by about u times the root of the sum of squared products, and eight
    times that is hardly ever passed.  That sum is the same gradient over squared inputs.
    """
    u = 2.0 ** -14 if q.dtype == torch.bfloat16 else 2.0 ** -19
    sq = lambda t: None if t is None else t.double() ** 2  # noqa: E731
    ref = backward(q, k, v, g, do, scale, s0, dlast, lengths)["dlog_decay"]
    squares = backward(sq(q), sq(k), sq(v), 2 * g.double(), sq(do), scale ** 2, sq(s0), sq(dlast), lengths)["dlog_decay"]
    return ref, 8 * u * squares.sqrt()


def decay_grad_wrong(got, ref, slack, dtype):
    """How many elements of a decay's gradient are further off than the bound and one rounding to `dtype`."""
    half = torch.finfo(dtype).eps / 2
    over = (got.double() - ref).abs() - (1 + half) * slack - half * ref.abs()
    # an exponential below the smallest normal number is zero, whatever up to 2^16 it multiplies
    return int((~(over <= 2.0 ** -110)).sum())
