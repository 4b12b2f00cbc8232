"""Attention over a window with sinks in 64 bits, its gradients, the paged cache and the
rotation, token by token where that is affordable; and what a result may be off by,
counted from magnitudes.

The bounds, element by element.  u is the rounding of an operand that the kernel forms
itself (probabilities, their gradients) to the inputs' type on the way into a product:
eps / 2 = 2^-8 for bf16, nothing for fp32.  e32 = 2^-23 is an fp32 addition or product on
the tensor core (which may truncate).

  scores       a sum of d products: |s'_tj - s_tj| <= scale (d + 8) e32 sum |q||k|
  exponents    s log2 e - m and its power of two, ex2 good to 2^-22: with the error of the
               score e_tj = scale (d + 8) e32 sum|q||k| + 4 e32 (|s_tj| + |m_t|) + 2^-21 of
               a probability, e_t the largest of a row's
  outputs      o: sum_j p|v| (2 e_t + u + (n + 64) e32), numerator and normaliser each off
               by e_t, n additions and as many rescalings as tiles; lse: e_t + (n + 64) e32
               + 4 e32 (|lse| + 1)
  gradients    the probability from the saved normaliser: g_t = e_t + the lse's bound;
               do.v: a = (d + 8) e32 sum|do||v|;  do.o: D = sum|do| (bound of o) + (d + 8)
               e32 sum|do||o|;  ds: p (a + D) (1 + g + u) + |ds| (g + u + 4 e32);
               dq: scale sum_j (ds's)|k| + n e32 sum|ds||k|, dk alike over t, dv: sum_t
               p|do| (g + u + (n + 64) e32)
  underflow    powers of two, and operands, below 2^-126 may come out as zero: that much of
               every p and of every ds, absolutely
  the end      half a step of the output's type, of the value and of the bound
"""
from __future__ import annotations

import math

import torch

E32 = 2.0 ** -23
TINY = 2.0 ** -126


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def mask(L, window, sinks, device):
    t = torch.arange(L, device=device)
    return (t[None, :] <= t[:, None]) & ((t[:, None] - t[None, :] < window) | (t[None, :] < sinks))


def attention(q, k, v, window, sinks=0, scale=None, lengths=None, do=None):
    """{name: (value, bound)} for o, lse and, with do, dq, dk, dv; zero behind a row's length."""
    batch, L, heads, d = q.shape
    kv_heads, dtype = k.shape[2], q.dtype
    share, scale = heads // kv_heads, d ** -0.5 if scale is None else scale
    u = half_step(dtype) if dtype == torch.bfloat16 else 0.0
    f64 = dict(dtype=torch.float64, device=q.device)
    names = [("o", q.shape), ("lse", (batch, heads, L))]
    if do is not None:
        names += [("dq", q.shape), ("dk", k.shape), ("dv", v.shape)]
    out = {n: (torch.zeros(s, **f64), torch.zeros(s, **f64)) for n, s in names}
    for b in range(batch):
        n = L if lengths is None else min(max(int(lengths[b]), 0), L)
        if n == 0:
            continue
        seen = mask(n, window, sinks, q.device)
        count = int(seen.sum(-1).max())
        for h in range(heads):
            Q, K, V = q[b, :n, h].double(), k[b, :n, h // share].double(), v[b, :n, h // share].double()
            s = (Q @ K.T * scale).masked_fill(~seen, -math.inf)
            lse = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[:, None])
            o = p @ V
            top = s.amax(-1)
            e = scale * (d + 8) * E32 * (Q.abs() @ K.abs().T) + 4 * E32 * (s.abs() + top.abs()[:, None]) + 2.0 ** -21
            e = e.masked_fill(~seen, 0).amax(-1, keepdim=True)
            bo = (p @ V.abs()) * (2 * e + u + (count + 64) * E32) + 2 * TINY * (seen.double() @ V.abs())
            bl = e[:, 0] + (count + 64) * E32 + 4 * E32 * (lse.abs() + 1)
            out["o"][0][b, :n, h], out["o"][1][b, :n, h] = o, bo
            out["lse"][0][b, h, :n], out["lse"][1][b, h, :n] = lse, bl
            if do is None:
                continue
            G = do[b, :n, h].double()
            dp, delta = G @ V.T, (G * o).sum(-1, keepdim=True)
            ds = p * (dp - delta)
            g = e + bl[:, None]
            rounded = bo + half_step(dtype) * (o.abs() + bo)
            a = (d + 8) * E32 * (G.abs() @ V.abs().T)
            D = (G.abs() * rounded).sum(-1, keepdim=True) + (d + 8) * E32 * (G.abs() * o.abs()).sum(-1, keepdim=True)
            eds = p * (a + D) * (1 + g + u) + ds.abs() * (g + u + 4 * E32) + TINY * (dp.abs() + delta.abs() + a + D + 1) * seen
            for name, at, value, bound in (
                    ("dq", h, scale * ds @ K, scale * (eds @ K.abs() + count * E32 * (ds.abs() @ K.abs()))),
                    ("dk", h // share, scale * ds.T @ Q, scale * (eds.T @ Q.abs() + n * share * E32 * (ds.abs().T @ Q.abs()))),
                    ("dv", h // share, p.T @ G, (p * (g + u + (n * share + 64) * E32) + TINY * seen).T @ G.abs())):
                out[name][0][b, :n, at] += value
                out[name][1][b, :n, at] += bound
    return out


def check(name, got, ref, by):
    """got against a value with its bound, rounded to got's type at the end."""
    got, half = got.double(), half_step(got.dtype)
    assert torch.isfinite(got).all(), name
    over = (got - ref).abs() - by * (1 + half) - half * ref.abs() - 1e-37
    assert (over <= 0).all(), f"{name}: {float(over.max()):.3g} over a bound of {float(by.max()):.3g}"


def step(q, k_pages, v_pages, table, lengths, window, sinks=0, scale=None):
    """(o, bound) of the newest tokens over the cache; tokens in no page are not seen."""
    batch, tokens, heads, d = q.shape
    pages, page, kv_heads, _ = k_pages.shape
    share, scale = heads // kv_heads, d ** -0.5 if scale is None else scale
    u = half_step(q.dtype) if q.dtype == torch.bfloat16 else 0.0
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    by = torch.zeros_like(o)
    table = table.tolist()
    for b in range(batch):
        n = min(max(int(lengths[b]), 0), len(table[b]) * page)
        for i in range(tokens):
            t = n - tokens + i
            js = [j for j in range(t + 1) if (t - j < window or j < sinks) and 0 <= table[b][j // page] < pages]
            if not js:
                continue
            at = torch.tensor([table[b][j // page] for j in js], device=q.device), torch.tensor([j % page for j in js], device=q.device)
            K, V = (x[at].double().repeat_interleave(share, 1) for x in (k_pages, v_pages))
            Q = q[b, i].double()
            s = torch.einsum("hd,jhd->hj", Q, K) * scale
            p = torch.softmax(s, -1)
            e = scale * (d + 8) * E32 * torch.einsum("hd,jhd->hj", Q.abs(), K.abs()) + 8 * E32 * s.abs().amax(-1, keepdim=True) + 2.0 ** -21
            e = e.amax(-1, keepdim=True)
            o[b, i] = torch.einsum("hj,jhd->hd", p, V)
            # the walk may be cut in 16 parts, each joined by two more products
            by[b, i] = torch.einsum("hj,jhd->hd", p, V.abs()) * (2 * e + u + (len(js) + 96) * E32 + 2.0 ** -21)
    return o, by


def rotate(x, starts, inv_freq, interleaved=False, inverse=False):
    """(value, bound): the turned pairs, off by the fp32 of sine and cosine and two products."""
    y, by = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    half = 0 if inv_freq is None else inv_freq.shape[0]
    if half == 0:
        return y, by
    at = torch.as_tensor(starts, device=x.device).double()[:, None] + torch.arange(x.shape[1], device=x.device).double()
    angle = at[..., None] * inv_freq.double() * (-1 if inverse else 1)
    c, s = angle.cos()[..., None, :], angle.sin()[..., None, :]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    xa, xb = x[..., a].double(), x[..., b].double()
    y[..., a], y[..., b] = xa * c - xb * s, xa * s + xb * c
    # sine and cosine: half a step of fp32 and, of a wide angle brought into +-pi, 2^-50 of it
    by[..., a] = by[..., b] = (xa.abs() + xb.abs()) * (3 * 2.0 ** -24 + angle.abs()[..., None, :] * 2.0 ** -50)
    return y, by
