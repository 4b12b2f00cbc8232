"""Attention over a window with sinks, its paged cache and the rotation of positions, as cases to measure.

What a hybrid model has between its recurrent layers: attention of token t to the
tokens j <= t with t - j < window, and to the first few (the sinks) however far:

    s_tj = scale * q_t . k_j,    o_t = sum_j softmax_j(s_tj) v_j

over a prompt (``ss_winattn_fwd``), its gradients (``ss_winattn_bwd``), the newest
tokens of each sequence over a paged cache (``ss_winattn_step``), keys and values
brought into that cache with their positions' rotation (``ss_kv_append``), and the
rotation by itself with its inverse, for training (``ss_rotate``).

``own`` false: the plain forms, elementary torch operations in 32 bits (angles in
64).  ``own`` true: the package's entry points.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_BASE = 10000.0


def _attn(op, name, batch, seqlen, heads, kv_heads, d, window, sinks, dtype, ragged=False):
    return {"name": name, "op": op, "batch": batch, "seqlen": seqlen, "heads": heads, "kv_heads": kv_heads, "d": d,
            "window": window, "sinks": sinks, "dtype": dtype, "ragged": ragged}


def _step(name, batch, context, heads, kv_heads, d, window, sinks, page, dtype, tokens=1):
    return {"name": name, "op": "step", "batch": batch, "context": context, "heads": heads, "kv_heads": kv_heads,
            "d": d, "window": window, "sinks": sinks, "page": page, "dtype": dtype, "tokens": tokens}


def _append(name, batch, seqlen, heads, kv_heads, d, rot, page, dtype, context, interleaved=False):
    return {"name": name, "op": "append", "batch": batch, "seqlen": seqlen, "heads": heads, "kv_heads": kv_heads,
            "d": d, "rot": rot, "page": page, "dtype": dtype, "context": context, "interleaved": interleaved}


def _rotate(name, batch, seqlen, heads, kv_heads, d, rot, dtype, inverse, interleaved=False):
    return {"name": name, "op": "rotate", "batch": batch, "seqlen": seqlen, "heads": heads, "kv_heads": kv_heads,
            "d": d, "rot": rot, "dtype": dtype, "inverse": inverse, "interleaved": interleaved}


def listed():
    return [
        # a short question, a prompt of odd length: latency counts
        _attn("fwd", "fwd_turn_b1_l203_h8_bf16", 1, 203, 8, 8, 64, 128, 4, "bf16"),
        # a 5120-wide model's batch of long prompts, the largest call
        _attn("fwd", "fwd_b4_l8192_h40_d128_w2048_bf16", 4, 8192, 40, 8, 128, 2048, 4, "bf16"),
        # a padded batch in fp32, the numerics reference of a training run
        _attn("fwd", "fwd_ragged_b6_l1000_h8_f32", 6, 1000, 8, 4, 64, 256, 16, "f32", ragged=True),
        # training steps: a 512-wide model in fp32, a 1536-wide one with shared keys and values, long and odd sequences
        _attn("bwd", "bwd_b2_l1024_h8_f32", 2, 1024, 8, 8, 64, 256, 0, "f32"),
        _attn("bwd", "bwd_b8_l2048_h24_shared_bf16", 8, 2048, 24, 8, 64, 512, 4, "bf16"),
        _attn("bwd", "bwd_b2_l4097_h16_d128_bf16", 2, 4097, 16, 4, 128, 1024, 64, "bf16"),
        # generation: a few users (latency) and a full batch behind long contexts (bandwidth)
        _step("step_b4_h24_bf16", 4, 700, 24, 8, 64, 512, 4, 16, "bf16"),
        _step("step_b64_h40_d128_w4096_bf16", 64, 8192, 40, 8, 128, 4096, 16, 64, "bf16"),
        # the cache's side of the same: a token for each of a few users, a batch of prompts behind a shared beginning
        _append("append_b4_h24_bf16", 4, 1, 24, 8, 64, 64, 16, "bf16", 700),
        _append("append_b8_l2048_h40_d128_bf16", 8, 2048, 40, 8, 128, 128, 64, "bf16", 301),
        # training: queries and keys before the attention, and their gradients behind it
        _rotate("rotate_b8_l2048_h24_bf16", 8, 2048, 24, 8, 64, 64, "bf16", False),
        _rotate("rotate_grad_b2_l4097_h16_d128_bf16", 2, 4097, 16, 4, 128, 64, "bf16", True, interleaved=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "step", "append", "rotate"])
    kv_heads = _spread(rng, 1, 10)
    case = {"op": op, "kv_heads": kv_heads, "heads": kv_heads * rng.choice([1, 2, 3, 5, 8]),
            "d": rng.choice([32, 64, 64, 128, 128, 8 * rng.randint(2, 15), rng.randint(9, 127)]),
            "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"])}
    heads, d = case["heads"], case["d"]
    if op in ("append", "rotate"):
        case["rot"] = rng.choice([d // 2 * 2, d // 4 * 2])
        case["interleaved"] = rng.random() < 0.3
        case["seqlen"] = _spread(rng, 1, 4000)
        case["batch"] = _spread(rng, 1, max(1, min(64, 4_000_000 // (case["seqlen"] * heads))))
        if op == "rotate":
            return {**case, "inverse": rng.random() < 0.5}
        return {**case, "page": rng.choice([16, 32, 64, 100]), "context": _spread(rng, 1, 5000) - 1}
    case["sinks"] = rng.choice([0, 1, 4, 16, rng.randint(0, 200)])
    if op == "step":
        case["window"] = _spread(rng, 1, 70000)
        case["page"] = rng.choice([16, 32, 64, 100])
        case["tokens"] = rng.choice([1, 1, 1, 1, 2, 5])
        most = 500_000_000 // (kv_heads * d)
        case["context"] = _spread(rng, 8, min(70000, most))
        case["batch"] = _spread(rng, 1, max(1, min(128, most // case["context"])))
        return case
    case["window"] = _spread(rng, 1, 9000)
    case["ragged"] = rng.random() < 0.3
    pairs = (2_000_000_000 if op == "fwd" else 600_000_000) // (4 if case["dtype"] == "f32" or d % 8 else 1)
    seqlen = _spread(rng, 1, 20000)
    while heads * seqlen * min(seqlen, case["window"] + 500) > pairs:
        seqlen = seqlen * 2 // 3
    most = pairs // (heads * seqlen * min(seqlen, case["window"] + 500))
    return {**case, "seqlen": seqlen, "batch": rng.randint(1, max(1, min(8, most)))}


def _frequencies(rot):
    return (_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = _TYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=gen, dtype=dtype)

    def randint(lo, hi, *shape):
        return torch.randint(lo, hi, shape, device="cuda", generator=gen).int()

    op = case["op"]
    batch, heads, kv_heads, d = (case[n] for n in ("batch", "heads", "kv_heads", "d"))
    s = {"op": op, "scale": d ** -0.5}
    if op in ("fwd", "bwd"):
        seqlen = case["seqlen"]
        s["q"] = randn(batch, seqlen, heads, d)
        s["k"], s["v"] = randn(batch, seqlen, kv_heads, d), randn(batch, seqlen, kv_heads, d)
        s["window"], s["sinks"] = case["window"], case["sinks"]
        s["lengths"] = randint(0, seqlen + 1, batch) if case["ragged"] else None
        if op == "bwd":
            s["do"] = randn(batch, seqlen, heads, d)
            # a training step has these from its forward pass
            o, s["lse"] = _plain_fwd(s["q"].float(), s["k"].float(), s["v"].float(), s["scale"], s["window"], s["sinks"],
                                     s["lengths"])
            s["o"] = o.to(dtype)
        return s
    if op == "rotate":
        s["q"], s["k"] = randn(batch, case["seqlen"], heads, d), randn(batch, case["seqlen"], kv_heads, d)
        s["inv_freq"], s["interleaved"], s["inverse"] = _frequencies(case["rot"]), case["interleaved"], case["inverse"]
        return s
    # a pool whose pages lie in any order, with some that belong to nobody
    page = case["page"]
    longest = case["context"] + (case["seqlen"] if op == "append" else 0)
    per_row = -(-longest // page)
    pages = batch * per_row + 3
    s["k_pages"], s["v_pages"] = randn(pages, page, kv_heads, d), randn(pages, page, kv_heads, d)
    s["page_table"] = torch.randperm(pages, device="cuda", generator=gen)[:batch * per_row].int().view(batch, per_row)
    if op == "append":
        s["q"] = randn(batch, case["seqlen"], heads, d)
        s["k"], s["v"] = randn(batch, case["seqlen"], kv_heads, d), randn(batch, case["seqlen"], kv_heads, d)
        s["starts"] = randint(case["context"] // 2, case["context"] + 1, batch)
        s["inv_freq"], s["interleaved"] = _frequencies(case["rot"]), case["interleaved"]
        return s
    s["q"] = randn(batch, case["tokens"], heads, d)
    s["lengths"] = randint(min(case["context"], max(case["tokens"], case["context"] // 2)), case["context"] + 1, batch)
    s["window"], s["sinks"] = case["window"], case["sinks"]
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import selective_state_space_ss_b200 as ss

    if s["op"] == "fwd":
        o, lse = ss.ss_winattn_fwd(s["q"], s["k"], s["v"], s["window"], sinks=s["sinks"], scale=s["scale"],
                                   lengths=s["lengths"])
        return {"o": o, "lse": lse}
    if s["op"] == "bwd":
        return ss.ss_winattn_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["window"], sinks=s["sinks"],
                                 scale=s["scale"], lengths=s["lengths"])
    if s["op"] == "step":
        return ss.ss_winattn_step(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["lengths"], s["window"],
                                  sinks=s["sinks"], scale=s["scale"])
    if s["op"] == "append":
        q, _ = ss.ss_kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["page_table"], s["starts"],
                               inv_freq=s["inv_freq"], q=s["q"], interleaved=s["interleaved"])
        return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    q, k = ss.ss_rotate(s["q"], s["inv_freq"], k=s["k"], interleaved=s["interleaved"], inverse=s["inverse"])
    return {"q": q, "k": k}


# ---- the plain forms ------------------------------------------------------------------------------

_ROWS = 512


def _sees(rows, cols, window, sinks):
    """[rows, cols] truth values: the token at a row's position sees the one at the column's."""
    rows, cols = rows[:, None], cols[None, :]
    return (cols <= rows) & ((rows - cols < window) | (cols < sinks))


def _plain_fwd(q, k, v, scale, window, sinks, lengths):
    """Blocks of queries against the keys that any of them sees: products, a masked softmax, a product."""
    batch, seqlen, heads, d = q.shape
    kv_heads = k.shape[2]
    q = q.transpose(1, 2).unflatten(1, (kv_heads, heads // kv_heads))  # [batch, kv_heads, share, seqlen, d]
    k, v = k.transpose(1, 2)[:, :, None], v.transpose(1, 2)[:, :, None]
    at = torch.arange(seqlen, device=q.device)
    os, ls = [], []
    for r0 in range(0, seqlen, _ROWS):
        r1 = min(r0 + _ROWS, seqlen)
        first = max(0, r0 - window + 1)
        cols = torch.cat([at[:min(sinks, first)], at[first:r1]])
        kb, vb = k[..., cols, :], v[..., cols, :]
        scores = (q[..., r0:r1, :] @ kb.mT) * scale
        scores = scores.masked_fill(~_sees(at[r0:r1], cols, window, sinks), -math.inf)
        top = scores.amax(-1, keepdim=True)
        e = torch.exp(scores - top)
        total = e.sum(-1, keepdim=True)
        os.append((e @ vb) / total)
        ls.append((top + torch.log(total))[..., 0])
    o = torch.cat(os, -2).flatten(1, 2).transpose(1, 2)
    lse = torch.cat(ls, -1).flatten(1, 2)
    if lengths is not None:  # nothing behind a row's length
        real = at < lengths[:, None]
        o = torch.where(real[..., None, None], o, torch.zeros_like(o))
        lse = torch.where(real[:, None], lse, torch.zeros_like(lse))
    return o.contiguous(), lse.contiguous()


def _turn(x, positions, inv_freq, interleaved, inverse=False):
    """Pairs of the first 2 * len(inv_freq) values of each head turned by position * inv_freq."""
    half = inv_freq.shape[0]
    angle = positions.double()[..., None] * inv_freq.double() * (-1 if inverse else 1)
    cos, sin = torch.cos(angle).float()[..., None, :], torch.sin(angle).float()[..., None, :]
    y = x.float().clone()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    ya, yb = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = ya * cos - yb * sin, ya * sin + yb * cos
    return y.to(x.dtype)


def _run_plain(s):
    op, dtype = s["op"], s["q"].dtype
    if op == "fwd":
        o, lse = _plain_fwd(s["q"].float(), s["k"].float(), s["v"].float(), s["scale"], s["window"], s["sinks"], s["lengths"])
        return {"o": o.to(dtype), "lse": lse}
    if op == "bwd":
        leaves = [s[n].float().requires_grad_() for n in ("q", "k", "v")]
        with torch.enable_grad():
            o, _ = _plain_fwd(*leaves, s["scale"], s["window"], s["sinks"], s["lengths"])
        grads = torch.autograd.grad(o, leaves, s["do"].float())
        return {n: x.to(dtype).contiguous() for n, x in zip(("dq", "dk", "dv"), grads)}
    if op == "rotate":
        at = torch.arange(s["q"].shape[1], device="cuda").expand(s["q"].shape[:2])
        return {n: _turn(s[n], at, s["inv_freq"], s["interleaved"], s["inverse"]) for n in ("q", "k")}
    page = s["k_pages"].shape[1]
    if op == "append":
        at = s["starts"].long()[:, None] + torch.arange(s["q"].shape[1], device="cuda")
        where = s["page_table"].long().gather(1, at // page), at % page
        s["k_pages"][where] = _turn(s["k"], at, s["inv_freq"], s["interleaved"])
        s["v_pages"][where] = s["v"]
        return {"q": _turn(s["q"], at, s["inv_freq"], s["interleaved"]), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    # step: the sinks and the last window of every row, out of their pages
    batch, tokens, heads, d = s["q"].shape
    kv_heads, window, sinks = s["k_pages"].shape[2], s["window"], s["sinks"]
    longest = s["page_table"].shape[1] * page
    lengths = s["lengths"].long()[:, None]
    recent = lengths - torch.arange(min(window + tokens - 1, longest), 0, -1, device="cuda")
    kept = torch.arange(min(sinks, longest), device="cuda").expand(batch, -1)
    kept = torch.where(kept < recent[:, :1], kept, -1)  # a sink that the window holds counts once
    cols = torch.cat([kept, recent], 1)
    read = cols.clamp(min=0)
    where = s["page_table"].long().gather(1, read // page), read % page
    k, v = (s[n][where].float().transpose(1, 2)[:, :, None] for n in ("k_pages", "v_pages"))
    rows = (lengths - tokens + torch.arange(tokens, device="cuda"))[..., None]
    cols = cols[:, None]
    seen = (cols >= 0) & (cols <= rows) & ((rows - cols < window) | (cols < sinks))
    q = s["q"].float().transpose(1, 2).unflatten(1, (kv_heads, heads // kv_heads))
    scores = ((q @ k.mT) * s["scale"]).masked_fill(~seen[:, None, None], -math.inf)
    e = torch.exp(scores - scores.amax(-1, keepdim=True))
    o = (e @ v) / e.sum(-1, keepdim=True)
    return o.flatten(1, 2).transpose(1, 2).to(dtype).contiguous()


# ---- what the definitions give in 64 bits -----------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "step":
        return _exact_step(case, s)
    if op in ("fwd", "bwd"):
        return _exact_attention(case, s)
    # the rotation as a product of complex numbers
    seqlen, sign = case["seqlen"], -1 if op == "rotate" and case["inverse"] else 1
    starts = s["starts"].tolist() if op == "append" else [0] * case["batch"]

    def turned(x):
        y, half = x.double(), s["inv_freq"].shape[0]
        for b, start in enumerate(starts):
            angle = torch.arange(start, start + seqlen, dtype=torch.float64, device="cuda")[:, None] * s["inv_freq"].double()
            by = torch.polar(torch.ones_like(angle), sign * angle)[:, None]
            z = y[b, :, :, :2 * half]
            if case["interleaved"]:
                z = torch.view_as_complex(z.unflatten(-1, (half, 2)).contiguous()) * by
                y[b, :, :, :2 * half] = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(z[..., :half], z[..., half:]) * by
                y[b, :, :, :2 * half] = torch.cat([z.real, z.imag], -1)
        return y

    if op == "rotate":
        return {"q": turned(s["q"]), "k": turned(s["k"])}
    pools = {n: s[n].double() for n in ("k_pages", "v_pages")}
    new = {"k_pages": turned(s["k"]), "v_pages": s["v"].double()}
    page, table = case["page"], s["page_table"].tolist()
    for b, start in enumerate(starts):
        at = start
        while at < start + seqlen:  # page by page
            n = min(page - at % page, start + seqlen - at)
            for name, pool in pools.items():
                pool[table[b][at // page], at % page:at % page + n] = new[name][b, at - start:at - start + n]
            at += n
    return {"q": turned(s["q"]), **pools}


def _exact_step(case, s):
    tokens, share, page = case["tokens"], case["heads"] // case["kv_heads"], case["page"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lengths"].tolist()):
        pages = s["page_table"][b, :-(-n // page)].long()
        k, v = (s[x][pages].flatten(0, 1)[:n].double().repeat_interleave(share, 1) for x in ("k_pages", "v_pages"))
        for i in range(tokens):
            t = n - tokens + i
            near = max(0, t - case["window"] + 1)
            far = list(range(min(case["sinks"], near)))
            kt, vt = (torch.cat([x[far], x[near:t + 1]]) for x in (k, v))
            w = torch.softmax(torch.einsum("hd,jhd->hj", s["q"][b, i].double(), kt) * s["scale"], -1)
            o[b, i] = torch.einsum("hj,jhd->hd", w, vt)
    return o


def _exact_attention(case, s):
    batch, seqlen, heads, kv_heads, d = (case[n] for n in ("batch", "seqlen", "heads", "kv_heads", "d"))
    if batch * heads * seqlen * seqlen * d > 1.5e13:
        return None
    share, scale = heads // kv_heads, s["scale"]
    f64 = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros(batch, seqlen, heads, d, **f64), torch.zeros(batch, heads, seqlen, **f64)
    dq, dk, dv = (torch.zeros(s[n].shape, **f64) for n in ("q", "k", "v"))
    ends = s["lengths"].tolist() if s["lengths"] is not None else [seqlen] * batch
    for b, end in enumerate(ends):
        for h in range(heads):
            q, k, v = s["q"][b, :end, h].double(), s["k"][b, :end, h // share].double(), s["v"][b, :end, h // share].double()
            for r0 in range(0, end, 4096):
                rows = slice(r0, min(r0 + 4096, end))
                i = torch.arange(r0, min(r0 + 4096, end), device="cuda")[:, None] - torch.arange(end, device="cuda")[None, :]
                hidden = (i < 0) | ((i >= case["window"]) & (torch.arange(end, device="cuda") >= case["sinks"]))
                x = torch.where(hidden, -math.inf, scale * torch.einsum("id,jd->ij", q[rows], k))
                z = torch.logsumexp(x, -1)
                p = torch.exp(x - z[:, None])
                out = p @ v
                if case["op"] == "fwd":
                    o[b, rows, h], lse[b, h, rows] = out, z
                    continue
                g = s["do"][b, rows, h].double()
                dv[b, :end, h // share] += p.T @ g
                ds = p * (g @ v.T - (g * out).sum(-1, keepdim=True)) * scale
                dq[b, rows, h] = ds @ k
                dk[b, :end, h // share] += ds.T @ q[rows]
    return {"o": o, "lse": lse} if case["op"] == "fwd" else {"dq": dq, "dk": dk, "dv": dv}


def _visible(last, window, sinks):
    """Tokens that those at the positions below `last` see, all told."""
    near = sum_to(min(last, window)) + max(0, last - window) * window
    far = sum(max(0, last - window - j) for j in range(min(sinks, last)))
    return near + far


def sum_to(n):
    return n * (n + 1) // 2


def work(case):
    op = case["op"]
    batch, heads, kv_heads, d = (case[n] for n in ("batch", "heads", "kv_heads", "d"))
    size = 2 if case["dtype"] == "bf16" else 4
    if op in ("fwd", "bwd"):
        seqlen, part = case["seqlen"], 0.5 if case["ragged"] else 1  # lengths are uniform between none and all
        pairs = batch * heads * part * _visible(seqlen, case["window"], case["sinks"])
        tokens = batch * seqlen * part
        if op == "fwd":  # q, k, v in, o and its normaliser out
            return {"bytes": tokens * (size * d * 2 * (heads + kv_heads) + 4 * heads), "flops": 4 * d * pairs}
        # q, k, v, o, do and the normaliser in, three gradients out; five products
        return {"bytes": tokens * (size * d * 4 * (heads + kv_heads) + 4 * heads), "flops": 10 * d * pairs}
    if op == "step":
        tokens, mean = case["tokens"], 0.75 * case["context"]
        seen = min(mean, case["window"] + case["sinks"] + tokens - 1)
        return {"bytes": batch * size * d * (2 * kv_heads * seen + 2 * heads * tokens), "flops": 4 * d * batch * heads * tokens * seen}
    rows = heads + kv_heads + (kv_heads if op == "append" else 0)
    values = batch * case["seqlen"] * rows * d
    turned = batch * case["seqlen"] * (heads + kv_heads) * case["rot"]
    return {"bytes": 2 * size * values, "flops": 3 * turned}
