"""The linear-attention operators and the 8-bit state cache, as cases to measure.

Beside the selective scan, whose state decays channel by channel, stands the
recurrence with one decay per head, a linear attention whose state is a matrix:

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,      o_t = scale * S_t^T q_t

over a prompt (``ss_linattn_fwd``), its gradients (``ss_linattn_bwd``), one token
at a time (``ss_linattn_step``), and the states of sequences that wait, kept in a
pool in 8 bits with a scale for each row (``ss_state_store8``, ``ss_state_load8``).

``own`` false: the plain forms, elementary torch operations in 32 bits (sums of
log decays in 64).  ``own`` true: the package's entry points.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _attn(op, name, batch, seqlen, heads, qk_heads, dk, dv, dtype, state=False, ragged=False):
    return {"name": name, "op": op, "batch": batch, "seqlen": seqlen, "heads": heads, "qk_heads": qk_heads,
            "dk": dk, "dv": dv, "dtype": dtype, "state": state, "ragged": ragged}


def _pool(name, batch, slots, rows, width):
    return {"name": name, "op": "park", "batch": batch, "slots": slots, "rows": rows, "width": width}


def listed():
    return [
        # a short question after earlier turns: one prompt of odd length from the kept state, latency counts
        _attn("fwd", "fwd_turn_b1_l203_h8_bf16", 1, 203, 8, 8, 64, 64, "bf16", state=True),
        # prompts or a training batch of a 1536-wide model: 24 heads of 64 that share queries and keys
        _attn("fwd", "fwd_b8_l2048_h24_shared_bf16", 8, 2048, 24, 1, 128, 64, "bf16"),
        # a 5120-wide model's batch of long prompts, the largest call
        _attn("fwd", "fwd_b4_l8192_h40_d128_bf16", 4, 8192, 40, 40, 128, 128, "bf16"),
        # one long document: few heads, many tokens, an odd end
        _attn("fwd", "fwd_b1_l65001_h16_bf16", 1, 65001, 16, 16, 64, 64, "bf16", state=True),
        # a padded batch in fp32, the numerics reference of a training run
        _attn("fwd", "fwd_ragged_b6_l1000_h8_f32", 6, 1000, 8, 4, 64, 128, "f32", state=True, ragged=True),
        # training steps: a 512-wide model in fp32, a 1536-wide one with shared queries and keys, long and odd sequences
        _attn("bwd", "bwd_b2_l1024_h8_f32", 2, 1024, 8, 8, 64, 64, "f32"),
        _attn("bwd", "bwd_b8_l2048_h24_shared_bf16", 8, 2048, 24, 8, 64, 64, "bf16"),
        _attn("bwd", "bwd_b2_l4097_h16_d128_bf16", 2, 4097, 16, 16, 128, 128, "bf16", state=True),
        # generation: a few users (latency) and a full batch (bandwidth)
        _attn("step", "step_b4_h24_bf16", 4, 1, 24, 24, 64, 64, "bf16"),
        _attn("step", "step_b128_h40_d128_bf16", 128, 1, 40, 8, 128, 128, "bf16"),
        # sequences parked in the pool and woken: a few selective-scan states (1536 channels of 16), many matrix states
        _pool("park_b6_d1536_n16", 6, 96, 1536, 16),
        _pool("park_b64_h40_d128", 64, 100, 40 * 128, 128),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "park"])
    if op == "park":
        batch, rows, width = _spread(rng, 1, 128), _spread(rng, 64, 6000), rng.choice([16, 32, 64, 128, rng.randint(5, 128)])
        return {"op": op, "batch": batch, "slots": batch + rng.randint(0, 60), "rows": rows, "width": width}
    qk_heads = _spread(rng, 1, 16)
    heads = qk_heads * rng.choice([1, 1, 2, 3])
    dk, dv = (rng.choice([16, 32, 64, 128, 128, rng.randint(9, 127)]) for _ in range(2))
    case = {"op": op, "heads": heads, "qk_heads": qk_heads, "dk": dk, "dv": dv, "dtype": rng.choice(["bf16", "bf16", "f32"]),
            "state": rng.random() < 0.5, "ragged": op != "step" and rng.random() < 0.3}
    if op == "step":
        case["state"] = False
        return {**case, "batch": _spread(rng, 1, 128), "seqlen": 1}
    most = (300_000 if op == "fwd" else 100_000) // heads
    seqlen = _spread(rng, 1, min(20000, most))
    return {**case, "batch": rng.randint(1, min(8, most // seqlen)), "seqlen": seqlen}


def _decay(shape, gen, dtype):
    """Log decays -Delta * a: steps of 1e-3 to 1e-1 and rates of 1 to 16 for each head, varied from token to token."""
    heads = shape[-1]
    dt = torch.exp(torch.empty(heads, device="cuda").uniform_(math.log(1e-3), math.log(1e-1), generator=gen))
    rate = torch.empty(heads, device="cuda").uniform_(1, 16, generator=gen)
    vary = torch.exp(0.5 * torch.randn(shape, device="cuda", generator=gen))
    return (-dt * rate * vary).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, device="cuda", generator=gen).to(dtype)

    op = case["op"]
    if op == "park":
        batch, slots, rows, width = (case[k] for k in ("batch", "slots", "rows", "width"))
        # rows of very different sizes, as states of channels with different decays are
        return {"op": op, "state": randn(batch, rows, width) * torch.exp(randn(batch, rows, 1)),
                "where": torch.randperm(slots, device="cuda", generator=gen)[:batch].int(),
                "codes": torch.zeros(slots, rows, width, dtype=torch.int8, device="cuda"),
                "scales": torch.zeros(slots, rows, device="cuda")}
    batch, seqlen, heads, qk_heads, dk, dv = (case[k] for k in ("batch", "seqlen", "heads", "qk_heads", "dk", "dv"))
    dtype = _TYPES[case["dtype"]]
    s = {"op": op, "scale": dk ** -0.5}
    if op == "step":
        s["state"] = randn(batch, heads, dk, dv)
        s["q"], s["k"] = (randn(batch, qk_heads, dk, dtype=dtype) for _ in range(2))
        s["v"] = randn(batch, heads, dv, dtype=dtype)
        s["log_decay"] = _decay((batch, heads), gen, dtype)
        return s
    s["q"], s["k"] = (randn(batch, seqlen, qk_heads, dk, dtype=dtype) for _ in range(2))
    s["v"] = randn(batch, seqlen, heads, dv, dtype=dtype)
    s["log_decay"] = _decay((batch, seqlen, heads), gen, dtype)
    s["initial_state"] = randn(batch, heads, dk, dv) if case["state"] else None
    s["lengths"] = None
    if case["ragged"]:
        s["lengths"] = torch.randint(0, seqlen + 1, (batch,), device="cuda", generator=gen).int()
    if op == "bwd":
        s["do"] = randn(batch, seqlen, heads, dv, dtype=dtype)
        s["dlast_state"] = randn(batch, heads, dk, dv) if case["state"] else None
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import selective_state_space_ss_b200 as ss

    if s["op"] == "fwd":
        o, last = ss.ss_linattn_fwd(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"],
                                    initial_state=s["initial_state"], lengths=s["lengths"])
        return {"o": o, "last_state": last}
    if s["op"] == "bwd":
        return ss.ss_linattn_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["do"], scale=s["scale"],
                                 initial_state=s["initial_state"], dlast_state=s["dlast_state"], lengths=s["lengths"])
    if s["op"] == "step":
        o = ss.ss_linattn_step(s["state"], s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"])
        return {"o": o, "state": s["state"]}
    # parked, then woken: the codes come back as the values they stand for
    ss.ss_state_store8(s["state"], s["codes"], s["scales"], slots=s["where"])
    return {"state": ss.ss_state_load8(s["codes"], s["scales"], slots=s["where"]), "scales": s["scales"]}


# ---- the plain forms ------------------------------------------------------------------------------

_CHUNK = 128


def _chunks(x, n):
    """[batch, seqlen, heads, d] to [batch, heads, n, chunk, d], zeros behind the end."""
    x = torch.nn.functional.pad(x.transpose(1, 2), (0, 0, 0, n * _CHUNK - x.shape[1]))
    return x.unflatten(2, (n, _CHUNK))


def _plain_fwd(q, k, v, g, scale, s0, lengths):
    """Chunks of the sequence as masked products, chunk states joined by a product with the decays between chunks."""
    batch, seqlen, heads = g.shape
    n = -(-seqlen // _CHUNK)
    q, k = (x.repeat_interleave(heads // x.shape[2], dim=2) for x in (q, k))
    real = None
    if lengths is not None:  # tokens behind a row's length add nothing and decay nothing
        real = torch.arange(seqlen, device=g.device) < lengths[:, None]
        q, k, v = (torch.where(real[..., None, None], x, torch.zeros_like(x)) for x in (q, k, v))
        g = torch.where(real[..., None], g, torch.zeros_like(g))
    q, k, v = (_chunks(x, n) for x in (q, k, v))
    g = _chunks(g.double()[..., None], n)[..., 0].cumsum(-1)
    total = g[..., -1]
    seen = torch.ones(_CHUNK, _CHUNK, dtype=torch.bool, device=g.device).tril()
    between = torch.exp((g[..., :, None] - g[..., None, :]).masked_fill(~seen, -math.inf).float())
    o = ((q @ k.mT) * between) @ v
    local = (k * torch.exp((total[..., None] - g).float())[..., None]).mT @ v
    upto = total.cumsum(-1)
    earlier = torch.ones(n, n, dtype=torch.bool, device=g.device).tril(-1)
    before = torch.exp(((upto - total)[..., :, None] - upto[..., None, :]).masked_fill(~earlier, -math.inf).float())
    states = (before @ local.flatten(3)).unflatten(3, local.shape[3:])
    if s0 is not None:
        states = states + torch.exp((upto - total).float())[..., None, None] * s0[:, :, None]
    o = (o + (q * torch.exp(g.float())[..., None]) @ states) * scale
    last = states[:, :, -1] * torch.exp(total[:, :, -1].float())[..., None, None] + local[:, :, -1]
    o = o.flatten(2, 3)[:, :, :seqlen].transpose(1, 2)
    return o if real is None else torch.where(real[..., None, None], o, torch.zeros_like(o)), last


def _run_plain(s):
    if s["op"] == "fwd":
        o, last = _plain_fwd(s["q"].float(), s["k"].float(), s["v"].float(), s["log_decay"].float(), s["scale"],
                             s["initial_state"], s["lengths"])
        return {"o": o.to(s["q"].dtype).contiguous(), "last_state": last}
    if s["op"] == "bwd":
        leaves = [s[n].float().requires_grad_() for n in ("q", "k", "v", "log_decay")]
        s0 = s["initial_state"]
        if s0 is not None:
            s0 = s0.detach().requires_grad_()
        with torch.enable_grad():
            out, last = _plain_fwd(*leaves, s["scale"], s0, s["lengths"])
        of, by = [out], [s["do"].float()]
        if s["dlast_state"] is not None:
            of, by = of + [last], by + [s["dlast_state"]]
        grads = torch.autograd.grad(of, leaves + ([] if s0 is None else [s0]), by)
        dtype = s["q"].dtype
        names = ("dq", "dk", "dv", "dlog_decay")
        return {**{n: x.to(dtype).contiguous() for n, x in zip(names, grads)},
                "dinitial_state": None if s0 is None else grads[4]}
    if s["op"] == "step":
        q, k = (s[n].float().repeat_interleave(s["v"].shape[1] // s[n].shape[1], dim=1) for n in ("q", "k"))
        new = s["state"] * torch.exp(s["log_decay"].float())[..., None, None] + k[..., :, None] * s["v"].float()[..., None, :]
        s["state"].copy_(new)
        o = (q[..., None, :] @ new)[..., 0, :] * s["scale"]
        return {"o": o.to(s["q"].dtype), "state": s["state"]}
    where = s["where"].long()
    scale = s["state"].abs().amax(-1) / 127
    # the steps in 64 bits, so that a value next to the border of two codes gets the nearer one
    s["codes"][where] = torch.round(s["state"].double() / scale.double()[..., None]).to(torch.int8)
    s["scales"][where] = scale
    return {"state": s["codes"][where].float() * s["scales"][where][..., None], "scales": s["scales"]}


# ---- what the definitions give in 64 bits -----------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "park":
        values, scales = torch.empty_like(s["state"], dtype=torch.float64), s["scales"].double()
        for b, slot in enumerate(s["where"].tolist()):
            x = s["state"][b].double()
            step = x.abs().max(-1).values / 127
            held = step.float().double()[:, None]  # the pool's scale is a number of 32 bits, and a code counts its steps
            values[b], scales[slot] = torch.round(x / held) * held, step
        return {"state": values, "scales": scales}
    share = case["heads"] // case["qk_heads"]
    if case["op"] == "step":
        q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
        state = s["state"].double() * s["log_decay"].double().exp()[..., None, None]
        state += torch.einsum("bhk,bhv->bhkv", k.repeat_interleave(share, 1), v)
        return {"o": torch.einsum("bhk,bhkv->bhv", q.repeat_interleave(share, 1), state) * s["scale"], "state": state}
    return _exact_fwd(case, s, share) if case["op"] == "fwd" else _exact_bwd(case, s, share)


def _tokens(case, s, share):
    """Each token's q, k, v, decay in 64 bits; behind a row's length k and v are zero and the decay is one."""
    batch, seqlen = case["batch"], case["seqlen"]
    ends = s["lengths"].tolist() if s["lengths"] is not None else [seqlen] * batch
    live = torch.zeros(batch, seqlen, 1, 1, dtype=torch.float64, device="cuda")
    for b, e in enumerate(ends):
        live[b, :e] = 1

    def at(t):
        m = live[:, t]
        q, k = (s[n][:, t].double().repeat_interleave(share, 1) * m for n in ("q", "k"))
        return q, k, s["v"][:, t].double() * m, torch.exp(s["log_decay"][:, t].double()[..., None, None] * m[..., None])

    return live, at


def _start(case, s):
    if s["initial_state"] is not None:
        return s["initial_state"].double().clone()
    return torch.zeros(case["batch"], case["heads"], case["dk"], case["dv"], dtype=torch.float64, device="cuda")


def _exact_fwd(case, s, share):
    _, at = _tokens(case, s, share)
    state = _start(case, s)
    o = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    for t in range(case["seqlen"]):
        q, k, v, a = at(t)
        state.mul_(a).addcmul_(k[..., :, None], v[..., None, :])
        o[:, t] = torch.matmul(q[..., None, :], state)[..., 0, :] * s["scale"]
    return {"o": o, "last_state": state}


def _exact_bwd(case, s, share):
    live, at = _tokens(case, s, share)
    batch, seqlen, heads, dk, dv = (case[n] for n in ("batch", "seqlen", "heads", "dk", "dv"))
    if 8 * batch * (seqlen + 1) * heads * dk * dv > 60e9:
        return None
    states = torch.empty(seqlen + 1, batch, heads, dk, dv, dtype=torch.float64, device="cuda")
    states[0] = _start(case, s)
    for t in range(seqlen):
        _, k, v, a = at(t)
        torch.mul(states[t], a, out=states[t + 1])
        states[t + 1].addcmul_(k[..., :, None], v[..., None, :])
    dq, dk_ = (torch.zeros(batch, seqlen, heads, dk, dtype=torch.float64, device="cuda") for _ in range(2))
    dv_ = torch.zeros(batch, seqlen, heads, dv, dtype=torch.float64, device="cuda")
    dg = torch.zeros(batch, seqlen, heads, dtype=torch.float64, device="cuda")
    r = torch.zeros_like(states[0]) if s["dlast_state"] is None else s["dlast_state"].double().clone()
    for t in reversed(range(seqlen)):
        q, k, v, a = at(t)
        do = s["do"][:, t].double() * live[:, t] * s["scale"]
        dq[:, t] = torch.matmul(states[t + 1], do[..., None])[..., 0]
        r.addcmul_(q[..., :, None], do[..., None, :])
        dk_[:, t] = torch.matmul(r, v[..., None])[..., 0] * live[:, t]
        dv_[:, t] = torch.matmul(k[..., None, :], r)[..., 0, :] * live[:, t]
        r.mul_(a)
        dg[:, t] = (r * states[t]).sum((-1, -2)) * live[:, t, :, 0]
    return {"dq": dq.unflatten(2, (case["qk_heads"], share)).sum(3), "dk": dk_.unflatten(2, (case["qk_heads"], share)).sum(3),
            "dv": dv_, "dlog_decay": dg, "dinitial_state": None if s["initial_state"] is None else r}


def work(case):
    op = case["op"]
    if op == "park":  # written: 4 bytes in and 1 out, and a scale; read: the other way
        n = case["batch"] * case["rows"]
        return {"bytes": n * (10 * case["width"] + 8), "flops": 4 * n * case["width"]}
    batch, seqlen, heads, qk_heads, dk, dv = (case[k] for k in ("batch", "seqlen", "heads", "qk_heads", "dk", "dv"))
    size, tokens, states = (2 if case["dtype"] == "bf16" else 4), batch * seqlen, 4 * batch * heads * dk * dv
    if case["ragged"]:
        tokens = tokens / 2  # lengths are uniform between none and all
    per_token = 2 * qk_heads * dk + heads * (dv + 1)  # q, k, v and the decay
    if op == "bwd":
        # q, k, v, g and do in, four gradients out; products for the two states and for dq, dk, dv
        moved = tokens * size * (2 * per_token + heads * dv) + (3 * states if case["state"] else 0)
        return {"bytes": moved, "flops": 10 * tokens * heads * dk * dv}
    moved = tokens * size * (per_token + heads * dv) + states * (2 if case["state"] or op == "step" else 1)
    return {"bytes": moved, "flops": 4 * tokens * heads * dk * dv}
