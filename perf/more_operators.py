"""The operators of a linear-attention layer around the ternary products: the
norms before and after a block, the short causal convolution, and the gated
delta rule with its state.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end) where ``own`` is false, and through the
framework's entry points where it is true.  ``exact`` is the definition in 64
bits, written apart from both.

A call holds the new tokens of ``seqs`` sequences in a row.  Each sequence has a
slot in a pool of states; it reads the state in slots[b] (zeros where it has no
past) and writes the new one to dst_slots[b].

  short_conv   y[t] = silu(bias + sum_w weight[:, w] x[t - (W - 1) + w]), the inputs
               before the first token from the state (the last W - 1 inputs);
  gated_delta  per value head, S [Dv, Dk] in 32 bits:  a = exp(g),
               u = beta (v - a S k),  S <- a S + u k^T,  o = scale S q,
               queries and keys divided by their length where qk_norm says so, and with
               "raw" gates  g = -exp(a_log) softplus(g + dt_bias), beta = sigmoid(beta);
  rms_norm     before a block  h = residual + s x,  y = h / rms(h) w act(gate),
               after it        y = residual + s (x / rms(x) w act(gate)).
"""
import math

import torch

own = False

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def _delta(name, seqs, new, ragged, past, k_heads, v_heads, dk, dv, raw, qk_norm):
    c = dict(op="delta", seqs=seqs, new=new, ragged=ragged, past=past, k_heads=k_heads, v_heads=v_heads, dk=dk, dv=dv,
             raw=raw, qk_norm=qk_norm)
    return dict(c, name=name) if name else c


def _conv(name, seqs, new, ragged, past, channels, width, in_f32, bias):
    c = dict(op="conv", seqs=seqs, new=new, ragged=ragged, past=past, channels=channels, width=width, in_f32=in_f32,
             bias=bias)
    return dict(c, name=name) if name else c


def _norm(name, tokens, heads, dim, in_f32, residual, gate, after):
    c = dict(op="norm", tokens=tokens, heads=heads, dim=dim, in_f32=in_f32, residual=residual, gate=gate, after=after)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one generated token of one conversation: the smallest call, all latency
        _delta("delta_token", 1, 1, False, True, 16, 32, 128, 128, True, True),
        # one token for each of 64 conversations: the serving step, bound by reading and writing the states
        _delta("delta_batch", 64, 1, False, True, 16, 48, 128, 128, True, True),
        # a speculative verify step: five tokens for each of eight conversations
        _delta("delta_verify", 8, 5, False, True, 16, 32, 128, 128, True, True),
        # one prompt alone: as many chains of chunks as there are heads
        _delta("delta_prompt", 1, 2048, False, False, 16, 32, 128, 128, True, True),
        # a batch of prompts of unlike length: bound by the products
        _delta("delta_prompts", 6, 4096, True, False, 16, 48, 128, 128, True, True),
        # conversations that go on, narrow keys and uneven heads, gates and keys prepared by the caller
        _delta("delta_narrow", 3, 700, True, True, 5, 15, 64, 96, False, False),
        # sixteen generated tokens, the fp32 output of the decode product
        _conv("conv_token", 16, 1, False, True, 8192, 4, True, False),
        # prompts of unlike length, the bf16 output of the prefill product
        _conv("conv_prompt", 4, 4096, True, False, 8192, 4, False, True),
        # before a block, one generated token: the residual stream and the last product's output, both fp32
        _norm("norm_token", 1, 1, 5120, True, "f32", False, False),
        # before a block, a prompt
        _norm("norm_prompt", 4096, 1, 5120, False, "bf16", False, False),
        # the delta rule's output, head by head, under its gate
        _norm("norm_gated", 2048, 48, 128, False, "none", True, False),
        # after a block, scaled into the residual stream, odd sizes
        _norm("norm_after", 777, 1, 4104, True, "f32", True, True),
    ]


_HEADS = [(16, 32, 128, 128), (16, 48, 128, 128), (16, 16, 128, 128), (4, 8, 64, 128), (5, 15, 64, 96), (8, 8, 64, 64),
          (3, 12, 128, 64), (2, 6, 128, 176), (1, 7, 128, 256)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(c):
    w, pad = work(c), 0
    if c["op"] == "delta":   # what the padded plain form makes of it, and its steps one after another
        pad = c["seqs"] * max(_lengths(c)) * c["v_heads"] * c["dv"] + 2e4 * max(_lengths(c))
    if c["op"] == "conv":
        pad = c["seqs"] * max(_lengths(c)) * c["channels"]
    return max(w["bytes"] / 6e12, w["flops"] / 1e15), pad


def draw(rng):
    """One more case: sizes spread over their range (over its logarithm), odd ones among them."""
    every = [c for c in listed()]
    while True:
        op = rng.choice(["delta", "delta", "delta", "conv", "norm"])
        ragged, past = rng.random() < 0.5, rng.random() < 0.6
        if op == "delta":
            kind = rng.choice(["token", "few", "prompt", "prompt"])
            new = {"token": 1, "few": rng.randint(2, 40), "prompt": _log(rng, 30, 4096)}[kind]
            seqs = _log(rng, 1, 80) if kind != "prompt" else rng.randint(1, 6)
            c = _delta(None, seqs, new, ragged, past, *rng.choice(_HEADS), rng.random() < 0.5, rng.random() < 0.7)
        elif op == "conv":
            new = rng.choice([1, _log(rng, 1, 4096)])
            c = _conv(None, _log(rng, 1, 64), new, ragged, past, 8 * _log(rng, 8, 1536), rng.randint(2, 4),
                      rng.random() < 0.5, rng.random() < 0.5)
        else:
            heads = rng.choice([1, 1, rng.randint(2, 48)])
            dim = 8 * (_log(rng, 8, 32) if heads > 1 else _log(rng, 16, 2048))
            c = _norm(None, _log(rng, 1, 8192), heads, dim, rng.random() < 0.5, rng.choice(["none", "f32", "bf16"]),
                      rng.random() < 0.5, rng.random() < 0.4)
        most, most_pad = (max(v) for v in zip(*(_cost(x) for x in every if x["op"] == op)))
        cost, pad = _cost(c)
        if cost <= most and pad <= most_pad:
            return c


def _lengths(c):
    """The new tokens of each sequence: ragged ones from a fifth of the full length up to it, in no order."""
    out = []
    for b in range(c["seqs"]):
        f = 0.2 + 0.8 * ((b * 5 + 2) % c["seqs"] + 1) / c["seqs"] if c["ragged"] else 1.0
        out.append(max(1, min(c["new"], int(c["new"] * f))))
    return out


def work(c):
    if c["op"] == "norm":
        n = c["tokens"] * c["heads"] * c["dim"]
        kinds = {"none": 0, "f32": 4, "bf16": 2}
        # x, residual (and, before a block, the new one), gate, output
        out = kinds[c["residual"]] or 2
        per = (4 if c["in_f32"] else 2) + kinds[c["residual"]] + (2 if c["gate"] else 0) + \
            (out if c["after"] else 2 + kinds[c["residual"]])
        return {"bytes": n * per + 4 * c["dim"], "flops": 6 * n}
    t, b = sum(_lengths(c)), c["seqs"]
    read = b if c["past"] else 0   # (about one in eight of them has none all the same)
    if c["op"] == "conv":
        ch, w = c["channels"], c["width"]
        return {"bytes": t * ch * ((4 if c["in_f32"] else 2) + 2) + (read + b) * (w - 1) * ch * 4 + 4 * ch * (w + 1),
                "flops": t * ch * (2 * w + 4)}
    hk, hv, dk, dv = c["k_heads"], c["v_heads"], c["dk"], c["dv"]
    return {"bytes": t * (4 * hk * dk + 4 * hv * dv + 8 * hv) + (read + b) * hv * dk * dv * 4,
            "flops": 6 * t * hv * dk * dv}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _normal(shape, gen):
    return torch.empty(shape, device="cuda").normal_(generator=gen)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "norm":
        t, h, d = c["tokens"], c["heads"], c["dim"]
        kind = torch.float32 if c["in_f32"] else torch.bfloat16
        s["x"] = (_normal((t, h, d), gen) * 3.0).to(kind)
        s["weight"] = 1.0 + 0.2 * _normal(d, gen)
        s["scale"] = 0.5 if c["after"] else 1.0
        s["residual"] = s["residual_out"] = s["gate"] = None
        if c["residual"] != "none":
            kind = torch.float32 if c["residual"] == "f32" else torch.bfloat16
            s["residual"] = (_normal((t, h, d), gen) * 5.0).to(kind)
            s["residual_out"] = None if c["after"] else torch.empty_like(s["residual"])
        if c["gate"]:   # a part of a projection's output
            wide = _normal((t, h * d + 64), gen).to(torch.bfloat16)
            s["gate"] = wide[:, 64:].view(t, h, d) if h == 1 else wide[:, 64:].unflatten(1, (h, d))
        out = s["residual"].dtype if c["after"] and s["residual"] is not None else torch.bfloat16
        s["out"] = torch.empty((t, h, d), dtype=out, device=dev)
        return s
    lens, b = _lengths(c), c["seqs"]
    t = sum(lens)
    s["lens_host"], s["max_new"] = lens, max(lens)
    s["q_start"] = torch.tensor([sum(lens[:i]) for i in range(b + 1)], dtype=torch.int32, device=dev)
    order = torch.randperm(2 * b + 3, generator=gen, device=dev).to(torch.int32)
    s["slots"], s["dst_slots"] = order[:b].contiguous(), order[b:2 * b].contiguous()
    past = torch.randint(1, 9, (b,), generator=gen, device=dev, dtype=torch.int32) - 1   # one in eight begins
    s["past"] = past if c["past"] else torch.zeros_like(past)
    if c["op"] == "conv":
        ch, w = c["channels"], c["width"]
        x = _normal((t, ch + 128), gen)   # beside the gate's part of the projection
        s["x"] = (x if c["in_f32"] else x.to(torch.bfloat16))[:, :ch]
        s["weight"] = _normal((ch, w), gen) * w ** -0.5
        s["bias"] = 0.1 * _normal(ch, gen) if c["bias"] else None
        s["state"] = _normal((2 * b + 3, w - 1, ch), gen)
        s["out"] = torch.empty((t, ch), dtype=torch.bfloat16, device=dev)
        return s
    hk, hv, dk, dv = c["k_heads"], c["v_heads"], c["dk"], c["dv"]
    x = _normal((t, 2 * hk * dk + hv * dv), gen)
    x = x * torch.sigmoid(x)                                   # the convolution's output, [q | k | v]
    if not c["qk_norm"]:
        qk = x[:, :2 * hk * dk].view(t, 2 * hk, dk)
        qk /= (qk * qk).sum(dim=-1, keepdim=True).sqrt() + 1e-3
    x = x.to(torch.bfloat16)
    s["q"], s["k"], s["v"] = x[:, :hk * dk].view(t, hk, dk), x[:, hk * dk:2 * hk * dk].view(t, hk, dk), \
        x[:, 2 * hk * dk:].view(t, hv, dv)
    gates = _normal((t, 2 * hv), gen)                          # one small projection's output
    s["g"], s["beta"] = gates[:, :hv], gates[:, hv:]
    s["a_log"] = s["dt_bias"] = None
    # decay rates from 1 to 16, steps from 1e-3 to 0.1
    rate = 1.0 + 15.0 * torch.rand(hv, generator=gen, device=dev)
    step = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(hv, generator=gen, device=dev))
    if c["raw"]:
        s["a_log"], s["dt_bias"] = rate.log(), step + torch.log(-torch.expm1(-step))
    else:
        s["g"].copy_(-rate * step * s["g"].exp())
        s["beta"].copy_(torch.sigmoid(s["beta"]))
    s["scale"] = dk ** -0.5
    s["state"] = 0.3 * _normal((2 * b + 3, hv, dv, dk), gen)
    s["out"] = torch.empty((t, hv, dv), dtype=torch.bfloat16, device=dev)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _padded(s, n):
    """Where each sequence's tokens stand, [B, n] rows (clamped), and which of them are its own."""
    start = s["q_start"].long()
    i = torch.arange(n, device=start.device)
    live = i < (start[1:] - start[:-1])[:, None]
    return torch.where(live, start[:-1, None] + i, 0), live


def _plain_norm(s):
    c, x = s["case"], s["x"].float()
    y = x if c["after"] or s["residual"] is None else s["residual"].float() + s["scale"] * x
    if s["residual_out"] is not None:
        s["residual_out"].copy_(y)
    y = y * torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + 1e-6) * s["weight"]
    if s["gate"] is not None:
        z = s["gate"].float()
        y = y * (z * torch.sigmoid(z))
    if c["after"]:
        y = s["scale"] * y if s["residual"] is None else s["residual"].float() + s["scale"] * y
    s["out"].copy_(y)
    return {"out": s["out"]} if s["residual_out"] is None else {"out": s["out"], "residual": s["residual_out"]}


def _plain_conv(s):
    c, start = s["case"], s["q_start"].long()
    w = c["width"]
    at, live = _padded(s, s["max_new"])
    old = s["state"][s["slots"].long()] * (s["past"] > 0)[:, None, None]
    x = torch.cat((old, s["x"][at].float()), dim=1)                              # [B, W - 1 + n, C]
    y = (x.unfold(1, w, 1) * s["weight"]).sum(dim=-1)
    y = y if s["bias"] is None else y + s["bias"]
    y = y * torch.sigmoid(y)
    s["out"][at[live]] = y[live].to(torch.bfloat16)
    last = (start[1:] - start[:-1])[:, None] + torch.arange(w - 1, device=x.device)
    s["state"][s["dst_slots"].long()] = x.gather(1, last[..., None].expand(-1, -1, x.shape[2]))
    return {"out": s["out"], "state": s["state"]}


def _plain_delta(s):
    c = s["case"]
    size = min(64, 1 << (s["max_new"] - 1).bit_length())                          # tokens of a chunk
    at, live = _padded(s, -(-s["max_new"] // size) * size)
    group = c["v_heads"] // c["k_heads"]

    def chunks(x, fill=True):   # [T, heads, ...] -> [B, heads, chunks, size, ...], zeros past a sequence's end
        x = x[at].float() * live.reshape(live.shape + (1,) * (x.dim() - 1))
        return x.transpose(1, 2).unflatten(2, (-1, size))

    g, beta = s["g"], s["beta"]
    if c["raw"]:
        g = g + s["dt_bias"]
        g = -s["a_log"].exp() * (g.clamp(min=0) + torch.log1p(torch.exp(-g.abs())))
        beta = torch.sigmoid(beta)
    g, beta = chunks(g), chunks(beta)[..., None]
    q, k, v = chunks(s["q"]), chunks(s["k"]), chunks(s["v"])
    if c["qk_norm"]:
        q, k = (x * torch.rsqrt((x * x).sum(dim=-1, keepdim=True) + 1e-6) for x in (q, k))
    total = g.double().cumsum(dim=-1)
    below = torch.tril(torch.ones(size, size, dtype=torch.bool, device=g.device))
    decay = (total[..., :, None] - total[..., None, :]).masked_fill_(~below, -math.inf).exp_().float()
    near, left = total.exp().float()[..., None], (total[..., -1:] - total).exp().float()[..., None]
    kk, qk = ((x @ k.transpose(-1, -2)).repeat_interleave(group, dim=1) for x in (k, q))
    # (I + a)^-1 of a strictly lower a: (I - a)(I + a^2)(I + a^4) ...
    a = (beta * decay * kk).tril_(-1)
    inverse, span = torch.eye(size, device=a.device) - a, 2
    while span < size:
        a = a @ a
        inverse, span = inverse + inverse @ a, 2 * span
    del kk, a
    p = qk.mul_(decay)
    q, k = (x.repeat_interleave(group, dim=1) for x in (q, k))
    value, reach = inverse @ (beta * v), inverse @ (beta * near * k)
    q, kept = near * q, (left * k).transpose(-1, -2)
    state = (s["state"][s["slots"].long()] * (s["past"] > 0)[:, None, None, None]).transpose(-1, -2)
    out = torch.empty_like(v)
    for i in range(v.shape[2]):
        u = value[:, :, i] - reach[:, :, i] @ state
        out[:, :, i] = q[:, :, i] @ state + p[:, :, i] @ u
        state = near[:, :, i, -1:] * state + kept[:, :, i] @ u
    out = out.flatten(2, 3).transpose(1, 2)
    s["out"][at[live]] = (out[live] * s["scale"]).to(torch.bfloat16)
    s["state"][s["dst_slots"].long()] = state.transpose(-1, -2)
    return {"out": s["out"], "state": s["state"]}


def run(s):
    c = s["case"]
    if not own:
        return {"norm": _plain_norm, "conv": _plain_conv, "delta": _plain_delta}[c["op"]](s)
    import bit_gemv_gemm_gb300 as tern
    if c["op"] == "norm":
        tern.rms_norm(s["x"], s["weight"], residual=s["residual"], scale=s["scale"], gate=s["gate"], eps=1e-6,
                      after=c["after"], residual_out=s["residual_out"], out=s["out"])
        return {"out": s["out"]} if s["residual_out"] is None else {"out": s["out"], "residual": s["residual_out"]}
    if c["op"] == "conv":
        tern.short_conv(s["x"], s["weight"], s["state"], s["slots"], q_start=s["q_start"], max_new=s["max_new"],
                        bias=s["bias"], past=s["past"], dst_slots=s["dst_slots"], out=s["out"])
        return {"out": s["out"], "state": s["state"]}
    tern.gated_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["slots"], q_start=s["q_start"],
                     max_new=s["max_new"], scale=s["scale"], qk_norm=c["qk_norm"], a_log=s["a_log"],
                     dt_bias=s["dt_bias"], past=s["past"], dst_slots=s["dst_slots"], out=s["out"])
    return {"out": s["out"], "state": s["state"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        x, w = s["x"].double(), s["weight"].double()
        z = 1.0 if s["gate"] is None else s["gate"].double() / (1.0 + torch.exp(-s["gate"].double()))
        r = torch.zeros_like(x) if s["residual"] is None else s["residual"].double()
        if c["after"]:
            return {"out": r + s["scale"] * z * w * x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()}
        h = x if s["residual"] is None else r + s["scale"] * x
        out = {"out": z * w * h / (h.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()}
        return out if s["residual_out"] is None else {**out, "residual": h}
    state, slots, to = s["state"].double(), s["slots"].tolist(), s["dst_slots"].tolist()
    past, first = s["past"].tolist(), s["q_start"].tolist()
    if c["op"] == "conv":
        w, out, new = c["width"], [], state.clone()
        for b in range(c["seqs"]):
            x = s["x"][first[b]:first[b + 1]].double()
            x = torch.cat((state[slots[b]] if past[b] else torch.zeros_like(state[0]), x))
            y = sum(s["weight"][:, i].double() * x[i:i + len(x) - w + 1] for i in range(w))
            y = y if s["bias"] is None else y + s["bias"].double()
            out.append(y / (1.0 + torch.exp(-y)))
            new[to[b]] = x[len(x) - w + 1:]
        return {"out": torch.cat(out), "state": new}
    q, k, v, g, beta = (s[n].double() for n in ("q", "k", "v", "g", "beta"))
    if c["raw"]:
        g = -torch.exp(s["a_log"].double()) * torch.nn.functional.softplus(g + s["dt_bias"].double(), threshold=700.0)
        beta = 1.0 / (1.0 + torch.exp(-beta))
    if c["qk_norm"]:
        q, k = q / (q.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt(), k / (k.pow(2).sum(-1, keepdim=True) + 1e-6).sqrt()
    head = torch.arange(c["v_heads"], device=q.device) // (c["v_heads"] // c["k_heads"])
    S = state[s["slots"].long()]
    S[s["past"] == 0] = 0.0
    out = torch.zeros(v.shape, dtype=torch.float64, device=v.device)
    # the longest sequences first, so that those still running are always the first ones
    order = sorted(range(c["seqs"]), key=lambda b: -s["lens_host"][b])
    S, n = S[order], [s["lens_host"][b] for b in order]
    begin = torch.tensor([first[b] for b in order], device=q.device)
    for i in range(n[0]):
        m = sum(x > i for x in n)
        rows = begin[:m] + i
        kt, qt, R = k[rows][:, head, :, None], q[rows][:, head, :, None], S[:m]
        R *= g[rows].exp()[..., None, None]
        u = beta[rows][..., None, None] * (v[rows][..., None] - R @ kt)
        R += u * kt.transpose(-1, -2)
        out[rows] = s["scale"] * (R @ qt)[..., 0]
    state[s["dst_slots"].long()[order]] = S
    return {"out": out, "state": state}
