"""The serving operators around the ternary products: rotary positions that fill
a paged key/value cache, attention of new tokens over that cache, the attention
weight each cached key has received, and eviction by that weight.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end) where ``own`` is false, and through the
framework's entry points where it is true.  ``exact`` is the definition in 64
bits, written apart from both.

Layout of the cache: pages of ``page`` slots, one slot a token, ``kv_heads``
heads of ``head_dim`` bf16 values; key j of sequence b sits in slot j % page of
page table[b][j // page].  "hnd" pages hold [head][slot][value], "nhd" pages
[slot][head][value].  Sequence b brings new_b tokens whose keys are already the
last new_b of its lens[b] cached ones; query i sees key j where
j <= lens[b] - new_b + i (and, with a window, j > that - window).
"""
import math

import torch

own = False

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def _rope(name, seqs, new, ctx, q_heads, kv_heads, head_dim, rot_dim, interleaved, in_f32, page, layout, scaling):
    c = dict(op="rope", seqs=seqs, new=new, ctx=ctx, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
             rot_dim=rot_dim, interleaved=interleaved, in_f32=in_f32, page=page, layout=layout, scaling=scaling)
    return dict(c, name=name) if name else c


def _attn(name, op, seqs, new, ctx, ragged, q_heads, kv_heads, head_dim, page, layout, window):
    c = dict(op=op, seqs=seqs, new=new, ctx=ctx, ragged=ragged, q_heads=q_heads, kv_heads=kv_heads,
             head_dim=head_dim, page=page, layout=layout, window=window)
    return dict(c, name=name) if name else c


def _evict(name, seqs, ctx, ragged, kv_heads, head_dim, page, layout, budget, recent):
    c = dict(op="evict", seqs=seqs, ctx=ctx, ragged=ragged, kv_heads=kv_heads, head_dim=head_dim, page=page,
             layout=layout, budget=budget, recent=recent)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one generated token: the fp32 output of the decode product goes to the cache; latency is all
        _rope("rope_token", 1, 1, 1000, 32, 8, 128, 128, False, True, 16, "hnd", "none"),
        # a prompt's bf16 projections, a quarter of a wide head rotated in pairs, a context stretched by parts
        _rope("rope_prompt", 4, 2048, 30000, 16, 4, 256, 64, True, False, 32, "nhd", "yarn"),
        # one generated token of one short conversation: the smallest attention call
        _attn("attn_token_short", "attn", 1, 1, 500, False, 32, 8, 128, 16, "hnd", 0),
        # one token for each of 32 conversations of unlike length: the serving step, bound by reading the cache
        _attn("attn_token_batch", "attn", 32, 1, 16383, True, 32, 8, 128, 16, "hnd", 0),
        # a speculative verify step: five tokens each over long contexts of an odd length
        _attn("attn_verify", "attn", 4, 5, 31994, False, 32, 8, 128, 64, "nhd", 0),
        # a chunk of 512 prompt tokens over a long cache: bound by the tensor cores
        _attn("attn_chunk", "attn", 1, 512, 32000, False, 32, 8, 128, 64, "hnd", 0),
        # whole prompts of unlike length, small heads in groups of seven
        _attn("attn_prompts", "attn", 4, 4000, 0, True, 28, 4, 64, 16, "hnd", 0),
        # wide heads and a sliding window
        _attn("attn_window", "attn", 2, 300, 10000, False, 16, 4, 256, 32, "nhd", 4096),
        # one step's weights added to the running sums, a token for each of 8 conversations
        _attn("mass_token", "mass", 8, 1, 16383, True, 32, 8, 128, 16, "hnd", 0),
        # the weights that a chunk of 512 prompt tokens gives to the cache
        _attn("mass_chunk", "mass", 1, 512, 16000, False, 32, 8, 128, 64, "hnd", 0),
        # one conversation that just passed its budget
        _evict("evict_short", 1, 1100, False, 8, 128, 16, "hnd", 1024, 128),
        # sixteen long conversations of unlike length cut to 4096 keys
        _evict("evict_batch", 16, 20000, True, 8, 128, 32, "nhd", 4096, 512),
    ]


_HEADS = [(32, 8, 128), (16, 4, 256), (28, 4, 64), (8, 8, 128), (40, 8, 128), (16, 1, 64), (20, 4, 256), (22, 2, 128)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    pad = 0.0
    if case["op"] in ("attn", "mass"):  # what the padded plain form makes of it
        n, c = _lengths(case)
        pad = 4.0 * case["seqs"] * case["q_heads"] * max(n) * max(c) * case["head_dim"] / 60e12
    return max(w["bytes"] / 6e12, w["flops"] / 1e15), pad


def draw(rng):
    """One more case: sizes spread over their range (over its logarithm), odd ones among them."""
    most, most_pad = (max(v) for v in zip(*(_cost(c) for c in listed())))
    while True:
        op = rng.choice(["rope", "attn", "attn", "attn", "mass", "evict"])
        hq, hk, d = rng.choice(_HEADS)
        page, layout = rng.choice([16, 32, 48, 64, 128, 256]), rng.choice(["hnd", "nhd"])
        if op == "rope":
            new = rng.choice([1, _log(rng, 1, 4096)])
            c = _rope(None, _log(rng, 1, 64), new, _log(rng, 1, 60000), hq, hk, d,
                      rng.choice([d, d // 2, d // 4]), rng.random() < 0.5, rng.random() < 0.5, page, layout,
                      rng.choice(["none", "linear", "ntk", "yarn"]))
        elif op == "evict":
            ctx = _log(rng, 40, 40000)
            budget = _log(rng, 16, 8192)
            c = _evict(None, _log(rng, 1, 32), ctx, rng.random() < 0.5, hk, d, page, layout, budget,
                       rng.randint(0, budget))
        else:
            kind = rng.choice(["token", "verify", "chunk", "prompt"])
            new = {"token": 1, "verify": rng.randint(2, 16), "chunk": _log(rng, 17, 1024),
                   "prompt": _log(rng, 30, 4000)}[kind]
            seqs = _log(rng, 1, 48) if kind in ("token", "verify") else rng.randint(1, 4)
            ctx = 0 if kind == "prompt" else _log(rng, 1, 32000)
            window = _log(rng, 16, 8192) if rng.random() < 0.25 else 0
            c = _attn(None, op, seqs, new, ctx, rng.random() < 0.5, hq, hk, d, page, layout, window)
        cost, pad = _cost(c)
        if cost <= most and pad <= most_pad and _tokens(c) <= 65536:
            return c


def _tokens(c):
    return c["seqs"] * c.get("new", 1)


def _lengths(c):
    """(new tokens, cached keys) of each sequence; the cached keys include the new ones."""
    n, lens = [], []
    for b in range(c["seqs"]):
        new, ctx = c.get("new", 0), c["ctx"]
        if c.get("ragged"):  # from about a fifth of the full length up to it, in no order
            f = 0.2 + 0.8 * ((b * 7 + c["seqs"] - 1) % c["seqs"] + 1) / c["seqs"] if math.gcd(7, c["seqs"]) == 1 else \
                0.2 + 0.8 * (b + 1) / c["seqs"]
            ctx = int(ctx * f)
            if new > 16:
                new = max(1, int(new * (1.2 - f)))
        n.append(new)
        lens.append(ctx + new)
    return n, lens


def _pairs(c):
    """Query-key pairs that see each other, per head."""
    total = 0
    for n, length in zip(*_lengths(c)):
        w, lo = c["window"] or length, length - n   # position p, from lo on, sees min(p + 1, w) keys
        full = max(0, min(length, w) - lo)          # of them those below w see p + 1
        total += full * (2 * lo + full + 1) // 2 + (n - full) * w
    return total


def work(c):
    d, hk = c["head_dim"], c["kv_heads"]
    if c["op"] == "rope":
        t, width = _tokens(c), (c["q_heads"] + 2 * hk) * d
        return {"bytes": t * width * ((4 if c["in_f32"] else 2) + 2) + 12 * t + 2 * c["rot_dim"],
                "flops": 3 * t * (c["q_heads"] + hk) * c["rot_dim"]}
    if c["op"] == "evict":
        _, lens = _lengths(c)
        kept = sum(min(x, c["budget"]) for x in lens)
        return {"bytes": hk * (4 * sum(lens) + kept * (2 * 2 * 2 * d + 4 + 4)), "flops": hk * sum(lens)}
    n, lens = _lengths(c)
    keys = sum(min(x, c["window"] + a - 1) if c["window"] else x for a, x in zip(n, lens))
    rows = sum(n) * c["q_heads"]
    if c["op"] == "attn":
        return {"bytes": rows * (4 * d + 4) + 4 * d * hk * keys, "flops": 4 * d * c["q_heads"] * _pairs(c)}
    return {"bytes": rows * (2 * d + 4) + hk * (2 * d * keys + 8 * sum(lens)), "flops": 2 * d * c["q_heads"] * _pairs(c)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _frequencies(c):
    """Rotary frequencies (fp32) and the factor on cos and sin, for a context stretched four times."""
    r, base, factor, original = c["rot_dim"], 10000.0, 4.0, 8192
    if c["scaling"] == "ntk":
        base *= factor ** (r / max(r - 2, 1))
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if c["scaling"] == "linear":
        f = [x / factor for x in f]
    if c["scaling"] == "yarn":
        def at(turns):
            return r * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(0, math.floor(at(32.0))), min(r // 2 - 1, math.ceil(at(1.0)))
        for i in range(r // 2):
            ramp = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            f[i] = f[i] / factor * ramp + f[i] * (1 - ramp)
        return f, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _pool(c, pages, gen, dev):
    d, hk, page = c["head_dim"], c["kv_heads"], c["page"]
    shape = (pages, hk, page, d) if c["layout"] == "hnd" else (pages, page, hk, d)
    if gen is None:
        x = torch.zeros(shape, dtype=torch.bfloat16, device=dev)
    else:
        x = torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(generator=gen)
    return x if c["layout"] == "hnd" else x.permute(0, 2, 1, 3)


def _table(lens, page, gen, dev):
    """Scattered pages: [B, W] ids, entries past a sequence's last page 0, and how many pages there are."""
    need = [-(-x // page) for x in lens]
    w, total = max(max(need), 1), sum(need)
    ids = torch.randperm(total + 3, generator=gen, device=dev)[:max(total, 1)].to(torch.int32)
    first = torch.tensor([sum(need[:b]) for b in range(len(need))], device=dev)
    col = torch.arange(w, device=dev)
    at = (first[:, None] + col[None, :]).clamp(max=max(total, 1) - 1)
    used = col[None, :] < torch.tensor(need, device=dev)[:, None]
    return torch.where(used, ids[at], 0).to(torch.int32).contiguous(), total + 3


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    d, hk, page = c["head_dim"], c["kv_heads"], c["page"]
    n, lens = _lengths(c)
    table, pages = _table(lens, page, gen, dev)
    s = {"case": c, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
         "lens_host": lens, "new_host": n}
    if c["op"] == "evict":
        s["k_cache"], s["v_cache"] = _pool(c, pages, gen, dev), _pool(c, pages, gen, dev)
        # running sums: a few heavy keys, many light ones, and some that no query has met (ties at zero)
        u = torch.rand((pages, hk, page), generator=gen, device=dev)
        s["mass"] = torch.where(u < 0.05, 0.0, u ** 8 * 50.0)
        dst, dst_pages = _table([c["budget"]] * c["seqs"], page, gen, dev)
        s["dst_table"] = dst
        s["dst_k"], s["dst_v"] = _pool(c, dst_pages, None, dev), _pool(c, dst_pages, None, dev)
        s["dst_mass"] = torch.zeros((dst_pages, hk, page), device=dev)
        s["keep"] = torch.zeros((c["seqs"], hk, c["budget"]), dtype=torch.int32, device=dev)
        s["dst_lens"] = torch.zeros(c["seqs"], dtype=torch.int32, device=dev)
        s["scratch"] = torch.zeros(1 << 24, dtype=torch.uint8, device=dev)
        return s
    hq, t = c["q_heads"], sum(n)
    s["q_start"] = torch.tensor([sum(n[:b]) for b in range(len(n) + 1)], dtype=torch.int32, device=dev)
    s["max_new"] = max(n)
    if c["op"] == "rope":
        # one projection's output, [q heads | k heads | v heads] side by side
        x = torch.empty((t, (hq + 2 * hk) * d), device=dev).normal_(generator=gen)
        x = x if c["in_f32"] else x.to(torch.bfloat16)
        s["q"] = x[:, :hq * d].view(t, hq, d)
        s["k"] = x[:, hq * d:(hq + hk) * d].view(t, hk, d)
        s["v"] = x[:, (hq + hk) * d:].view(t, hk, d)
        seq = torch.bucketize(torch.arange(t, device=dev), s["q_start"][1:].long(), right=True)
        pos = torch.arange(t, device=dev) - s["q_start"].long()[seq] + (s["lens"] - torch.tensor(n, device=dev))[seq]
        s["positions"] = pos.to(torch.int32)
        s["slots"] = table[seq, pos // page].long() * page + pos % page
        f, s["factor"] = _frequencies(c)
        s["inv_freq"] = torch.tensor(f, dtype=torch.float32, device=dev)
        s["k_cache"], s["v_cache"] = _pool(c, pages, None, dev), _pool(c, pages, None, dev)
        s["q_out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev)
        return s
    # scores of a standard deviation near two: some hundreds of keys share a long row's weight
    s["q"] = torch.empty((t, hq, d), device=dev).normal_(generator=gen).mul_(2.0).to(torch.bfloat16)
    s["k_cache"] = _pool(c, pages, gen, dev)
    s["scale"] = d ** -0.5
    if c["op"] == "attn":
        s["v_cache"] = _pool(c, pages, gen, dev)
        s["out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty((t, hq), dtype=torch.float32, device=dev)
        s["scratch"] = torch.zeros(1 << 27, dtype=torch.uint8, device=dev)
    else:
        scores, seq, i = _scores(s)
        s["lse"] = torch.logsumexp(scores, dim=-1)[seq, :, :, i].reshape(t, hq).contiguous()
        s["mass"] = torch.rand((pages, hk, page), generator=gen, device=dev) * 4.0
        s["mass_out"] = torch.zeros((pages, hk, page), device=dev)
        s["decay"] = 0.9375
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------


def _scores(s):
    """Scaled scores [B, kv_heads, group, new, keys] in 32 bits, -inf where masked, and where each token is."""
    c, q, table = s["case"], s["q"], s["table"].long()
    hk, d, w = c["kv_heads"], c["head_dim"], c["window"]
    start, lens, t = s["q_start"].long(), s["lens"].long(), q.shape[0]
    row = torch.arange(t, device=q.device)
    seq = torch.bucketize(row, start[1:], right=True)
    i = torch.arange(s["max_new"], device=q.device)
    at = (start[:-1, None] + i).clamp(max=t - 1)
    x = q[at].float().unflatten(2, (hk, -1)).permute(0, 2, 3, 1, 4)             # [B, hk, group, new, d]
    keys = s["k_cache"][table].permute(0, 2, 1, 3, 4).flatten(2, 3).float()     # [B, hk, keys, d]
    scores = (x.flatten(2, 3) @ keys.transpose(-1, -2)).unflatten(2, x.shape[2:4]).mul_(s["scale"])
    pos = (lens - (start[1:] - start[:-1]))[:, None] + i                         # [B, new]
    j = torch.arange(keys.shape[2], device=q.device)
    seen = (j <= pos[..., None]) & (i < (start[1:] - start[:-1])[:, None])[..., None]
    if w:
        seen &= j > pos[..., None] - w
    return scores.masked_fill_(~seen[:, None, None], -math.inf), seq, row - start[seq]


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].float()[:, None] * s["inv_freq"]
    cos, sin = (angle.cos() * s["factor"])[:, None], (angle.sin() * s["factor"])[:, None]
    r = c["rot_dim"]

    def turned(x):
        x = x.float()
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])
        y = (a * cos - b * sin, b * cos + a * sin)
        y = torch.stack(y, dim=-1).flatten(-2) if c["interleaved"] else torch.cat(y, dim=-1)
        return torch.cat((y, x[..., r:]), dim=-1).to(torch.bfloat16)

    page, slot = s["slots"] // c["page"], s["slots"] % c["page"]
    s["k_cache"][page, :, slot] = turned(s["k"])
    s["v_cache"][page, :, slot] = s["v"].to(torch.bfloat16)
    return {"q": turned(s["q"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attn(s):
    scores, seq, i = _scores(s)
    top = scores.amax(dim=-1, keepdim=True)
    p = scores.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    values = s["v_cache"][s["table"].long()].permute(0, 2, 1, 3, 4).flatten(2, 3).float()
    o = (p.flatten(2, 3) @ values).unflatten(2, p.shape[2:4]) / total.clamp(min=1e-30)
    lse = (top + total.log()).squeeze(-1)
    t, hq = s["q"].shape[:2]
    return {"out": o[seq, :, :, i].reshape(t, hq, -1).to(torch.bfloat16), "lse": lse[seq, :, :, i].reshape(t, hq)}


def _plain_mass(s):
    c = s["case"]
    scores, seq, i = _scores(s)
    hk, group = scores.shape[1:3]
    lse = torch.full(scores.shape[:4], math.inf, device=scores.device)
    lse[seq, :, :, i] = s["lse"].view(-1, hk, group)
    got = scores.sub_(lse[..., None]).exp_().sum(dim=(2, 3))                     # [B, hk, keys]
    table, page = s["table"].long(), c["page"]
    j = torch.arange(got.shape[2], device=got.device).expand(got.shape[0], -1)
    # every key of a sequence has a slot of its own; the keys past a sequence's end go to slot 0 of a spare row
    live = j < s["lens"][:, None]
    rows = s["mass"].shape[0]
    where = torch.where(live, table.gather(1, j // page) * page + j % page, rows * page)
    sums = torch.zeros((rows + 1) * page, hk, device=got.device)
    sums[where.flatten()] = got.permute(0, 2, 1).flatten(0, 1)
    touched = torch.zeros((rows + 1) * page, dtype=torch.bool, device=got.device)
    touched[where.flatten()] = True
    new = s["mass"] * s["decay"] + sums[:rows * page].view(rows, page, hk).transpose(1, 2)
    s["mass_out"].copy_(torch.where(touched[:rows * page].view(rows, 1, page), new, s["mass_out"]))
    return {"mass": s["mass_out"]}


def _plain_evict(s):
    c = s["case"]
    table, page, budget = s["table"].long(), c["page"], c["budget"]
    mass = s["mass"][table].permute(0, 2, 1, 3).flatten(2)                       # [B, hk, keys]
    lens = s["lens"].long()[:, None, None]
    j = torch.arange(mass.shape[2], device=mass.device)
    key = torch.where(j >= lens - c["recent"], math.inf, mass)
    key = torch.where(j < lens, key, -math.inf)
    order = key.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    live = torch.arange(order.shape[2], device=mass.device) < lens.clamp(max=budget)
    keep = torch.where(live, order, mass.shape[2]).sort(dim=-1).values           # ascending, the rest at the end
    keep = torch.nn.functional.pad(keep, (0, budget - keep.shape[2]), value=mass.shape[2])
    live = torch.arange(budget, device=mass.device).expand_as(keep) < lens.clamp(max=budget)
    at = torch.where(live, keep, 0)
    b = torch.arange(table.shape[0], device=mass.device)[:, None, None]
    h = torch.arange(c["kv_heads"], device=mass.device)[None, :, None]
    src, slot = table[b, at // page], at % page
    i = torch.arange(budget, device=mass.device).expand_as(keep)
    dst, dslot = s["dst_table"].long()[b, i // page], i % page
    h, live1 = h.expand_as(dst), live[..., None]
    for to, of in (("dst_k", "k_cache"), ("dst_v", "v_cache")):
        s[to][dst, h, dslot] = torch.where(live1, s[of][src, h, slot], s[to][dst, h, dslot])
    s["dst_mass"][dst, h, dslot] = torch.where(live, s["mass"][src, h, slot], s["dst_mass"][dst, h, dslot])
    s["keep"].copy_(torch.where(live, keep, -1))
    s["dst_lens"].copy_(s["lens"].clamp(max=budget))
    return {"keep": s["keep"], "lens": s["dst_lens"], "k": s["dst_k"], "v": s["dst_v"], "mass": s["dst_mass"]}


def run(s):
    c = s["case"]
    if not own:
        return {"rope": _plain_rope, "attn": _plain_attn, "mass": _plain_mass, "evict": _plain_evict}[c["op"]](s)
    import bit_gemv_gemm_gb300 as tern
    if c["op"] == "rope":
        tern.rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"], s["k_cache"],
                         s["v_cache"], q_out=s["q_out"], interleaved=c["interleaved"], attn_factor=s["factor"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["op"] == "attn":
        tern.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], q_start=s["q_start"],
                             max_new=s["max_new"], scale=s["scale"], window=c["window"], out=s["out"], lse=s["lse"],
                             ws=s["scratch"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "mass":
        tern.attention_mass(s["q"], s["k_cache"], s["table"], s["lens"], s["lse"], s["mass"], out=s["mass_out"],
                            q_start=s["q_start"], max_new=s["max_new"], scale=s["scale"], window=c["window"],
                            decay=s["decay"])
        return {"mass": s["mass_out"]}
    tern.cache_evict(s["k_cache"], s["v_cache"], s["mass"], s["table"], s["lens"], c["budget"], c["recent"],
                     s["dst_k"], s["dst_v"], s["dst_mass"], s["dst_table"], keep=s["keep"], dst_lens=s["dst_lens"],
                     ws=s["scratch"])
    return {"keep": s["keep"], "lens": s["dst_lens"], "k": s["dst_k"], "v": s["dst_v"], "mass": s["dst_mass"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one sequence at a time
# ---------------------------------------------------------------------------


def _rows_of(pool, table_row, length, page):
    """Keys 0 .. length - 1 of one sequence, [heads, length, ...], in 64 bits."""
    j = torch.arange(length, device=pool.device)
    return pool[table_row.long()[j // page], :, j % page].transpose(0, 1).double()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    page, hk, d = c["page"], c["kv_heads"], c["head_dim"]
    if c["op"] == "rope":
        r, t = c["rot_dim"], s["q"].shape[0]
        angle = torch.outer(s["positions"].double(), s["inv_freq"].double())
        turn = torch.polar(torch.full_like(angle, s["factor"]), angle)[:, None]   # a pair as a complex number

        def turned(x):
            x = x.double().clone()
            re, im = (slice(0, r, 2), slice(1, r, 2)) if c["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
            z = torch.complex(x[..., re], x[..., im]) * turn
            x[..., re], x[..., im] = z.real, z.imag
            return x

        caches = []
        for x, like in ((turned(s["k"]), s["k_cache"]), (s["v"].double(), s["v_cache"])):
            flat = torch.zeros(like.shape[0] * page, hk, d, dtype=torch.float64, device=x.device)
            flat[s["slots"]] = x
            caches.append(flat.view(-1, page, hk, d).transpose(1, 2))
        return {"q": turned(s["q"]), "k_cache": caches[0], "v_cache": caches[1]}
    if c["op"] == "evict":
        keep, k, v, mass = s["keep"].cpu(), s["dst_k"].double(), s["dst_v"].double(), s["dst_mass"].double()
        for b, length in enumerate(s["lens_host"]):
            m, n = _rows_of(s["mass"], s["table"][b], length, page), min(length, c["budget"])
            safe = min(c["recent"], n)
            kk, vv = (_rows_of(s[x], s["table"][b], length, page) for x in ("k_cache", "v_cache"))
            j = torch.arange(n, device=k.device)
            to = s["dst_table"][b].long()[j // page], j % page
            for h in range(hk):
                values = m[h, :length - safe].tolist()
                best = sorted(range(length - safe), key=lambda x: (-values[x], x))[:n - safe]
                chosen = torch.tensor(sorted(best) + list(range(length - safe, length)), dtype=torch.long)
                keep[b, h] = -1
                keep[b, h, :n] = chosen.to(torch.int32)
                chosen = chosen.to(k.device)
                k[to[0], h, to[1]], v[to[0], h, to[1]] = kk[h, chosen], vv[h, chosen]
                mass[to[0], h, to[1]] = m[h, chosen]
        lens = torch.tensor([min(x, c["budget"]) for x in s["lens_host"]], dtype=torch.int32)
        return {"keep": keep, "lens": lens, "k": k, "v": v, "mass": mass}
    group, parts = c["q_heads"] // hk, []
    new_mass = s["mass_out"].double() if c["op"] == "mass" else None
    for b, (n, length) in enumerate(zip(s["new_host"], s["lens_host"])):
        keys = _rows_of(s["k_cache"], s["table"][b], length, page)
        vals = _rows_of(s["v_cache"], s["table"][b], length, page) if c["op"] == "attn" else None
        sums = torch.zeros(hk, length, dtype=torch.float64, device=keys.device)
        first, step = int(sum(s["new_host"][:b])), max(1, (1 << 27) // (length * hk * group))
        j = torch.arange(length, device=keys.device)
        for lo in range(0, n, step):
            hi = min(n, lo + step)
            x = s["q"][first + lo:first + hi].double().view(hi - lo, hk, group, d)
            z = torch.einsum("nhgd,hld->nhgl", x, keys) * s["scale"]
            p = torch.arange(length - n + lo, length - n + hi, device=keys.device)[:, None]
            hide = (j > p) | (j <= p - c["window"]) if c["window"] else j > p
            z.masked_fill_(hide[:, None, None], -math.inf)
            if c["op"] == "attn":
                lse = torch.logsumexp(z, dim=-1)
                parts.append((torch.einsum("nhgl,hld->nhgd", (z - lse[..., None]).exp_(), vals), lse))
            else:
                known = s["lse"][first + lo:first + hi].double().view(hi - lo, hk, group, 1)
                sums += (z - known).exp_().sum(dim=(0, 2))
        if c["op"] == "mass":
            old = _rows_of(s["mass"], s["table"][b], length, page)
            new_mass[s["table"][b].long()[j // page], :, j % page] = (s["decay"] * old + sums).transpose(0, 1)
    if c["op"] == "mass":
        return {"mass": new_mass}
    t = s["q"].shape[0]
    return {"out": torch.cat([x[0] for x in parts]).reshape(t, -1, d),
            "lse": torch.cat([x[1] for x in parts]).reshape(t, -1)}
