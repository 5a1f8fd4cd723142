"""The decoder-block operators as they are measured.

Five operators around the frozen-NF4 linears of a decoder block:

  norm   the residual update between two branches of a block: the branch
         output normalised (optional), gated per channel (optional), scaled
         and added to the residual stream, and the stream normalised for the
         next branch; forward and backward
  rope   rotary positions on queries and keys, both pair layouts, part of the
         head, frequencies scaled for long contexts; forward and backward
  write  the serving form of rope: queries rotated, keys rotated and stored
         with the values into the slots of a paged key-value cache
  attn   attention of one new token per sequence over the paged cache
  plan   pages, block tables, slots and positions of a batch of requests

`run` computes them in elementary torch operations (32 bits inside, angles in
64, one rounding at the end) when `own` is false and calls the package when it
is true.  `exact` is the definition in 64 bits.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # --- norm: a decode step of 16 sequences at the 65B-shaped width, the plain pre-norm block
        # (no norm behind the branch, no gate): where latency counts
        {"name": "norm_fwd_16x8192", "op": "norm", "bwd": False, "tokens": 16, "width": 8192, "x": "bf16",
         "h": "bf16", "post": False, "gate": False, "alpha": 1.0},
        # a training batch of 8192 tokens at that width, every part on
        {"name": "norm_fwd_8192x8192", "op": "norm", "bwd": False, "tokens": 8192, "width": 8192, "x": "bf16",
         "h": "bf16", "post": True, "gate": True, "alpha": 0.5},
        # the backward with a 32-bit residual stream and 16-bit branches (what the block keeps) at the
        # 7B width, an odd number of tokens, with the gradients of the gains and the gate
        {"name": "norm_bwd_8191x4096", "op": "norm", "bwd": True, "tokens": 8191, "width": 4096, "x": "f32",
         "h": "bf16", "post": True, "gate": True, "alpha": 0.5},
        # --- rope: 4 sequences of 1024 tokens, 32 heads of 128 (the 7B attention shape)
        {"name": "rope_fwd_4096x32x128", "op": "rope", "bwd": False, "tokens": 4096, "seq": 1024, "start": 0,
         "heads": 32, "kv_heads": 32, "dim": 128, "rot": 128, "dtype": "bf16", "interleaved": False,
         "scaling": "none", "factor": 1.0},
        # the backward at far positions of a context stretched 16 times: pairs interleaved, half of each
        # head rotated, shared key heads, 32 bits, an odd number of tokens
        {"name": "rope_bwd_8191x64x128", "op": "rope", "bwd": True, "tokens": 8191, "seq": 8191, "start": 122880,
         "heads": 64, "kv_heads": 8, "dim": 128, "rot": 64, "dtype": "f32", "interleaved": True,
         "scaling": "yarn", "factor": 16.0},
        # --- write: one token of each of 16 sequences, 64 query heads on 8 key heads
        {"name": "write_16x64x128", "op": "write", "tokens": 16, "seq": 1, "start": 1000, "heads": 64,
         "kv_heads": 8, "dim": 128, "rot": 128, "page": 16, "slots": 32768, "interleaved": False,
         "scaling": "none", "factor": 1.0},
        # the prompts of 8 sequences of 1024 tokens, 32 heads
        {"name": "write_8192x32x128", "op": "write", "tokens": 8192, "seq": 1024, "start": 0, "heads": 32,
         "kv_heads": 32, "dim": 128, "rot": 128, "page": 64, "slots": 16384, "interleaved": False,
         "scaling": "none", "factor": 1.0},
        # --- attn: one sequence of 512 tokens (few rows, the length has to be split)
        {"name": "attn_1x512_32on32", "op": "attn", "seqs": 1, "low": 512, "high": 512, "heads": 32,
         "kv_heads": 32, "dim": 128, "page": 16},
        # 16 sequences of very different lengths up to 4096, every head its own keys
        {"name": "attn_16x4096_32on32", "op": "attn", "seqs": 16, "low": 1, "high": 4096, "heads": 32,
         "kv_heads": 32, "dim": 128, "page": 16},
        # long contexts: 8 sequences up to 65536 tokens, 64 query heads on 8 key heads
        {"name": "attn_8x65536_64on8", "op": "attn", "seqs": 8, "low": 32768, "high": 65536, "heads": 64,
         "kv_heads": 8, "dim": 128, "page": 64},
        # --- plan: one decode step of 16 running sequences
        {"name": "plan_16x1", "op": "plan", "seqs": 16, "cached_high": 4096, "new_low": 1, "new_high": 1,
         "page": 16, "pad": 0},
        # 1024 prompts of up to 511 tokens, some of them continuing a cached prefix, with padded rows behind
        {"name": "plan_1024x511", "op": "plan", "seqs": 1024, "cached_high": 1500, "new_low": 0, "new_high": 511,
         "page": 16, "pad": 1000},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "rope", "write", "attn", "attn", "plan"])
    if op == "norm":
        width = rng.choice([128, 256, 1000, 2048, 4096, 4097, 8192])
        x = rng.choice(["bf16", "f32"])
        return {"op": op, "bwd": rng.random() < 0.5, "tokens": _log_int(rng, 1, 8192), "width": width, "x": x,
                "h": "bf16" if x == "bf16" else rng.choice(["bf16", "f32"]), "post": rng.random() < 0.6,
                "gate": rng.random() < 0.6, "alpha": rng.choice([1.0, 0.5, 0.22])}
    if op in ("rope", "write"):
        dim = rng.choice([64, 80, 96, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        tokens = _log_int(rng, 1, 4096)
        case = {"op": op, "tokens": tokens, "seq": _log_int(rng, 1, tokens), "start": _log_int(rng, 1, 200000) - 1,
                "heads": kv * rng.choice([1, 2, 4, 8]), "kv_heads": kv, "dim": dim,
                "rot": dim // rng.choice([1, 1, 2]), "interleaved": rng.random() < 0.5, "scaling": scaling,
                "factor": 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 16.0])}
        if op == "rope":
            case.update(bwd=rng.random() < 0.5, dtype=rng.choice(["bf16", "f32"]))
        else:
            case.update(page=rng.choice([16, 32, 64, 128]), slots=8192)
        return case
    if op == "attn":
        seqs, kv = _log_int(rng, 1, 64), rng.choice([1, 2, 4, 8])
        high = _log_int(rng, 1, 262144 // (seqs * kv) * 2)
        return {"op": op, "seqs": seqs, "low": rng.choice([0, high // 2, high]), "high": high,
                "heads": kv * rng.choice([1, 2, 3, 4, 7, 8, 16]), "kv_heads": kv, "dim": rng.choice([64, 80, 96, 128]),
                "page": rng.choice([16, 32, 64, 128])}
    high = _log_int(rng, 1, 256)
    return {"op": op, "seqs": _log_int(rng, 1, 1024), "cached_high": rng.choice([0, 100, 1500]),
            "new_low": rng.choice([0, 1, high]), "new_high": high, "page": rng.choice([1, 16, 32, 64, 128]),
            "pad": rng.choice([0, 1, 333])}


# ------------------------------------------------------------------ inputs

def _spread(n, low, high):
    """n whole numbers spread evenly over [low, high] (both ends taken when n > 1)."""
    return [high] if n == 1 else [low + (high - low) * i // (n - 1) for i in range(n)]


def _frequencies(case):
    """Angle per position of each pair, in radians (fp64), and the factor on the rotated values."""
    rot, base, factor = case["rot"], 10000.0, case["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    if case["scaling"] == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "yarn":
        turns = f * 8192 / (2 * math.pi)               # turns a pair makes over the trained length
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _table(case):
    """The rotary table that a program builds once."""
    if own:
        from bit_nf4_quantized_quantize_amd import RopeTable
        return RopeTable(case["rot"], base=10000.0, scaling=case["scaling"], factor=case["factor"],
                         original_len=8192, interleaved=case["interleaved"], device=torch.device("cuda"))
    f, m = _frequencies(case)
    return f.cuda(), m


def _positions(case):
    t = torch.arange(case["tokens"], device="cuda")
    return (case["start"] + t % case["seq"]).to(torch.int32)


def _shuffled(g, values, dtype=torch.int32):
    v = torch.tensor(values, dtype=torch.int64, device="cuda")
    return v[torch.randperm(v.numel(), generator=g, device="cuda")].to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        return (mean + std * torch.randn(*shape, generator=g, device="cuda")).to(dtype)

    op, st = case["op"], {"case": case}
    if op == "norm":
        T, D, xt, ht = case["tokens"], case["width"], _DT[case["x"]], _DT[case["h"]]
        st["x"], st["h"] = n(T, D, dtype=xt), n(T, D, dtype=ht, std=0.3)
        st["w_post"] = n(D, std=0.1, mean=1.0) if case["post"] else None
        st["gate"] = n(D, std=0.2, mean=0.5) if case["gate"] else None
        st["w_pre"] = n(D, std=0.1, mean=1.0)
        if case["bwd"]:
            st["dxo"], st["dn"] = n(T, D, dtype=xt), n(T, D, dtype=ht)
        return st
    if op in ("rope", "write"):
        T, d = case["tokens"], case["dim"]
        dt = _DT[case.get("dtype", "bf16")]
        st["q"], st["k"] = n(T, case["heads"], d, dtype=dt), n(T, case["kv_heads"], d, dtype=dt)
        st["positions"] = _positions(case)
        st["table"] = _table(case)
        if op == "write":
            st["v"] = n(T, case["kv_heads"], d, dtype=dt)
            pages = case["slots"] // case["page"]
            shape = (pages, case["kv_heads"], case["page"], d)
            st["k_cache"], st["v_cache"] = n(*shape, dtype=dt), n(*shape, dtype=dt)
            order = torch.randperm(case["slots"], generator=g, device="cuda")[:T] if case["seq"] == 1 else None
            if order is None:   # prompts fill whole pages, the pages in any order
                page = torch.randperm(pages, generator=g, device="cuda")
                t = torch.arange(T, device="cuda")
                order = page[t // case["page"]] * case["page"] + t % case["page"]
            st["slots"] = order.to(torch.int32)
        return st
    if op == "attn":
        S, page = case["seqs"], case["page"]
        lens = _spread(S, case["low"], case["high"])
        most = max(1, -(-case["high"] // page))
        pages = S * most
        st["q"] = n(S, case["heads"], case["dim"], dtype=torch.bfloat16)
        shape = (pages, case["kv_heads"], page, case["dim"])
        st["k_cache"], st["v_cache"] = n(*shape, dtype=torch.bfloat16), n(*shape, dtype=torch.bfloat16)
        st["table"] = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(S, most)
        st["lengths"] = _shuffled(g, lens)
        return st
    S, page = case["seqs"], case["page"]
    cached, new = _spread(S, 0, case["cached_high"]), _spread(S, case["new_low"], case["new_high"])
    st["cached"], st["new"] = _shuffled(g, cached), _shuffled(g, new)
    most = -(-(case["cached_high"] + case["new_high"]) // page) + 1
    pages = S * most
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    have = (st["cached"] + page - 1) // page
    col = torch.arange(most, device="cuda")
    taken = torch.cumsum(have, 0) - have
    st["block_table"] = torch.where(col < have[:, None], ids[(taken[:, None] + col).clamp(max=pages - 1)],
                                    torch.full_like(ids[:1], -1))
    st["free"] = ids[int(have.sum()):].contiguous()
    st["tokens"] = sum(new) + case["pad"]
    return st


# --------------------------------------------------------- the plain forms

def _norm_plain(st):
    c = st["case"]
    h, a = st["h"].float(), c["alpha"]
    u = h
    if c["post"]:
        u = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * st["w_post"]
    x = st["x"].float() + a * (u * st["gate"] if c["gate"] else u)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * st["w_pre"]
    return x.to(st["x"].dtype), y.to(st["h"].dtype)


def _norm_bwd_plain(st):
    # st["x"] is the residual stream after the update, as the forward returned it
    c = st["case"]
    x, h, a = st["x"].float(), st["h"].float(), c["alpha"]
    dn = st["dn"].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    dw_pre = (dn * xh).sum(0)
    t = dn * st["w_pre"]
    gx = st["dxo"].float() + r * (t - xh * (t * xh).mean(-1, keepdim=True))
    du = a * gx
    if c["post"]:
        rh = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
        hh = h * rh
        u = hh * st["w_post"]
    else:
        u = h
    dgate = (du * u).sum(0) if c["gate"] else None
    if c["gate"]:
        du = du * st["gate"]
    dw_post = None
    if c["post"]:
        dw_post = (du * hh).sum(0)
        t = du * st["w_post"]
        du = rh * (t - hh * (t * hh).mean(-1, keepdim=True))
    out = [gx.to(st["x"].dtype), du.to(st["h"].dtype), dw_pre]
    return out + [d for d in (dw_post, dgate) if d is not None]


def _rotate_plain(z, positions, table, case, sign):
    f, m = table
    rot = case["rot"]
    ang = positions.double()[:, None] * f
    cos, sin = (ang.cos() * m).float()[:, None, :], (sign * ang.sin() * m).float()[:, None, :]
    zf = z.float()
    out = zf.clone()
    if case["interleaved"]:
        a, b = zf[..., 0:rot:2], zf[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = zf[..., :rot // 2], zf[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    return out.to(z.dtype)


def _write_plain(st):
    c = st["case"]
    q = _rotate_plain(st["q"], st["positions"], st["table"], c, 1.0)
    k = _rotate_plain(st["k"], st["positions"], st["table"], c, 1.0)
    s = st["slots"].long()
    page, off = s // c["page"], s % c["page"]
    st["k_cache"][page, :, off] = k
    st["v_cache"][page, :, off] = st["v"]
    return q, st["k_cache"], st["v_cache"]


def _attn_plain(st):
    c = st["case"]
    S, H, KV, d, page = c["seqs"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    L = st["table"].shape[1] * page
    t = st["table"].long()
    k = st["k_cache"][t].float().permute(0, 2, 1, 3, 4).reshape(S, KV, L, d)
    v = st["v_cache"][t].float().permute(0, 2, 1, 3, 4).reshape(S, KV, L, d)
    q = st["q"].float().view(S, KV, H // KV, d).transpose(2, 3).contiguous() / math.sqrt(d)
    s = torch.matmul(k, q).transpose(2, 3).contiguous()                  # [S, KV, G, L]
    out = torch.arange(L, device=s.device) >= st["lengths"][:, None, None, None]
    s = s.masked_fill(out, float("-inf"))
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - top.masked_fill(top == float("-inf"), 0.0))
    den = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / den.masked_fill(den == 0, 1.0)              # a sequence of no tokens gives zeros
    return o.reshape(S, H, d).to(st["q"].dtype)


def _plan_plain(st):
    page, free, table = st["case"]["page"], st["free"], st["block_table"]
    cached, new = st["cached"].long(), st["new"].long()
    total = cached + new
    have, need = (cached + page - 1) // page, (total + page - 1) // page
    take = need - have
    first = torch.cumsum(take, 0) - take
    col = torch.arange(table.shape[1], device=table.device)
    index = first[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    pick = free[index.clamp(0, free.numel() - 1)]
    table.copy_(torch.where(fresh, pick, table))
    starts = torch.zeros(new.numel() + 1, dtype=torch.int64, device=new.device)
    starts[1:] = torch.cumsum(new, 0)
    t = torch.arange(st["tokens"], device=new.device)
    seq = torch.searchsorted(starts, t, right=True) - 1
    real = t < starts[-1]
    seq = seq.clamp(max=new.numel() - 1)
    pos = torch.where(real, cached[seq] + t - starts[seq], torch.zeros_like(t))
    slot = table[seq, torch.where(real, pos // page, torch.zeros_like(pos))].long() * page + pos % page
    slot = torch.where(real, slot, torch.full_like(slot, -1))
    i32 = torch.int32
    return table, total.to(i32), starts.to(i32), slot.to(i32), pos.to(i32)


# ------------------------------------------------------------------- a pass

def run(st):
    c = st["case"]
    op = c["op"]
    if not own:
        if op == "norm":
            return _norm_bwd_plain(st) if c["bwd"] else _norm_plain(st)
        if op == "rope":
            sign = -1.0 if c["bwd"] else 1.0
            return tuple(_rotate_plain(st[z], st["positions"], st["table"], c, sign) for z in ("q", "k"))
        return {"write": _write_plain, "attn": _attn_plain, "plan": _plan_plain}[op](st)
    from bit_nf4_quantized_quantize_amd import decoder as D
    if op == "norm":
        if not c["bwd"]:
            return D.qlora_norm_residual_fwd(st["x"], st["h"], w_pre=st["w_pre"], w_post=st["w_post"],
                                             gate=st["gate"], alpha=c["alpha"], eps=EPS)
        gr = D.qlora_norm_residual_bwd(st["dxo"], st["dn"], st["x"], st["h"], w_pre=st["w_pre"],
                                       w_post=st["w_post"], gate=st["gate"], alpha=c["alpha"], eps=EPS,
                                       need_gains=True)
        return [t for t in (gr.dx, gr.dh, gr.dw_pre, gr.dw_post, gr.dgate) if t is not None]
    if op == "rope":
        return D.qlora_rope(st["q"], st["k"], st["table"], st["positions"], inverse=c["bwd"])
    if op == "write":
        q = D.qlora_rope_cache_write(st["q"], st["k"], st["v"], st["table"], st["positions"], st["slots"],
                                     st["k_cache"], st["v_cache"])
        return q, st["k_cache"], st["v_cache"]
    if op == "attn":
        return D.qlora_paged_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lengths"])
    p = D.qlora_paged_plan(st["cached"], st["new"], st["free"], st["block_table"], c["page"], st["tokens"])
    return st["block_table"], p.total_lens, p.starts, p.slots, p.positions


# ------------------------------------------------ the definitions in 64 bits

def _norm_exact(st):
    c = st["case"]
    x, h, w = st["x"].double(), st["h"].double(), st["w_pre"].double()
    D = c["width"]
    one = torch.ones(D, dtype=torch.float64, device=x.device)
    wp = st["w_post"].double() if c["post"] else one
    gate = st["gate"].double() if c["gate"] else one

    def unit(z):
        return z / torch.sqrt((z ** 2).sum(-1, keepdim=True) / D + EPS)

    if not c["bwd"]:
        u = (unit(h) if c["post"] else h) * wp
        xo = x + c["alpha"] * gate * u
        return xo, unit(xo) * w

    def unit_grad(z, dy):   # of sum(dy * unit(z)) for z
        s = torch.sqrt((z ** 2).sum(-1, keepdim=True) / D + EPS)
        return dy / s - z * (dy * z).sum(-1, keepdim=True) / (D * s ** 3)

    dn = st["dn"].double()
    dx = st["dxo"].double() + unit_grad(x, dn * w)
    y = unit(h) if c["post"] else h
    dy = c["alpha"] * dx * gate * wp
    out = [dx, unit_grad(h, dy) if c["post"] else dy, (dn * unit(x)).sum(0)]
    if c["post"]:
        out.append((c["alpha"] * dx * gate * y).sum(0))
    if c["gate"]:
        out.append((c["alpha"] * dx * wp * y).sum(0))
    return out


def _rotate_exact(z, case, st):
    f, m = _frequencies(case)
    r = case["rot"]
    ang = torch.outer(st["positions"].double(), f.to(z.device))
    if case.get("bwd"):
        ang = -ang
    turn = torch.polar(torch.full_like(ang, m), ang)[:, None]
    z = z.double()
    p = z[..., :r]
    p = p.unflatten(-1, (r // 2, 2)) if case["interleaved"] else p.unflatten(-1, (2, r // 2)).transpose(-1, -2)
    p = torch.view_as_real(torch.view_as_complex(p.contiguous()) * turn)
    p = p.flatten(-2) if case["interleaved"] else p.transpose(-1, -2).flatten(-2)
    return torch.cat([p, z[..., r:]], -1)


def _attn_exact(st):
    c = st["case"]
    S, H, KV, d, page = c["seqs"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    out = torch.zeros(S, H, d, dtype=torch.float64, device="cuda")
    for s, n in enumerate(st["lengths"].tolist()):
        if n == 0:
            continue
        rows = st["table"][s, :-(-n // page)].long()
        for j in range(KV):
            k = st["k_cache"][rows, j].reshape(-1, d)[:n].double()
            v = st["v_cache"][rows, j].reshape(-1, d)[:n].double()
            for i in range(j * (H // KV), (j + 1) * (H // KV)):
                p = torch.softmax((k * st["q"][s, i].double()).sum(-1) * d ** -0.5, 0)
                out[s, i] = (p[:, None] * v).sum(0)
    return out


def _plan_exact(st):
    page = st["case"]["page"]
    free, table = st["free"].tolist(), st["block_table"].tolist()
    cached, new = st["cached"].tolist(), st["new"].tolist()
    total, starts, slots, positions, used = [], [0], [], [], 0
    for s, (c, n) in enumerate(zip(cached, new)):
        for j in range(-(-c // page), -(-(c + n) // page)):
            table[s][j] = free[used]
            used += 1
        for p in range(c, c + n):
            slots.append(table[s][p // page] * page + p % page)
            positions.append(p)
        total.append(c + n)
        starts.append(starts[-1] + n)
    pad = st["tokens"] - len(slots)
    return tuple(torch.tensor(v, dtype=torch.int32, device="cuda")
                 for v in (table, total, starts, slots + [-1] * pad, positions + [0] * pad))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _norm_exact(st)
    if op == "rope":
        return _rotate_exact(st["q"], case, st), _rotate_exact(st["k"], case, st)
    if op == "write":
        caches = []
        for z, cache in ((_rotate_exact(st["k"], case, st), st["k_cache"]), (st["v"].double(), st["v_cache"])):
            flat = cache.double().transpose(1, 2).reshape(-1, case["kv_heads"], case["dim"])  # [slot, head, dim]
            flat[st["slots"].long()] = z
            caches.append(flat.view(-1, case["page"], case["kv_heads"], case["dim"]).transpose(1, 2))
        return _rotate_exact(st["q"], case, st), caches[0], caches[1]
    if op == "attn":
        return _attn_exact(st)
    return _plan_exact(st)


# -------------------------------------------------------------- what it costs

def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "norm":
        T, D, sx, sh = case["tokens"], case["width"], size[case["x"]], size[case["h"]]
        gains = 4 * D * (1 + case["post"] + case["gate"])
        if case["bwd"]:   # dxo, dn, xo in, dx, dh out; h in where the gradients need it
            h_in = sh if case["post"] or case["gate"] else 0
            return {"bytes": T * D * (3 * sx + 2 * sh + h_in) + 2 * gains, "flops": 30 * T * D}
        return {"bytes": T * D * 2 * (sx + sh) + gains, "flops": 12 * T * D}
    if op in ("rope", "write"):
        T, d, H, KV = case["tokens"], case["dim"], case["heads"], case["kv_heads"]
        sz = size[case.get("dtype", "bf16")]
        rows = H + KV * (2 if op == "write" else 1)
        return {"bytes": 2 * T * rows * d * sz + T * (8 if op == "write" else 4) + 4 * case["rot"],
                "flops": 3 * T * (H + KV) * case["rot"]}
    if op == "attn":
        n = sum(_spread(case["seqs"], case["low"], case["high"]))
        pages = sum(-(-v // case["page"]) for v in _spread(case["seqs"], case["low"], case["high"]))
        io = 4 * case["seqs"] * case["heads"] * case["dim"]
        return {"bytes": 4 * n * case["kv_heads"] * case["dim"] + io + 4 * (pages + case["seqs"]),
                "flops": 4 * n * case["heads"] * case["dim"]}
    S, page = case["seqs"], case["page"]
    tokens = sum(_spread(S, case["new_low"], case["new_high"])) + case["pad"]
    pages = S + tokens // page      # about: pages taken, read from the free list and written to the table
    return {"bytes": 8 * S + 8 * S + 8 * tokens + 8 * pages, "flops": 4 * tokens}
