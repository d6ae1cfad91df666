"""Measured cases of the 8-bit paged cache and of the pass that feeds it: the
norm and rotation of a step's queries and keys, the cache that is quantised as
it is written, its rows read back, and the attention that reads it.

  norm_rope           an RMS norm of every head of q and k, then op "rope" at
                      positions of one to four axes, in one pass
  paged_write_q8      new K and V rows into an 8-bit pool by a slot map
  paged_read_q8       rows of such a pool back as f32
  paged_attention_q8  ragged batches against the 8-bit pool: single tokens,
                      prompt chunks, and trees of drafted (f32) tokens

A pool holds int8 or e4m3 codes [pages * pageSize, kvHeads * headDim] and a
scale [pages * pageSize, kvHeads] for K and for V; an element is code x scale.
An int8 scale is the head's largest |element| / 127, an e4m3 scale the least
power of two with which the largest |element| is at most 448; neither is below
2^-126, and a code is the nearest one, ties to even.  Rows are packed and pages
named as in the f32 paged cache: rows cu_rows[b] .. cu_rows[b + 1] - 1 are request
b's, row s of it is pool row block_table[b, s // pageSize] * pageSize + s %
pageSize.  With `own` the library's entry points run; without it the same
results come from elementary torch operations.
"""
import math

import torch

own = False

GOLD = 0.6180339887498949
LEAST = 2.0 ** -126


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One user's next token on a short chat: latency alone.
        dict(name="attn_one_token", op="attn", form="int8", requests=1, len_lo=211, len_hi=211, rows_lo=1, rows_hi=1,
             tree=False, heads=16, kv_heads=4, head_dim=128, page=16, window=0, sinks=0, softcap=0.0, scale=0.0),
        # A serving batch's ordinary step: one token each, ragged contexts.
        dict(name="attn_batch_tokens", op="attn", form="int8", requests=32, len_lo=517, len_hi=8111, rows_lo=1,
             rows_hi=1, tree=False, heads=32, kv_heads=8, head_dim=128, page=16, window=0, sinks=0, softcap=0.0,
             scale=0.0),
        # Long documents that only fit because the cache is small: one token each.
        dict(name="attn_long_tokens", op="attn", form="e4m3", requests=24, len_lo=8192, len_hi=32704, rows_lo=1,
             rows_hi=1, tree=False, heads=32, kv_heads=8, head_dim=128, page=64, window=0, sinks=0, softcap=0.0,
             scale=0.0),
        # Small drafted trees, headDim 64, an odd group, a sliding window with sinks and a softcap.
        dict(name="attn_small_trees", op="attn", form="e4m3", requests=5, len_lo=90, len_hi=3001, rows_lo=5,
             rows_hi=21, tree=True, heads=12, kv_heads=4, head_dim=64, page=32, window=1024, sinks=4, softcap=30.0,
             scale=0.11),
        # The largest trees over long contexts: 64 nodes x 4 heads per KV head.
        dict(name="attn_large_trees", op="attn", form="int8", requests=8, len_lo=16384, len_hi=32704, rows_lo=64,
             rows_hi=64, tree=True, heads=32, kv_heads=8, head_dim=128, page=64, window=0, sinks=0, softcap=0.0,
             scale=0.0),
        # Chunks of prompts over what is cached of them, beside each other in one step.
        dict(name="attn_chunks", op="attn", form="int8", requests=3, len_lo=1000, len_hi=5003, rows_lo=129,
             rows_hi=509, tree=False, heads=40, kv_heads=8, head_dim=128, page=16, window=0, sinks=0, softcap=0.0,
             scale=0.0),
        # A decode batch's new rows, one per request.
        dict(name="write_tokens", op="write", form="int8", rows=32, kv_heads=8, head_dim=128, page=16, pages=4096,
             skipped=0.1),
        # The rows of a batch of prompts.
        dict(name="write_prompts", op="write", form="e4m3", rows=32003, kv_heads=8, head_dim=128, page=16, pages=4096,
             skipped=0.02),
        # A few rows of another head width, to be looked at or moved.
        dict(name="read_rows", op="read", form="e4m3", rows=67, kv_heads=5, head_dim=96, page=16, pages=256,
             skipped=0.1),
        # A long request's rows, out of the cache for a pass that takes f32.
        dict(name="read_request", op="read", form="int8", rows=31999, kv_heads=8, head_dim=128, page=16, pages=4096,
             skipped=0.0),
        # Queries and keys of one small tree.
        dict(name="norm_rope_tree", op="rope", rows=23, heads=32, kv_heads=8, head_dim=128, rotary=128,
             interleaved=False, base=500000.0, pos_hi=32768, axes=1, dealt=False, norm=True, offset=0.0),
        # Prompts with images: positions in time, height and width.
        dict(name="norm_rope_images", op="rope", rows=8111, heads=32, kv_heads=8, head_dim=128, rotary=128,
             interleaved=False, base=1000000.0, pos_hi=32768, axes=3, dealt=True, norm=True, offset=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "attn", "write", "read", "rope", "rope"])
    if op == "attn":
        cost = [work(c) for c in listed() if c["op"] == "attn"]
        most_bytes, most_flops = max(w["bytes"] for w in cost), max(w["flops"] for w in cost)
        while True:
            kind = rng.choice(["token", "token", "run", "tree"])
            hk, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
            hi_len = _log(rng, 20, 32704)
            hi_rows = 1 if kind == "token" else _log(rng, 2, 509) if kind == "run" else _log(rng, 2, 64)
            if kind != "tree":
                hi_len = max(hi_len, hi_rows + 1)
            lo_rows = rng.randint(1, hi_rows)
            lo_len = rng.randint(hi_rows if kind != "tree" else 1, hi_len)
            c = dict(op="attn", form=rng.choice(["int8", "e4m3"]), requests=_log(rng, 1, 64), len_lo=lo_len,
                     len_hi=hi_len, rows_lo=lo_rows, rows_hi=hi_rows, tree=kind == "tree", heads=hk * g, kv_heads=hk,
                     head_dim=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 128]),
                     window=rng.choice([0, 0, 0, _log(rng, 8, 4096)]), sinks=rng.choice([0, 4, 37]),
                     softcap=rng.choice([0.0, 0.0, 0.0, 20.0]), scale=rng.choice([0.0, 0.0, 0.07]))
            w = work(c)
            # the plain form pads every request to the longest
            pad = c["requests"] * (hi_len + 64) * hk * c["head_dim"] * 8
            scores = 4.0 * c["requests"] * hk * g * hi_rows * (hi_len + 64)
            if w["bytes"] <= most_bytes and w["flops"] <= most_flops and pad <= 7e9 and scores <= 2.2e9:
                return c
    if op in ("write", "read"):
        pages = 4096 if op == "write" else _log(rng, 128, 4096)
        page = rng.choice([16, 64]) if pages <= 1024 else 16
        return dict(op=op, form=rng.choice(["int8", "e4m3"]), rows=min(_log(rng, 1, 32003), pages * page),
                    kv_heads=rng.randint(1, 8), head_dim=rng.choice([64, 80, 96, 128]), page=page, pages=pages,
                    skipped=rng.choice([0.0, 0.02, 0.3]))
    d = rng.choice([64, 96, 128, 128])
    axes = rng.choice([1, 1, 2, 3, 4])
    hk = rng.randint(1, 8)
    return dict(op="rope", rows=_log(rng, 1, 8111), heads=hk * rng.randint(1, 5), kv_heads=hk, head_dim=d,
                rotary=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.3,
                base=rng.choice([10000.0, 500000.0]), pos_hi=_log(rng, 100, 131072), axes=axes,
                dealt=axes > 1 and rng.random() < 0.5, norm=rng.random() < 0.8, offset=rng.choice([0.0, 0.0, 1.0]))


def _spread(n, lo, hi, salt):
    """n whole numbers over lo..hi, the same ones for every seed."""
    return [lo + int((hi - lo + 1) * ((i + 1) * GOLD + salt) % (hi - lo + 1)) if hi > lo else lo for i in range(n)]


def _sizes(case):
    """Request lengths and row counts of a case."""
    n = case["requests"]
    lens, rows = _spread(n, case["len_lo"], case["len_hi"], 0.0), _spread(n, case["rows_lo"], case["rows_hi"], 0.37)
    lens[0], rows[0] = case["len_hi"], case["rows_hi"]
    return lens, rows


def _sections(case):
    """Pairs of each position axis: the first gets what the equal shares of the others leave."""
    half, axes = case["rotary"] // 2, case["axes"]
    share = half // axes - (1 if axes > 1 and half // axes > 2 else 0)
    return [half - share * (axes - 1)] + [share] * (axes - 1)


def _seen(case, length, t):
    """(keys that some row of a request sees, keys seen summed over its rows), at least."""
    ctx = length if case["tree"] else length - t
    total = ctx + t
    w, k = case["window"], case["sinks"]
    if not w:
        return total, (t * total if not case["tree"] else t * (ctx + 1)) - (t * (t - 1) // 2 if not case["tree"] else 0)
    return min(total, w + t + k), t * min(max(1, ctx), w)


def work(case):
    op = case["op"]
    if op == "attn":
        lens, rows = _sizes(case)
        hd, hk = case["heads"] * case["head_dim"], case["kv_heads"]
        kd = hk * case["head_dim"]
        b = f = 0
        for length, t in zip(lens, rows):
            union, pairs = _seen(case, length, t)
            cached, fresh = (union, 0) if not case["tree"] else (max(union - t, 0), t)
            b += 2 * cached * (kd + 4 * hk) + 8 * fresh * kd + 8 * t * hd + 4 * (-(-cached // case["page"])) + 8
            b += 12 * t if case["tree"] else 0
            f += 4 * pairs * hd
        return {"bytes": b, "flops": f}
    n = case["rows"]
    if op == "rope":
        heads = case["heads"] + case["kv_heads"]
        return {"bytes": 8 * n * heads * case["head_dim"] + 4 * n * case["axes"],
                "flops": n * heads * (3 * case["rotary"] + 4 * case["head_dim"])}
    width, hk = case["kv_heads"] * case["head_dim"], case["kv_heads"]
    live = 1 - case["skipped"]
    if op == "read":  # rows of no slot are zeros
        return {"bytes": int(2 * n * (live * (width + 4 * hk) + 4 * width)) + 4 * n, "flops": 2 * n * width}
    return {"bytes": int(2 * n * live * (5 * width + 4 * hk)) + 4 * n, "flops": 4 * n * width}


# ------------------------------------------------------------------ inputs
def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    cpu = torch.Generator()
    cpu.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case=case)
    op = case["op"]
    if op == "rope":
        n, d = case["rows"], case["head_dim"]
        pos = torch.randint(0, case["pos_hi"], (case["axes"], n), generator=g, device="cuda", dtype=torch.int32)
        s.update(q=normal(n, case["heads"] * d) * 3, k=normal(n, case["kv_heads"] * d) * 5,
                 positions=pos if case["axes"] > 1 else pos[0].contiguous(),
                 qw=1 + 0.2 * normal(d) - case["offset"], kw=1 + 0.2 * normal(d) - case["offset"])
        return s
    hk, d, form = case["kv_heads"], case["head_dim"], case["form"]
    # Keys of trained models have a few channels that are much larger than the rest, and
    # heads differ in size.
    gain = torch.ones(hk * d, device="cuda")
    gain[torch.randperm(hk * d, generator=cpu)[: max(1, hk * d // 32)].cuda()] = 4.0
    gain = gain * torch.exp2(torch.linspace(-3, 2, hk, device="cuda")).repeat_interleave(d)
    if op in ("write", "read"):
        total, n = case["pages"] * case["page"], case["rows"]
        slots = torch.randperm(total, generator=g, device="cuda")[:n].to(torch.int32)
        slots[torch.rand(n, generator=g, device="cuda") < case["skipped"]] = -1
        kp, ks = _quantise(normal(total, hk * d) * gain, hk, form)
        vp, vs = _quantise(normal(total, hk * d), hk, form)
        s.update(slots=slots, k_pool=kp, k_scale=ks, v_pool=vp, v_scale=vs)
        if op == "write":
            s.update(k_new=normal(n, hk * d) * gain, v_new=normal(n, hk * d))
        return s
    lens, rows = _sizes(case)
    perm = torch.randperm(len(lens), generator=cpu).tolist()  # the seed orders the batch
    lens, rows = [lens[i] for i in perm], [rows[i] for i in perm]
    cu = [0]
    for t in rows:
        cu.append(cu[-1] + t)
    s.update(lens=_ints(lens), cu_rows=_ints(cu), rows=cu[-1])
    page = case["page"]
    held = [-(-n // page) for n in lens]
    pages = sum(held) + 3
    ids = torch.randperm(pages, generator=cpu, dtype=torch.int64).to(torch.int32)
    table, at = torch.full((len(lens), max(max(held), 1)), -1, dtype=torch.int32), 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    # Scores of trained models reach ten or so, whatever the heads' sizes.
    heads_gain = torch.exp2(torch.linspace(3, -2, hk, device="cuda")).repeat_interleave(case["heads"] // hk * d)
    kp, ks = _quantise(normal(pages * page, hk * d) * gain, hk, form)
    vp, vs = _quantise(normal(pages * page, hk * d), hk, form)
    s.update(table=table.cuda(), k_pool=kp, k_scale=ks, v_pool=vp, v_scale=vs,
             q=normal(s["rows"], case["heads"] * d) * heads_gain)
    if case["tree"]:
        parents, u = torch.zeros(cu[-1], dtype=torch.int32), torch.rand(cu[-1], generator=cpu)
        for a, b in zip(cu, cu[1:]):  # a node hangs below an earlier one; now and then another root
            j = torch.arange(b - a)
            par = (u[a:b] * j).to(torch.int32)
            par[(u[a:b] > 0.97) | (j == 0)] = -1
            parents[a:b] = par
        s["parents"] = parents.cuda()
        s.update(k_new=normal(s["rows"], hk * d) * gain, v_new=normal(s["rows"], hk * d))
        s["masks"], s["positions"] = _paths(s["parents"], s["cu_rows"], s["lens"])
    return s


def _paths(parents, cu, lens):
    """Ancestor masks and positions of the drafted rows."""
    r = torch.arange(parents.numel(), device=cu.device)
    b = torch.searchsorted(cu.long(), r, right=True) - 1
    j, p = r - cu.long()[b], parents.long()
    up = torch.where((p >= 0) & (p < j), cu.long()[b] + p, torch.full_like(p, -1))
    mask = torch.ones_like(j) << j
    for _ in range(6):  # each pass doubles the length of the path that a mask covers
        at = up.clamp(min=0)
        mask = torch.where(up >= 0, mask | mask[at], mask)
        up = torch.where(up >= 0, up[at], up)
    depth = ((mask[:, None] >> torch.arange(64, device=mask.device)) & 1).sum(1) - 1
    return mask, (lens.long()[b] + depth).to(torch.int32)


# ------------------------------------------------------------- plain forms
def _quantise(x, kv_heads, form):
    """(codes, scales) of rows; quotients next to a border in 64 bits."""
    h = x.view(x.shape[0], kv_heads, -1)
    top = h.abs().amax(-1)
    fine = torch.isfinite(top)
    if form == "int8":
        scale = (top.double() / 127.0).float().clamp_min(LEAST)
        code = torch.round(h.double() / scale.double()[..., None]).to(torch.int8)
    else:
        part, e = torch.frexp(top)  # top = part 2^e, part in [1/2, 1); 448 = 7/8 2^9
        e = torch.where(top > 0, torch.where(part <= 0.875, e - 9, e - 8), torch.full_like(e, -126)).clamp(min=-126)
        scale = torch.ldexp(torch.ones_like(top), e)
        code = (h / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    code = torch.where(fine[..., None], code, torch.zeros_like(code)).view(x.shape)
    scale = torch.where(fine, scale, torch.full_like(scale, math.nan))
    return (code if form == "int8" else code.view(torch.float8_e4m3fn)), scale


def _values(pool, scale, rows):
    """Rows of a pool as f32, [.., kv_heads, head_dim]."""
    code = pool.view(torch.uint8)[rows].view(pool.dtype).float()
    return code.view(*rows.shape, scale.shape[1], -1) * scale[rows][..., None]


def _write(s):
    case, live = s["case"], s["slots"] >= 0
    at = s["slots"][live].long()
    for a in ("k", "v"):
        code, scale = _quantise(s[a + "_new"][live], case["kv_heads"], case["form"])
        s[a + "_pool"].view(torch.uint8)[at] = code.view(torch.uint8)
        s[a + "_scale"][at] = scale
    return [s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"]]


def _read(s):
    live = s["slots"] >= 0
    at = s["slots"].long().clamp(min=0)
    out = []
    for a in ("k", "v"):
        x = _values(s[a + "_pool"], s[a + "_scale"], at)
        out.append(torch.where(live[:, None, None], x, torch.zeros_like(x)).flatten(1))
    return out


def _axis_of(case):
    """The axis of each rotated pair: runs of pairs, or pairs dealt out in turn."""
    sec, axes = _sections(case), case["axes"]
    if not case["dealt"]:
        return torch.arange(axes).repeat_interleave(torch.tensor(sec))
    j = torch.arange(case["rotary"] // 2)
    return torch.where(j < axes * torch.tensor(sec)[j % axes], j % axes, torch.zeros_like(j))


def _norm_rope(s):
    case = s["case"]
    d, rd = case["head_dim"], case["rotary"]
    pos = s["positions"].view(case["axes"], -1).double()
    dev = pos.device
    j = torch.arange(rd // 2, device=dev, dtype=torch.float64)
    th = pos[_axis_of(case).to(dev)].T * torch.pow(torch.tensor(case["base"], dtype=torch.float64, device=dev), -2.0 * j / rd)
    c, n = th.cos().float()[:, None, :], th.sin().float()[:, None, :]
    res = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        h = x.view(x.shape[0], -1, d)
        if case["norm"]:
            h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * (w + case["offset"])
        out = h.clone()
        if case["interleaved"]:
            a, b = h[..., 0:rd:2], h[..., 1:rd:2]
            out[..., 0:rd:2], out[..., 1:rd:2] = a * c - b * n, b * c + a * n
        else:
            a, b = h[..., : rd // 2], h[..., rd // 2:rd]
            out[..., : rd // 2], out[..., rd // 2:rd] = a * c - b * n, b * c + a * n
        res.append(out.view_as(x))
    return res


def _attention(s):
    case = s["case"]
    hk, d = case["kv_heads"], case["head_dim"]
    g, page = case["heads"] // hk, case["page"]
    cu, lens, table = s["cu_rows"].long(), s["lens"].long(), s["table"]
    n, most = lens.numel(), case["rows_hi"]
    t = cu[1:] - cu[:-1]
    i = torch.arange(most, device=cu.device)
    row = (cu[:-1, None] + i).clamp(max=s["rows"] - 1)                       # [n, most]
    alive = i < t[:, None]
    q = s["q"][row].view(n, most, hk, g, d).permute(0, 2, 1, 3, 4).reshape(n, hk, most * g, d)
    key = torch.arange(table.shape[1] * page, device=cu.device)
    at = (table.long()[:, key // page].clamp(min=0) * page + key % page)     # [n, keys]
    there = key < lens[:, None]
    kk, vv = _values(s["k_pool"], s["k_scale"], at), _values(s["v_pool"], s["v_scale"], at)
    if case["tree"]:
        pos = s["positions"].long()[row]                                     # [n, most]
        kpos = torch.cat([key.expand(n, -1), pos], 1)
        see = there[:, None, :].expand(n, most, -1)
        anc = ((s["masks"][row][:, :, None] >> i) & 1).bool() & alive[:, None, :]
        see = torch.cat([see, anc], 2)
        kk = torch.cat([kk, s["k_new"][row].view(n, most, hk, d)], 1)
        vv = torch.cat([vv, s["v_new"][row].view(n, most, hk, d)], 1)
    else:
        pos = lens[:, None] - t[:, None] + i
        kpos = key.expand(n, -1)
        see = there[:, None, :] & (key <= pos[:, :, None])
    if case["window"]:
        ctx = torch.arange(kpos.shape[1], device=cu.device) < key.numel()
        near = kpos[:, None, :] > pos[:, :, None] - case["window"]
        see = see & (near | ((kpos < case["sinks"]) & ctx)[:, None, :])
    x = torch.matmul(q, kk.permute(0, 2, 3, 1)) * (case["scale"] or 1.0 / math.sqrt(d))
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    see = see[:, None, :, None, :].expand(n, hk, most, g, -1).reshape(n, hk, most * g, -1)
    x = x.masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    den = p.sum(-1, keepdim=True)
    o = torch.matmul(p, vv.permute(0, 2, 1, 3)) / torch.where(den > 0, den, torch.ones_like(den))
    o = o.view(n, hk, most, g, d).permute(0, 2, 1, 3, 4).reshape(n, most, hk * g * d)
    return o[alive]


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"attn": _attention, "write": _write, "read": _read, "rope": _norm_rope}[op](state)
    import f32_gqa_attention_gb300 as vtmu
    if op == "rope":
        return list(vtmu.norm_rope(state["q"], state["k"], state["positions"], headDim=case["head_dim"],
                                   norm=case["norm"], qWeight=state["qw"] if case["norm"] else None,
                                   kWeight=state["kw"] if case["norm"] else None, weightOffset=case["offset"],
                                   sections=_sections(case) if case["axes"] > 1 else None, dealt=case["dealt"],
                                   base=case["base"], rotaryDim=case["rotary"], interleaved=case["interleaved"]))
    pools = [state[a] for a in ("k_pool", "v_pool", "k_scale", "v_scale")]
    if op == "attn":
        tree = (state["k_new"], state["v_new"], state["masks"], state["positions"]) if case["tree"] else None
        return vtmu.paged_attention_q8(state["q"], *pools, state["table"], state["lens"], state["cu_rows"], tree=tree,
                                       heads=case["heads"], kvHeads=case["kv_heads"], headDim=case["head_dim"],
                                       pageSize=case["page"], maxRows=case["rows_hi"], window=case["window"],
                                       sinks=case["sinks"], softcap=case["softcap"], scale=case["scale"] or None)
    if op == "read":
        return list(vtmu.paged_read_q8(*pools, state["slots"]))
    vtmu.paged_write_q8(*pools, state["k_new"], state["v_new"], state["slots"])
    return pools


# ---------------------------------------------------------- 64-bit answers
def _exact_codes(x, form):
    """One head's rows: codes as the numbers they are, scales."""
    top = x.abs().max(1, keepdim=True).values
    if form == "int8":
        scale = torch.clamp((top / 127).to(torch.float32).double(), min=LEAST)
        return torch.round(x / scale), scale[:, 0]
    scale = torch.exp2(torch.ceil(torch.log2((top / 448).clamp(min=LEAST))))
    y = x / scale
    # The spacing of e4m3 numbers: 2^-3 of the power of two below, at least 2^-9.
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, scale[:, 0]


def _rows64(pool, scale, rows, head, d):
    """Rows of one head of a pool."""
    code = pool.view(torch.uint8)[rows][:, head * d:(head + 1) * d].contiguous().view(pool.dtype)
    return code.to(torch.float32).double() * scale[rows, head].double()[:, None]


def exact(case, seed):
    """The definitions in 64 bits, request by request and head by head."""
    s = prepare(case, seed)
    op, d, hk = case["op"], case["head_dim"], case["kv_heads"]
    if op == "rope":
        rd, axis, res = case["rotary"], _axis_of(case).tolist(), []
        pos = s["positions"].view(case["axes"], -1).double()
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            out = x.double().clone()
            for h in range(x.shape[1] // d):
                y = out[:, h * d:(h + 1) * d]
                if case["norm"]:
                    y /= torch.sqrt((y * y).sum(1, keepdim=True) / d + 1e-6)
                    y *= w.double() + case["offset"]
                for j in range(rd // 2):
                    turn = pos[axis[j]] * float(case["base"]) ** (-2.0 * j / rd)
                    a, b = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + rd // 2)
                    z = torch.complex(y[:, a], y[:, b]) * torch.polar(torch.ones_like(turn), turn)
                    y[:, a], y[:, b] = z.real, z.imag
            res.append(out)
        return res
    if op == "write":
        live = (s["slots"] >= 0).nonzero()[:, 0]
        at, pools, scales = s["slots"].long()[live], [], []
        for a in ("k", "v"):
            pool, scale = s[a + "_pool"].to(torch.float32).double(), s[a + "_scale"].double()
            for h in range(hk):
                code, sc = _exact_codes(s[a + "_new"][live][:, h * d:(h + 1) * d].double(), case["form"])
                pool[at, h * d:(h + 1) * d], scale[at, h] = code, sc
            pools.append(pool if case["form"] == "e4m3" else pool.to(torch.int8))
            scales.append(scale)
        return pools + scales
    if op == "read":
        live = (s["slots"] >= 0).nonzero()[:, 0]
        at, res = s["slots"].long()[live], []
        for a in ("k", "v"):
            out = torch.zeros(case["rows"], hk * d, dtype=torch.float64, device="cuda")
            for h in range(hk):
                out[live, h * d:(h + 1) * d] = _rows64(s[a + "_pool"], s[a + "_scale"], at, h, d)
            res.append(out)
        return res
    page, g = case["page"], case["heads"] // hk
    cu, lens = s["cu_rows"].tolist(), s["lens"].tolist()
    out = torch.zeros(s["rows"], case["heads"] * d, dtype=torch.float64, device="cuda")
    for b, length in enumerate(lens):
        a, e = cu[b], cu[b + 1]
        if a == e:
            continue
        kpos = torch.arange(length, device="cuda")
        at = s["table"][b].long()[kpos // page] * page + kpos % page
        sink = kpos < case["sinks"]
        if case["tree"]:
            ppos = s["positions"][a:e].long()
            line = torch.zeros(e - a, e - a, dtype=torch.bool)
            for j, up in enumerate(s["parents"][a:e].tolist()):
                if 0 <= up < j:
                    line[j] = line[up]
                line[j, j] = True
            allowed = torch.cat([torch.ones(e - a, length, dtype=torch.bool), line], 1).cuda()
            kpos, sink = torch.cat([kpos, ppos]), torch.cat([sink, torch.zeros(e - a, dtype=torch.bool, device="cuda")])
        else:
            ppos = torch.arange(length - (e - a), length, device="cuda")
            allowed = kpos[None] <= ppos[:, None]
        if case["window"]:
            allowed = allowed & ((ppos[:, None] - kpos[None] < case["window"]) | sink[None])
        for m in range(hk):
            k, v = (_rows64(s[x + "_pool"], s[x + "_scale"], at, m, d) for x in ("k", "v"))
            if case["tree"]:
                k = torch.cat([k, s["k_new"][a:e, m * d:(m + 1) * d].double()])
                v = torch.cat([v, s["v_new"][a:e, m * d:(m + 1) * d].double()])
            for h in range(m * g, (m + 1) * g):
                x = s["q"][a:e, h * d:(h + 1) * d].double() @ k.T * (case["scale"] or d ** -0.5)
                if case["softcap"]:
                    x = torch.tanh(x / case["softcap"]) * case["softcap"]
                x = torch.where(allowed, x, torch.full_like(x, -math.inf))
                w = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
                out[a:e, h * d:(h + 1) * d] = torch.nan_to_num(w, nan=0.0) @ v
    return out
