"""Measured cases of the paged-cache operators: a batch of requests whose K and
V rows live in pages of one shared pool, decoded with drafted token trees.

  page_map         block tables, slot maps and positions from request lengths
  tree_plan        ancestor masks and positions of drafted trees from parents
  rope_at          op "rope" at a position given per row
  paged_write      new K and V rows into the pool by a slot map
  paged_attention  ragged batches against the paged cache: single tokens,
                   short runs, and trees of drafted tokens

Layouts are the library's: flat row-major f32 tensors, heads side by side in a
row; a pool is [pages * pageSize, kvHeads * headDim] and row s of request b is
pool row block_table[b, s // pageSize] * pageSize + s % pageSize.  Requests are
packed one after the other: rows cu_rows[b] .. cu_rows[b + 1] - 1 are request
b's.  With `own` the library's entry points run; without it the same results
come from elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

GOLD = 0.6180339887498949


# ------------------------------------------------------------------- cases
def listed():
    return [
        # One user's next token on a short chat: latency alone.
        dict(name="attn_one_token", op="attn", requests=1, len_lo=211, len_hi=211, rows_lo=1, rows_hi=1, tree=False,
             heads=16, kv_heads=4, head_dim=128, page=16, window=0, sinks=0, softcap=0.0, scale=0.0),
        # A serving batch's ordinary step: one token each, ragged contexts.
        dict(name="attn_batch_tokens", op="attn", requests=32, len_lo=517, len_hi=8111, rows_lo=1, rows_hi=1,
             tree=False, heads=32, kv_heads=8, head_dim=128, page=16, window=0, sinks=0, softcap=0.0, scale=0.0),
        # Small drafted trees, headDim 64, odd group counts, sliding window with sinks and a softcap.
        dict(name="attn_small_trees", op="attn", requests=5, len_lo=90, len_hi=3001, rows_lo=5, rows_hi=21, tree=True,
             heads=12, kv_heads=4, head_dim=64, page=32, window=1024, sinks=4, softcap=30.0, scale=0.11),
        # The largest trees over long contexts: 64 nodes x 4 heads per KV head.
        dict(name="attn_large_trees", op="attn", requests=8, len_lo=16384, len_hi=32704, rows_lo=64, rows_hi=64,
             tree=True, heads=32, kv_heads=8, head_dim=128, page=64, window=0, sinks=0, softcap=0.0, scale=0.0),
        # Slots of the rows that a step's verification kept, a handful of requests.
        dict(name="map_accepted", op="map", requests=7, len_lo=40, len_hi=5003, rows_lo=9, rows_hi=33, accept=True,
             page=16, max_pages=512),
        # A batch of prompts and chunks comes in: many rows and pages at once.
        dict(name="map_prompts", op="map", requests=256, len_lo=0, len_hi=3000, rows_lo=1, rows_hi=1021, accept=False,
             page=16, max_pages=1024),
        # One request's drafted tree.
        dict(name="tree_one", op="tree", requests=1, len_lo=300, len_hi=300, rows_lo=13, rows_hi=13),
        # The trees of a large batch.
        dict(name="tree_batch", op="tree", requests=512, len_lo=1, len_hi=30000, rows_lo=1, rows_hi=64),
        # The queries of one small tree.
        dict(name="rope_tree", op="rope", rows=23, heads=32, head_dim=128, rotary=128, interleaved=False, base=500000.0,
             pos_hi=32768),
        # Queries and keys side by side for a batch of prompts.
        dict(name="rope_prompts", op="rope", rows=8111, heads=40, head_dim=128, rotary=128, interleaved=False,
             base=500000.0, pos_hi=131072),
        # A decode batch's new rows, one per request.
        dict(name="write_tokens", op="write", rows=32, width=1024, page=16, pages=4096, skipped=0.1),
        # The rows of a batch of prompts.
        dict(name="write_prompts", op="write", rows=32003, width=1024, page=16, pages=4096, skipped=0.02),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "attn", "map", "tree", "rope", "write"])
    if op == "attn":
        top = work(next(c for c in listed() if c["name"] == "attn_large_trees"))
        while True:
            kind = rng.choice(["token", "run", "tree", "tree"])
            hk, g = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8])
            hi_len = _log(rng, 20, 32768)
            hi_rows = 1 if kind == "token" else _log(rng, 2, 12) if kind == "run" else _log(rng, 2, 64)
            if kind != "tree":
                hi_len = max(hi_len, hi_rows + 1)
            lo_rows = rng.randint(1, hi_rows)
            lo_len = rng.randint(hi_rows if kind != "tree" else 1, hi_len)
            c = dict(op="attn", requests=_log(rng, 1, 64), len_lo=lo_len, len_hi=hi_len, rows_lo=lo_rows,
                     rows_hi=hi_rows, tree=kind == "tree", heads=hk * g, kv_heads=hk,
                     head_dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
                     window=rng.choice([0, 0, 0, _log(rng, 8, 4096)]), sinks=rng.choice([0, 4, 37]),
                     softcap=rng.choice([0.0, 0.0, 0.0, 20.0]), scale=rng.choice([0.0, 0.0, 0.07]))
            w = work(c)
            # the plain form pads every request to the longest
            pad = c["requests"] * (hi_len + 64) * hk * c["head_dim"] * 8
            scores = 4.0 * c["requests"] * hk * g * hi_rows * (hi_len + 64)
            if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"] and pad <= 2.2e9 and scores <= 2.2e9:
                return c
    if op == "map":
        acc = rng.random() < 0.5
        hi = _log(rng, 1, 64 if acc else 1021)
        return dict(op="map", requests=_log(rng, 1, 256), len_lo=0, len_hi=_log(rng, 1, 3000), rows_lo=rng.randint(0, hi),
                    rows_hi=hi, accept=acc, page=rng.choice([16, 32, 64, 128]), max_pages=rng.choice([256, 509, 1024]))
    if op == "tree":
        hi = _log(rng, 1, 64)
        return dict(op="tree", requests=_log(rng, 1, 512), len_lo=0, len_hi=_log(rng, 1, 100000),
                    rows_lo=rng.randint(0, hi), rows_hi=hi)
    if op == "rope":
        d = rng.choice([64, 96, 128])
        return dict(op="rope", rows=_log(rng, 1, 8111), heads=rng.randint(1, 40), head_dim=d,
                    rotary=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.3, base=rng.choice([10000.0, 500000.0]),
                    pos_hi=_log(rng, 100, 131072))
    return dict(op="write", rows=_log(rng, 1, 32003), width=64 * rng.randint(1, 16), page=rng.choice([16, 64]),
                pages=4096, skipped=rng.choice([0.0, 0.02, 0.3]))


def _spread(n, lo, hi, salt):
    """n whole numbers over lo..hi, the same ones for every seed."""
    return [lo + int((hi - lo + 1) * ((i + 1) * GOLD + salt) % (hi - lo + 1)) if hi > lo else lo for i in range(n)]


def _sizes(case):
    """Request lengths and row counts of a case."""
    n = case["requests"]
    lens, rows = _spread(n, case["len_lo"], case["len_hi"], 0.0), _spread(n, case["rows_lo"], case["rows_hi"], 0.37)
    lens[0] = case["len_hi"]
    rows[0] = case["rows_hi"]
    return lens, rows


def _seen(case, length, t):
    """(keys that some row of a request sees, keys seen summed over its rows), at least."""
    ctx = length if case["tree"] else length - t
    total = ctx + t
    w, k = case["window"], case["sinks"]
    if not w:
        return total, (t * total if not case["tree"] else t * (ctx + 1)) - (t * (t - 1) // 2 if not case["tree"] else 0)
    reach = min(total, w + t + k)
    return reach, t * min(max(1, ctx), w)


def work(case):
    op = case["op"]
    if op == "attn":
        lens, rows = _sizes(case)
        hd, kd = case["heads"] * case["head_dim"], case["kv_heads"] * case["head_dim"]
        b = f = 0
        for length, t in zip(lens, rows):
            union, pairs = _seen(case, length, t)
            b += 8 * union * kd + 8 * t * hd + 4 * (-(-union // case["page"])) + 8 + (12 * t if case["tree"] else 0)
            f += 4 * pairs * hd
        return {"bytes": b, "flops": f}
    if op == "map":
        lens, rows = _sizes(case)
        return {"bytes": sum(8 * t + 8 * (-(-t // case["page"])) + 20 for t in rows), "flops": 0}
    if op == "tree":
        lens, rows = _sizes(case)
        return {"bytes": sum(16 * t + 8 for t in rows), "flops": 0}
    if op == "rope":
        return {"bytes": 8 * case["rows"] * case["heads"] * case["head_dim"] + 4 * case["rows"],
                "flops": 3 * case["rows"] * case["heads"] * case["rotary"]}
    return {"bytes": int(16 * case["rows"] * case["width"] * (1 - case["skipped"])) + 4 * case["rows"], "flops": 0}


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
    if op in ("attn", "map", "tree"):
        lens, rows = _sizes(case)
        perm = torch.randperm(len(lens), generator=cpu).tolist()  # the seed orders the batch
        lens, rows = [lens[i] for i in perm], [rows[i] for i in perm]
        cu = [0]
        for t in rows:
            cu.append(cu[-1] + t)
        s.update(lens=_ints(lens), cu_rows=_ints(cu), rows=cu[-1])
    if op == "tree" or (op == "attn" and case["tree"]):
        s["parents"] = _parents(s, cpu)
    if op == "attn":
        page, kd = case["page"], case["kv_heads"] * case["head_dim"]
        held = [-(-n // page) for n in lens]
        pages = sum(held) + 3
        ids = torch.randperm(pages, generator=cpu, dtype=torch.int64).to(torch.int32)
        table, at = torch.full((len(lens), max(max(held), 1)), -1, dtype=torch.int32), 0
        for b, n in enumerate(held):
            table[b, :n] = ids[at:at + n]
            at += n
        # Keys of trained models have a few channels that are much larger than the rest.
        gain = torch.ones(kd, device="cuda")
        gain[torch.randperm(kd, generator=cpu)[: max(1, kd // 32)].cuda()] = 4.0
        s.update(table=table.cuda(), k_pool=normal(pages * page, kd) * gain, v_pool=normal(pages * page, kd),
                 q=normal(s["rows"], case["heads"] * case["head_dim"]))
        if case["tree"]:
            s.update(k_new=normal(s["rows"], kd) * gain, v_new=normal(s["rows"], kd))
            s["masks"], s["positions"] = _tree_plan(s["parents"], s["cu_rows"], s["lens"])
    elif op == "map":
        page = case["page"]
        held = [min(-(-n // page), case["max_pages"]) for n in lens]
        more = sum(-(-(n + t) // page) + 1 for n, t in zip(lens, rows))
        ids = torch.randperm(sum(held) + more, generator=cpu, dtype=torch.int64).to(torch.int32)
        table, at = torch.full((len(lens), case["max_pages"]), -1, dtype=torch.int32), 0
        for b, n in enumerate(held):
            table[b, :n] = ids[at:at + n]
            at += n
        s.update(table=table.cuda(), free=ids[at:].cuda(), n_free=_ints([len(ids) - at]), accept=None)
        if case["accept"]:
            kept = [sum(1 << j for j in torch.randperm(t, generator=cpu)[: 1 + t // 4].tolist()) for t in rows]
            s["accept"] = torch.from_numpy(np.array(kept, dtype=np.uint64).view(np.int64)).cuda()
    elif op == "rope":
        s.update(x=normal(case["rows"], case["heads"] * case["head_dim"]),
                 positions=torch.randint(0, case["pos_hi"], (case["rows"],), generator=g, device="cuda", dtype=torch.int32))
    elif op == "write":
        total = case["pages"] * case["page"]
        slots = torch.randperm(total, generator=g, device="cuda")[: case["rows"]].to(torch.int32)
        slots[torch.rand(case["rows"], generator=g, device="cuda") < case["skipped"]] = -1
        s.update(slots=slots, k_pool=normal(total, case["width"]), v_pool=normal(total, case["width"]),
                 k_new=normal(case["rows"], case["width"]), v_new=normal(case["rows"], case["width"]))
    return s


def _parents(s, cpu):
    """Random trees as drafting makes them: each node's parent is an earlier node, the first one a root; now and then another root."""
    cu = s["cu_rows"].tolist()
    p = torch.zeros(cu[-1], dtype=torch.int32)
    u = torch.rand(cu[-1], generator=cpu)
    for a, b in zip(cu, cu[1:]):
        j = torch.arange(b - a)
        par = (u[a:b] * j).to(torch.int32)
        par[(u[a:b] > 0.97) | (j == 0)] = -1
        p[a:b] = par
    return p.cuda()


# ------------------------------------------------------------- plain forms
def _place(cu, rows):
    """Request and index in it of each packed row; request -1 behind the last."""
    r = torch.arange(rows, device=cu.device)
    b = torch.searchsorted(cu.long(), r, right=True) - 1
    inside = r < cu[-1]
    b = torch.where(inside, b, torch.zeros_like(b))
    return b, r - cu.long()[b], inside


def _tree_plan(parents, cu, lens):
    b, j, inside = _place(cu, parents.numel())
    p = parents.long()
    up = torch.where((p >= 0) & (p < j), cu.long()[b] + p, torch.full_like(p, -1))
    mask = torch.where(inside & (j < 64), torch.ones_like(j) << j.clamp(max=63), torch.zeros_like(j))
    for _ in range(6):  # each pass doubles the length of the path that a mask covers
        at = up.clamp(min=0)
        mask = torch.where(up >= 0, mask | mask[at], mask)
        up = torch.where(up >= 0, up[at], up)
    depth = ((mask[:, None] >> torch.arange(64, device=mask.device)) & 1).sum(1) - 1
    pos = torch.where(inside & (j < 64), lens.long()[b] + depth, torch.full_like(depth, -1))
    return mask, pos.to(torch.int32)


def _page_map(s):
    case, cu, lens = s["case"], s["cu_rows"].long(), s["lens"].long()
    page, table, dev = case["page"], s["table"], s["lens"].device
    t = cu[1:] - cu[:-1]
    bits = torch.arange(64, device=dev)
    if s["accept"] is not None:
        kept = ((s["accept"][:, None] >> bits) & 1) * (bits < t[:, None])
        add = kept.sum(1)
    else:
        add = t
    most = table.shape[1]
    held = ((lens + page - 1) // page).clamp(max=most)
    want = ((lens + add + page - 1) // page).clamp(max=most)
    first = torch.cumsum(want - held, 0) - (want - held)
    col = torch.arange(most, device=dev)
    new = (col >= held[:, None]) & (col < want[:, None])
    k = first[:, None] + col - held[:, None]
    n_free = s["n_free"].long()
    took = s["free"].long()[(n_free - 1 - k).clamp(0, s["free"].numel() - 1)]
    table.copy_(torch.where(new, torch.where(k < n_free, took, torch.full_like(took, -1)), table.long()).to(torch.int32))
    b, j, inside = _place(s["cu_rows"], s["rows"])
    if s["accept"] is not None:
        before = torch.cumsum(kept, 1) - kept
        in_mask = inside & (j < 64)
        jj = j.clamp(max=63)
        rank, live = before[b, jj], in_mask & (kept[b, jj] > 0)
    else:
        rank, live = j, inside
    pos = lens[b] + rank
    col = pos // page
    pg = table.long()[b, col.clamp(max=most - 1)]
    slot = torch.where(live & (col < most) & (pg >= 0), pg * page + pos % page, torch.full_like(pos, -1))
    pos = torch.where(live, pos, torch.full_like(pos, -1))
    return dict(slots=slot.to(torch.int32), positions=pos.to(torch.int32), new_lens=(lens + add).to(torch.int32),
                n_free=(n_free - (want - held).sum()).to(torch.int32), table=table)


def _rope(s):
    case, x = s["case"], s["x"]
    d, rd = case["head_dim"], case["rotary"]
    j = torch.arange(rd // 2, device=x.device, dtype=torch.float64)
    th = s["positions"].double()[:, None] * torch.pow(torch.tensor(case["base"], dtype=torch.float64, device=x.device), -2.0 * j / rd)
    c, n = th.cos().float()[:, None, :], th.sin().float()[:, None, :]
    h = x.view(x.shape[0], -1, d)
    out = h.clone()
    if case["interleaved"]:
        a, b = h[..., 0:rd:2], h[..., 1:rd:2]
        out[..., 0:rd:2], out[..., 1:rd:2] = a * c - b * n, b * c + a * n
    else:
        a, b = h[..., : rd // 2], h[..., rd // 2:rd]
        out[..., : rd // 2], out[..., rd // 2:rd] = a * c - b * n, b * c + a * n
    return out.view_as(x)


def _write(s):
    live = s["slots"] >= 0
    at = s["slots"][live].long()
    s["k_pool"][at] = s["k_new"][live]
    s["v_pool"][at] = s["v_new"][live]
    return [s["k_pool"], s["v_pool"]]


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
    kk, vv = s["k_pool"][at].view(n, -1, hk, d), s["v_pool"][at].view(n, -1, hk, d)
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
        if op == "attn":
            return _attention(state)
        if op == "map":
            return _page_map(state)
        if op == "tree":
            return list(_tree_plan(state["parents"], state["cu_rows"], state["lens"]))
        return _rope(state) if op == "rope" else _write(state)
    import f32_gqa_attention_gb300 as vtmu
    if op == "attn":
        tree = (state["k_new"], state["v_new"], state["masks"], state["positions"]) if case["tree"] else None
        return vtmu.paged_attention(state["q"], state["k_pool"], state["v_pool"], state["table"], state["lens"],
                                    state["cu_rows"], tree=tree, heads=case["heads"], kvHeads=case["kv_heads"],
                                    headDim=case["head_dim"], pageSize=case["page"], maxRows=case["rows_hi"],
                                    window=case["window"], sinks=case["sinks"], softcap=case["softcap"],
                                    scale=case["scale"] or None)
    if op == "map":
        slots, positions, new_lens, n_free = vtmu.page_map(
            state["lens"], state["cu_rows"], state["table"], state["free"], state["n_free"], rows=state["rows"],
            pageSize=case["page"], accept=state["accept"])
        return dict(slots=slots, positions=positions, new_lens=new_lens, n_free=n_free, table=state["table"])
    if op == "tree":
        return list(vtmu.tree_plan(state["parents"], state["cu_rows"], state["lens"]))
    if op == "rope":
        return vtmu.rope_at(state["x"], state["positions"], headDim=case["head_dim"], base=case["base"],
                            rotaryDim=case["rotary"], interleaved=case["interleaved"])
    vtmu.paged_write(state["k_pool"], state["v_pool"], state["k_new"], state["v_new"], state["slots"])
    return [state["k_pool"], state["v_pool"]]


# ---------------------------------------------------------- 64-bit answers
def exact(case, seed):
    """The definitions in 64 bits, request by request and head by head."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        x, d, rd = s["x"].double(), case["head_dim"], case["rotary"]
        out = x.clone()
        for j in range(rd // 2):
            turn = s["positions"].double() * float(case["base"]) ** (-2.0 * j / rd)
            z = torch.polar(torch.ones_like(turn), turn)
            a, b = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + rd // 2)
            for h in range(case["heads"]):
                w = torch.complex(x[:, h * d + a], x[:, h * d + b]) * z
                out[:, h * d + a], out[:, h * d + b] = w.real, w.imag
        return out
    if op == "write":
        live = (s["slots"] >= 0).nonzero()[:, 0]
        return [s[a].double().index_copy_(0, s["slots"].long()[live], s[b].double()[live])
                for a, b in (("k_pool", "k_new"), ("v_pool", "v_new"))]
    if op != "attn":
        return None  # whole numbers: compared as they are
    hk, d, page = case["kv_heads"], case["head_dim"], case["page"]
    g = case["heads"] // hk
    cu, lens = s["cu_rows"].tolist(), s["lens"].tolist()
    out = torch.zeros(s["rows"], case["heads"] * d, dtype=torch.float64, device="cuda")
    for b, length in enumerate(lens):
        a, e = cu[b], cu[b + 1]
        if a == e:
            continue
        at = torch.arange(length, device="cuda")
        at = s["table"][b].long()[at // page] * page + at % page
        kpos = torch.arange(length, device="cuda")
        k, v = s["k_pool"][at], s["v_pool"][at]
        sink = kpos < case["sinks"]
        if case["tree"]:
            ppos = s["positions"][a:e].long()
            par = s["parents"][a:e].tolist()
            line = torch.zeros(e - a, e - a, dtype=torch.bool)
            for j, up in enumerate(par):
                if 0 <= up < j:
                    line[j] = line[up]
                line[j, j] = True
            allowed = torch.cat([torch.ones(e - a, length, dtype=torch.bool), line], 1).cuda()
            k, v = torch.cat([k, s["k_new"][a:e]]), torch.cat([v, s["v_new"][a:e]])
            kpos, sink = torch.cat([kpos, ppos]), torch.cat([sink, torch.zeros(e - a, dtype=torch.bool, device="cuda")])
        else:
            ppos = torch.arange(length - (e - a), length, device="cuda")
            allowed = kpos[None] <= ppos[:, None]
        if case["window"]:
            allowed = allowed & ((ppos[:, None] - kpos[None] < case["window"]) | sink[None])
        for h in range(case["heads"]):
            c = (h // g) * d
            x = s["q"][a:e, h * d:(h + 1) * d].double() @ k[:, c:c + d].double().T
            x = x * (case["scale"] or d ** -0.5)
            if case["softcap"]:
                x = torch.tanh(x / case["softcap"]) * case["softcap"]
            x = torch.where(allowed, x, torch.full_like(x, -math.inf))
            w = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
            out[a:e, h * d:(h + 1) * d] = torch.nan_to_num(w, nan=0.0) @ v[:, c:c + d].double()
    return out
