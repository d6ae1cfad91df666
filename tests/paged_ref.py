"""Plain 64-bit numpy implementations of the paged-cache operators, written
from their definitions in include/vtmu_attention.h, and makers of small ragged
batches.  Test infrastructure: shares no code with the library."""
import numpy as np


def ancestors(parents):
    """[n, n] bool: row j's own path in a tree given by parents."""
    n = len(parents)
    line = np.zeros((n, n), bool)
    for j, p in enumerate(parents):
        if 0 <= p < j:
            line[j] = line[p]
        line[j, j] = True
    return line


def tree_plan(parents, cu, lens):
    rows = len(parents)
    masks, pos = np.zeros(rows, np.uint64), np.full(rows, -1, np.int32)
    for b in range(len(lens)):
        a, e = int(cu[b]), int(cu[b + 1])
        line = ancestors(parents[a:min(e, a + 64)])
        for j in range(line.shape[0]):
            masks[a + j] = sum(1 << int(i) for i in np.flatnonzero(line[j]))
            pos[a + j] = max(int(lens[b]), 0) + int(line[j].sum()) - 1
    return masks, pos


def page_map(lens, cu, table, free, n_free, rows, page, accept=None):
    table = table.copy()
    most = table.shape[1]
    slots, pos = np.full(rows, -1, np.int32), np.full(rows, -1, np.int32)
    new_lens = np.zeros(len(lens), np.int32)
    left = int(n_free)
    for b in range(len(lens)):
        a, e, at = int(cu[b]), int(cu[b + 1]), max(int(lens[b]), 0)
        held = min(-(-at // page), most)
        for j in range(e - a):
            if accept is not None and not (j < 64 and (int(accept[b]) >> j) & 1):
                continue
            col = at // page
            if col < most:
                if col >= held:
                    table[b, col] = free[left - 1] if left > 0 else -1
                    left -= 1
                    held = col + 1
                if table[b, col] >= 0:
                    slots[a + j] = table[b, col] * page + at % page
            pos[a + j] = at
            at += 1
        new_lens[b] = at
    return slots, pos, new_lens, left, table


def rope_at(x, positions, *, headDim, base=10000.0, rotaryDim=None, interleaved=False):
    out = x.astype(np.float64)
    rd = rotaryDim or headDim
    for t, p in enumerate(positions):
        for h in range(x.shape[1] // headDim):
            for j in range(rd // 2):
                a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rd // 2)
                a, b = h * headDim + a, h * headDim + b
                th = float(p) * base ** (-2.0 * j / rd)
                u, v = float(x[t, a]), float(x[t, b])
                out[t, a], out[t, b] = u * np.cos(th) - v * np.sin(th), v * np.cos(th) + u * np.sin(th)
    return out


def attention(q, k_pool, v_pool, table, lens, cu, *, heads, headDim, kvHeads, pageSize, tree=None, scale=None,
              softcap=None, window=None, sinks=None):
    """Request by request, head by head; keys a row does not see are left out."""
    out = np.zeros(q.shape, np.float64)
    D, G = headDim, heads // kvHeads
    for b in range(len(lens)):
        a, e, n = int(cu[b]), int(cu[b + 1]), int(lens[b])
        s = np.arange(n)
        rows = table[b, s // pageSize].astype(np.int64) * pageSize + s % pageSize if n else np.zeros(0, np.int64)
        kk, vv, kpos = k_pool[rows], v_pool[rows], s
        if tree is not None:
            k_new, v_new, masks, positions = tree
            kk, vv = np.concatenate([kk, k_new[a:e]]), np.concatenate([vv, v_new[a:e]])
            if window:
                kpos = np.concatenate([s, positions[a:e]])
        for t in range(e - a):
            if tree is not None:
                bits = np.array([(int(masks[a + t]) >> j) & 1 for j in range(e - a)], bool)
                see = np.concatenate([np.ones(n, bool), bits])
                p = int(positions[a + t]) if window else 0
            else:
                p = n - (e - a) + t
                see = s <= p
            if window:
                near = kpos > p - window
                near[:n] |= s < (sinks or 0)
                see = see & near
            at = np.flatnonzero(see)
            if not len(at):
                continue
            for h in range(heads):
                c = (h // G) * D
                x = kk[at, c:c + D].astype(np.float64) @ q[a + t, h * D:(h + 1) * D].astype(np.float64)
                x = x * (D ** -0.5 if scale is None else scale)
                if softcap:
                    x = softcap * np.tanh(x / softcap)
                w = np.exp(x - x.max())
                out[a + t, h * D:(h + 1) * D] = w @ vv[at, c:c + D].astype(np.float64) / w.sum()
    return out


def batch(seed, lens, counts, *, heads, kvHeads, headDim, pageSize, tree=False, extra_cols=2, extra_rows=0, waste=float("nan")):
    """A ragged batch with shuffled pages.  Everything that no row may see
    (pool rows of no request, table entries past a request's pages, rows behind
    the last request) holds `waste` or -1."""
    g = np.random.default_rng(seed)
    kd = kvHeads * headDim
    held = [-(-n // pageSize) for n in lens]
    pages = sum(held) + 2
    ids = g.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(held + [0]) + extra_cols), -1, np.int32)
    k, v = (np.full((pages * pageSize, kd), waste, np.float32) for _ in range(2))
    at = 0
    for b, n in enumerate(lens):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
        s = np.arange(n)
        rows = table[b, s // pageSize].astype(np.int64) * pageSize + s % pageSize
        k[rows] = g.standard_normal((n, kd), dtype=np.float32)
        v[rows] = g.standard_normal((n, kd), dtype=np.float32)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(cu[-1]) + extra_rows
    q = g.standard_normal((rows, heads * headDim), dtype=np.float32)
    q[int(cu[-1]):] = waste
    d = dict(q=q, k_pool=k, v_pool=v, table=table, lens=np.array(lens, np.int32), cu=cu, tree=None)
    if tree:
        parents = np.full(rows, -1, np.int32)
        for a, e in zip(cu, cu[1:]):
            for j in range(1, e - a):
                parents[a + j] = g.integers(-1 if g.random() < 0.1 else 0, j)
        masks, pos = tree_plan(parents, cu, d["lens"])
        kn, vn = (g.standard_normal((rows, kd), dtype=np.float32) for _ in range(2))
        kn[int(cu[-1]):] = vn[int(cu[-1]):] = waste
        d.update(parents=parents, tree=(kn, vn, masks, pos))
    return d
