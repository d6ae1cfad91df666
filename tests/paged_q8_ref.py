"""Plain numpy implementations, in 64 bits, of the 8-bit cache's formats and of
norm_rope, written from include/vtmu_attention.h.  Test infrastructure: shares no
code with the library."""
import numpy as np

import paged_ref as ref

INT8, E4M3 = 1, 2


def e4m3_values():
    """The number that each code stands for (OCP e4m3: bias 7, no infinities, 0x7f NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 7.0), m / 8.0 * 2.0 ** -6)
    v[(c & 127) == 127] = np.nan
    return np.where(c & 128, -v, v)


def _e4m3_code(y):
    """Nearest code, ties to the even one; |y| <= 448."""
    v = e4m3_values()[:127]  # ascending
    a = np.abs(y)
    hi = np.clip(np.searchsorted(v, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = v[hi] - a, a - v[lo]
    code = np.where(up < down, hi, np.where(up > down, lo, np.where(hi % 2 == 0, hi, lo)))
    return (code | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def quantise(x, kv_heads, form):
    """(codes uint8 [rows, width], scales f32 [rows, kv_heads]) of rows."""
    h = x.astype(np.float64).reshape(x.shape[0], kv_heads, -1)
    with np.errstate(all="ignore"):
        top = np.abs(h).max(-1) if h.size else np.zeros(h.shape[:2])
        if form == INT8:
            scale = np.maximum((top / 127.0).astype(np.float32), np.float32(2.0 ** -126))
            code = np.rint(h / scale[..., None].astype(np.float64))
            code = np.where(np.isfinite(code), code, 0).astype(np.int8).view(np.uint8)
        else:
            part, e = np.frexp(np.where(np.isfinite(top), top, 0))
            k = np.where(top > 0, np.where(part <= 0.875, e - 9, e - 8), -126)
            scale = (2.0 ** np.maximum(k, -126)).astype(np.float32)
            y = h / scale[..., None].astype(np.float64)
            code = _e4m3_code(np.where(np.isfinite(y), y, 0))
    bad = ~np.isfinite(top)
    scale = np.where(bad, np.float32(np.nan), scale).astype(np.float32)
    return np.where(bad[..., None], 0, code).astype(np.uint8).reshape(x.shape), scale


def values(codes, scale, form):
    """f64 rows of codes."""
    v = codes.view(np.int8).astype(np.float64) if form == INT8 else e4m3_values()[codes]
    n, hk = scale.shape
    return (v.reshape(n, hk, -1) * scale.astype(np.float64)[..., None]).reshape(codes.shape)


def batch(seed, lens, counts, *, form, gain=None, **kw):
    """paged_ref.batch with pools of codes (kc, ks, vc, vs), and k_pool, v_pool the numbers
    they stand for; what no row may see is NaN (scale NaN)."""
    d = ref.batch(seed, lens, counts, **kw)
    if gain is not None:
        d["k_pool"], d["v_pool"] = gain(d["k_pool"], d["v_pool"])
    for a in "kv":
        d[a + "c"], d[a + "s"] = quantise(d[a + "_pool"], kw["kvHeads"], form)
        d[a + "_pool"] = values(d[a + "c"], d[a + "s"], form)
    d["form"] = form
    return d


def axis_of(half, sections, dealt):
    if sections is None:
        return [0] * half
    if not dealt:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    n = len(sections)
    return [j % n if j < n * sections[j % n] else 0 for j in range(half)]


def norm_rope(x, positions, *, headDim, weight=None, norm=True, eps=1e-6, weightOffset=0.0, sections=None, dealt=False,
              base=10000.0, rotaryDim=None, interleaved=False):
    """(result, the size |a| + |b| of the pair behind each element)."""
    T, rd = x.shape[0], rotaryDim or headDim
    pos = np.asarray(positions).reshape(-1, T).astype(np.float64)
    h = x.astype(np.float64).reshape(T, -1, headDim)
    if norm:
        h = h / np.sqrt((h * h).mean(-1, keepdims=True) + float(np.float32(eps)))
        if weight is not None:
            h = h * (weight.astype(np.float64) + weightOffset)
    out, size = h.copy(), np.abs(h)
    axis = axis_of(rd // 2, sections, dealt)
    for j in range(rd // 2):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rd // 2)
        th = (pos[axis[j]] * base ** (-2.0 * j / rd))[:, None]
        u, v = h[..., a], h[..., b]
        out[..., a], out[..., b] = u * np.cos(th) - v * np.sin(th), v * np.cos(th) + u * np.sin(th)
        size[..., a] = size[..., b] = np.abs(u) + np.abs(v)
    return out.reshape(x.shape), size.reshape(x.shape)
