"""The 8-bit paged cache and norm_rope on the GPU against plain 64-bit
implementations.

Tolerances.  Codes and scales are exact.  A row read back is one product: off by at
most half a step, 2^-24 of itself.  norm_rope: a head's squares are summed by at most
D / 32 + 5 additions in a row (8 + 5 up to D = 256), whose roundings the root halves;
rsqrt is off by at most 2 ulp (2^-22), the mean and eps by 2^-24, the weight, its
offset and the two products by 3 2^-24: (13 / 2 + 4 + 1 + 3) 2^-24 < 2^-20 of the
element.  The rotation adds 2^-21 (sine and cosine) and 2^-22 (two products, a sum) of
|a| + |b|: 2^-20 + 2^-21 + 2^-22 in all.  Attention: as of the f32 paged cache (1e-4,
and 2^-17 in the 2-norm); the codes add nothing, they are exact operands, and the scales
one rounding each."""
import numpy as np
import pytest

import paged_q8_ref as q8
import paged_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import f32_gqa_attention_gb300 as vtmu  # noqa: E402
from test_gpu_paged import check, dev  # noqa: E402

FORMS = [q8.INT8, q8.E4M3]
DTYPE = {q8.INT8: torch.int8, q8.E4M3: torch.float8_e4m3fn}
CUDA, TENSOR = vtmu.VTMU_PAGED_CUDA_CORES, vtmu.VTMU_PAGED_TENSOR_CORES


def codes(a, form):
    return dev(a).view(DTYPE[form])


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


# --------------------------------------------------------------------- write
def edge_rows(g, n, width):
    """Rows of every size: subnormal, tiny, ordinary, huge, zero; exact ties; not finite."""
    x = g.standard_normal((n, width), dtype=np.float32)
    x *= (2.0 ** g.integers(-4, 4, (n, 1))).astype(np.float32)
    special = [x[0] * 1e-40, x[0] * 1e-30, x[0] * 1e37, x[0] * 0, np.round(x[0] * 20) * 0.5]
    for i, row in enumerate(special):
        x[i % n] = row
    if n > 6:
        x[5, 0], x[6, -1] = np.inf, np.nan
    if n > 8:
        x[7] = 0.5 * np.arange(width) % 128 - 63.5  # ties of an int8 scale of 1
        x[7, :2] = 127.0, -127.0
        x[8] = np.float32(448.0) * (1 - np.arange(width) % 97 / 64.0)
    return x


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows,hk,d", [(1, 1, 1), (3, 2, 8), (9, 3, 64), (40, 8, 128), (17, 2, 96), (12, 1, 256), (11, 5, 7),
                                       (300, 3, 80), (20, 2, 132), (10, 1, 250)])
@pytest.mark.parametrize("shift", [0, 1])
def test_write(form, rows, hk, d, shift):
    """Codes and scales bit by bit; rows without a slot and slots outside the pool change nothing.
    `shift`: new rows off the 16-byte grid, codes at an odd address."""
    g = np.random.default_rng(rows * d)
    total = rows + 9
    x = [edge_rows(g, rows, hk * d) for _ in range(2)]
    slots = g.permutation(total)[:rows].astype(np.int32)
    if rows > 3:
        slots[1], slots[2] = -1, total
    pools = [g.integers(0, 256, (total, hk * d), dtype=np.uint8) for _ in range(2)]
    scales = [g.standard_normal((total, hk), dtype=np.float32) for _ in range(2)]

    def moved(a):  # the same tensor, one element off the allocation's start
        t = torch.empty(a.size + shift, dtype=torch.from_numpy(a[:0]).dtype, device="cuda")[shift:].view(a.shape)
        return t.copy_(torch.from_numpy(a))

    kp, vp = (moved(p).view(DTYPE[form]) for p in pools)
    ks, vs = (moved(s) for s in scales)
    vtmu.paged_write_q8(kp, vp, ks, vs, moved(x[0]), moved(x[1]), dev(slots))
    for got, scale, new, pool, old in ((kp, ks, x[0], pools[0], scales[0]), (vp, vs, x[1], pools[1], scales[1])):
        c, s = q8.quantise(new, hk, form)
        live = (slots >= 0) & (slots < total)
        pool, old = pool.copy(), old.copy()
        pool[slots[live]], old[slots[live]] = c[live], s[live]
        assert np.array_equal(scale.cpu().numpy(), old, equal_nan=True)
        assert np.array_equal(raw(got), pool)


@pytest.mark.parametrize("form", FORMS)
def test_write_of_quotients_next_to_a_tie(form):
    """int8: x / scale within an f32 rounding of a half; the exact quotient decides."""
    g = np.random.default_rng(8)
    d, rows = 128, 2000
    top = g.uniform(1, 2, (rows, 1)).astype(np.float32)
    scale = (top.astype(np.float64) / 127).astype(np.float32)
    x = ((g.integers(-126, 126, (rows, d)) + 0.5) * scale.astype(np.float64)).astype(np.float32)  # to the nearest f32
    x = np.where(g.random((rows, d)) < 0.5, x, np.nextafter(x, np.float32(0)))
    x = x.astype(np.float32)
    x[:, 0] = top[:, 0]
    pool, sc = torch.zeros(rows, d, dtype=DTYPE[form], device="cuda"), torch.zeros(rows, 1, device="cuda")
    slots = torch.arange(rows, dtype=torch.int32, device="cuda")
    vtmu.paged_write_q8(pool, torch.zeros_like(pool), sc, torch.zeros_like(sc), dev(x), dev(x), slots)
    c, s = q8.quantise(x, 1, form)
    assert np.array_equal(sc.cpu().numpy(), s) and np.array_equal(raw(pool), c)


# ---------------------------------------------------------------------- read
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows,hk,d", [(1, 1, 1), (5, 2, 64), (70, 8, 128), (13, 5, 96), (6, 3, 7), (8, 1, 250), (1000, 2, 256)])
@pytest.mark.parametrize("shift", [0, 1])
def test_read(form, rows, hk, d, shift):
    g = np.random.default_rng(rows + d)
    total = 50
    c = [g.integers(0, 256, (total, hk * d), dtype=np.uint8) for _ in range(2)]
    s = [np.abs(g.standard_normal((total, hk), dtype=np.float32)) for _ in range(2)]
    s[0][3] = np.nan
    slots = g.integers(-3, total + 3, rows).astype(np.int32)  # some twice, some outside

    def moved(a):
        t = torch.empty(a.size + shift, dtype=torch.from_numpy(a[:0]).dtype, device="cuda")[shift:].view(a.shape)
        return t.copy_(torch.from_numpy(a))

    out = tuple(moved(np.full((rows, hk * d), np.nan, np.float32)) for _ in range(2))
    got = vtmu.paged_read_q8(moved(c[0]).view(DTYPE[form]), moved(c[1]).view(DTYPE[form]), moved(s[0]), moved(s[1]), dev(slots),
                             out=out)
    assert got[0] is out[0] and got[1] is out[1]
    for y, cc, ss in zip(got, c, s):
        live = (slots >= 0) & (slots < total)
        want = np.zeros((rows, hk * d))
        want[live] = q8.values(cc, ss, form)[slots[live]]
        assert np.array_equal(np.isnan(y.cpu().numpy()), np.isnan(want))
        ok = ~np.isnan(want)
        assert np.all(np.abs(y.cpu().numpy().astype(np.float64) - want)[ok] <= 2.0 ** -24 * np.abs(want)[ok])


# ----------------------------------------------------------------- norm_rope
ROPE = [  # T, heads, kv, D, rope and norm arguments
    (1, 1, 1, 2, dict()), (3, 5, 1, 128, dict(base=500000.0)), (7, 4, 2, 96, dict(rotaryDim=48)),
    (5, 6, 3, 64, dict(interleaved=True)), (4, 3, 1, 10, dict(rotaryDim=6)), (9, 2, 1, 256, dict(interleaved=True)),
    (300, 32, 8, 128, dict(sections=[24, 20, 20], dealt=True, base=1e6)), (40, 8, 2, 128, dict(sections=[16, 24, 24])),
    (11, 4, 4, 64, dict(sections=[8, 8, 8, 8], interleaved=True)), (6, 7, 7, 64, dict(rotaryDim=32, sections=[0, 16])),
    (13, 2, 1, 80, dict(sections=[30, 10])), (5, 3, 0, 128, dict()), (8, 2, 2, 7, dict(rotaryDim=4)),
    (6, 9, 3, 32, dict(weightOffset=1.0)), (2000, 4, 1, 16, dict()), (4, 2, 1, 24, dict(rotaryDim=8)),
    (3, 2, 1, 128, dict(rotaryDim=0, eps=0.0)),
]


@pytest.mark.parametrize("case", range(len(ROPE)))
@pytest.mark.parametrize("norm,weights", [(True, True), (True, False), (False, False)])
@pytest.mark.parametrize("place", ["new", "in place", "shifted"])
def test_norm_rope(case, norm, weights, place):
    T, H, hk, D, kw = ROPE[case]
    g = np.random.default_rng(case)
    q, k = (g.standard_normal((T, n * D), dtype=np.float32) * 3 for n in (H, hk))
    axes = len(kw.get("sections", [0]))
    pos = g.integers(0, 100000, (axes, T)).astype(np.int32)
    pos[:, 0] = 0
    if T > 2:
        pos[-1, 2] = -1  # left as it was
    w = [(1 + 0.3 * g.standard_normal(D, dtype=np.float32)).astype(np.float32) if weights else None for _ in range(2)]
    shift = 1 if place == "shifted" else 0

    def moved(a):
        t = torch.empty(a.size + shift, device="cuda")[shift:].view(a.shape)
        return t.copy_(torch.from_numpy(a))

    tq, tk = moved(q), moved(k) if hk else None
    out = (tq, tk) if place == "in place" else (torch.full_like(tq, 7.0), torch.full_like(tk, 7.0) if hk else None)
    kk = dict(kw, norm=norm)
    got = vtmu.norm_rope(tq, tk, dev(pos if axes > 1 else pos[0]), headDim=D, qWeight=None if w[0] is None else moved(w[0]),
                         kWeight=None if w[1] is None or not hk else moved(w[1]), out=out, **kk)
    assert got[0] is out[0] and got[1] is out[1]
    live = (pos >= 0).all(0)
    if kk.get("rotaryDim") == 0:  # the default: every channel turns
        kk.pop("rotaryDim")
    for y, x, ww in ((got[0], q, w[0]), (got[1], k, w[1])):
        if y is None:
            continue
        want, size = q8.norm_rope(x, pos, headDim=D, weight=ww, **kk)
        y = y.cpu().numpy()
        assert np.array_equal(y[~live], x[~live] if place == "in place" else np.full_like(x[~live], 7.0))
        err = np.abs(y.astype(np.float64) - want)[live] - (2.0 ** -20 + 2.0 ** -21 + 2.0 ** -22) * size[live]
        assert err.size == 0 or err.max() <= 0, err.max()


@pytest.mark.parametrize("D", [128, 100])
@pytest.mark.parametrize("size,eps", [(1e25, 1e-6), (3e38, 0.0), (1e-30, 0.0), (1e-30, 1e-6), (1e-38, 0.0), (0.0, 1e-6)])
def test_norm_of_far_sizes(D, size, eps):
    """Elements whose squares leave f32's range."""
    g = np.random.default_rng(1)
    x = (g.uniform(-1, 1, (5, 3 * D)) * size).astype(np.float32)
    x[3] = g.standard_normal(3 * D)  # an ordinary row beside them
    pos = np.arange(5, dtype=np.int32)
    y, _ = vtmu.norm_rope(dev(x), None, dev(pos), headDim=D, eps=eps)
    want, big = q8.norm_rope(x, pos, headDim=D, eps=eps)
    err = np.abs(y.cpu().numpy() - want)
    # Elements far below 2^-126 have fewer bits of their own: x times the factor is exact from there.
    assert np.all(err <= (2.0 ** -20 + 2.0 ** -21 + 2.0 ** -22) * big + 1e-37), (err - 2.0 ** -19 * big).max()


def test_norm_of_rows_that_are_not_finite():
    x = np.ones((4, 2 * 64), np.float32)
    x[1, 3], x[2, 70], x[3, :64] = np.inf, np.nan, 0.0
    y, _ = vtmu.norm_rope(dev(x), None, dev(np.zeros(4, np.int32)), headDim=64, eps=0.0)
    y = y.cpu().numpy().reshape(4, 2, 64)
    assert np.all(np.isfinite(y[0])) and np.all(np.isfinite(y[1, 1])) and np.all(np.isfinite(y[2, 0]))
    assert np.isnan(y[1, 0, 3]) and np.isnan(y[2, 1]).all() and np.isnan(y[3, 0]).all() and np.all(np.isfinite(y[3, 1]))


def test_norm_rope_with_no_norm_is_rope_at():
    """Both turn by the same angles; sine and cosine are off by at most 2^-21 in rope_at, and products
    and sums by 2^-22 in each, so two results differ by less than 2^-20 of |a| + |b| <= 2 max |x|."""
    g = np.random.default_rng(3)
    x, pos = dev(g.standard_normal((50, 6 * 128), dtype=np.float32)), dev(g.integers(0, 500000, 50).astype(np.int32))
    for kw in (dict(), dict(interleaved=True), dict(rotaryDim=64), dict(scaling={"type": "linear", "factor": 3.0}),
               dict(invFreq=[1.0 / (j + 1) for j in range(64)]), dict(invFreq=[-3.0 * j for j in range(64)], attentionFactor=1.2)):
        y, _ = vtmu.norm_rope(x, None, pos, headDim=128, norm=False, **kw)
        want = vtmu.rope_at(x, pos, headDim=128, **kw)
        assert float((y - want).abs().max()) <= 1.2 * 2.0 ** -20 * 2 * float(x.abs().max())


@pytest.mark.parametrize("D,kw", [(128, dict()), (128, dict(sections=[24, 20, 20], dealt=True)), (10, dict())])
def test_norm_rope_at_far_positions(D, kw):
    """Positions up to 2^31 - 1.  The plain angle is a double that rounds at 2^31 2^-53, the kernel's a
    fixed-point number off by 2^31 2^-65 turns: 2^-21 more."""
    g = np.random.default_rng(2)
    axes = len(kw.get("sections", [0]))
    pos = (2 ** 31 - 1 - g.integers(0, 50, (axes, 6))).astype(np.int32)
    x = g.standard_normal((6, 4 * D), dtype=np.float32)
    y, _ = vtmu.norm_rope(dev(x), None, dev(pos if axes > 1 else pos[0]), headDim=D, **kw)
    want, size = q8.norm_rope(x, pos, headDim=D, **kw)
    assert np.all(np.abs(y.cpu().numpy() - want) <= (2.0 ** -20 + 2.0 ** -21 + 2.0 ** -22 + 2.0 ** -21) * size)


def test_norm_rope_wrong_arguments():
    x, p = torch.zeros(4, 256, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    w = torch.ones(128, device="cuda")
    for kw in (dict(headDim=96), dict(headDim=128, qWeight=w[:64]), dict(headDim=128, sections=[32, 32]),
               dict(headDim=128, out=(x, x)), dict(headDim=128, qWeight=w.double())):
        with pytest.raises(ValueError):
            vtmu.norm_rope(x, None, p, **kw)
    with pytest.raises(vtmu.VtmuError):
        vtmu.norm_rope(x, None, p, headDim=128, norm=False, qWeight=w)


# ----------------------------------------------------------------- attention
def attend(d, *, kernel, out=None, maxRows=None, **kw):
    tree = None if d["tree"] is None else tuple(dev(x) for x in d["tree"])
    counts = np.diff(d["cu"])
    o = vtmu.paged_attention_q8(dev(d["q"]), codes(d["kc"], d["form"]), codes(d["vc"], d["form"]), dev(d["ks"]), dev(d["vs"]),
                                dev(d["table"]), dev(d["lens"]), dev(d["cu"]), tree=tree, kernel=kernel, out=out,
                                maxRows=int(counts.max()) if maxRows is None else maxRows, **kw)
    torch.cuda.synchronize()
    assert vtmu.vtmu_device_error() == 0
    return o.cpu().numpy()


def expect(d, **kw):
    return ref.attention(d["q"], d["k_pool"], d["v_pool"], d["table"], d["lens"], d["cu"], tree=d["tree"], **kw)


SHAPES = [  # lens, counts, heads, kvHeads, D, page, tree, attention arguments
    ([1], [1], 1, 1, 64, 16, False, {}),
    ([211], [1], 16, 4, 128, 16, False, {}),
    ([17, 300, 64, 65], [1, 1, 1, 1], 8, 2, 128, 16, False, {}),
    ([40, 0, 129, 7], [5, 0, 1, 7], 12, 4, 64, 32, False, dict(scale=0.2)),
    ([3, 260], [5, 2], 4, 4, 64, 64, False, {}),                    # rows before the request's first position
    ([100, 1000], [33, 70], 6, 2, 64, 16, False, dict(window=50, sinks=3)),
    ([90, 700, 33], [7, 21, 1], 12, 4, 64, 32, True, dict(window=128, sinks=4, softcap=30.0, scale=0.11)),
    ([0, 500], [64, 64], 8, 2, 128, 16, True, {}),
    ([1500, 31], [64, 3], 7, 1, 128, 128, True, dict(softcap=5.0)),
    ([700], [260], 5, 1, 128, 16, False, {}),
    ([129], [3], 8, 8, 128, 8, False, dict(window=1)),
    ([77, 500], [2, 3], 3, 3, 96, 16, False, {}),
    ([77, 50], [2, 3], 6, 2, 40, 5, True, dict(window=20)),
    ([30], [2], 2, 1, 7, 3, False, {}),
    ([600, 20], [9, 4], 16, 1, 64, 24, False, {}),                  # pages that end inside a tile
    ([64] * 40, [1] * 40, 4, 2, 64, 16, False, {}),
    ([33], [4], 2, 2, 256, 16, False, {}),
]


def kernels_of(D):
    return [CUDA, TENSOR] if D in (64, 128) else [CUDA, vtmu.VTMU_PAGED_AUTO]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_attention(case, form):
    lens, counts, H, hk, D, page, tree, kw = SHAPES[case]
    size = dict(heads=H, kvHeads=hk, headDim=D, pageSize=page)
    d = q8.batch(case, lens, counts, form=form, tree=tree, extra_rows=3, **size)
    want = expect(d, **size, **kw)
    live = int(d["cu"][-1])
    for kernel in kernels_of(D):
        out = torch.full(d["q"].shape, 5.0, device="cuda")
        got = attend(d, kernel=kernel, out=out, **size, **kw)
        check(got, want, live)
        assert np.all(got[live:] == 5.0)  # rows of no request


def test_heads_of_far_sizes():
    """K and V heads whose sizes differ by 2^80, rows of a cache that do by 2^30; outliers in K."""
    size = dict(heads=8, kvHeads=4, headDim=64, pageSize=16)

    def gain(k, v):
        g = np.random.default_rng(9)
        heads = np.repeat(2.0 ** np.array([-40.0, 0, 3, 40]), 64).astype(np.float32)
        k = k * heads
        k[:, ::32] *= 8
        return k, v * heads[::-1] * (2.0 ** g.integers(-15, 15, (v.shape[0], 1))).astype(np.float32)

    for form in FORMS:
        d = q8.batch(5, [300, 70], [3, 2], form=form, gain=gain, **size)
        d["q"] *= np.repeat(2.0 ** np.array([40.0, 40, 0, 0, -3, -3, -40, -40]), 64).astype(np.float32)
        want = expect(d, **size)
        for kernel in kernels_of(64):
            got = attend(d, kernel=kernel, **size).astype(np.float64)
            for h in range(8):  # by heads, whose outputs differ in size
                c = slice(64 * h, 64 * h + 64)
                for t in range(5):
                    n = np.linalg.norm(want[t, c])
                    assert np.linalg.norm(got[t, c] - want[t, c]) <= 2.0 ** -15 * n, (form, kernel, h, t)


def test_keys_and_values_that_are_not_finite():
    """Unseen ones change nothing; a seen key makes the row's head NaN, a seen value the head's columns."""
    size = dict(heads=4, kvHeads=2, headDim=64, pageSize=16)
    for form in FORMS:
        d = q8.batch(6, [100], [6], form=form, **size)
        rows = [d["table"][0, s // 16] * 16 + s % 16 for s in range(100)]
        want = expect(d, **size)
        d["ks"][rows[97], 0] = np.nan   # seen by rows 3, 4, 5 (positions 97 ..)
        d["vs"][rows[98], 1] = np.nan   # by rows 4, 5
        for kernel in kernels_of(64):
            got = attend(d, kernel=kernel, **size)
            nan = np.zeros_like(want, bool)
            nan[3:, :128], nan[4:, 128:] = True, True
            assert np.array_equal(np.isnan(got), nan)
            assert np.abs(got - want)[~nan].max() <= 1e-4


def test_bad_pages_and_lengths():
    """Page ids outside the pool stand for zeros; lengths past the table are clamped."""
    size = dict(heads=4, kvHeads=2, headDim=64, pageSize=16)
    for form in FORMS:
        d = q8.batch(7, [100, 60], [2, 1], form=form, extra_cols=0, **size)
        t = d["table"].copy()
        t[0, 2], t[1, 0] = 10 ** 6, -5
        d["lens"] = np.array([112, 10 ** 9], np.int32)
        cols = t.shape[1]
        kf, vf = np.concatenate([d["k_pool"], np.zeros((16, 128))]), np.concatenate([d["v_pool"], np.zeros((16, 128))])
        zero = len(d["k_pool"]) // 16
        full = np.where((t < 0) | (t >= zero), zero, t)
        # rows of the pool that no request owns hold NaN scales: name them zeros for this test
        kf, vf = np.nan_to_num(kf), np.nan_to_num(vf)
        d["ks"], d["vs"] = np.nan_to_num(d["ks"]), np.nan_to_num(d["vs"])
        want = ref.attention(d["q"], kf, vf, full, np.array([112, cols * 16]), d["cu"], **size)
        d["table"] = t
        for kernel in kernels_of(64):
            check(attend(d, kernel=kernel, **size), want)


# Calls of more than 16 rows x heads of a group take kernels of their own: each of the
# following comes with few rows and with many.
def size_of(H, hk, D, page):
    return dict(heads=H, kvHeads=hk, headDim=D, pageSize=page)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows", [3, 20])
@pytest.mark.parametrize("Hk", [1, 3])
@pytest.mark.parametrize("lens", [[4 * 64], [3 * 64 + 1, 1], [64 * 151], [64 * 152, 64], [64 * 304 + 5], [64 * 609]])
def test_units_cut_at_every_kind_of_boundary(lens, Hk, rows, form):
    size = size_of(Hk, Hk, 64, 16)
    d = q8.batch(31, lens, [rows] * len(lens), form=form, **size)
    check(attend(d, kernel=TENSOR, **size), expect(d, **size))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hk", list(range(1, 10)) + [17])
def test_numbers_of_heads(Hk, D):
    size = size_of(2 * Hk, Hk, D, 16)
    for counts, tree in (([4, 1, 7], False), ([3, 8, 2], True), ([30, 9, 1], True)):
        d = q8.batch(Hk, [300, 33, 1000], counts, form=FORMS[Hk % 2], tree=tree, **size)
        check(attend(d, kernel=TENSOR, **size), expect(d, **size))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [1, 2, 5, 7, 12, 24, 48, 256, 1000])
def test_page_sizes(page, D, form):
    size = size_of(4, 2, D, page)
    for counts, tree in (([2, 5], False), ([40, 33], False), ([30, 12], True)):
        d = q8.batch(page, [77, 501], counts, form=form, tree=tree, **size)
        check(attend(d, kernel=TENSOR, **size), expect(d, **size))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("counts", [[5, 6], [40, 61]])
@pytest.mark.parametrize("kw", [dict(window=1), dict(window=33, sinks=70), dict(window=700, softcap=3.0),
                                dict(window=64, sinks=1, scale=1.0), dict(softcap=50.0)])
def test_windows_and_caps(kw, counts, tree, form):
    """Rows before a request's first position and rows whose window leaves nothing are zeros."""
    size = size_of(6, 2, 128, 16)
    d = q8.batch(17, [3, 640], counts, form=form, tree=tree, **size)
    want = expect(d, **size, **kw)
    for kernel in (CUDA, TENSOR):
        got = attend(d, kernel=kernel, **size, **kw)
        check(got, want)
        assert np.all(got[np.abs(want).max(1) == 0] == 0)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("counts", [[4], [30]])
@pytest.mark.parametrize("bad", [np.nan, np.inf, 3e38])
def test_what_a_row_does_not_see_does_not_reach_it(bad, counts, form):
    """Scales of any kind, and any codes, at keys that a window, causality or the end hides."""
    size = size_of(4, 2, 64, 16)
    n = counts[0]
    d = q8.batch(41, [400], counts, form=form, **size)
    at = d["table"][0, np.arange(400) // 16].astype(np.int64) * 16 + np.arange(400) % 16
    want = expect(d, **size, window=100)
    last = 400 - n  # the first row's position
    hidden = np.arange(400) < last - 99  # from every row; the newest key, from all but the last row
    d["ks"][at[hidden]], d["vs"][at[hidden]] = bad, bad
    d["ks"][at[399]], d["vs"][at[399]] = bad, bad
    unowned = np.setdiff1d(np.arange(len(d["ks"])), at)
    d["ks"][unowned], d["vs"][unowned] = bad, bad
    d["kc"][unowned], d["vc"][unowned] = 0x7f, 0xff  # NaN as e4m3
    for kernel in (CUDA, TENSOR):
        got = attend(d, kernel=kernel, **size, window=100)
        check(got[:n - 1], want[:n - 1])  # the last row alone sees key 399
        if np.isnan(bad):
            assert np.all(np.isnan(got[n - 1]))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("counts", [[3, 2], [20, 18]])
@pytest.mark.parametrize("which", ["spread", "tiny values", "subnormal values", "huge values", "huge keys", "zero heads"])
def test_rows_of_any_size(which, counts, form):
    """By heads, whose outputs differ in size: 2^-15 in the 2-norm, as of test_heads_of_far_sizes, and
    for values below 2^-126 the last place of theirs."""
    size = size_of(8, 4, 64, 16)
    mul = np.ones(8)

    def gain(k, v):
        g = np.random.default_rng(9)
        heads = 2.0 ** np.array([-40.0, 0, 3, 40])
        if which == "spread":
            k, v = k * np.repeat(heads, 64), v * np.repeat(heads[::-1], 64) * 2.0 ** g.integers(-15, 15, (v.shape[0], 1))
            k[:, ::32] *= 8
            mul[:] = np.repeat(1 / heads, 2) * [1, 1, 1, 1, 1, 1, 1, 1]
        elif which == "tiny values":
            v = v * 2.0 ** -112 * np.repeat([1.0, 2.0 ** -3, 2.0 ** 4, 2.0 ** 10], 64)
        elif which == "subnormal values":
            v = v * 2.0 ** -121
        elif which == "huge values":
            v = v * 2.0 ** 121
        elif which == "huge keys":
            k, mul[:] = k * 2.0 ** 100, 2.0 ** -100
        else:
            v = v.copy()
            v[:, 64:128] = 0
            v[::3, 128:192] = 0
        return k.astype(np.float32), v.astype(np.float32)

    d = q8.batch(5, [300, 70], counts, form=form, gain=gain, **size)
    d["q"] = (d["q"] * np.repeat(mul, 64)).astype(np.float32)
    want = expect(d, **size)
    for kernel in (CUDA, TENSOR):
        got = attend(d, kernel=kernel, **size).astype(np.float64)
        for h in range(8):
            c = slice(64 * h, 64 * h + 64)
            for t in range(sum(counts)):
                n = np.linalg.norm(want[t, c])
                e = np.linalg.norm(got[t, c] - want[t, c])
                assert e <= 2.0 ** -15 * n + 64 * 2.0 ** -149, (kernel, h, t, e, n)


@pytest.mark.parametrize("counts", [[6], [40]])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_drafted_rows_that_are_not_finite(bad, counts):
    size = size_of(4, 2, 64, 16)
    for form in FORMS:
        d = q8.batch(16, [100], counts, form=form, tree=True, **size)
        kn, vn, masks, pos = d["tree"]
        want = expect(d, **size)
        sees = [np.array([(int(m) >> j) & 1 for m in masks], bool) for j in (2, 3)]
        kn[2, 5], vn[3, 64 + 7] = bad, bad  # a key of KV head 0, a value of head 1
        got = attend(d, kernel=TENSOR, **size)
        assert np.all(np.isnan(got[sees[0]][:, :128])) and np.all(np.isnan(got[sees[1]][:, 128:]))
        good = np.ones(got.shape, bool)
        good[np.ix_(sees[0], range(128))] = False
        good[np.ix_(sees[1], range(128, 256))] = False
        assert np.all(np.isfinite(got[good])) and np.abs(got - want)[good].max() <= 1e-4


@pytest.mark.parametrize("counts", [[6], [40]])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("tree", [False, True])
def test_queries_that_are_not_finite(bad, counts, tree):
    size = size_of(4, 2, 128, 16)
    for form in FORMS:
        d = q8.batch(16, [100], counts, form=form, tree=tree, **size)
        want = expect(d, **size)
        d["q"][3, 130] = bad  # head 1
        got = attend(d, kernel=TENSOR, **size)
        assert np.all(np.isnan(got[3, 128:256]))
        got[3, 128:256] = want[3, 128:256]
        check(got, want)


@pytest.mark.parametrize("counts,tree", [([2, 1], False), ([40, 9], False), ([3, 4], True), ([40, 9], True)])
def test_bad_pages(counts, tree):
    """Page ids outside the pool stand for zeros, as do all of them where the pool has none."""
    size = size_of(4, 2, 128, 16)
    for form in FORMS:
        d = q8.batch(7, [100, 60], counts, form=form, tree=tree, extra_cols=0, **size)
        t = d["table"].copy()
        t[0, 2], t[1, 0], t[0, 4] = 10 ** 6, -5, 2 ** 31 - 1
        zero = len(d["k_pool"]) // 16
        kf, vf = (np.concatenate([np.nan_to_num(d[x]), np.zeros((16, 256))]) for x in ("k_pool", "v_pool"))
        want = ref.attention(d["q"], kf, vf, np.where((t < 0) | (t >= zero), zero, t), d["lens"], d["cu"], tree=d["tree"], **size)
        d["table"] = t
        for kernel in (CUDA, TENSOR):
            check(attend(d, kernel=kernel, **size), want)
        d["kc"], d["vc"], d["ks"], d["vs"] = (d[x][:0] for x in ("kc", "vc", "ks", "vs"))
        want = ref.attention(d["q"], 0 * kf, 0 * vf, np.minimum(np.maximum(t, 0), 0), d["lens"], d["cu"], tree=d["tree"], **size)
        check(attend(d, kernel=vtmu.VTMU_PAGED_AUTO, **size), want)


@pytest.mark.parametrize("counts", [[5, 9, 2], [50, 33, 2]])
def test_rows_past_max_rows_stay_as_they_were(counts):
    size = size_of(4, 2, 64, 16)
    for most in (1, counts[1] - 2):
        d = q8.batch(9, [200, 90, 500], counts, form=q8.INT8, **size)
        want = expect(d, **size)
        for kernel in (CUDA, TENSOR):
            got = attend(d, kernel=kernel, out=torch.full(d["q"].shape, 3.0, device="cuda"), maxRows=most, **size)
            for b in range(3):
                a, e = d["cu"][b], d["cu"][b + 1]
                check(got[a:min(e, a + most)], want[a:min(e, a + most)])
                assert np.all(got[min(e, a + most):e] == 3.0)


def test_many_small_requests():
    size = size_of(2, 1, 64, 16)
    for counts in ([1] * 1024, [20] * 700 + [0] * 324):
        d = q8.batch(12, [(7 * b) % 90 for b in range(1024)], counts, form=q8.E4M3, **size)
        check(attend(d, kernel=TENSOR, **size), expect(d, **size))


@pytest.mark.parametrize("counts,tree", [([3, 2], False), ([40, 30], False), ([3, 2], True), ([40, 30], True)])
def test_same_call_gives_the_same_bits(counts, tree):
    size = size_of(8, 2, 128, 16)
    d = q8.batch(13, [5000, 3000], counts, form=q8.INT8, tree=tree, **size)
    first = attend(d, kernel=TENSOR, **size)
    for _ in range(4):
        assert np.array_equal(attend(d, kernel=TENSOR, **size), first)


@pytest.mark.parametrize("which", ["q", "kc", "vc", "out", "k_new", "ks"])
def test_misaligned_tensors(which):
    """They take the CUDA cores (scales off the 16-byte grid do not)."""
    size = size_of(8, 4, 64, 16)
    d = q8.batch(14, [150], [20], form=q8.E4M3, tree=True, **size)
    want = expect(d, **size)

    def shifted(t):
        raw_ = torch.empty(t.numel() + 4, dtype=t.dtype, device="cuda")
        return raw_[1:1 + t.numel()].view(t.shape).copy_(t)

    ts = dict(q=dev(d["q"]), kc=codes(d["kc"], d["form"]), vc=codes(d["vc"], d["form"]), ks=dev(d["ks"]), out=torch.zeros(d["q"].shape, device="cuda"),
              k_new=dev(d["tree"][0]))
    ts[which] = shifted(ts[which])

    def call(kernel):
        return vtmu.paged_attention_q8(ts["q"], ts["kc"], ts["vc"], ts["ks"], dev(d["vs"]), dev(d["table"]), dev(d["lens"]),
                                       dev(d["cu"]), tree=(ts["k_new"], *(dev(x) for x in d["tree"][1:])), maxRows=20,
                                       kernel=kernel, out=ts["out"], **size)

    check(call(vtmu.VTMU_PAGED_AUTO).cpu().numpy(), want)
    if which != "ks":
        with pytest.raises(vtmu.VtmuError) as e:
            call(TENSOR)
        assert e.value.status == vtmu.VTMU_ERR_UNSUPPORTED


def test_offsets_past_32_bits():
    """Pools of 4.3 GB of codes: written, read and attended over at their end."""
    hk, D, P = 8, 128, 16
    size = size_of(8, hk, D, P)
    pages = (1 << 32) // (hk * D * P) + 40
    d = q8.batch(15, [200, 330], [3, 2], form=q8.INT8, extra_cols=0, **size)
    many = q8.batch(15, [200, 330], [30, 20], form=q8.INT8, extra_cols=0, **size)
    kp, vp = (torch.zeros(pages * P, hk * D, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(pages * P, hk, device="cuda") for _ in range(2))
    used = len(d["ks"])
    rows = slice(pages * P - used, pages * P)
    up = pages - used // P
    for x in (d, many):
        kp[rows], vp[rows] = codes(x["kc"], q8.INT8), codes(x["vc"], q8.INT8)
        ks[rows], vs[rows] = dev(x["ks"]), dev(x["vs"])
        table = np.where(x["table"] >= 0, x["table"] + up, -1).astype(np.int32)
        want = expect(x, **size)
        for kernel in (CUDA, TENSOR):
            got = vtmu.paged_attention_q8(dev(x["q"]), kp, vp, ks, vs, dev(table), dev(x["lens"]), dev(x["cu"]), kernel=kernel,
                                          maxRows=int(np.diff(x["cu"]).max()), **size)
            check(got.cpu().numpy(), want)
    g = np.random.default_rng(2)
    x = [g.standard_normal((2, hk * D), dtype=np.float32) for _ in range(2)]
    slots = dev(np.array([pages * P - 1, pages * P - 7], np.int32))
    vtmu.paged_write_q8(kp, vp, ks, vs, dev(x[0]), dev(x[1]), slots)
    for y, new in zip(vtmu.paged_read_q8(kp, vp, ks, vs, slots), x):
        want = q8.values(*q8.quantise(new, hk, q8.INT8), q8.INT8)
        assert np.all(np.abs(y.cpu().numpy() - want) <= 2.0 ** -24 * np.abs(want))


@pytest.mark.parametrize("counts,tree", [([3, 2], False), ([40, 30], False), ([3, 2], True), ([40, 30], True)])
@pytest.mark.parametrize("given", [False, True])
def test_captured_and_replayed_with_other_lengths(counts, tree, given):
    """Two graphs of one workspace, replayed with other contents of the same buffers."""
    size = size_of(8, 2, 128, 16)
    cases = [q8.batch(50 + i, lens, counts, form=q8.INT8, tree=tree, extra_cols=0, **size)
             for i, lens in enumerate(([900, 64], [1, 880], [300, 300]))]
    pages, cols = max(len(d["ks"]) for d in cases), max(d["table"].shape[1] for d in cases)

    def fit(d):
        pad = lambda a, n, v: np.concatenate([a, np.full((n - len(a),) + a.shape[1:], v, a.dtype)])
        table = np.full((2, cols), -1, np.int32)
        table[:, :d["table"].shape[1]] = d["table"]
        t = [dev(d["q"]), codes(pad(d["kc"], pages, 0), q8.INT8), codes(pad(d["vc"], pages, 0), q8.INT8),
             dev(pad(d["ks"], pages, np.nan)), dev(pad(d["vs"], pages, np.nan)), dev(table), dev(d["lens"]), dev(d["cu"])]
        return t + ([dev(x) for x in d["tree"]] if tree else [])

    fitted = [fit(d) for d in cases]
    static = [t.clone() for t in fitted[0]]
    ws = vtmu.Workspace() if given else None
    kw = dict(size, maxRows=max(counts), tree=tuple(static[8:]) if tree else None, workspace=ws)
    if given:  # grown before the capture
        vtmu.paged_attention_q8(*static[:8], **kw)
    graphs = []
    for _ in range(2):
        out = torch.zeros_like(static[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            vtmu.paged_attention_q8(*static[:8], out=out, **kw)
        graphs.append((g, out))
    for i in (1, 0, 2, 1):
        for s, x in zip(static, fitted[i]):
            s.copy_(x)
        want = expect(cases[i], **size)
        for g, out in graphs:
            g.replay()
            check(out.cpu().numpy(), want)
    assert vtmu.vtmu_device_error() == 0


@pytest.mark.parametrize("given", [False, True])
def test_two_streams(given):
    """Calls in flight together, few rows and many, with a workspace each or none."""
    size = size_of(8, 2, 128, 16)
    ds = [q8.batch(19 + i, [2000, 700], counts, form=q8.E4M3, tree=True, **size) for i, counts in enumerate(([2, 1], [3, 30]))]
    streams = [torch.cuda.Stream() for _ in ds]
    spaces = [vtmu.Workspace() if given else None for _ in ds]
    ins = [([dev(d["q"]), codes(d["kc"], d["form"]), codes(d["vc"], d["form"])] + [dev(d[k]) for k in ("ks", "vs", "table", "lens", "cu")],
            tuple(dev(x) for x in d["tree"])) for d in ds]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(vtmu.paged_attention_q8(*ins[i][0], tree=ins[i][1], maxRows=30 if i else 2, workspace=spaces[i], **size))
    torch.cuda.synchronize()
    for i, d in enumerate(ds):
        want = expect(d, **size)
        for o in outs[i]:
            check(o.cpu().numpy(), want)


def test_a_captured_step():
    """norm_rope, paged_write_q8, attention and paged_read_q8 of one token in a graph; the same bits as eager."""
    H, hk, D, P, cols = 8, 2, 64, 16, 30
    size = size_of(H, hk, D, P)
    g = np.random.default_rng(4)
    pages = 64
    pools = [torch.zeros(pages * P, hk * D, dtype=torch.int8, device="cuda") for _ in range(2)]
    pools += [torch.zeros(pages * P, hk, device="cuda") for _ in range(2)]
    table = dev(g.permutation(pages)[:2 * cols].reshape(2, cols).astype(np.int32))
    cu = dev(np.arange(3, dtype=np.int32))
    q, k, v = (torch.zeros(2, n * D, device="cuda") for n in (H, hk, hk))
    lens, pos, slots = (torch.zeros(2, dtype=torch.int32, device="cuda") for _ in range(3))

    def step():
        qt, kt = vtmu.norm_rope(q, k, pos, headDim=D)
        vtmu.paged_write_q8(*pools, kt, v, slots)
        out = vtmu.paged_attention_q8(qt, *pools, table, lens, cu, maxRows=1, **size)
        return (out, *vtmu.paged_read_q8(*pools, slots))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for t in range(40):
        for x in (q, k, v):
            x.copy_(dev(g.standard_normal(x.shape, dtype=np.float32)))
        pos.fill_(t)
        lens.fill_(t + 1)
        slots.copy_(table[:, t // P] * P + t % P)
        before = [p.clone() for p in pools]
        graph.replay()
        one = [x.clone() for x in got]
        after = [p.clone() for p in pools]
        for p, x in zip(pools, before):
            p.copy_(x)
        two = step()
        assert all(torch.equal(x, y) for x, y in zip(one + after, list(two) + pools))
    assert vtmu.vtmu_device_error() == 0


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("form", FORMS)
def test_a_serving_run(form):
    """Prompts, then steps of single tokens, then a drafted tree whose accepted rows are written:
    norm_rope, page_map, tree_plan, paged_write_q8, paged_attention_q8 and paged_read_q8 as a
    worker calls them, against plain arrays that hold every request's f32 rows."""
    H, hk, D, P = 8, 2, 64, 16
    g = np.random.default_rng(11)
    pages = 60
    kp, vp = (torch.zeros(pages * P, hk * D, dtype=DTYPE[form], device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(pages * P, hk, device="cuda") for _ in range(2))
    table = torch.full((2, 20), -1, dtype=torch.int32, device="cuda")
    free, n_free = dev(np.arange(pages, dtype=np.int32)), dev(np.array([pages], np.int32))
    lens = dev(np.zeros(2, np.int32))
    qw, kw = (dev((1 + 0.2 * g.standard_normal(D)).astype(np.float32)) for _ in range(2))
    rope = dict(headDim=D, base=10000.0, sections=[12, 10, 10], dealt=True, qWeight=qw, kWeight=kw)
    size = dict(heads=H, kvHeads=hk, headDim=D, pageSize=P)
    held = [[np.zeros((0, hk * D))] * 2 for _ in range(2)]  # what the cache stands for

    def step(counts, tree=False):
        nonlocal lens, n_free
        cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        rows = int(cu[-1])
        q, k, v = (g.standard_normal((rows, n * D), dtype=np.float32) for n in (H, hk, hk))
        if not tree:
            slots, pos, new_lens, left = vtmu.page_map(lens, dev(cu), table, free, n_free, rows=rows, pageSize=P)
        else:
            parents = np.concatenate([[-1] + [int(g.integers(0, j)) for j in range(1, n)] for n in counts]).astype(np.int32)
            masks, pos = vtmu.tree_plan(dev(parents), dev(cu), lens)
        pos3 = torch.stack([pos, pos // 2, pos // 3])
        qt, kt = vtmu.norm_rope(dev(q), dev(k), pos3, **rope)
        kn, vn = kt.cpu().numpy(), v
        old = lens.cpu().numpy().copy()
        if not tree:
            vtmu.paged_write_q8(kp, vp, ks, vs, kt, dev(v), slots)
            lens, n_free = new_lens, left
            for b in range(2):
                for i, x in enumerate((kn, vn)):
                    x = x[cu[b]:cu[b + 1]]
                    held[b][i] = np.concatenate([held[b][i], q8.values(*q8.quantise(x, hk, form), form)])
            out = vtmu.paged_attention_q8(qt, kp, vp, ks, vs, table, lens, dev(cu), maxRows=max(counts), **size)
        else:
            out = vtmu.paged_attention_q8(qt, kp, vp, ks, vs, table, lens, dev(cu), maxRows=max(counts),
                                          tree=(kt, dev(v), masks, pos), **size)
        # the same from plain arrays: each request's rows are its own pages
        flat = np.zeros((2, 320, hk * D)), np.zeros((2, 320, hk * D))
        for b in range(2):
            for i in range(2):
                flat[i][b, :len(held[b][i])] = held[b][i]
        now = np.array([len(held[b][0]) for b in range(2)])
        want = ref.attention(qt.cpu().numpy(), flat[0].reshape(640, -1), flat[1].reshape(640, -1),
                             np.arange(40).reshape(2, 20), now, cu,
                             tree=None if not tree else (kn, vn, masks.cpu().numpy().view(np.uint64), pos.cpu().numpy()), **size)
        check(out.cpu().numpy(), want)
        if tree:  # every other node of the first path is kept
            accept = np.array([0b1011, 0b1], np.uint64)
            slots, pos, lens, n_free = vtmu.page_map(lens, dev(cu), table, free, n_free, rows=rows, pageSize=P, accept=dev(accept))
            vtmu.paged_write_q8(kp, vp, ks, vs, kt, dev(v), slots)
            for b in range(2):
                keep = [j for j in range(counts[b]) if (int(accept[b]) >> j) & 1]
                for i, x in enumerate((kn, vn)):
                    held[b][i] = np.concatenate([held[b][i], q8.values(*q8.quantise(x[cu[b]:cu[b + 1]][keep], hk, form), form)])
        assert lens.cpu().numpy().tolist() == [len(held[b][0]) for b in range(2)] and old.size == 2

    step([70, 33])
    for _ in range(3):
        step([1, 1])
    step([9, 5], tree=True)
    step([1, 2])
    for b in range(2):  # every row read back
        n = int(lens[b])
        s = np.arange(n)
        slots = table.cpu().numpy()[b, s // P] * P + s % P
        k, v = vtmu.paged_read_q8(kp, vp, ks, vs, dev(slots.astype(np.int32)))
        for y, x in zip((k, v), held[b]):
            assert np.all(np.abs(y.cpu().numpy() - x) <= 2.0 ** -24 * np.abs(x))
