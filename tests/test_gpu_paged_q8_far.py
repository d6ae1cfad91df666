"""The 8-bit caches' attention and norm_rope at the ends of f32's range, against plain 64-bit
implementations.

Tolerance of attention, by row and head, whose outputs differ in size: 2^-15 of the 2-norm, as of
test_rows_of_any_size (a score's products are each off by 2^-20 of their size, sizes add up to less
than 2^3, so a weight is off by less than 2^-17 of itself and an output by 2^-16)."""
import numpy as np
import pytest

import paged_q8_ref as q8

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import f32_gqa_attention_gb300 as vtmu  # noqa: E402
from test_gpu_paged import check, dev  # noqa: E402
from test_gpu_paged_q8 import CUDA, FORMS, TENSOR, attend, codes, expect, size_of  # noqa: E402


def check_heads(got, want, D):
    got, want = (x.reshape(-1, D).astype(np.float64) for x in (got, want))
    assert np.all(np.isfinite(got)), np.flatnonzero(~np.isfinite(got).all(1))
    biggest = np.abs(want).max(1, keepdims=True) + (np.abs(want).max(1, keepdims=True) == 0)  # squares would overflow
    err, norm = (np.linalg.norm(x / biggest, axis=1) for x in (got - want, want))
    assert np.all(err <= 2.0 ** -15 * norm), (err / norm).max()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows", [3, 20])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("power,q_power", [(118, -100), (112, -96), (100, -90)])
def test_scores_of_large_keys_stay_in_range(power, q_power, D, rows, form):
    """Keys all alike but for their sign: those of the larger score weigh the same, the others nothing.
    The codes times the scaled queries times the keys' scale alone would leave f32."""
    size = size_of(4, 2, D, 16)

    def gain(k, v):
        g = np.random.default_rng(5)
        k[:] = np.where(g.random((k.shape[0], 1)) < 0.5, -1, 1) * 2.0 ** power
        return k, v

    d = q8.batch(20, [300, 70], [rows, 2], form=form, gain=gain, waste=0.0, **size)
    d["q"][:] = 2.0 ** q_power
    check_heads(attend(d, kernel=TENSOR, **size), expect(d, **size), D)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows", [3, 20])
@pytest.mark.parametrize("power", [118, 124])
@pytest.mark.parametrize("softcap", [None, 20.0])
@pytest.mark.parametrize("D,tree", [(64, False), (128, False), (64, True)])
def test_large_keys_and_small_queries(D, tree, softcap, power, rows, form):
    """Scores of ordinary size, on the tensor cores."""
    size = size_of(4, 2, D, 16)
    d = q8.batch(21, [300, 70], [rows, 2], form=form, tree=tree, gain=lambda k, v: (k * np.float32(2.0 ** power), v), **size)
    d["q"] = d["q"] * np.float32(2.0 ** -power)
    if tree:
        d["tree"][0][:] *= np.float32(2.0 ** power)
    check_heads(attend(d, kernel=TENSOR, softcap=softcap, **size), expect(d, softcap=softcap, **size), D)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows", [3, 20])
@pytest.mark.parametrize("kernel", [CUDA, TENSOR])
def test_some_large_keys_beside_small_ones(kernel, rows, form):
    """Keys of 2^120 that a window hides, or that are orthogonal to the queries, in the tiles of ordinary ones."""
    size = size_of(4, 2, 64, 16)

    def gain(k, v):
        k[:, ::64] = 0
        k[::3, 1:] = 0
        k[::3, ::64] = 2.0 ** 120  # beside a query of 0 there
        return k, v

    d = q8.batch(22, [300, 70], [rows, 2], form=form, gain=gain, waste=0.0, **size)
    d["q"][:, ::64] = 0
    check_heads(attend(d, kernel=kernel, **size), expect(d, **size), 64)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows", [3, 20])
@pytest.mark.parametrize("power", [118, 124, -118, -124])
def test_far_queries_and_keys_on_the_cuda_cores(power, rows, form):
    size = size_of(4, 2, 64, 16)
    d = q8.batch(23, [300, 70], [rows, 2], form=form, gain=lambda k, v: (k * np.float32(2.0 ** -power), v), **size)
    d["q"] = d["q"] * np.float32(2.0 ** power)
    check_heads(attend(d, kernel=CUDA, **size), expect(d, **size), 64)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows", [3, 20])
@pytest.mark.parametrize("power", [118, 124])
def test_large_queries_and_small_keys(power, rows, form):
    size = size_of(4, 2, 64, 16)
    d = q8.batch(24, [300, 70], [rows, 2], form=form, gain=lambda k, v: (k * np.float32(2.0 ** -power), v), **size)
    d["q"] = d["q"] * np.float32(2.0 ** power)
    check_heads(attend(d, kernel=TENSOR, **size), expect(d, **size), 64)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows", [3, 20])
def test_scores_of_zero_between_large_rows(rows, form, tree):
    """Queries along one channel, keys along another: every key weighs the same."""
    size = size_of(4, 2, 64, 16)

    def gain(k, v):
        k[:] = 0
        k[:, 1::64] = 2.0 ** 100
        return k, v

    d = q8.batch(25, [90, 40], [rows, 2], form=form, tree=tree, gain=gain, **size)
    d["q"][:] = 0
    d["q"][:, ::64] = 2.0 ** 100
    if tree:
        gain(d["tree"][0], None)
    check_heads(attend(d, kernel=TENSOR, **size), expect(d, **size), 64)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows", [3, 20])
@pytest.mark.parametrize("Hk", [1, 2, 8])
@pytest.mark.parametrize("D", [64, 128])
def test_outputs_up_to_the_end_of_the_range(D, Hk, rows, form, tree):
    """Values of 2e38 to 3e38, of one sign a column: any sum of two leaves f32."""
    size = size_of(Hk, Hk, D, 16)

    def gain(k, v):
        g = np.random.default_rng(3)
        sign = np.where(g.random(v.shape[1]) < 0.5, -1, 1)
        v[:] = g.uniform(2e38, 3e38, v.shape) * sign
        return k, v

    d = q8.batch(26, [3000, 70], [rows, 2], form=form, tree=tree, gain=gain, **size)
    if tree:
        gain(None, d["tree"][1])
    check_heads(attend(d, kernel=TENSOR, **size), expect(d, **size), D)


# ----------------------------------------------------------------- norm_rope
@pytest.mark.parametrize("D", [128, 100, 2])
@pytest.mark.parametrize("size,eps", [(3e19, 3e38), (1e18, 1e38), (2e19, 1e36), (1e20, 3.4e38), (1e18, 3.4e38), (1.5e19, 3e38)])
def test_an_eps_beside_squares_that_leave_the_range(D, size, eps):
    g = np.random.default_rng(1)
    x = (g.uniform(-1, 1, (5, 3 * D)) * size).astype(np.float32)
    pos = np.arange(5, dtype=np.int32)
    y, _ = vtmu.norm_rope(dev(x), None, dev(pos), headDim=D, eps=eps)
    want, big = q8.norm_rope(x, pos, headDim=D, eps=eps)
    # As in test_gpu_paged_q8: 2^-20 of the norm, 2^-20 of sine and cosine, 2^-22 of products and sum.
    assert np.all(np.abs(y.cpu().numpy() - want) <= (2.0 ** -19 + 2.0 ** -22) * big)


@pytest.mark.parametrize("D", [128, 100])
@pytest.mark.parametrize("top,rest", [(2.0 ** 70, 2.0 ** -50), (2.0 ** 120, 2.0 ** 5), (2.0 ** 64, 2.0 ** -55)])
def test_small_elements_of_a_head_of_large_ones(D, top, rest):
    """At position 0, where nothing turns: each element to 2^-20 of itself."""
    g = np.random.default_rng(2)
    x = (g.uniform(0.5, 1, (4, 2 * D)) * rest).astype(np.float32)
    x[:, ::D] = top
    pos = np.zeros(4, np.int32)
    y, _ = vtmu.norm_rope(dev(x), None, dev(pos), headDim=D)
    want, _ = q8.norm_rope(x, pos, headDim=D)
    assert np.abs(want).min() >= 2.0 ** -126
    assert np.all(np.abs(y.cpu().numpy() - want) <= 2.0 ** -20 * np.abs(want))


def turns(freqs, positions):
    """position x frequency / (2 pi) less its whole part, from whole numbers of 2000 bits."""
    bits = 2000

    def atan_inv(n):  # atan(1 / n), in units of 2^-bits
        total, term, k = 0, (1 << bits) // n, 0
        while term:
            total += (-term if k & 1 else term) // (2 * k + 1)
            term //= n * n
            k += 1
        return total

    two_pi = 8 * (4 * atan_inv(5) - atan_inv(239))  # Machin's formula
    out = np.zeros((len(positions), len(freqs)))
    for j, f in enumerate(freqs):
        num, den = float(f).as_integer_ratio()
        for t, p in enumerate(positions):
            part = (((int(p) * num << 2 * bits) // (den * two_pi)) % (1 << bits)) >> (bits - 64)
            out[t, j] = part / 2.0 ** 64
    return out


@pytest.mark.parametrize("size", [1e-20, 1e-3, 1.0, 1e9, 6e16, 3e17, 1e20, 1e30, 3e38])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("D", [64, 10])
def test_explicit_frequencies_of_any_size(D, sign, size):
    """Sine and cosine to 2^-20 (the angle's and the sine's own error), 2^-22 of products and sum."""
    g = np.random.default_rng(4)
    half = D // 2
    freqs = (sign * size * g.uniform(0.3, 1, half)).astype(np.float32)
    pos = np.array([0, 1, 2, 77, 100003, 2 ** 31 - 1], np.int32)
    x = g.standard_normal((len(pos), 2 * D), dtype=np.float32)
    y, _ = vtmu.norm_rope(dev(x), None, dev(pos), headDim=D, norm=False, invFreq=freqs.tolist())
    th = 2 * np.pi * turns(freqs, pos)[:, None, :]
    a, b = np.split(x.reshape(len(pos), 2, D).astype(np.float64), 2, axis=2)
    want = np.concatenate([a * np.cos(th) - b * np.sin(th), b * np.cos(th) + a * np.sin(th)], 2)
    bound = (2.0 ** -20 + 2.0 ** -22) * np.concatenate([np.abs(a) + np.abs(b)] * 2, 2)
    assert np.all(np.abs(y.cpu().numpy().reshape(want.shape) - want) <= bound)


@pytest.mark.parametrize("D", [128, 100])
@pytest.mark.parametrize("kw", [dict(), dict(interleaved=True), dict(sections="dealt")])
def test_rotation_alone(D, kw):
    """Without a norm.  The angle in f32 is off by 2^-25 (its turn), 2^-25 (the factor) and 2^-24 (the product) of
    pi at most, 3.8e-7; the sine by 2^-21.41 and the cosine by 2^-21.19 more, 4.2e-7: 8.0e-7.  A product and an FMA
    round at 2^-24 each of |a| + |b|: 9.2e-7, below 2^-20."""
    g = np.random.default_rng(6)
    T, half = 3000, D // 2
    kw = dict(kw, sections=[half - 2 * (half // 3), half // 3, half // 3], dealt=True) if "sections" in kw else kw
    axes = len(kw.get("sections", [0]))
    pos = g.integers(0, 2 ** 20, (axes, T)).astype(np.int32)
    x = g.standard_normal((T, 2 * D), dtype=np.float32)
    y, _ = vtmu.norm_rope(dev(x), None, dev(pos if axes > 1 else pos[0]), headDim=D, norm=False, **kw)
    want, size = q8.norm_rope(x, pos, headDim=D, norm=False, **kw)
    assert np.all(np.abs(y.cpu().numpy() - want) <= 2.0 ** -20 * size)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[0, 0], [40, 0]])
def test_a_drafted_row_alone_is_its_value(D, lens):
    """A request whose one drafted row sees nothing else gives its value, of 22 bits or fewer, as it is,
    whatever its size."""
    size = size_of(2, 2, D, 16)
    d = q8.batch(27, lens, [3, 1], form=q8.INT8, tree=True, **size)
    g = np.random.default_rng(7)
    for e in range(-120, 127, 3):
        for power in (e, e + 1):
            v = np.ldexp(g.integers(2 ** 21, 2 ** 22, 2 * D).astype(np.float32), power - 21).astype(np.float32)
            d["tree"][1][3] = v
            got = attend(d, kernel=TENSOR, **size)
            assert np.array_equal(got[3], v), power


@pytest.mark.parametrize("kernel", [CUDA, TENSOR])
@pytest.mark.parametrize("rows", [3, 20])
@pytest.mark.parametrize("page", [8, 32, 64])
@pytest.mark.parametrize("tree", [False, True])
def test_a_request_as_long_as_its_table_allows(tree, page, rows, kernel):
    """Row numbers up to 2^31 - 1: the last rows of the longest request, seen through a window,
    are those of a short one with the same last rows."""
    last, window = 256, 100
    size = size_of(4, 2, 64, page)
    d = q8.batch(54, [last], [rows], form=q8.INT8, tree=tree, **size)
    want = expect(d, window=window, **size)
    cols = (1 << 31) // page - 1
    n = cols * page
    table = torch.zeros(1, cols, dtype=torch.int32, device="cuda")
    table[0, cols - last // page:] = dev(d["table"][0, :last // page])
    drafted = None
    if tree:
        kn, vn, masks, positions = d["tree"]
        drafted = tuple(dev(x) for x in (kn, vn, masks, (positions.astype(np.int64) + n - last).astype(np.int32)))
        if int(positions.max()) + n - last >= 2 ** 31:
            pytest.skip("no position is left for rows as deep as these")
    got = vtmu.paged_attention_q8(dev(d["q"]), codes(d["kc"], q8.INT8), codes(d["vc"], q8.INT8), dev(d["ks"]), dev(d["vs"]), table,
                                  dev(np.array([n], np.int32)), dev(d["cu"]), tree=drafted, maxRows=rows, kernel=kernel,
                                  window=window, **size)
    check(got.cpu().numpy(), want)
    assert vtmu.vtmu_device_error() == 0
