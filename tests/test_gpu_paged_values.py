"""Paged attention on rows of very different size, scores past what 16 bits hold and
numbers that are not finite, on both kernels, against plain 64-bit implementations.

Tolerance: NORM of test_gpu_paged in the 2-norm of a request's output.  It is for
scores of up to 2^3; where a test's weights come from larger ones, a score x is off by
at most 2^-20 sum |q k| scale, so its weight by that of itself: `far` adds 2^-20 |x|
for keys that point along the query (sum |q k| scale = |x|)."""
import numpy as np
import pytest

import paged_ref as ref

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from test_gpu_paged import BOTH, NORM, TENSOR, attend, check, expect, kw_of  # noqa: E402

pytestmark = pytest.mark.gpu

# A row's context: inside one CTA, and cut into pieces by many.
WHOLE, CUT = 130, 64 * 400 + 7


def close(got, want, extra=0.0):
    assert np.all(np.isfinite(got))
    size = np.max(np.abs(want))
    err = np.linalg.norm((got.astype(np.float64) - want) / size) / np.linalg.norm(want / size)
    assert err <= NORM + extra, f"relative error {err:.3e}"


def cache_rows(d, b, page):
    s = np.arange(int(d["lens"][b]))
    return d["table"][b, s // page].astype(np.int64) * page + s % page


def aim(d, kw, b, key, log2_weight):
    """Points the first KV head's key `key` of request b along row 0, head 0 of its query,
    with a score of log2_weight * ln 2."""
    D, page = kw["headDim"], kw["pageSize"]
    q = d["q"][d["cu"][b], :D].astype(np.float64)
    x = log2_weight * np.log(2.0)
    d["k_pool"][cache_rows(d, b, page)[key], :D] = q * (x / (q @ q) * D ** 0.5)


# ---------------------------------------------------------- values of any size
@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [WHOLE, CUT])
@pytest.mark.parametrize("size", [1.0, 600.0, 1e4, 1e5, 1e6, 1e9, 1e20])
def test_a_large_value_row_that_weighs_nothing(kernel, D, n, size):
    """It is seen, and its product with its weight is far below the output."""
    kw = kw_of(2, 2, D, 16)
    d = ref.batch(41, [n, 40], [1, 1], **kw)
    for b, key in ((0, 5), (0, 70), (1, 33)):
        aim(d, kw, b, key, -120.0)
        d["v_pool"][cache_rows(d, b, 16)[key], :D] *= np.float32(size)
    close(attend(d, kernel=kernel, **kw), expect(d, **kw))


@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [WHOLE, CUT])
@pytest.mark.parametrize("bits", [12, 20, 30, 60, 90])
def test_a_large_value_row_whose_product_counts(kernel, D, n, bits):
    """A weight of 2^-bits times a value of 2^bits: as large as the ordinary products."""
    kw = kw_of(2, 2, D, 16)
    d = ref.batch(42, [n, 40], [1, 1], **kw)
    for b, key in ((0, 5), (0, 70), (1, 33)):
        aim(d, kw, b, key, -float(bits))
        d["v_pool"][cache_rows(d, b, 16)[key], :D] *= np.float32(2.0 ** bits)
    close(attend(d, kernel=kernel, **kw), expect(d, **kw), extra=bits * np.log(2.0) * 2.0 ** -20)


@BOTH
@pytest.mark.parametrize("small", [1e-4, 1e-12, 1e-30])
def test_a_tile_of_which_the_heaviest_key_has_a_small_value(kernel, small):
    """One key takes nearly all of the weight and brings next to nothing."""
    kw = kw_of(2, 2, 128, 16)
    d = ref.batch(43, [WHOLE, 40], [1, 1], **kw)
    for b, key in ((0, 0), (1, 0)):
        aim(d, kw, b, key, 14.0)
        d["v_pool"][cache_rows(d, b, 16)[key], :128] *= np.float32(small)
    close(attend(d, kernel=kernel, **kw), expect(d, **kw), extra=14 * np.log(2.0) * 2.0 ** -20)


@BOTH
def test_large_value_rows_in_trees(kernel):
    """Context and drafted rows of the trees, seen with weights of every size."""
    kw = kw_of(8, 2, 128, 32)
    d = ref.batch(44, [300, 70], [30, 64], tree=True, **kw)
    g = np.random.default_rng(44)
    for v, rows in ((d["v_pool"], len(d["v_pool"])), (d["tree"][1], len(d["q"]))):
        v *= np.where(g.random((rows, 1)) < 0.1, 10.0 ** g.uniform(2, 6, (rows, 1)), 1.0).astype(np.float32)
    got, want = attend(d, kernel=kernel, **kw), expect(d, **kw)
    for t in range(94):  # row by row: the large ones do not hide the others
        for h in range(8):
            close(got[t, h * 128:(h + 1) * 128], want[t, h * 128:(h + 1) * 128], extra=2.0 ** -17)


# ----------------------------------------------------- values at f32's far end
@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [30, 60])
@pytest.mark.parametrize("size", [1e30, 1e33, 1e36])
def test_values_near_the_largest(kernel, D, n, size):
    """At most 60 keys and |N(0, 1)| below 4.5: sums of weights times values stay below 2.7e38."""
    kw = kw_of(4, 2, D, 16)
    d = ref.batch(45, [n], [2], **kw)
    d["v_pool"] = np.clip(d["v_pool"], -4.5, 4.5) * np.float32(size)
    close(attend(d, kernel=kernel, **kw), expect(d, **kw))


@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [1e-30, 1e-34, 1e-36])
def test_values_near_the_smallest(kernel, D, size):
    """Products of weights and values go down to 2^-149 in steps of that: below 2^-24 of these outputs."""
    kw = kw_of(4, 2, D, 16)
    d = ref.batch(53, [WHOLE, 40], [2, 1], **kw)
    d["v_pool"] *= np.float32(size)
    close(attend(d, kernel=kernel, **kw), expect(d, **kw))


@pytest.mark.parametrize("size", [1e30, 1e33, 1e37])
def test_values_near_the_largest_on_many_tiles(size):
    """The tensor cores' sums are kept in units that such values fit, whatever their number;
    ordinary rows come before and after."""
    kw = kw_of(4, 2, 64, 64)
    d = ref.batch(46, [CUT, 300], [2, 2], **kw)
    rows = cache_rows(d, 0, 64)
    d["v_pool"][rows[1000:9000]] = np.clip(d["v_pool"][rows[1000:9000]], -4.5, 4.5) * np.float32(size)
    close(attend(d, kernel=TENSOR, **kw)[:2], expect(d, **kw)[:2])
    check(attend(d, kernel=TENSOR, **kw)[2:], expect(d, **kw)[2:])


@BOTH
@pytest.mark.parametrize("n", [WHOLE, CUT])
@pytest.mark.parametrize("weight", [-100.0, -200.0])
def test_the_largest_values_with_a_negligible_weight(kernel, n, weight):
    kw = kw_of(2, 2, 128, 16)
    d = ref.batch(47, [n, 40], [1, 1], **kw)
    for b, key in ((0, 5), (0, 70), (1, 33)):
        aim(d, kw, b, key, weight)
        d["v_pool"][cache_rows(d, b, 16)[key], :128] = np.float32(1e37)
    close(attend(d, kernel=kernel, **kw), expect(d, **kw), extra=-weight * np.log(2.0) * 2.0 ** -20)


def test_a_large_row_that_later_keys_leave_behind():
    """It sets the units of the running sum, then rising scores take its weight away."""
    kw = kw_of(2, 2, 128, 64)
    d = ref.batch(48, [64 * 6], [1], **kw)
    aim(d, kw, 0, 3, 10.0)
    d["v_pool"][cache_rows(d, 0, 64)[3], :128] *= np.float32(2.0 ** 100)
    for i, bits in enumerate((60.0, 110.0, 160.0)):
        aim(d, kw, 0, 64 * (i + 2) + 9, bits)
    close(attend(d, kernel=TENSOR, **kw), expect(d, **kw), extra=160 * np.log(2.0) * 2.0 ** -20)


# ------------------------------------------------------------------ far scores
def best_key_leads(d, D, cap):
    """True where in every row the best score leads the runner-up by more than 2^10, and by
    more than 2^-17 of itself, which no rounding of a score turns round."""
    for b in range(len(d["lens"])):
        k = d["k_pool"][cache_rows(d, b, 16)].astype(np.float64)
        for t in range(int(d["cu"][b]), int(d["cu"][b + 1])):
            lim = len(k) - (int(d["cu"][b + 1]) - 1 - t)
            for h in range(4):
                x = k[:lim, (h // 2) * D:(h // 2 + 1) * D] @ d["q"][t, h * D:(h + 1) * D].astype(np.float64) * D ** -0.5
                x = np.unique(cap * np.tanh(x / cap) if cap else x)
                if not x[-1] - x[-2] > max(2.0 ** 10, 2.0 ** -17 * abs(x[-1])):
                    return False
    return True


@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [50, CUT])
@pytest.mark.parametrize("q_size,k_size", [
    (2e3, 1e3), (3e3, 2e3), (3e3, 4e3), (5e3, 5e3), (1e4, 1e4), (5e5, 20.0), (1e7, 40.0), (1e15, 1e15), (1e30, 1.0)])
@pytest.mark.parametrize("capped", [False, True])
def test_far_scores_take_one_key(kernel, D, n, q_size, k_size, capped):
    """Scores of q_size * k_size: the output is the value of the best key, half of each where
    two keys are the same (some are, in one tile, in two and in two pieces of a unit)."""
    kw = kw_of(4, 2, D, 16)
    d = ref.batch(49, [n, 40], [2, 1], **kw)
    d["q"] *= np.float32(q_size)
    d["k_pool"] *= np.float32(k_size)
    for b, i, j in ((0, 7, 33), (0, 9, n - 5), (1, 2, 35)):
        rows = cache_rows(d, b, 16)
        d["k_pool"][rows[i]] *= np.float32(3)
        d["k_pool"][rows[j]] = d["k_pool"][rows[i]]
    if capped:  # a cap that the scores do not come near
        kw["softcap"] = 1e3 * q_size * k_size
    assert best_key_leads(d, D, kw.get("softcap"))
    close(attend(d, kernel=kernel, **kw), expect(d, **kw))


# ------------------------------------------------------ numbers that are not finite
@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [WHOLE, CUT])
@pytest.mark.parametrize("where", ["query", "a key", "an early key", "every key"])
@pytest.mark.parametrize("softcap", [None, 3.0])
def test_nan_scores_make_their_rows_nan(kernel, D, n, where, softcap):
    """Whether the row's unit is cut or not, and no other row or head."""
    kw = kw_of(4, 2, D, 16)
    d = ref.batch(50, [n, 90], [3, 2], **kw)
    kw["softcap"] = softcap
    want = expect(d, **kw)
    nan = np.zeros(want.shape, bool)
    if where == "query":
        d["q"][1, D + 3] = np.nan
        nan[1, D:2 * D] = True
    else:
        rows = cache_rows(d, 0, 16)
        rows = {"a key": rows[n - 40:n - 39], "an early key": rows[:1], "every key": rows}[where]
        d["k_pool"][rows, D + 5] = np.nan
        nan[:3, 2 * D:] = True
    got = attend(d, kernel=kernel, **kw)
    assert np.array_equal(np.isnan(got), nan)
    check(np.where(nan, 0.0, got), np.where(nan, 0.0, want))


@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [WHOLE, CUT])
@pytest.mark.parametrize("weight", [-20.0, -400.0])
@pytest.mark.parametrize("others", [False, True])
def test_a_value_that_is_not_finite_counts_whatever_its_weight(kernel, D, n, weight, others):
    """Its column of the row that sees it is not finite, whether the unit is cut or not."""
    kw = kw_of(2, 2, D, 16)
    d = ref.batch(51, [n, 40], [2, 1], **kw)
    for key in (*range(min(n - 20, 1000) if others else 0), 5, n - 1):  # whole tiles and pieces with it; the last key
        aim(d, kw, 0, key, weight)                                        # is the second row's alone
    want = expect(d, **kw)
    d["v_pool"][cache_rows(d, 0, 16)[5], 9] = np.inf
    d["v_pool"][cache_rows(d, 0, 16)[n - 1], 11] = np.nan
    lost = np.zeros(want.shape, bool)
    lost[:2, 9] = lost[1, 11] = True
    got = attend(d, kernel=kernel, **kw)
    assert np.array_equal(~np.isfinite(got), lost)
    extra = -weight * np.log(2.0) * 2.0 ** -20
    close(np.where(lost, 0.0, got), np.where(lost, 0.0, want), extra=extra)
