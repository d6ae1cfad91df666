"""Short windows and sinks of paged attention, on both kernels, against the plain 64-bit
implementation; tolerances as in test_gpu_paged."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import f32_gqa_attention_gb300 as vtmu  # noqa: E402
import paged_ref as ref  # noqa: E402
from test_gpu_paged import BOTH, attend, check, dev, expect, kw_of, run_case  # noqa: E402

pytestmark = pytest.mark.gpu


@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [1, 2, 5])
@pytest.mark.parametrize("sinks", [1, 4, 70, 100, 128, 1000])
@pytest.mark.parametrize("tree", [False, True])
def test_sinks_beside_a_short_window(kernel, D, window, sinks, tree):
    """The first rows stay visible, those in the cache's last tile too, although the window
    leaves none of the others."""
    run_case(([3, 64, 100, 128, 191], [3, 2, 5, 1, 64], 4, 2, D, 16, tree, dict(window=window, sinks=sinks)), kernel, seed=52)


@BOTH
@pytest.mark.parametrize("page", [8, 32])
@pytest.mark.parametrize("tree", [False, True])
def test_a_request_as_long_as_its_table_allows(kernel, page, tree):
    """Row numbers up to 2^31 - 1: the last rows of the longest request, seen through a window,
    are those of a short one with the same last rows."""
    last, window = 256, 100
    kw = kw_of(4, 2, 64, page, window=window)
    d = ref.batch(54, [last], [3], tree=tree, heads=4, kvHeads=2, headDim=64, pageSize=page)
    want = expect(d, **kw)
    cols = (1 << 31) // page - 1
    n = cols * page
    table = torch.zeros(1, cols, dtype=torch.int32, device="cuda")
    table[0, cols - last // page:] = dev(d["table"][0, :last // page])
    drafted = None
    if tree:
        kn, vn, masks, positions = d["tree"]
        drafted = tuple(dev(x) for x in (kn, vn, masks, (positions.astype(np.int64) + n - last).astype(np.int32)))
        assert int(positions.max()) + n - last < 2 ** 31
    got = vtmu.paged_attention(dev(d["q"]), dev(d["k_pool"]), dev(d["v_pool"]), table, dev(np.array([n], np.int32)), dev(d["cu"]),
                               tree=drafted, maxRows=3, kernel=kernel, **kw)
    check(got.cpu().numpy(), want)
    assert vtmu.vtmu_device_error() == 0


@BOTH
@pytest.mark.parametrize("n", [0, 2, 5, 6, 70])
def test_drafted_rows_are_no_sinks(kernel, n):
    """Only rows of the cache are, in a chain that is deeper than the window too."""
    kw = kw_of(4, 2, 64, 16, window=3, sinks=6)
    d = ref.batch(55, [n, 40], [9, 4], heads=4, kvHeads=2, headDim=64, pageSize=16, tree=True)
    kn, vn, masks, positions = d["tree"]
    masks[:9] = [(2 << j) - 1 for j in range(9)]  # a chain
    positions[:9] = n + np.arange(9)
    got = attend(d, kernel=kernel, **kw)
    check(got, expect(d, **kw))
    # Row 8 at position n + 8 sees its window, drafted rows 6 to 8, and the cache's first rows.
    keys = min(n, 6)
    at = d["table"][0, np.arange(keys) // 16].astype(np.int64) * 16 + np.arange(keys) % 16
    k, v = np.concatenate([d["k_pool"][at], kn[6:9]]), np.concatenate([d["v_pool"][at], vn[6:9]])
    for h in range(4):
        c = (h // 2) * 64
        x = k[:, c:c + 64].astype(np.float64) @ d["q"][8, 64 * h:64 * h + 64].astype(np.float64) / 8.0
        w = np.exp(x - x.max())
        assert np.max(np.abs(got[8, 64 * h:64 * h + 64] - w @ v[:, c:c + 64] / w.sum())) <= 1e-4
