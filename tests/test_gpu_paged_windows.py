"""Short windows and sinks of paged attention, on both kernels, against the plain 64-bit
implementation; tolerances as in test_gpu_paged."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import f32_gqa_attention_gb300 as vtmu  # noqa: E402
import paged_ref as ref  # noqa: E402
from test_gpu_paged import BOTH, check, dev, expect, kw_of, run_case  # noqa: E402

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
