"""Short windows and sinks of paged attention, on both kernels, against the plain 64-bit
implementation; tolerances as in test_gpu_paged."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from test_gpu_paged import BOTH, run_case  # noqa: E402

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
