"""The paged-cache operators on the GPU against plain 64-bit implementations.

Tolerances.  Whole numbers (tables, slots, positions, masks) and copied rows
are exact.  rope_at: the angle is reduced in double, cos and sin are off by at
most 2^-21 and two products and a sum round at 2^-24 each, so an element is off
by less than (2^-21 + 2^-22) (|a| + |b|), |a| + |b| below 2^4 here: 2^-16.5;
1e-5 is asked (2^-16.6), as of op rope.  Attention: the library's 1e-4 on
outputs of order 1, and 2^-17 in the 2-norm: a score is a sum of products that
are each off by at most 2^-20 of their size (operands kept to 22 bits) plus f32
sums; sizes add up to less than 2^3 for unit rows, so a weight is off by less
than 2^-17 of itself before the normalisation takes out the common part."""
import numpy as np
import pytest

import paged_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import f32_gqa_attention_gb300 as vtmu  # noqa: E402

TOL, NORM = 1e-4, 2.0 ** -17
CUDA, TENSOR = vtmu.VTMU_PAGED_CUDA_CORES, vtmu.VTMU_PAGED_TENSOR_CORES


def dev(a):
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int64) if a.dtype == np.uint64 else a).cuda()


def check(got, want, live=None):
    got, want = got.astype(np.float64), want if live is None else want[:live]
    got = got if live is None else got[:live]
    assert np.all(np.isfinite(got))
    if want.size:
        err = np.max(np.abs(got - want))
        assert err <= TOL, f"max |err| {err:.3e}"
        n = np.linalg.norm(want)
        rel = np.linalg.norm(got - want) / n if n else 0.0
        assert rel <= NORM, f"relative error {rel:.3e}"


def attend(d, *, kernel, out=None, maxRows=None, **kw):
    tree = None if d["tree"] is None else tuple(dev(x) for x in d["tree"])
    counts = np.diff(d["cu"])
    o = vtmu.paged_attention(dev(d["q"]), dev(d["k_pool"]), dev(d["v_pool"]), dev(d["table"]), dev(d["lens"]),
                             dev(d["cu"]), tree=tree, kernel=kernel, out=out,
                             maxRows=int(counts.max()) if maxRows is None else maxRows, **kw)
    torch.cuda.synchronize()
    assert vtmu.vtmu_device_error() == 0
    return o.cpu().numpy()


def expect(d, **kw):
    return ref.attention(d["q"], d["k_pool"], d["v_pool"], d["table"], d["lens"], d["cu"], tree=d["tree"], **kw)


# ------------------------------------------------------------------ page_map
MAPS = [  # lens, counts, page, max_pages, accept, pages short
    ([0], [1], 16, 4, False, 0),
    ([15], [1], 16, 4, False, 0),
    ([16], [1], 16, 4, False, 0),
    ([0, 0, 7], [0, 0, 0], 16, 3, False, 0),
    ([5, 0, 31, 100], [3, 70, 1, 0], 8, 40, False, 0),
    ([5, 0, 31, 100], [3, 70, 1, 29], 1, 200, False, 0),
    ([40, 3], [30, 500], 16, 6, False, 0),           # past the table
    ([10, 20, 30], [64, 64, 33], 16, 20, True, 0),
    ([10, 20, 30], [70, 5, 33], 16, 20, True, 0),     # rows past the 64th are never accepted
    ([10, 20, 30], [50, 50, 50], 16, 20, False, 4),   # the stack runs out
    ([-3, 4], [5, 5], 4, 8, False, 0),
    (list(range(300)), [i % 7 for i in range(300)], 16, 30, False, 0),
    ([1], [5000], 7, 1000, False, 0),
]


@pytest.mark.parametrize("case", range(len(MAPS)))
def test_page_map(case):
    lens, counts, page, most, accepted, short = MAPS[case]
    g = np.random.default_rng(case)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(cu[-1]) + 5  # some rows behind the last request
    held = [min(-(-max(n, 0) // page), most) for n in lens]
    need = sum(min(-(-(max(n, 0) + t) // page), most) - h for n, t, h in zip(lens, counts, held))
    total = sum(held) + need + 3
    ids = g.permutation(total).astype(np.int32)
    table, at = np.full((len(lens), most), -7, np.int32), 0
    for b, h in enumerate(held):
        table[b, :h] = ids[at:at + h]
        at += h
    free = ids[at:]
    n_free = len(free) if not short else max(need - short, 0)
    accept = np.array([int(g.integers(0, 1 << 63)) * 2 + 1 for _ in lens], np.uint64) if accepted else None
    lens = np.array(lens, np.int32)
    want = ref.page_map(lens, cu, table, free, n_free, rows, page, accept)
    t = dev(table)
    slots, pos, new_lens, left = vtmu.page_map(dev(lens), dev(cu), t, dev(free), dev(np.array([n_free], np.int32)),
                                               rows=rows, pageSize=page, accept=dev(accept))
    assert np.array_equal(slots.cpu().numpy(), want[0])
    assert np.array_equal(pos.cpu().numpy(), want[1])
    assert np.array_equal(new_lens.cpu().numpy(), want[2])
    assert int(left) == want[3]
    assert np.array_equal(t.cpu().numpy(), want[4])


# ----------------------------------------------------------------- tree_plan
@pytest.mark.parametrize("counts", [[1], [64], [0, 3, 0], [2, 33, 64, 1, 32, 31], [70, 4], [5] * 700])
@pytest.mark.parametrize("shape", ["random", "chain", "star", "bad"])
def test_tree_plan(counts, shape):
    g = np.random.default_rng(len(counts))
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(cu[-1]) + 3
    j = np.concatenate([np.arange(n) for n in counts] + [np.zeros(3, np.int64)])
    parents = {"random": g.integers(-1, np.maximum(j, 1)), "chain": j - 1, "star": np.zeros_like(j),
               "bad": g.integers(-100, 100, rows)}[shape].astype(np.int32)
    lens = g.integers(-2, 1000, len(counts)).astype(np.int32)
    masks, pos = vtmu.tree_plan(dev(parents), dev(cu), dev(lens))
    want = ref.tree_plan(parents, cu, lens)
    assert np.array_equal(masks.cpu().numpy().view(np.uint64), want[0])
    assert np.array_equal(pos.cpu().numpy(), want[1])


# ------------------------------------------------------------------- rope_at
@pytest.mark.parametrize("T,heads,D,rd,inter,base", [
    (1, 1, 2, 2, False, 10000.0), (3, 5, 128, 128, False, 500000.0), (7, 2, 96, 48, False, 10000.0),
    (5, 3, 64, 64, True, 10000.0), (4, 3, 10, 6, False, 10000.0), (9, 1, 256, 256, True, 10000.0),
    (300, 2, 64, 32, False, 10000.0), (2, 3, 7, 4, True, 10000.0)])
@pytest.mark.parametrize("inplace", [False, True])
def test_rope_at(T, heads, D, rd, inter, base, inplace):
    g = np.random.default_rng(T * D)
    x = g.standard_normal((T, heads * D), dtype=np.float32)
    pos = g.integers(0, 200000, T).astype(np.int32)
    pos[0] = 0
    if T > 2:
        pos[2] = -1  # left as it was
    want = ref.rope_at(x, pos, headDim=D, base=base, rotaryDim=rd, interleaved=inter)
    xd = dev(x)
    out = xd if inplace else torch.full_like(xd, 7.0)
    vtmu.rope_at(xd, dev(pos), headDim=D, base=base, rotaryDim=rd, interleaved=inter, out=out)
    got = out.cpu().numpy()
    keep = pos >= 0
    assert np.max(np.abs(got[keep] - want[keep])) <= 1e-5
    assert np.array_equal(got[~keep], x[~keep] if inplace else np.full_like(x[~keep], 7.0))


def test_rope_at_consecutive_positions_equal_rope():
    x = torch.randn(33, 6 * 128, device="cuda")
    a = vtmu.rope(x, headDim=128, offset=1000)
    b = vtmu.rope_at(x, torch.arange(1000, 1033, dtype=torch.int32, device="cuda"), headDim=128)
    assert torch.allclose(a, b, rtol=0, atol=1e-5)


# --------------------------------------------------------------- paged_write
@pytest.mark.parametrize("rows,kw,vw,shift", [(1, 1, 1, 0), (5, 1024, 1024, 0), (33, 96, 32, 0), (7, 5, 3, 0),
                                              (600, 256, 256, 0), (9, 64, 64, 1), (6000, 4, 4, 0), (3, 0, 8, 0)])
def test_paged_write(rows, kw, vw, shift):
    """Rows bit for bit, the others untouched; `shift` moves the new rows off the 16-byte grid."""
    g = np.random.default_rng(rows)
    pool = rows + 40
    slots = g.permutation(pool)[:rows].astype(np.int32)
    slots[::4] = [-1, pool, 1 << 30, -(1 << 31)][rows % 4]
    kn, vn = (torch.randn(rows * w + 4, device="cuda")[shift:shift + rows * w].view(rows, w) for w in (kw, vw))
    kp, vp = torch.randn(pool, kw, device="cuda"), torch.randn(pool, vw, device="cuda")
    wk, wv = kp.cpu().numpy().copy(), vp.cpu().numpy().copy()
    for r, s in enumerate(slots):
        if 0 <= s < pool:
            wk[s], wv[s] = kn[r].cpu().numpy(), vn[r].cpu().numpy()
    vtmu.paged_write(kp, vp, kn, vn, dev(slots))
    assert np.array_equal(kp.cpu().numpy(), wk) and np.array_equal(vp.cpu().numpy(), wv)


# ----------------------------------------------------------- paged_attention
SHAPES = [  # lens, counts, heads, kvHeads, headDim, page, tree, params
    ([1], [1], 4, 1, 128, 16, False, {}),
    ([211], [1], 16, 4, 128, 16, False, {}),
    ([64, 128, 63, 65, 1, 300], [1, 1, 1, 1, 1, 1], 8, 2, 128, 16, False, {}),
    ([500, 77, 130, 0], [3, 77, 1, 0], 8, 8, 64, 32, False, {}),
    ([500, 77, 130], [40, 77, 1], 6, 2, 64, 64, False, {}),              # G = 3, several row blocks
    ([700], [130], 16, 2, 128, 128, False, {}),                          # 1040 virtual rows per KV head
    ([3, 9], [5, 9], 4, 2, 128, 16, False, {}),                          # more rows than the cache holds: empty rows
    ([0, 1, 63, 64, 65], [1, 5, 64, 33, 2], 4, 1, 128, 16, True, {}),
    ([300, 17, 1000], [21, 64, 7], 12, 4, 64, 32, True, {}),
    ([129, 40], [64, 64], 8, 1, 128, 64, True, {}),
    ([2000, 0, 333], [13, 60, 1], 14, 2, 64, 16, True, {}),
    ([900, 200], [1, 9], 8, 2, 128, 16, False, dict(window=100)),
    ([900, 200, 64], [4, 20, 3], 8, 2, 128, 16, False, dict(window=33, sinks=5)),
    ([900, 150], [4, 2], 4, 2, 64, 64, False, dict(window=1)),
    ([900, 150], [4, 2], 4, 2, 64, 64, False, dict(window=200, sinks=700)),
    ([900, 150, 3], [33, 20, 5], 4, 2, 64, 32, True, dict(window=64, sinks=4)),
    ([900, 150, 3], [33, 20, 5], 4, 2, 128, 32, True, dict(window=2)),
    ([333], [5], 4, 4, 128, 16, True, dict(softcap=5.0, scale=0.2)),
    ([333], [5], 4, 4, 64, 16, False, dict(softcap=5.0, window=70, sinks=1)),
    ([333], [5], 4, 4, 128, 16, False, dict(scale=-0.05)),
    ([333], [5], 4, 4, 128, 16, True, dict(scale=0.0)),
    ([5000], [1], 2, 1, 128, 256, False, {}),
    ([130, 70], [6, 3], 4, 2, 64, 8, True, {}),
]
OTHER = [  # shapes of the CUDA-core kernel alone
    ([100, 7], [3, 7], 4, 2, 96, 16, False, {}),
    ([100, 7], [3, 7], 4, 2, 32, 5, True, {}),
    ([100, 7], [3, 7], 3, 1, 7, 3, True, dict(window=9, sinks=2)),
    ([400], [2], 4, 4, 256, 32, False, dict(softcap=4.0)),
    ([100, 50], [3, 7], 4, 2, 128, 24, False, {}),
]


def run_case(c, kernel, seed=0):
    lens, counts, H, Hk, D, page, tree, kw = c
    d = ref.batch(seed, lens, counts, heads=H, kvHeads=Hk, headDim=D, pageSize=page, tree=tree, extra_rows=2)
    kw = dict(heads=H, kvHeads=Hk, headDim=D, pageSize=page, **kw)
    out = torch.full(d["q"].shape, 5.0, device="cuda")
    got = attend(d, kernel=kernel, out=out, **kw)
    live = int(d["cu"][-1])
    check(got, expect(d, **kw), live)
    assert np.all(got[live:] == 5.0)  # rows of no request stay as they were


@pytest.mark.parametrize("case", range(len(OTHER)))
def test_attention_cuda_core_shapes(case):
    run_case(OTHER[case], vtmu.VTMU_PAGED_AUTO)


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_attention_cuda_cores(case):
    run_case(SHAPES[case], CUDA)


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_attention_tensor_cores(case):
    run_case(SHAPES[case], TENSOR)
