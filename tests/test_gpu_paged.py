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


BOTH = pytest.mark.parametrize("kernel", [CUDA, TENSOR], ids=["cuda_cores", "tensor_cores"])
KW = dict(heads=8, kvHeads=2, headDim=128, pageSize=16)


def kw_of(H, Hk, D, page, **more):
    return dict(heads=H, kvHeads=Hk, headDim=D, pageSize=page, **more)


@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), 3.0e38, -3.4e38])
def test_what_a_row_does_not_see_does_not_reach_it(kernel, D, bad):
    """Keys and values of drafted rows that are no ancestors, and of a run's later
    rows, hold anything."""
    kw = kw_of(8, 2, D, 16)
    d = ref.batch(1, [100, 40], [30, 12], tree=True, **kw)
    node = 5  # of the first request
    seen = (d["tree"][2][:30] >> np.uint64(node)) & np.uint64(1)
    want = expect(d, **kw)
    d["tree"][0][node] = d["tree"][1][node] = bad
    got = attend(d, kernel=kernel, **kw)
    keep = np.concatenate([seen == 0, np.ones(12, bool)])
    assert keep.sum() > 20 and not keep.all()
    check(got[keep], want[keep])
    d = ref.batch(2, [100, 40], [30, 12], tree=False, **kw)
    want = expect(d, **kw)
    s = 100 - 30 + 7  # position of the first request's row 7
    row = d["table"][0, s // 16] * 16 + s % 16
    d["k_pool"][row] = d["v_pool"][row] = bad
    got = attend(d, kernel=kernel, **kw)
    keep = np.ones(42, bool)
    keep[7:30] = False
    check(got[keep], want[keep])


@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tree", [False, True])
def test_values_that_are_not_finite_stay_in_their_columns(kernel, D, tree):
    """A value that a row sees and that is not finite makes that column of the row not finite, and no other."""
    kw = kw_of(4, 2, D, 32)
    d = ref.batch(3, [200, 90], [9, 3], tree=tree, **kw)
    d["v_pool"][d["table"][0, 1] * 32 + 3, 5] = np.inf       # cache row 35
    d["v_pool"][d["table"][0, 2] * 32 + 1, D + 7] = np.nan   # the other KV head
    if tree:
        d["tree"][1][0, 11] = -np.inf                         # the first request's root
    want = expect(d, **kw)
    got = attend(d, kernel=kernel, **kw)
    fine = np.isfinite(want)
    assert not fine.all() and np.array_equal(np.isfinite(got), fine)
    assert np.array_equal(np.sign(got[np.isinf(want)]), np.sign(want[np.isinf(want)]))
    check(np.where(fine, got, 0.0), np.where(fine, want, 0.0))


@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("which", ["keys", "values", "both", "tiny values", "huge values"])
def test_rows_of_any_size(kernel, D, which):
    """Rows of keys and values between 1e-30 and 1e30 beside ordinary ones: in the
    2-norm of the output's column scale, as close as ordinary ones."""
    kw = kw_of(8, 2, D, 16)
    g = np.random.default_rng(5)
    d = ref.batch(6, [300, 77], [6, 3], tree=True, **kw)
    n = len(d["k_pool"])
    if which in ("keys", "both"):
        d["k_pool"] *= np.where(g.random((n, 1)) < 0.1, 10.0 ** g.uniform(-30, -1, (n, 1)), 1.0).astype(np.float32)
        d["k_pool"][d["table"][1, 0] * 16] *= np.float32(2e3)  # one key that rules where it is seen
    if which in ("values", "both"):
        d["v_pool"] *= np.where(g.random((n, 1)) < 0.1, 10.0 ** g.uniform(-30, 4, (n, 1)), 1.0).astype(np.float32)
    scale = {"tiny values": 1e-20, "huge values": 1e30}.get(which, 1.0)
    d["v_pool"] *= np.float32(scale)
    d["tree"][1][:] *= np.float32(scale)
    want = expect(d, **kw)
    got = attend(d, kernel=kernel, **kw).astype(np.float64)
    assert np.all(np.isfinite(got))
    assert np.linalg.norm((got - want) / scale) <= NORM * np.linalg.norm(want / scale)


@BOTH
def test_bad_page_ids_read_as_zeros(kernel):
    d = ref.batch(7, [100, 60, 200], [1, 5, 2], **KW)
    d["table"][1, 1], d["table"][1, 3] = -1, 1 << 30
    d["table"][0, 6] = len(d["k_pool"]) // 16  # the first id past the pool
    e = {k: v for k, v in d.items()}
    pages = len(d["k_pool"]) // 16
    e["k_pool"] = np.concatenate([d["k_pool"], np.zeros((16, 256), np.float32)])
    e["v_pool"] = np.concatenate([d["v_pool"], np.zeros((16, 256), np.float32)])
    e["table"] = np.where((d["table"] < 0) | (d["table"] >= pages), pages, d["table"])
    check(attend(d, kernel=kernel, **KW), expect(e, **KW))


@BOTH
def test_lengths_out_of_range_are_clamped(kernel):
    """Lengths past the table and below zero, decreasing and overlong cu_rows: no
    row that is not a request's is written, the others come out right."""
    d = ref.batch(8, [96, 50, 33], [2, 3, 1], extra_cols=0, **KW)
    want = expect(d, **KW)
    d["lens"] = np.array([96, -5, 33], np.int32)
    want[2:5] = 0.0  # nothing to see
    out = torch.full(d["q"].shape, 5.0, device="cuda")
    check(attend(d, kernel=kernel, out=out, **KW), want)
    d["lens"][1] = 50
    d["cu"] = np.array([0, 2, 1, 1000000], np.int32)  # request 1 has no rows, request 2 rows 1 .. the end
    out = torch.full(d["q"].shape, 5.0, device="cuda")
    got = attend(d, kernel=kernel, out=out, maxRows=3, **KW)
    assert np.all(np.isfinite(got)) and np.all(got[4:] == 5.0)  # past max_rows: as they were
    check(got[:1], want[:1])


@BOTH
def test_rows_past_max_rows_stay_as_they_were(kernel):
    d = ref.batch(9, [90, 40], [7, 2], **KW)
    out = torch.full(d["q"].shape, 5.0, device="cuda")
    got = attend(d, kernel=kernel, out=out, maxRows=4, **KW)
    want = expect(d, **KW)
    check(got[:4], want[:4])
    check(got[7:9], want[7:9])
    assert np.all(got[4:7] == 5.0)


@BOTH
def test_many_small_requests(kernel):
    g = np.random.default_rng(10)
    lens = g.integers(0, 40, 1024).tolist()
    counts = [min(int(c), n) for c, n in zip(g.integers(0, 3, 1024), lens)]
    kw = kw_of(4, 2, 64, 16)
    d = ref.batch(10, lens, counts, **kw)
    check(attend(d, kernel=kernel, **kw), expect(d, **kw))


@pytest.mark.parametrize("lens", [[4 * 64], [3 * 64 + 1, 1], [64 * 151], [64 * 152, 64], [64 * 304 + 5], [64 * 609]])
@pytest.mark.parametrize("Hk", [1, 3])
def test_units_cut_at_every_kind_of_boundary(lens, Hk):
    """Whole, started, continued and finished pieces, pieces of one to a few tiles."""
    kw = kw_of(2 * Hk, Hk, 64, 64)
    d = ref.batch(11, lens, [1] * len(lens), **kw)
    check(attend(d, kernel=TENSOR, **kw), expect(d, **kw))


def test_rising_scores_move_the_reference():
    """Keys whose scores grow along the cache, in steps and slowly: references move in
    many tiles, in some rows only."""
    kw = kw_of(4, 1, 128, 64)
    d = ref.batch(12, [64 * 40], [5], **kw)
    s = np.arange(64 * 40)
    rows = d["table"][0, s // 64].astype(np.int64) * 64 + s % 64
    for q in range(5):  # one direction for each query row
        d["k_pool"][rows, q] = s / 64.0 * (q + 1) / 2
        d["q"][q, :] *= 0.2
        for h in range(4):
            d["q"][q, h * 128 + q] = 3.0 * (-1) ** h
    check(attend(d, kernel=TENSOR, **kw), expect(d, **kw))


def test_same_call_gives_the_same_bits():
    d = ref.batch(13, [3000, 900, 4100], [5, 33, 64], tree=True, **KW)
    a, b = (attend(d, kernel=TENSOR, **KW) for _ in range(2))
    assert np.array_equal(a, b)


def test_both_kernels_agree_with_flat_attention():
    """A run of rows at the end of one request equals op attention on the flat cache."""
    T, n, H, Hk, D = 150, 700, 8, 2, 128
    kw = kw_of(H, Hk, D, 64)
    d = ref.batch(14, [n], [T], **kw)
    s = np.arange(n)
    rows = d["table"][0, s // 64].astype(np.int64) * 64 + s % 64
    flat = vtmu.attention(dev(d["q"]), dev(d["k_pool"][rows]), dev(d["v_pool"][rows]), heads=H, kvHeads=Hk, headDim=D,
                          posOffset=n - T).cpu().numpy()
    for kernel in (CUDA, TENSOR):
        assert np.max(np.abs(attend(d, kernel=kernel, **kw) - flat)) <= TOL


@pytest.mark.parametrize("which", ["q", "k_pool", "out", "k_new"])
def test_misaligned_tensors_take_the_cuda_cores(which):
    """AUTO falls back where the tensor cores want 16-byte aligned tensors; forced, they refuse."""
    d = ref.batch(15, [77], [5], tree=True, **KW)

    def shifted(x):
        b = torch.empty(x.numel() + 1, device="cuda")[1:].view(x.shape)
        return b.copy_(x)

    t = {"q": dev(d["q"]), "k_pool": dev(d["k_pool"]), "k_new": dev(d["tree"][0]), "out": torch.zeros(d["q"].shape, device="cuda")}
    t[which] = shifted(t[which])
    tree = (t["k_new"], *(dev(x) for x in d["tree"][1:]))

    def call(kernel):
        return vtmu.paged_attention(t["q"], t["k_pool"], dev(d["v_pool"]), dev(d["table"]), dev(d["lens"]), dev(d["cu"]),
                                    tree=tree, maxRows=5, kernel=kernel, out=t["out"], **KW)

    check(call(vtmu.VTMU_PAGED_AUTO).cpu().numpy(), expect(d, **KW))
    with pytest.raises(vtmu.VtmuError) as e:
        call(TENSOR)
    assert e.value.status == vtmu.VTMU_ERR_UNSUPPORTED


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements, its last pages in use."""
    kw = kw_of(8, 8, 128, 16)
    pages = (1 << 31) // (16 * 1024) + 40
    kp, vp = (torch.empty(pages * 16, 1024, device="cuda") for _ in range(2))
    d = ref.batch(16, [0], [3], tree=True, **kw)
    g = np.random.default_rng(16)
    k, v = (g.standard_normal((100, 1024), dtype=np.float32) for _ in range(2))
    table = np.arange(pages - 7, pages, dtype=np.int32)[None]
    slots = np.arange(100, dtype=np.int32) + (pages - 7) * 16
    vtmu.paged_write(kp, vp, dev(k), dev(v), dev(slots))
    assert torch.equal(kp[(pages - 7) * 16:(pages - 7) * 16 + 100], dev(k))
    d.update(k_pool=k, v_pool=v, table=np.arange(7, dtype=np.int32)[None], lens=np.array([100], np.int32))
    want = expect(d, **kw)
    for kernel in (CUDA, TENSOR):
        got = vtmu.paged_attention(dev(d["q"]), kp, vp, dev(table), dev(d["lens"]), dev(d["cu"]),
                                   tree=tuple(dev(x) for x in d["tree"]), maxRows=3, kernel=kernel, **kw)
        check(got.cpu().numpy(), want)


def test_captured_and_replayed_with_other_lengths():
    """One graph serves steps of other lengths, row counts and tables; two graphs share a workspace in turn."""
    kw = kw_of(8, 2, 64, 16)
    a = ref.batch(17, [300, 40, 5], [4, 9, 1], tree=True, extra_cols=4, extra_rows=6, **kw)
    b = ref.batch(18, [10, 299, 60], [10, 2, 8], tree=True, **kw)
    cols, pages = a["table"].shape[1], max(len(a["k_pool"]), len(b["k_pool"])) // 16
    assert b["table"].shape[1] <= cols and b["cu"][-1] == len(a["q"])

    def fit(d):
        t = np.full((3, cols), -1, np.int32)
        t[:, :d["table"].shape[1]] = d["table"]
        k, v = (np.zeros((pages * 16, 128), np.float32) for _ in range(2))
        k[:len(d["k_pool"])], v[:len(d["v_pool"])] = d["k_pool"], d["v_pool"]
        return [dev(x) for x in (d["q"], k, v, t, d["lens"], d["cu"], *d["tree"])]

    ta, tb = fit(a), fit(b)
    static = [x.clone() for x in ta]
    ws = vtmu.Workspace()
    ws.get(vtmu.vtmu_paged_workspace_size(vtmu.vtmu_paged_params(rows=20, pages=pages, requests=3, max_rows=16, page_size=16,
                                                                 max_pages=cols, heads=8, kv_heads=2, head_dim=64, tree=1)))
    outs, graphs = [], []
    for kernel in (TENSOR, TENSOR, CUDA):
        out = torch.zeros_like(static[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            q, k, v, t, lens, cu, kn, vn, masks, pos = static
            vtmu.paged_attention(q, k, v, t, lens, cu, tree=(kn, vn, masks, pos), maxRows=16, kernel=kernel, out=out,
                                 workspace=ws, **kw)
        outs.append(out)
        graphs.append(g)
    for d, src in ((b, tb), (a, ta), (b, tb)):
        for s, x in zip(static, src):
            s.copy_(x)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out in outs:
            check(out.cpu().numpy(), expect(d, **kw), int(d["cu"][-1]))
    assert vtmu.vtmu_device_error() == 0


def test_two_streams_with_a_workspace_each():
    kw = kw_of(8, 2, 128, 64)
    ds = [ref.batch(19 + i, [2000, 700], [3, 30], tree=True, **kw) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in ds]
    spaces = [vtmu.Workspace() for _ in ds]
    ins = [[dev(d[k]) for k in ("q", "k_pool", "v_pool", "table", "lens", "cu")] + [tuple(dev(x) for x in d["tree"])] for d in ds]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                *t, tree = ins[i]
                outs[i].append(vtmu.paged_attention(*t, tree=tree, maxRows=30, workspace=spaces[i], **kw))
    torch.cuda.synchronize()
    for i, d in enumerate(ds):
        want = expect(d, **kw)
        for o in outs[i]:
            check(o.cpu().numpy(), want)


@pytest.mark.parametrize("D", [64, 128, 96])
def test_serving_loop(D):
    """Prompts, a verified tree and a single token, as a worker runs them: page_map,
    rope_at, paged_write and paged_attention, tree_plan and a map of the accepted rows;
    against dense per-request keys and values in 64 bits."""
    H, Hk, P, B = 4, 2, 16, 3
    kw = kw_of(H, Hk, D, P)
    g = np.random.default_rng(21)
    pages, cols = 60, 20
    kp, vp = (torch.zeros(pages * P, Hk * D, device="cuda") for _ in range(2))
    table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    free, left = dev(g.permutation(pages).astype(np.int32)), dev(np.array([pages], np.int32))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    dense = [[np.zeros((0, Hk * D)), np.zeros((0, Hk * D))] for _ in range(B)]

    def fresh(n, width):
        return g.standard_normal((n, width), dtype=np.float32)

    def dense_want(q, b, n_rows, pos0, tree=None):
        k, v = dense[b]
        t = np.arange(len(k) + 1, dtype=np.int32)[None]
        d = dict(q=q, k_pool=k, v_pool=v, table=t, lens=np.array([len(k)], np.int32), cu=np.array([0, n_rows], np.int32), tree=tree)
        return ref.attention(d["q"], d["k_pool"], d["v_pool"], d["table"], d["lens"], d["cu"], tree=tree,
                             heads=H, kvHeads=Hk, headDim=D, pageSize=1)

    for counts in ([37, 1, 90], [1, 1, 1], [5, 17, 2]):  # prompts, tokens, chunks
        cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        n = int(cu[-1])
        q, k, v = fresh(n, H * D), fresh(n, Hk * D), fresh(n, Hk * D)
        slots, pos, lens, left = vtmu.page_map(lens, dev(cu), table, free, left, rows=n, pageSize=P)
        qr, kr = vtmu.rope_at(dev(q), pos, headDim=D), vtmu.rope_at(dev(k), pos, headDim=D)
        vtmu.paged_write(kp, vp, kr, dev(v), slots)
        got = vtmu.paged_attention(qr, kp, vp, table, lens, dev(cu), maxRows=max(counts), **kw).cpu().numpy()
        p = pos.cpu().numpy()
        for b in range(B):
            a, e = cu[b], cu[b + 1]
            assert np.array_equal(p[a:e], len(dense[b][0]) + np.arange(counts[b]))
            dense[b][0] = np.concatenate([dense[b][0], ref.rope_at(k[a:e], p[a:e], headDim=D)])
            dense[b][1] = np.concatenate([dense[b][1], v[a:e]])
            check(got[a:e], dense_want(ref.rope_at(q[a:e], p[a:e], headDim=D), b, counts[b], p[a]))
    for step in range(2):  # trees, of which some path is accepted
        counts = [13, 1, 30] if step == 0 else [2, 64, 7]
        cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        n = int(cu[-1])
        q, k, v = fresh(n, H * D), fresh(n, Hk * D), fresh(n, Hk * D)
        parents = np.concatenate([[-1] + [int(g.integers(0, j)) for j in range(1, c)] for c in counts]).astype(np.int32)
        masks, pos = vtmu.tree_plan(dev(parents), dev(cu), lens)
        qr, kr = vtmu.rope_at(dev(q), pos, headDim=D), vtmu.rope_at(dev(k), pos, headDim=D)
        got = vtmu.paged_attention(qr, kp, vp, table, lens, dev(cu), tree=(kr, dev(v), masks, pos), maxRows=max(counts),
                                   **kw).cpu().numpy()
        p = pos.cpu().numpy()
        accept = np.zeros(B, np.uint64)
        for b in range(B):
            a, e = cu[b], cu[b + 1]
            m = masks.cpu().numpy().view(np.uint64)[a:e]
            kd, qd = ref.rope_at(k[a:e], p[a:e], headDim=D), ref.rope_at(q[a:e], p[a:e], headDim=D)
            check(got[a:e], dense_want(qd, b, counts[b], 0, (kd, v[a:e], m, p[a:e])))
            accept[b] = m[g.integers(0, counts[b])]  # a node's path from the root
            path = [j for j in range(counts[b]) if (int(accept[b]) >> j) & 1]
            dense[b][0] = np.concatenate([dense[b][0], kd[path]])
            dense[b][1] = np.concatenate([dense[b][1], v[a:e][path]])
        slots, pos2, lens, left = vtmu.page_map(lens, dev(cu), table, free, left, rows=n, pageSize=P, accept=dev(accept))
        kept = slots.cpu().numpy() >= 0
        assert np.array_equal(pos2.cpu().numpy()[kept], p[kept])  # a path's rows land at their own positions
        vtmu.paged_write(kp, vp, kr, dev(v), slots)
        assert lens.cpu().tolist() == [len(x[0]) for x in dense]
    assert int(left) == pages - sum(-(-len(x[0]) // P) for x in dense)
    assert vtmu.vtmu_device_error() == 0


# --------------------------------------------------------------- far corners
@BOTH
@pytest.mark.parametrize("c", [
    ([100, 70], [64, 40], 64, 1, 128, 16, True, {}),     # 4096 virtual rows per KV head: four rounds of a team
    ([100, 70], [64, 3], 71, 1, 64, 32, True, {}),        # a prime group
    ([1300], [1100], 8, 1, 64, 64, False, {}),            # a prompt's chunk
    ([40, 90], [3, 5], 130, 1, 128, 8, False, {}),        # more heads than a row block has rows
])
def test_many_virtual_rows(kernel, c):
    run_case(c, kernel, seed=31)


@BOTH
@pytest.mark.parametrize("tree", [False, True])
def test_a_window_beyond_every_position_is_none(kernel, tree):
    d = ref.batch(32, [150, 20], [5, 9], tree=tree, **KW)
    whole = attend(d, kernel=kernel, **KW)
    for window in (1 << 20, (1 << 63) - 1):
        assert np.array_equal(attend(d, kernel=kernel, window=window, sinks=3, **KW), whole)


@BOTH
def test_max_rows_far_above_the_rows(kernel):
    d = ref.batch(33, [150, 20], [1, 1], **KW)
    check(attend(d, kernel=kernel, maxRows=1 << 27, **KW), expect(d, **KW))


def test_paged_write_of_one_slot_twice():
    kp, vp = torch.zeros(4, 1024, device="cuda"), torch.zeros(4, 1024, device="cuda")
    kn = torch.arange(1., 4., device="cuda")[:, None].expand(3, 1024).contiguous()
    vtmu.paged_write(kp, vp, kn, -kn, dev(np.array([2, 2, 0], np.int32)))
    k, v = kp.cpu().numpy(), vp.cpu().numpy()
    assert np.all((k[2] == 1) | (k[2] == 2)) and np.all((v[2] == -1) | (v[2] == -2))
    assert np.all(k[0] == 3) and np.all(v[0] == -3) and not k[[1, 3]].any() and not v[[1, 3]].any()


def test_helpers_captured_and_replayed():
    """page_map, tree_plan, rope_at and paged_write in one graph, replayed with another step's inputs."""
    H, D, P, cols = 2, 64, 16, 6
    kw = dict(rows=9, pageSize=P)
    steps = [([5, 30], [0, 4, 9]), ([0, 47], [0, 1, 6])]
    lens, cu = dev(np.zeros(2, np.int32)), dev(np.zeros(3, np.int32))
    table0 = np.array([[0, 1, -1, -1, -1, -1], [2, 3, 4, -1, -1, -1]], np.int32)
    table, free, n_free = dev(table0), dev(np.arange(5, 13, dtype=np.int32)), dev(np.array([8], np.int32))
    parents = dev(np.array([-1, 0, 0, 1, -1, 0, 1, 2, 3], np.int32))
    x = torch.randn(9, H * D, device="cuda")
    kp, vp = torch.zeros(13 * P, H * D, device="cuda"), torch.zeros(13 * P, H * D, device="cuda")

    def step():
        slots, pos, new, left = vtmu.page_map(lens, cu, table, free, n_free, **kw)
        masks, tpos = vtmu.tree_plan(parents, cu, lens)
        turned = vtmu.rope_at(x, pos, headDim=D, out=x.clone())
        vtmu.paged_write(kp, vp, turned, x, slots)
        return slots, pos, new, left, masks, tpos, turned

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = step()
    for l, c in steps + steps[:1]:
        lens.copy_(dev(np.array(l, np.int32)))
        cu.copy_(dev(np.array(c, np.int32)))
        outs, pools = [], []
        for run in (step, lambda: (g.replay(), got)[1]):
            table.copy_(dev(table0))
            kp.zero_()
            vp.zero_()
            outs.append([t.cpu().numpy() for t in run()])
            pools.append((kp.cpu().numpy(), vp.cpu().numpy(), table.cpu().numpy()))
        for a, b in zip(outs[0] + list(pools[0]), outs[1] + list(pools[1])):
            assert np.array_equal(a, b)
        want = ref.page_map(l, c, table0, np.arange(5, 13), 8, 9, P)
        assert np.array_equal(outs[0][0], want[0]) and np.array_equal(pools[0][2], want[4])
