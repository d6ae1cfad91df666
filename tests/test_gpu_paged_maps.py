"""Requests' rows from offsets that do not start at 0 or that fall, sizes past 32 bits,
and page_map after a call that ran out of pages, against what the definitions say.  Whole numbers are exact, attention as in test_gpu_paged."""
import numpy as np
import pytest

import paged_ref as ref

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import f32_gqa_attention_gb300 as vtmu  # noqa: E402
from test_gpu_paged import BOTH, CUDA, KW, attend, check, dev, expect  # noqa: E402

pytestmark = pytest.mark.gpu


def filled(n, dtype):
    """Outputs that hold something a call has to replace."""
    return torch.full((n,), 77, dtype=dtype, device="cuda")


def call_page_map(lens, cu, table, free, n_free, rows, page, accept=None):
    n, most = table.shape
    slots, pos, new, left = (filled(k, torch.int32) for k in (rows, rows, n, 1))
    vtmu.vtmu_page_map(dev(np.array(lens, np.int32)), dev(np.array(cu, np.int32)), dev(accept), table, dev(free), len(free),
                       dev(np.array([n_free], np.int32)), slots, pos, new, left, n, rows, page, most)
    return [t.cpu().numpy() for t in (slots, pos, new)] + [int(left), table.cpu().numpy()]


def call_tree_plan(parents, cu, lens):
    masks, pos = filled(len(parents), torch.int64), filled(len(parents), torch.int32)
    vtmu.vtmu_tree_plan(dev(parents), dev(np.array(cu, np.int32)), dev(np.array(lens, np.int32)), masks, pos, len(lens),
                        len(parents))
    return masks.cpu().numpy().view(np.uint64), pos.cpu().numpy()


def as_rising(cu, rows):
    """The rows that each request has: those from cu[b] to cu[b + 1] that lie between cu[0]
    and cu[-1]; (first, count) pairs."""
    cu = np.clip(np.asarray(cu, np.int64), 0, rows)
    out = []
    for a, e in zip(cu, cu[1:]):
        a, e = max(a, cu[0]), min(e, cu[-1])
        out.append((int(a), max(int(e - a), 0)))
    return out


OFFSETS = [[3, 8, 8, 12], [40, 45, 60], [1, 1], [70, 70, 70], [5, 600, 601]]                     # a slice of a larger batch's
FALLING = [[0, 5, 2], [4, 9, 3], [8, 3, 9, 6], [6, 2], [0, 9, 9, 4], [9, 20, 700, 11]]


@pytest.mark.parametrize("cu", OFFSETS + FALLING)
@pytest.mark.parametrize("accepted", [False, True])
def test_page_map_covers_every_row(cu, accepted):
    """Rows before the first request's, behind the last one's or of none get slot -1, position -1."""
    rows, page, n = 650, 4, len(cu) - 1
    lens = np.arange(3, 3 + n) * 5
    table = np.full((n, 300), -1, np.int32)
    ids = np.random.default_rng(1).permutation(400).astype(np.int32)
    held = [-(-int(x) // page) for x in lens]
    for b in range(n):
        table[b, :held[b]] = ids[b * 20:b * 20 + held[b]]
    accept = np.full(n, 0b1011011, np.uint64) if accepted else None
    have = as_rising(cu, rows)
    packed = np.concatenate([[0], np.cumsum([c for _, c in have])])  # the same requests one after the other from row 0 on
    total = int(packed[-1])
    want = ref.page_map(lens, packed, table, ids[100:], 300, total, page, accept)
    slots, pos = np.full(rows, -1, np.int32), np.full(rows, -1, np.int32)
    for (a, c), p in zip(have, packed):
        slots[a:a + c], pos[a:a + c] = want[0][p:p + c], want[1][p:p + c]
    got = call_page_map(lens, cu, dev(table), ids[100:], 300, rows, page, accept)
    assert np.array_equal(got[0], slots) and np.array_equal(got[1], pos)
    assert np.array_equal(got[2], want[2]) and got[3] == want[3] and np.array_equal(got[4], want[4])


@pytest.mark.parametrize("cu", OFFSETS + FALLING)
def test_tree_plan_covers_every_row(cu):
    """Rows of no request get mask 0, position -1."""
    rows, n = 650, len(cu) - 1
    parents = np.random.default_rng(2).integers(-1, 40, rows).astype(np.int32)
    lens = np.arange(n) * 9
    masks, pos = np.zeros(rows, np.uint64), np.full(rows, -1, np.int32)
    for b, (a, c) in enumerate(as_rising(cu, rows)):
        masks[a:a + c], pos[a:a + c] = ref.tree_plan(parents[a:a + c], [0, c], lens[b:b + 1])
    got = call_tree_plan(parents, cu, lens)
    assert np.array_equal(got[0], masks) and np.array_equal(got[1], pos)


@BOTH
@pytest.mark.parametrize("tree", [False, True])
def test_attention_writes_the_requests_rows_alone(kernel, tree):
    """Offsets that start above 0, and a falling pair at the end: the rows outside stay as they were."""
    d = ref.batch(34, [90, 40, 33], [7, 4, 0], tree=tree, **KW)
    want = expect(d, **KW)
    d["cu"] = np.array([7, 11, 9], np.int32)  # request 0: rows 7 and 8; request 1: none
    d["lens"], d["table"] = d["lens"][1:], d["table"][1:]
    out = torch.full(d["q"].shape, 5.0, device="cuda")
    got = attend(d, kernel=kernel, out=out, maxRows=7, **KW)
    assert np.all(got[:7] == 5.0) and np.all(got[9:] == 5.0)
    if tree:  # both rows' masks are of rows that they have
        check(got[7:9], want[7:9])
    else:     # two rows, where there were four: positions 38 and 39
        d["cu"] = np.array([0, 2], np.int32)
        d["q"], d["lens"], d["table"] = d["q"][7:9], d["lens"][:1], d["table"][:1]
        check(got[7:9], expect(d, **KW))


@BOTH
@pytest.mark.parametrize("most", [(1 << 31) - 1, 1 << 31, 1 << 32, (1 << 40) + 1])
def test_max_rows_past_32_bits(kernel, most):
    """A bound is a bound, whatever its size; a negative one is refused."""
    d = ref.batch(35, [150, 20], [4, 1], **KW)
    check(attend(d, kernel=kernel, maxRows=most, **KW), expect(d, **KW))
    with pytest.raises(vtmu.VtmuError):
        attend(d, kernel=kernel, maxRows=-most, **KW)


@pytest.mark.parametrize("page", [0, -16, 1 << 31, (1 << 32) + 16])
def test_page_sizes_out_of_range_are_refused(page):
    d = ref.batch(36, [150, 20], [4, 1], **KW)
    with pytest.raises((ValueError, vtmu.VtmuError)):
        vtmu.page_map(dev(d["lens"]), dev(d["cu"]), dev(d["table"]), dev(np.arange(9, dtype=np.int32)),
                      dev(np.array([9], np.int32)), rows=5, pageSize=page)
    with pytest.raises((ValueError, vtmu.VtmuError)):
        attend(dict(d, k_pool=d["k_pool"][:0], v_pool=d["v_pool"][:0]), kernel=CUDA, **dict(KW, pageSize=page))


def test_page_map_again_after_a_shortage():
    """A call that ran out of pages reads its inputs alone: once pages have come back, the same
    lengths and the same stack give every row its page, over the entries that were -1."""
    page, rows = 4, 40
    lens, cu = [6, 9, 0], [0, 15, 22, 40]
    ids = np.random.default_rng(3).permutation(40).astype(np.int32)
    table = np.full((3, 8), -1, np.int32)
    table[0, :2], table[1, :3] = ids[:2], ids[2:5]
    free = ids[5:].copy()
    t = dev(table)
    got = call_page_map(lens, cu, t, free, 5, rows, page)
    want = ref.page_map(lens, cu, table, free, 5, rows, page)
    assert got[3] == want[3] == -5  # pages for 21, 16 and 18 rows, less those held: 4 + 1 + 5, of 5
    assert all(np.array_equal(a, b) for a, b in zip(got[:3] + got[4:], want[:3] + want[4:]))
    assert (got[0][:40] == -1).sum() == (want[0] == -1).sum() > 0
    left = 5
    for page_id in free[30:35]:  # the pages come back, to the top of the stack
        free[left] = page_id
        left += 1
    got = call_page_map(lens, cu, t, free, left, rows, page)
    want = ref.page_map(lens, cu, table, free, left, rows, page)
    assert got[3] == want[3] == 0 and np.all(got[0] >= 0)
    assert all(np.array_equal(a, b) for a, b in zip(got[:3] + got[4:], want[:3] + want[4:]))
