"""The paged-cache operators on the host (no GPU): refusals before any launch, the
workspace's size, and the plain implementations that the GPU tests compare with."""
import numpy as np
import pytest

import f32_gqa_attention_gb300 as vtmu
import paged_ref as ref
from test_abi_host import FAKE, _err, host_only, lib  # noqa: F401

INV, UNS, WS = vtmu.VTMU_ERR_INVALID, vtmu.VTMU_ERR_UNSUPPORTED, vtmu.VTMU_ERR_WORKSPACE
A = [FAKE * (i + 1) for i in range(16)]  # addresses far from each other


def params(**kw):
    p = vtmu.vtmu_paged_params_init()
    for k, v in dict(dict(rows=5, pages=100, requests=2, max_rows=3, page_size=16, max_pages=10, heads=4, kv_heads=2,
                          head_dim=128), **kw).items():
        setattr(p, k, v)
    return p


def attend(p, q=A[0], k=A[1], v=A[2], table=A[3], lens=A[4], cu=A[5], kn=None, vn=None, masks=None, pos=None, out=A[6],
           ws=A[7], nbytes=1 << 40):
    vtmu.vtmu_paged_attention(q, k, v, table, lens, cu, kn, vn, masks, pos, out, p, ws, nbytes)


def test_params_init_writes_zeros(lib):  # noqa: F811
    p = vtmu.vtmu_paged_params_init()
    assert all(getattr(p, f[0]) == 0 for f in vtmu.vtmu_paged_params._fields_)


@pytest.mark.parametrize("kw,status,word", [
    (dict(rows=-1), INV, "rows"), (dict(pages=-1), INV, "pages"), (dict(requests=0), INV, "requests"),
    (dict(max_rows=-1), INV, "max_rows"), (dict(page_size=0), INV, "page_size"), (dict(max_pages=0), INV, "max_pages"),
    (dict(heads=0), INV, "heads"), (dict(heads=5), INV, "multiple of kvHeads"), (dict(kv_heads=-2), INV, "kvHeads"),
    (dict(head_dim=0), INV, "headDim"), (dict(head_dim=257), UNS, "headDim 257"), (dict(tree=2), INV, "tree"),
    (dict(has_scale=1, scale=float("inf")), INV, "scale"), (dict(softcap=-1.0), INV, "softcap"),
    (dict(softcap=float("nan")), INV, "softcap"), (dict(window=-1), INV, "window"), (dict(sinks=-1), INV, "sinks"),
    (dict(kernel=3), INV, "kernel"), (dict(requests=1025), UNS, "1025 requests"), (dict(tree=1, max_rows=65), UNS, "65 rows"),
    (dict(pages=1 << 30), UNS, "2^31"), (dict(max_pages=1 << 30), UNS, "2^31"), (dict(rows=1 << 31), UNS, "2^31"),
    (dict(heads=65536, kv_heads=1), UNS, "65535"),
    (dict(kernel=2, head_dim=96), UNS, "TENSOR_CORES"), (dict(kernel=2, page_size=24), UNS, "TENSOR_CORES"),
])
def test_parameters_are_refused(lib, kw, status, word):  # noqa: F811
    e = _err(lambda: vtmu.vtmu_paged_workspace_size(params(**kw)))
    assert e.status == status and word in str(e), str(e)
    assert word in vtmu.vtmu_last_error()


def test_workspace_size(lib):  # noqa: F811
    """Partials for the tensor cores whatever the lengths; none for the CUDA cores."""
    assert vtmu.vtmu_paged_workspace_size(params(kernel=1)) == 0
    assert vtmu.vtmu_paged_workspace_size(params(head_dim=96)) == 0
    n = vtmu.vtmu_paged_workspace_size(params())
    assert n > 64 * 1024 and n == vtmu.vtmu_paged_workspace_size(params(rows=1 << 20, requests=900, max_rows=4000))


@host_only
@pytest.mark.parametrize("kw,status,word", [
    (dict(q=None), INV, "NULL"), (dict(out=None), INV, "NULL"), (dict(lens=None), INV, "NULL"), (dict(cu=None), INV, "NULL"),
    (dict(table=None), INV, "NULL"), (dict(k=None), INV, "NULL"), (dict(v=None), INV, "NULL"),
    (dict(q=A[0] + 2), INV, "misaligned"), (dict(lens=A[4] + 1), INV, "misaligned"),
    (dict(kn=A[8]), INV, "disagree"), (dict(masks=A[8]), INV, "disagree"), (dict(pos=A[8]), INV, "disagree"),
    (dict(out=A[0]), INV, "overlaps"), (dict(out=A[1] + 64), INV, "overlaps"), (dict(out=A[3]), INV, "overlaps"),
    (dict(ws=None), WS, "workspace"), (dict(nbytes=100), WS, "workspace"), (dict(ws=A[7] + 128), WS, "aligned"),
])
def test_attention_pointers_are_refused(lib, kw, status, word):  # noqa: F811
    e = _err(lambda: attend(params(), **kw))
    assert e.status == status and word in str(e), str(e)


@host_only
@pytest.mark.parametrize("kw,word", [
    (dict(), "disagree"), (dict(kn=A[8], vn=A[9]), "disagree"), (dict(kn=A[8], masks=A[10]), "disagree"),
    (dict(kn=A[8], vn=A[9], masks=A[10]), "disagree"),  # a window needs the positions
    (dict(kn=A[8], vn=A[9], masks=A[10] + 4, pos=A[11]), "misaligned"),
])
def test_tree_arguments_are_refused(lib, kw, word):  # noqa: F811
    e = _err(lambda: attend(params(tree=1, window=4), **kw))
    assert e.status == INV and word in str(e), str(e)


@host_only
def test_forced_tensor_cores_want_aligned_tensors(lib):  # noqa: F811
    e = _err(lambda: attend(params(kernel=2), k=A[1] + 4))
    assert e.status == UNS and "16-byte" in str(e)


@host_only
def test_nothing_to_do(lib):  # noqa: F811
    attend(params(rows=0), q=None, out=None, lens=None)
    attend(params(max_rows=0), q=None, out=None, lens=None)
    vtmu.vtmu_rope_at(None, None, 0, 1, None, vtmu.make_rope_params(headDim=4))
    vtmu.vtmu_paged_write(None, None, 10, 4, 4, None, None, None, 0)
    vtmu.vtmu_tree_plan(None, A[0], A[1], None, None, 3, 0)


@host_only
@pytest.mark.parametrize("change,word", [
    (dict(requests=-1), "negative"), (dict(rows=-1), "negative"), (dict(cap=-1), "negative"), (dict(page=0), "page_size"),
    (dict(cols=0), "max_pages"), (dict(cu=None), "NULL"), (dict(lens=None), "NULL"), (dict(n_free=None), "NULL"),
    (dict(slots=None), "NULL"), (dict(free=None), "NULL"), (dict(out=None), "NULL"), (dict(accept=A[9] + 4), "misaligned"),
    (dict(slots=A[5] + 2), "misaligned"), (dict(slots=A[0]), "overlaps"), (dict(new=A[0]), "overlaps"),
    (dict(out=A[4]), "overlaps"), (dict(pos=A[5] + 16), "overlaps"), (dict(new=A[2]), "overlaps"),
])
def test_page_map_refusals(lib, change, word):  # noqa: F811
    c = dict(dict(lens=A[0], cu=A[1], accept=None, table=A[2], free=A[3], cap=50, n_free=A[4], slots=A[5], pos=A[6], new=A[7],
                  out=A[8], requests=4, rows=20, page=16, cols=8), **change)
    e = _err(lambda: vtmu.vtmu_page_map(c["lens"], c["cu"], c["accept"], c["table"], c["free"], c["cap"], c["n_free"],
                                        c["slots"], c["pos"], c["new"], c["out"], c["requests"], c["rows"], c["page"], c["cols"]))
    assert e.status == INV and word in str(e), str(e)


@host_only
@pytest.mark.parametrize("args,word", [
    ((A[0], A[1], A[2], A[3], A[4], -1, 5), "negative"), ((A[0], A[1], A[2], A[3], A[4], 2, -5), "negative"),
    ((None, A[1], A[2], A[3], A[4], 2, 5), "NULL"), ((A[0], None, A[2], A[3], A[4], 2, 5), "NULL"),
    ((A[0], A[1], None, A[3], A[4], 2, 5), "NULL"), ((A[0], A[1], A[2], A[3] + 4, A[4], 2, 5), "misaligned"),
    ((A[0], A[1], A[2], A[0], A[4], 2, 5), "overlaps"), ((A[0], A[1], A[2], A[3], A[3] + 8, 2, 5), "overlaps"),
])
def test_tree_plan_refusals(lib, args, word):  # noqa: F811
    e = _err(lambda: vtmu.vtmu_tree_plan(*args))
    assert e.status == INV and word in str(e), str(e)


@host_only
@pytest.mark.parametrize("args,status", [
    ((A[0], A[1], -1, 2, A[2]), INV), ((A[0], A[1], 3, 0, A[2]), INV), ((None, A[1], 3, 2, A[2]), INV),
    ((A[0], A[1], 3, 2, None), INV), ((A[0], A[1], 3, 2, A[2] + 2), INV), ((A[0], A[0] + 16, 3, 2, A[2]), INV),
    ((A[0], A[1], 3, 2, A[1] + 16), INV)])
def test_rope_at_refusals(lib, args, status):  # noqa: F811
    x, out, T, heads, pos = args
    e = _err(lambda: vtmu.vtmu_rope_at(x, out, T, heads, pos, vtmu.make_rope_params(headDim=64)))
    assert e.status == status


@host_only
def test_rope_at_checks_the_rope_parameters(lib):  # noqa: F811
    e = _err(lambda: vtmu.vtmu_rope_at(A[0], A[1], 3, 2, A[2], vtmu.make_rope_params(headDim=64, rotaryDim=65)))
    assert e.status == INV and "rotaryDim" in str(e)


@host_only
@pytest.mark.parametrize("args,status,word", [
    ((A[0], A[1], -1, 4, 4, A[2], A[3], A[4], 2), INV, "negative"), ((A[0], A[1], 9, 4, 4, A[2], A[3], A[4], -2), INV, "negative"),
    ((None, A[1], 9, 4, 4, A[2], A[3], A[4], 2), INV, "NULL"), ((A[0], A[1], 9, 4, 4, A[2], None, A[4], 2), INV, "NULL"),
    ((A[0], A[1], 9, 4, 4, A[2], A[3], None, 2), INV, "NULL"), ((A[0], A[1], 9, 4, 4, A[2] + 1, A[3], A[4], 2), INV, "aligned"),
    ((A[0], A[0] + 16, 9, 4, 4, A[2], A[3], A[4], 2), INV, "overlaps"), ((A[0], A[1], 9, 4, 4, A[0] + 16, A[3], A[4], 2), INV, "overlaps"),
    ((A[0], A[1], 9, 4, 4, A[2], A[3], A[1], 2), INV, "overlaps"), ((A[0], A[1], 1 << 31, 4, 4, A[2], A[3], A[4], 2), UNS, "2^31"),
])
def test_paged_write_refusals(lib, args, status, word):  # noqa: F811
    e = _err(lambda: vtmu.vtmu_paged_write(*args))
    assert e.status == status and word in str(e), str(e)


def test_other_kernels_do_not_include_the_paged_ones():
    """The profiles that the bench quotes record the sources of their kernels, headers included."""
    import glob
    import os
    csrc = os.path.join(os.path.dirname(vtmu.__file__), "csrc")
    for path in glob.glob(os.path.join(csrc, "*")):
        if not os.path.basename(path).startswith("paged") and path.endswith((".cu", ".cuh", ".h")):
            assert '#include "paged' not in open(path).read(), path


# -------------------------------------------------- the plain implementations
def test_plain_tree_plan_by_hand():
    #    0 -> 1 -> 3, 0 -> 2, and a second root 4 -> 5
    masks, pos = ref.tree_plan(np.array([-1, 0, 0, 1, -1, 4], np.int32), [0, 6], [10])
    assert masks.tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10000, 0b110000]
    assert pos.tolist() == [10, 11, 11, 12, 10, 11]


def test_plain_page_map_by_hand():
    """Two rows fit the held page of request 0, its third opens a page; request 1 opens one first."""
    table = np.array([[7, -1], [-1, -1]], np.int32)
    slots, pos, lens, left, t = ref.page_map([2, 0], [0, 3, 5], table, [1, 9, 5], 3, 6, 4)
    assert slots.tolist() == [30, 31, 20, 36, 37, -1] and pos.tolist() == [2, 3, 4, 0, 1, -1]
    assert lens.tolist() == [5, 2] and left == 1 and t.tolist() == [[7, 5], [9, -1]]
    slots, pos, lens, left, t = ref.page_map([2, 0], [0, 3, 5], table, [1, 9, 5], 3, 5, 4, [0b101, 0])
    assert slots.tolist() == [30, -1, 31, -1, -1] and lens.tolist() == [4, 0] and left == 3


def test_plain_attention_of_a_tree_is_a_chain_for_each_path():
    """A node's row equals plain causal attention over its own path."""
    kw = dict(heads=2, kvHeads=1, headDim=4, pageSize=2)
    d = ref.batch(3, [5], [7], tree=True, **kw)
    want = ref.attention(d["q"], d["k_pool"], d["v_pool"], d["table"], d["lens"], d["cu"], tree=d["tree"], **kw)
    for t in range(7):
        path = [j for j in range(7) if (int(d["tree"][2][t]) >> j) & 1]
        rows = [d["table"][0, s // 2] * 2 + s % 2 for s in range(5)]
        k = np.concatenate([d["k_pool"][rows], d["tree"][0][path]])
        v = np.concatenate([d["v_pool"][rows], d["tree"][1][path]])
        for h in range(2):
            x = k @ d["q"][t, 4 * h:4 * h + 4].astype(np.float64) / 2.0
            w = np.exp(x) / np.exp(x).sum()
            assert np.allclose(want[t, 4 * h:4 * h + 4], w @ v, atol=1e-6)
