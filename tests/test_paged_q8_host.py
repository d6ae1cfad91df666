"""The 8-bit paged cache and norm_rope on the host (no GPU): refusals before any
launch, defaults, and the plain implementations that the GPU tests compare with."""
import numpy as np
import pytest

import f32_gqa_attention_gb300 as vtmu
import paged_q8_ref as q8
from test_abi_host import FAKE, _err, host_only, lib  # noqa: F401
from test_paged_host import params

INV, UNS, WS = vtmu.VTMU_ERR_INVALID, vtmu.VTMU_ERR_UNSUPPORTED, vtmu.VTMU_ERR_WORKSPACE
A = [FAKE * (i + 1) for i in range(16)]


def call_write(kp=A[0], vp=A[1], ks=A[2], vs=A[3], total=64, hk=2, d=64, form=1, kn=A[4], vn=A[5], slots=A[6], rows=5):
    vtmu.vtmu_paged_write_q8(kp, vp, ks, vs, total, hk, d, form, kn, vn, slots, rows)


def call_read(kp=A[0], vp=A[1], ks=A[2], vs=A[3], total=64, hk=2, d=64, form=1, slots=A[6], kn=A[4], vn=A[5], rows=5):
    vtmu.vtmu_paged_read_q8(kp, vp, ks, vs, total, hk, d, form, slots, kn, vn, rows)


BOTH = [
    (dict(total=-1), INV, "bad size"), (dict(rows=-1), INV, "bad size"), (dict(hk=0), INV, "bad size"),
    (dict(d=0), INV, "bad size"), (dict(form=0), INV, "format 0"), (dict(form=3), INV, "format 3"),
    (dict(d=257), UNS, "257"), (dict(rows=1 << 31), UNS, "2^31"), (dict(total=1 << 31), UNS, "2^31"),
    (dict(hk=1 << 25), UNS, "2^31"), (dict(hk=1 << 24), UNS, "2^30"), (dict(rows=1 << 28, hk=8), UNS, "2^31"),
    (dict(kp=None), INV, "NULL"), (dict(vs=None), INV, "NULL"), (dict(kn=None), INV, "NULL"),
    (dict(slots=None), INV, "NULL"), (dict(ks=A[2] + 2), INV, "aligned"), (dict(kn=A[4] + 1), INV, "aligned"),
    (dict(kn=A[0] + 64), INV, "overlaps"), (dict(vn=A[6]), INV, "overlaps"), (dict(vn=A[3]), INV, "overlaps"),
]


@host_only
@pytest.mark.parametrize("call", [call_write, call_read])
@pytest.mark.parametrize("kw,status,word", BOTH)
def test_write_and_read_refusals(lib, call, kw, status, word):  # noqa: F811
    if call is call_write and kw == dict(vn=A[6]):
        return  # two inputs may overlap
    e = _err(lambda: call(**kw))
    assert e.status == status and word in str(e), str(e)


@host_only
def test_written_pools_are_apart(lib):  # noqa: F811
    for kw in (dict(vp=A[0]), dict(vs=A[2] + 4), dict(ks=A[0] + 8)):
        e = _err(lambda: call_write(**kw))
        assert e.status == INV and "overlaps" in str(e)


@host_only
def test_nothing_to_do(lib):  # noqa: F811
    call_write(kp=None, rows=0)
    call_write(kp=None, total=0)
    call_read(kp=None, rows=0)
    vtmu.vtmu_norm_rope(None, None, None, None, None, None, 0, 1, 0, None, vtmu.make_norm_rope_params(headDim=8))
    vtmu.vtmu_paged_attention_q8(None, None, None, None, None, 1, None, None, None, None, None, None, None, None,
                                 params(rows=0), None, 0)


def attend(p, q=A[0], k=A[1], v=A[2], ks=A[3], vs=A[4], form=1, table=A[5], lens=A[6], cu=A[7], kn=None, vn=None,
           masks=None, pos=None, out=A[8], ws=A[9], nbytes=1 << 40):
    vtmu.vtmu_paged_attention_q8(q, k, v, ks, vs, form, table, lens, cu, kn, vn, masks, pos, out, p, ws, nbytes)


@host_only
@pytest.mark.parametrize("kw,status,word", [
    (dict(q=None), INV, "NULL"), (dict(out=None), INV, "NULL"), (dict(lens=None), INV, "NULL"), (dict(cu=None), INV, "NULL"),
    (dict(table=None), INV, "NULL"), (dict(k=None), INV, "NULL"), (dict(vs=None), INV, "NULL"), (dict(form=0), INV, "format"),
    (dict(form=7), INV, "format"), (dict(q=A[0] + 2), INV, "misaligned"), (dict(ks=A[3] + 1), INV, "misaligned"),
    (dict(kn=A[10]), INV, "disagree"), (dict(masks=A[10]), INV, "disagree"), (dict(out=A[0]), INV, "overlaps"),
    (dict(out=A[1] + 64), INV, "overlaps"), (dict(out=A[4]), INV, "overlaps"), (dict(out=A[5]), INV, "overlaps"),
])
def test_attention_pointers_are_refused(lib, kw, status, word):  # noqa: F811
    e = _err(lambda: attend(params(), **kw))
    assert e.status == status and word in str(e), str(e)


@pytest.mark.parametrize("kw,status,word", [
    (dict(heads=5), INV, "multiple of kvHeads"), (dict(head_dim=257), UNS, "headDim 257"), (dict(rows=1 << 31), UNS, "2^31"),
    (dict(tree=1, max_rows=65), UNS, "65 rows"), (dict(kernel=2, head_dim=96), UNS, "TENSOR_CORES"),
    (dict(softcap=-1.0), INV, "softcap"),
])
def test_attention_parameters_are_refused(lib, kw, status, word):  # noqa: F811
    e = _err(lambda: vtmu.vtmu_paged_q8_workspace_size(params(**kw)))
    assert e.status == status and word in str(e), str(e)


def test_no_workspace_for_the_cuda_cores(lib):  # noqa: F811
    assert vtmu.vtmu_paged_q8_workspace_size(params(kernel=1)) == 0
    assert vtmu.vtmu_paged_q8_workspace_size(params(head_dim=96)) == 0


@host_only
def test_workspaces_are_refused(lib):  # noqa: F811
    for kw in (dict(), dict(max_rows=64, rows=64)):
        p = params(**kw)
        need = vtmu.vtmu_paged_q8_workspace_size(p)
        assert need > 0
        for ws, n in ((None, need), (A[9], need - 1), (A[9] + 128, need)):
            e = _err(lambda: attend(p, ws=ws, nbytes=n))
            assert e.status == WS, str(e)


@host_only
def test_forced_tensor_cores_are_refused(lib):  # noqa: F811
    for kw in (dict(q=A[0] + 4), dict(k=A[1] + 8), dict(v=A[2] + 1), dict(out=A[8] + 4)):
        e = _err(lambda: attend(params(kernel=2), **kw))
        assert e.status == UNS and "16-byte" in str(e), str(e)
    e = _err(lambda: vtmu.vtmu_paged_q8_workspace_size(params(kernel=2, pages=0)))
    assert e.status == UNS


def test_workspace_holds_the_drafted_rows_part(lib):  # noqa: F811
    for rows in (16, 64):
        more = [vtmu.vtmu_paged_q8_workspace_size(params(rows=n, max_rows=rows, tree=1)) for n in (64, 4096)]
        assert more[1] >= more[0] + (4096 - 64) * 8


def test_norm_rope_defaults(lib):  # noqa: F811
    p = vtmu.vtmu_norm_rope_params_init()
    assert (p.norm, p.axes, p.dealt, p.weight_offset, p.rope.base) == (1, 1, 0, 0.0, 0.0)  # base 0: 10000
    assert p.eps == np.float32(1e-6) and list(p.sections) == [0] * 4


def norm_rope(q=A[0], k=A[1], qw=A[2], kw=A[3], qo=A[4], ko=A[5], T=3, heads=4, kv=2, pos=A[6], **params_):
    vtmu.vtmu_norm_rope(q, k, qw, kw, qo, ko, T, heads, kv, pos, vtmu.make_norm_rope_params(**dict(dict(headDim=64), **params_)))


@host_only
@pytest.mark.parametrize("kw,status,word", [
    (dict(T=-1), INV, "T -1"), (dict(heads=0), INV, "heads 0"), (dict(kv=-1), INV, "kv_heads -1"),
    (dict(eps=-1.0), INV, "eps"), (dict(eps=float("nan")), INV, "eps"), (dict(weightOffset=float("inf")), INV, "weight_offset"),
    (dict(sections=[16] * 5), INV, "axes 5"), (dict(sections=[16, 15]), INV, "add up to 31"),
    (dict(sections=[40, -8]), INV, "negative"), (dict(sections=[10, 11, 11], dealt=True, T=3), INV, "dealt out"),
    (dict(rotaryDim=63), INV, "rotaryDim"), (dict(norm=False), INV, "weights without"), (dict(q=None), INV, "must be given"),
    (dict(pos=None), INV, "must be given"), (dict(k=None), INV, "must be given"), (dict(kv=0), INV, "must be given"),
    (dict(q=A[0] + 2), INV, "aligned"), (dict(qo=A[0] + 16), INV, "overlaps"), (dict(qo=A[1]), INV, "overlaps"),
    (dict(ko=A[4]), INV, "overlaps"), (dict(ko=A[6]), INV, "overlaps"), (dict(qo=A[2]), INV, "overlaps"),
    (dict(heads=1 << 25), UNS, "2^30"), (dict(heads=1 << 23, kv=1 << 23), UNS, "2^30"), (dict(T=1 << 31), UNS, "2^31"),
])
def test_norm_rope_refusals(lib, kw, status, word):  # noqa: F811
    e = _err(lambda: norm_rope(**kw))
    assert e.status == status and word in str(e), str(e)


# -------------------------------------------------- the plain implementations
def test_plain_e4m3_by_hand():
    v = q8.e4m3_values()
    assert v[0x38] == 1.0 and v[0x7e] == 448.0 and v[0x01] == 2.0 ** -9 and v[0xb8] == -1.0
    assert q8._e4m3_code(np.array([1.0, 1.0625, 1.1875, 448.0, -2.0 ** -10, 3 * 2.0 ** -10, 0.0])).tolist() == \
        [0x38, 0x38, 0x3a, 0x7e, 0x80, 2, 0]


def test_plain_quantise_by_hand():
    x = np.array([[1.27, -0.005, 0.015, 0.0, 448.5, 1.0, -449.0, 0.0]], np.float32)
    c, s = q8.quantise(x, 2, q8.INT8)
    assert s[0, 0] == np.float32(np.float32(1.27) / np.float64(127)) and c.view(np.int8)[0, [0, 3]].tolist() == [127, 0]
    c, s = q8.quantise(x, 2, q8.E4M3)
    assert s.tolist() == [[2.0 ** -8, 2.0]]  # 1.27 256 = 325 fits, 449 / 2 does and 449 does not
    c, s = q8.quantise(np.array([[np.inf, 1.0, 2.0, 0.0], [0, 0, 0, 0]], np.float32), 2, q8.E4M3)
    assert np.isnan(s[0, 0]) and s[0, 1] == 2.0 ** -7 and c[0, :2].tolist() == [0, 0] and s[1, 0] == 2.0 ** -126


def test_plain_axes_by_hand():
    assert q8.axis_of(4, None, False) == [0] * 4
    assert q8.axis_of(8, [3, 3, 2], False) == [0, 0, 0, 1, 1, 1, 2, 2]
    assert q8.axis_of(8, [4, 2, 2], True) == [0, 1, 2, 0, 1, 2, 0, 0]
