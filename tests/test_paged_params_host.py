"""What the paged attentions and norm_rope hand to the library, on the host: numbers are read at
every call, whatever type they come in, and equal calls are answered alike.  The library's launches
are replaced by a record of their parameters."""
import contextlib

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import f32_gqa_attention_gb300 as vtmu  # noqa: E402
from test_abi_host import lib  # noqa: E402,F401

TARGETS = ["paged_attention", "paged_attention_q8"]


@pytest.fixture
def record(lib, monkeypatch):  # noqa: F811
    """CPU tensors go through the helpers; the params of each launch, copied at the call."""
    seen = []

    def keep(kind, at):
        def launch(*args):
            p = args[at]
            seen.append({f[0]: (list(getattr(p, f[0])) if f[0] == "sections" else getattr(p, f[0])) for f in kind._fields_
                         if f[0] != "rope"} | ({"base": p.rope.base, "factor": p.rope.attention_factor} if hasattr(p, "rope") else {}))
        return launch

    monkeypatch.setattr(vtmu, "_need", lambda *a: None)
    monkeypatch.setattr(vtmu, "_on", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(vtmu, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(vtmu, "_scratch", lambda *a, **kw: (None, 0))
    monkeypatch.setattr(vtmu, "vtmu_paged_attention", keep(vtmu.vtmu_paged_params, 11))
    monkeypatch.setattr(vtmu, "vtmu_paged_attention_q8", keep(vtmu.vtmu_paged_params, 14))
    monkeypatch.setattr(vtmu, "vtmu_norm_rope", keep(vtmu.vtmu_norm_rope_params, 10))
    return seen


def attend(which, **kw):
    q = torch.zeros(2, 4 * 64)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    args = dict(dict(heads=4, kvHeads=2, headDim=64, pageSize=16, maxRows=2), **kw)
    if which == "paged_attention":
        pools = [torch.zeros(32, 2 * 64) for _ in range(2)]
    else:
        pools = [torch.zeros(32, 2 * 64, dtype=torch.int8) for _ in range(2)] + [torch.zeros(32, 2) for _ in range(2)]
    getattr(vtmu, which)(q, *pools, i32(0, 1).view(1, 2), i32(20), i32(0, 2), **args)


@pytest.mark.parametrize("which", TARGETS)
@pytest.mark.parametrize("name", ["scale", "softcap"])
def test_a_scale_that_changes_in_place(record, which, name):
    t = torch.tensor(0.5)
    attend(which, **{name: t})
    t.fill_(0.25)
    attend(which, **{name: t})
    a = np.array(0.5)
    attend(which, **{name: a})
    a[...] = 2.0
    attend(which, **{name: a})
    assert [r[name] for r in record] == [0.5, 0.25, 0.5, 2.0]


@pytest.mark.parametrize("which", TARGETS)
@pytest.mark.parametrize("name", ["heads", "kvHeads", "headDim", "pageSize", "maxRows", "window", "sinks", "kernel"])
def test_whole_numbers_are_taken_alike_before_and_after_an_equal_call(record, which, name):
    value = dict(heads=4, kvHeads=2, headDim=64, pageSize=16, maxRows=1, window=32, sinks=3, kernel=1)[name]
    kw = dict(window=32, maxRows=2) | {name: value}
    for _ in range(2):  # the second time after an int call
        with pytest.raises(TypeError):
            attend(which, **dict(kw, **{name: float(value)}))
        for same in (value, np.int64(value), np.array(value), torch.tensor(value)):
            attend(which, **dict(kw, **{name: same}))
    assert len(record) == 8 and all(r == record[0] for r in record)


@pytest.mark.parametrize("name,field", [("eps", "eps"), ("weightOffset", "weight_offset"), ("base", "base"),
                                        ("attentionFactor", "factor")])
def test_norm_rope_numbers_that_change_in_place(record, name, field):
    q, pos = torch.zeros(3, 2 * 64), torch.zeros(3, dtype=torch.int32)
    t, a = torch.tensor(0.5), np.array(0.5)
    for x in (t, a):
        vtmu.norm_rope(q, None, pos, headDim=64, **{name: x})
        x[...] = 4.0
        vtmu.norm_rope(q, None, pos, headDim=64, **{name: x})
    assert [r[field] for r in record] == [0.5, 4.0, 0.5, 4.0]


def test_norm_rope_sections_that_change_in_place(record):
    q, pos = torch.zeros(3, 2 * 64), torch.zeros(2, 3, dtype=torch.int32)
    for s in ([20, 12], torch.tensor([20, 12]), np.array([20, 12])):
        vtmu.norm_rope(q, None, pos, headDim=64, sections=s)
        s[0], s[1] = 10, 22
        vtmu.norm_rope(q, None, pos, headDim=64, sections=s)
    assert [r["sections"] for r in record] == [[20, 12, 0, 0], [10, 22, 0, 0]] * 3
