"""Calls without a workspace of their own: on two streams and threads, and in captured
graphs, none of which may share scratch with another.  Tolerances as in test_gpu_paged."""
import threading

import numpy as np
import pytest

import paged_ref as ref

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import f32_gqa_attention_gb300 as vtmu  # noqa: E402
from test_gpu_paged import check, dev, expect, kw_of  # noqa: E402

pytestmark = pytest.mark.gpu


def paged(seed, lens, counts, **shape):
    """(a paged call without a workspace, its 64-bit result): units of both kinds, whole and cut."""
    kw = kw_of(8, 2, 128, 64, **shape)
    d = ref.batch(seed, lens, counts, heads=8, kvHeads=2, headDim=128, pageSize=64, tree=True)
    ins = [dev(d[k]) for k in ("q", "k_pool", "v_pool", "table", "lens", "cu")]
    tree = tuple(dev(x) for x in d["tree"])
    return lambda **more: vtmu.paged_attention(*ins, tree=tree, maxRows=max(counts), **kw, **more), expect(d, **kw)


def decode(seed, S):
    """The same for op attention's split-KV decode, whose launches count arrivals in the workspace."""
    g = np.random.default_rng(seed)
    q, k, v = (g.standard_normal(s, dtype=np.float32) for s in ((1, 1024), (S, 256), (S, 256)))
    d = dict(q=q, k_pool=k, v_pool=v, table=np.arange(S, dtype=np.int32)[None], lens=np.array([S]), cu=np.array([0, 1]), tree=None)
    want = expect(d, heads=8, kvHeads=2, headDim=128, pageSize=1)
    t = [dev(x) for x in (q, k, v)]
    return lambda **more: vtmu.attention(*t, heads=8, kvHeads=2, headDim=128, posOffset=S - 1, **more), want


CALLS = [lambda: paged(60, [2000, 700], [3, 30]), lambda: paged(61, [9000], [64]), lambda: decode(62, 20000), lambda: decode(63, 333)]
PAIRS = [(0, 1), (2, 3), (0, 2), (1, 1)]


def warm(calls):
    for call, want in calls:
        check(call(workspace=vtmu.Workspace()).cpu().numpy(), want)


@pytest.mark.parametrize("pair", PAIRS)
def test_two_streams(pair):
    calls = [CALLS[i]() for i in pair]
    warm(calls)
    streams, outs = [torch.cuda.Stream() for _ in calls], [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for (call, _), st, out in zip(calls, streams, outs):
            with torch.cuda.stream(st):
                out.append(call())
    torch.cuda.synchronize()
    for (_, want), out in zip(calls, outs):
        for o in out:
            check(o.cpu().numpy(), want)
    assert vtmu.vtmu_device_error() == 0


def test_a_stream_given_as_a_handle():
    """`stream=` beside another current stream: the scratch is that stream's, cleared on it."""
    calls = [CALLS[i]() for i in (0, 2)]
    warm(calls)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty(want.shape, device="cuda") for _ in range(10)] for _, want in calls]
    torch.cuda.synchronize()
    for i in range(10):
        for (call, _), st, out in zip(calls, streams, outs):
            call(stream=st.cuda_stream, out=out[i])
    torch.cuda.synchronize()
    for (_, want), out in zip(calls, outs):
        for o in out:
            check(o.cpu().numpy(), want)


def test_two_threads_on_one_stream():
    calls = [CALLS[i]() for i in (0, 1)]
    warm(calls)
    outs, st = [[], []], torch.cuda.Stream()
    gate = threading.Barrier(2)

    def work(i):
        gate.wait()
        with torch.cuda.stream(st):
            for _ in range(50):
                outs[i].append(calls[i][0]())

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for (_, want), out in zip(calls, outs):
        assert len(out) == 50
        for o in out:
            check(o.cpu().numpy(), want)


def capture(call, st):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        out = call()
    return g, out


@pytest.mark.parametrize("pair", PAIRS)
def test_two_graphs_replayed_at_once(pair):
    """Captured on one stream, replayed on two, with calls on a third."""
    calls = [CALLS[i]() for i in pair]
    warm(calls)
    streams, side = [torch.cuda.Stream() for _ in range(2)], torch.cuda.Stream()
    graphs = [capture(call, side) for call, _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        with torch.cuda.stream(side):
            eager = calls[0][0]()
    torch.cuda.synchronize()
    for (_, want), (_, out) in zip(calls, graphs):
        check(out.cpu().numpy(), want)
    check(eager.cpu().numpy(), calls[0][1])
    assert vtmu.vtmu_device_error() == 0


@pytest.mark.parametrize("i", range(len(CALLS)))
def test_a_first_call_inside_a_capture(i):
    """The stream's own buffer comes later, outside the graph's memory, and cleared."""
    call, want = CALLS[i]()
    warm([(call, want)])
    st = torch.cuda.Stream()
    g, out = capture(call, st)
    for _ in range(2):
        with torch.cuda.stream(st):
            eager = call()
        g.replay()
        torch.cuda.synchronize()
        check(eager.cpu().numpy(), want)
        check(out.cpu().numpy(), want)
    del g, out
    torch.cuda.empty_cache()
    with torch.cuda.stream(st):
        eager = call()
    torch.cuda.synchronize()
    check(eager.cpu().numpy(), want)


@pytest.mark.parametrize("i", [0, 2])
def test_a_captured_workspace_that_grows_later(i):
    """The graph goes on with the buffer that it was captured with."""
    call, want = CALLS[i]()
    ws = vtmu.Workspace()
    check(call(workspace=ws).cpu().numpy(), want)
    g, out = capture(lambda: call(workspace=ws), torch.cuda.Stream())
    old = ws.buf.data_ptr()
    ws.get(4 * ws.buf.numel())
    assert ws.buf.data_ptr() != old
    torch.cuda.empty_cache()
    fill = [torch.full((ws.buf.numel() // 16,), -1, dtype=torch.int32, device="cuda") for _ in range(8)]
    assert all(not (f.data_ptr() <= old < f.data_ptr() + 4 * f.numel()) for f in fill)
    g.replay()
    torch.cuda.synchronize()
    check(out.cpu().numpy(), want)
    assert all(int(f.min()) == int(f.max()) == -1 for f in fill)


@pytest.mark.parametrize("i", [0, 2])
def test_a_workspace_that_is_too_small_in_a_capture(i):
    call, want = CALLS[i]()
    warm([(call, want)])
    ws = vtmu.Workspace()
    g, out = capture(lambda: call(workspace=ws), torch.cuda.Stream())
    assert ws.buf is None
    for _ in range(2):
        g.replay()
    check(call(workspace=ws).cpu().numpy(), want)
    torch.cuda.synchronize()
    check(out.cpu().numpy(), want)
