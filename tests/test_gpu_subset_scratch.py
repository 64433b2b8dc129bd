"""Calls over a part of the cache without workspace=, on streams that are not
joined, in graphs that are replayed beside one another and beside eager calls,
and after a wait that ran out in the binding's own buffer."""

import ctypes

import pytest
import torch

import paged_gqa_decode_reshape_gb300 as pg
from tests.test_gpu_subset import DEV, bf16, dev, pool, widened

pytestmark = pytest.mark.gpu
Hq, Hkv, D, SCALE = 28, 4, 128, 0.1
LENS = [6000, 5, 1700, 3000]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import paged_gqa_decode_reshape_gb300.build as b
    b.build()


def calls(seed):
    """Calls that cut their work and merge it by way of the workspace, writing to out; and out."""
    B = len(LENS)
    g, kc, vc, bt, _, _ = pool(seed, LENS + [900], Hkv, D)
    bt, pt = bt[:B].contiguous(), bt[B:].contiguous()
    w = torch.zeros(kc.shape[0], Hkv, 16)
    q_, kc_, vc_, bt_, pt_, w_ = dev(bf16(g, B, Hq, D), kc, vc, bt, widened(pt, B, Hkv, D), w)
    wide = widened(bt_, B, Hkv, D)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    ctx, cu, plen, cug = i32(*LENS), i32(0, 1, 2, 3, 4), i32(900), i32(0, 3)
    out = torch.zeros(4, B, Hq, D, dtype=torch.bfloat16, device=DEV)
    return [
        lambda: pg.pa_decode_window(out[0], q_, kc_, vc_, bt_, ctx, 5000, 4, SCALE),
        lambda: pg.pa_decode_window_multi(out[1], q_, kc_, vc_, wide, cu, ctx, 1 << 20, 0, SCALE),
        lambda: pg.pa_decode_prefix(out[2], q_, kc_, vc_, pt_, plen, cug, bt_, ctx, SCALE),
        lambda: pg.pa_decode_weights(out[3], w_, q_, kc_, vc_, bt_, ctx, SCALE),
    ], out


def bits(t):
    return t.view(torch.int16).clone()


def test_streams_that_are_not_joined():
    work = [calls(s) for s in (1, 2)]
    want = []
    for fs, out in work:
        for f in fs:
            f()
        torch.cuda.synchronize()
        want.append(bits(out))
        out.zero_()
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (fs, out) in zip(streams, work):
            with torch.cuda.stream(st):
                for f in fs:
                    f()
    torch.cuda.synchronize()
    for (fs, out), w in zip(work, want):
        assert torch.equal(bits(out), w)
    bufs = []
    for st in streams:
        with torch.cuda.stream(st):
            bufs.append(pg.partial_cache_workspace(torch.device(DEV)))
            assert pg.pa_workspace_status(bufs[-1]) == 0
    assert bufs[0].data_ptr() != bufs[1].data_ptr()


def test_graphs_beside_one_another_and_beside_eager_calls():
    work = [calls(s) for s in (3, 4, 5)]
    graphs, want, held = [], [], []
    for fs, out in work:
        for f in fs:
            f()
        torch.cuda.synchronize()
        want.append(bits(out))
        out.zero_()
    for fs, out in work[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for f in fs:
                f()
            held.append(pg.partial_cache_workspace())
        graphs.append(graph)
    assert held[0].data_ptr() != held[1].data_ptr()
    assert all(pg._in_graph_pool(h) for h in held) and not pg._in_graph_pool(pg.partial_cache_workspace())
    assert not any(t is h for t in pg._subset_ws._for_good for h in held)
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                if i < 2:
                    graphs[i].replay()
                else:
                    for f in work[2][0]:
                        f()
    torch.cuda.synchronize()
    for (fs, out), w in zip(work, want):
        assert torch.equal(bits(out), w)
    assert [pg.pa_workspace_status(h) for h in held] == [0, 0]


def test_a_forked_capture():
    """Two streams of one capture: a buffer each."""
    (fa, oa), (fb, ob) = calls(6), calls(7)
    for f in fa + fb:
        f()
    torch.cuda.synchronize()
    want = bits(oa), bits(ob)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        for f in fa:
            f()
        with torch.cuda.stream(side):
            for f in fb:
                f()
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(5):
        oa.zero_(), ob.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(oa), want[0]) and torch.equal(bits(ob), want[1])


def test_recovery_in_the_bindings_own_buffer():
    """A wait that ran out is seen in the buffer's status; zeroed, it serves again."""
    import paged_gqa_decode_reshape_gb300.build as pgb
    L, main = ctypes.CDLL(pgb.FAULT_LIB), pg.load_library()
    L.pa_decode_window.argtypes, L.pa_decode_window.restype = main.pa_decode_window.argtypes, ctypes.c_int
    L.pa_fault_test_configure.argtypes, L.pa_fault_test_configure.restype = [ctypes.c_int, ctypes.c_uint64], None
    B = len(LENS)
    g, kc, vc, bt, _, _ = pool(8, LENS, Hkv, D)
    q_, kc_, vc_, bt_, ctx_ = dev(bf16(g, B, Hq, D), kc, vc, bt, torch.tensor(LENS, dtype=torch.int32))
    out = torch.empty_like(q_)
    want = bits(pg.pa_decode_window(out, q_, kc_, vc_, bt_, ctx_, 5000, 4, SCALE))
    ws = pg.partial_cache_workspace(torch.device(DEV))
    assert pg.pa_workspace_status(ws) == 0
    torch.cuda.synchronize()
    L.pa_fault_test_configure(1, 200_000)
    rc = L.pa_decode_window(out.data_ptr(), q_.data_ptr(), kc_.data_ptr(), vc_.data_ptr(), bt_.data_ptr(), bt.shape[1],
                            ctx_.data_ptr(), B, Hq, Hkv, D, 16, kc.shape[0], 5000, 4, SCALE, ws.data_ptr(), ws.numel(),
                            torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and pg.pa_workspace_status(pg.partial_cache_workspace()) == -5
    L.pa_fault_test_configure(-1, 0)
    ws.zero_()
    assert torch.equal(bits(pg.pa_decode_window(out, q_, kc_, vc_, bt_, ctx_, 5000, 4, SCALE)), want)
    assert pg.pa_workspace_status(ws) == 0
