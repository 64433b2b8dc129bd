"""The bounded waits of the partial-cache decode kernels run out: the call
records PA_ERR_DEVICE, ends soon, and after zeroing the workspace the same
call gives the right result again. As in the dense decode's failure test, the
failure-test build stops the copies part-way, so that a wait for a stage that
is never filled runs out; nothing faults."""

import ctypes
import time

import pytest
import torch

import paged_gqa_decode_reshape_gb300 as pg
from tests import subset_reference as ref
from tests.test_gpu_subset import DEV, bf16, dev, pool

pytestmark = pytest.mark.gpu
PA_OK, PA_ERR_DEVICE = 0, -5
WAIT_NS = 200_000


@pytest.fixture(scope="module")
def flib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import paged_gqa_decode_reshape_gb300.build as pgb
    pgb.build()
    main = pg.load_library()
    L = ctypes.CDLL(pgb.FAULT_LIB)
    for n in ("pa_decode_window", "pa_decode_window_multi", "pa_decode_prefix", "pa_decode_weights",
              "pa_workspace_status"):
        getattr(L, n).argtypes = getattr(main, n).argtypes
        getattr(L, n).restype = ctypes.c_int
    L.pa_fault_test_configure.argtypes = [ctypes.c_int, ctypes.c_uint64]
    L.pa_fault_test_configure.restype = None
    yield L
    L.pa_fault_test_configure(-1, 0)


@pytest.mark.parametrize("stop_item", [0, 1])  # every warp and CTA here has at least two copies to make
@pytest.mark.parametrize("op", ["window", "window_many", "window_multi", "multi_many", "multi_each", "prefix", "prefix_each", "weights"])
def test_wait_runs_out_then_status_and_recovery(flib, op, stop_item):
    Hq, Hkv, D, scale = 28, 4, 128, 0.0884
    # window: a piece of a segment per CTA; window_many: a range of segments per warp
    # window_multi: cut units merged by a kernel of their own; multi_many: by the CTA of the last piece
    lens = [200] * 250 if op == "window_many" else [700] * 40 if op == "multi_many" else [3000, 1700, 2999, 800]
    B = len(lens)
    g, kc, vc, bt, _, _ = pool(7, lens + [900], Hkv, D)
    bt, pt = bt[:B].contiguous(), bt[B:].contiguous()
    # tables wide enough for the kernels that share reads between rows
    if op == "prefix":
        pt = torch.nn.functional.pad(pt, (0, 4096), value=-1)
    if op in ("window_multi", "multi_many"):
        bt = torch.nn.functional.pad(bt, (0, 4096), value=-1)
    q = bf16(g, B, Hq, D, std=2.0)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    q_, kc_, vc_, bt_, pt_ = dev(q, kc, vc, bt, pt)
    ctx, cu = i32(*lens), i32(*range(B + 1))
    w_ = torch.zeros(kc.shape[0], Hkv, 16, device=DEV)
    out = torch.empty_like(q_)
    MBS, NB = bt.shape[1], kc.shape[0]
    size = {"window_multi": lambda: pg.pa_decode_window_multi_workspace_size(B, B, Hq, Hkv, D),
            "multi_many": lambda: pg.pa_decode_window_multi_workspace_size(B, B, Hq, Hkv, D),
            "multi_each": lambda: pg.pa_decode_window_multi_workspace_size(B, B, Hq, Hkv, D),
            "prefix": lambda: pg.pa_decode_prefix_workspace_size(B, 1, Hq, Hkv, D),
            "prefix_each": lambda: pg.pa_decode_prefix_workspace_size(B, 1, Hq, Hkv, D),
            "weights": lambda: pg.pa_decode_weights_workspace_size(B, Hq, Hkv, D, MBS)}
    ws = torch.zeros(size.get(op, lambda: pg.pa_decode_window_workspace_size(B, Hq, Hkv, D))(), dtype=torch.uint8,
                     device=DEV)
    st = torch.cuda.current_stream().cuda_stream
    o, x, k, v, t, c = (y.data_ptr() for y in (out, q_, kc_, vc_, bt_, ctx))
    shape, tail = (Hq, Hkv, D, 16, NB), (scale, ws.data_ptr(), ws.numel(), st)

    def call():
        if op in ("window", "window_many"):
            rc = flib.pa_decode_window(o, x, k, v, t, MBS, c, B, *shape, 1 << 20, 0, *tail)
        elif op in ("window_multi", "multi_many", "multi_each"):
            rc = flib.pa_decode_window_multi(o, x, k, v, t, MBS, cu.data_ptr(), c, B, B, *shape, 1 << 20, 0, *tail)
        elif op in ("prefix", "prefix_each"):
            one, grp = i32(900), i32(0, B)
            rc = flib.pa_decode_prefix(o, x, k, v, pt_.data_ptr(), pt.shape[1], one.data_ptr(), grp.data_ptr(), 1, t,
                                       MBS, c, B, *shape, *tail)
        else:
            rc = flib.pa_decode_weights(o, w_.data_ptr(), x, k, v, t, MBS, c, B, *shape, *tail)
        assert rc == PA_OK
        return flib.pa_workspace_status(ws.data_ptr(), st)

    torch.cuda.synchronize()
    flib.pa_fault_test_configure(stop_item, WAIT_NS)
    t0 = time.perf_counter()
    status = call()
    elapsed = time.perf_counter() - t0
    flib.pa_fault_test_configure(-1, 0)
    assert status == PA_ERR_DEVICE, f"status {status}: the timeout was not recorded"
    assert elapsed < 5.0, f"the failed call took {elapsed:.2f} s"

    ws.zero_()
    assert call() == PA_OK
    for b in range(0, B, 1 if B < 10 else 49):
        pos = torch.arange(lens[b])
        kk, vv = ref.rows_at(kc, bt[b], pos)[0], ref.rows_at(vc, bt[b], pos)[0]
        if op in ("prefix", "prefix_each"):
            u = torch.arange(900)
            kk, vv = torch.cat([ref.rows_at(kc, pt[0], u)[0], kk]), torch.cat([ref.rows_at(vc, pt[0], u)[0], vv])
        want, bound, _, _ = ref.attend(q[b].double(), kk, vv, scale)
        ref.check(out[b], want, bound, f"after recovery, sequence {b}")
