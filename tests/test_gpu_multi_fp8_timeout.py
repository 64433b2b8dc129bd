"""The bounded waits of the kernels for several query rows over the 8-bit caches run out: the call records
PA_ERR_DEVICE, ends soon, and after zeroing the workspace the same call gives the right result again. The failure-test
build stops the copies part-way, so that a wait for a stage that is never filled runs out; nothing faults."""

import ctypes
import time

import pytest
import torch

import paged_gqa_decode_reshape_gb300 as pg
from tests.test_gpu_subset import DEV, bf16, dev, pool
from tests.test_gpu_window_multi_fp8 import check_rows, codes, filler, offsets, wide

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
    for n in ("pa_decode_window_multi_fp8", "pa_decode_window_multi_fp8_block", "pa_workspace_status"):
        getattr(L, n).argtypes = getattr(main, n).argtypes
        getattr(L, n).restype = ctypes.c_int
    L.pa_fault_test_configure.argtypes = [ctypes.c_int, ctypes.c_uint64]
    L.pa_fault_test_configure.restype = None
    yield L
    L.pa_fault_test_configure(-1, 0)


@pytest.mark.parametrize("stop_item", [0, 1])  # every warp and CTA here has at least two copies to make
@pytest.mark.parametrize("per_block", [False, True])
# each row for itself; units of several rows, those cut merged by a kernel of their own or by the CTA of the last piece
@pytest.mark.parametrize("op", ["each", "tiles", "tiles_many"])
def test_wait_runs_out_then_status_and_recovery(flib, op, per_block, stop_item):
    Hq, Hkv, D, scale = 28, 4, 128, 0.0884
    ctx = [700] * 40 if op == "tiles_many" else [3000, 1700, 2999, 800]
    ql = [1 if op == "each" else 8] * len(ctx)
    B, T = len(ctx), sum(ql)
    g, kc, vc, bt, _, _ = pool(7, ctx, Hkv, D)
    k8, v8, ks, vs, k64, v64 = codes(kc, vc, per_block, Hkv)
    table, cu, q = bt if op == "each" else wide(bt), offsets(ql), bf16(g, T, Hq, D, std=2.0)
    assert op == "each" or not filler(T, B, Hkv, 1 << 20, 0)
    args = dev(q, k8, v8, ks, vs, table, cu, torch.tensor(ctx, dtype=torch.int32))
    out = torch.empty_like(args[0])
    ws = torch.zeros(pg.pa_decode_window_multi_workspace_size(B, T, Hq, Hkv, D), dtype=torch.uint8, device=DEV)
    st = torch.cuda.current_stream().cuda_stream
    f = flib.pa_decode_window_multi_fp8_block if per_block else flib.pa_decode_window_multi_fp8
    o, x, k, v, a, b, t, c, n = (y.data_ptr() for y in (out, *args))

    def call():
        assert f(o, x, k, v, a, b, t, table.shape[1], c, n, B, T, Hq, Hkv, D, 16, k8.shape[0], 1 << 20, 0, scale,
                 ws.data_ptr(), ws.numel(), st) == PA_OK
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
    check_rows(out, q, k64, v64, bt, cu, ctx, ql, 1 << 20, 0, scale)
