"""A token that is not finite holds up nobody: rows whose result is not finite
are looked at once nothing waits for their warps any more, so that the kernels'
bounded waits, here a few milliseconds long, do not run out behind them."""

import ctypes

import pytest
import torch

import paged_gqa_decode_reshape_gb300 as pg
from tests import subset_reference as ref
from tests.subset_reference import BS
from tests.test_gpu_subset import DEV, NAN, bf16, dev, pool

pytestmark = pytest.mark.gpu
# far above what the call takes otherwise (under 1 ms), far below the time that 32 rows of 40000 tokens take a warp
# when it walks them one token after another (loads that depend on one another: 100 ns a token at the least, 128 ms)
WAIT_NS = 10_000_000


@pytest.fixture(scope="module")
def flib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import paged_gqa_decode_reshape_gb300.build as pgb
    pgb.build()
    main = pg.load_library()
    L = ctypes.CDLL(pgb.FAULT_LIB)
    for n in ("pa_decode_window_multi", "pa_workspace_status"):
        getattr(L, n).argtypes = getattr(main, n).argtypes
        getattr(L, n).restype = ctypes.c_int
    L.pa_fault_test_configure.argtypes = [ctypes.c_int, ctypes.c_uint64]
    L.pa_fault_test_configure.restype = None
    yield L
    L.pa_fault_test_configure(-1, 0)


@pytest.mark.parametrize("seen_by", ["all", "some"])
# rows of the long sequence: two units, cut and joined by a kernel of their own; 200, whole or merged by the last CTA
@pytest.mark.parametrize("rows", [36, 3600])
def test_a_token_that_is_not_finite_holds_up_nobody(flib, seen_by, rows):
    Hq, Hkv, D, scale = 14, 2, 128, 0.0884
    ctx, ql = [40000, 300, 70], [rows, 40, 3]
    g, kc, vc, bt, _, _ = pool(71, ctx, Hkv, D)
    # tokens that are not finite, each in dims of its own: one that every row sees, or one per 36 rows (a unit's)
    # that the later half of those rows see
    bad = {7: 64} if seen_by == "all" else {ctx[0] - rows + 18 + 36 * i: i for i in range(rows // 36)}
    for t, d in bad.items():
        vc[bt[0, t // BS], t % BS, 0, d] = NAN
    cu = torch.tensor([0] + torch.tensor(ql).cumsum(0).tolist(), dtype=torch.int32)
    T = int(cu[-1])
    q = bf16(g, T, Hq, D, std=2.0)
    q_, kc_, vc_, bt_, cu_, ctx_ = dev(q, kc, vc, bt, cu, torch.tensor(ctx, dtype=torch.int32))
    out = torch.full_like(q_, 7.0)
    ws = torch.zeros(pg.pa_decode_window_multi_workspace_size(len(ctx), T, Hq, Hkv, D), dtype=torch.uint8, device=DEV)
    st = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    flib.pa_fault_test_configure(-1, WAIT_NS)
    rc = flib.pa_decode_window_multi(out.data_ptr(), q_.data_ptr(), kc_.data_ptr(), vc_.data_ptr(), bt_.data_ptr(),
                                     bt_.shape[1], cu_.data_ptr(), ctx_.data_ptr(), len(ctx), T, Hq, Hkv, D, BS,
                                     kc.shape[0], 1 << 20, 0, scale, ws.data_ptr(), ws.numel(), st)
    status = flib.pa_workspace_status(ws.data_ptr(), st)
    flib.pa_fault_test_configure(-1, 0)
    assert (rc, status) == (0, 0)
    for b, r in [(0, x) for x in (0, 17, 18, 35, rows // 2 + 7, rows - 1)] + [(1, 0), (1, 39), (2, 0), (2, 2)]:
        u = torch.arange(ctx[b] - ql[b] + r + 1)
        row = int(cu[b]) + r
        want, bound, _, _ = ref.attend(q[row].double(), ref.rows_at(kc, bt[b], u)[0], ref.rows_at(vc, bt[b], u)[0],
                                       scale)
        got, fine = out[row].double().cpu(), torch.isfinite(want)
        assert (~fine).sum() == (0 if b else sum(t < len(u) for t in bad) * Hq // Hkv)
        assert torch.equal(torch.isfinite(got), fine), f"sequence {b} row {r}"
        assert ((got - want).abs() - bound)[fine].max() <= 0, f"sequence {b} row {r}"
