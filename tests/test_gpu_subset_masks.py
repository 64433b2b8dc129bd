"""Every token of a mask, on every kernel that may run a call over a part of the
cache. Queries are zero, so that each seen token has the same weight, and V is
1 in dim t mod D and 0 elsewhere: an output counts the seen tokens, and one
that is missing, doubled or too many shows, however long the window is. The
probabilities and their sums are exact (2^0 and whole numbers); the output is
rounded once to bf16 (2^-8) after a division (2^-24)."""

import pytest
import torch

import paged_gqa_decode_reshape_gb300 as pg
from tests import subset_reference as ref
from tests.subset_reference import BS
from tests.test_gpu_subset import CTX, DEV, HEADS, NAN, bf16, dev, pool, widened

pytestmark = pytest.mark.gpu
ROUNDING = 2.0 ** -8 + 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import paged_gqa_decode_reshape_gb300.build as b
    b.build()


def count_cache(seed, lens, Hkv, D, own=None):
    """A cache whose V rows are 1 (sequences from `own` on: 0.5) in dim t mod D; NaN where there is no token."""
    g, kc, vc, bt, perm, at = pool(seed, lens, Hkv, D)
    for b, n in enumerate(lens):
        t = torch.arange(n)
        v = torch.zeros(n, D).scatter_(1, (t % D)[:, None], 0.5 if own is not None and b >= own else 1.0)
        vc[bt[b][t // BS].long(), t % BS] = v[:, None].to(torch.bfloat16)
    return g, kc, vc, bt


def counts(t, D, value=1.0):
    return torch.bincount(t % D, minlength=D).double() * value


def check(out, want, what):
    """out [..., Hq, D]: the same counts in every head."""
    got = out.double().cpu()
    over = (got - want.unsqueeze(-2)).abs() - ROUNDING * want.unsqueeze(-2)
    assert torch.isfinite(got).all() and over.max() <= 0, f"{what}: {int((over > 0).sum())} elements"


def row_tiles(T, Hkv, D, MBS, window, sinks):
    """Does a call of these sizes go to the row tiles? (More rows than SMs.)"""
    assert T * Hkv > 152
    return T * Hkv * min(MBS * BS, window + sinks + 2 * BS) * D * 4 > (60 << 20) - (4 << 20)


WINDOWS = [(1, 0), (2, 3), (16, 0), (17, 1), (100, 4), (129, 63), (1000, 200), (1 << 30, 5)]
ROWS = [(28, 4, 128), (8, 8, 128), (8, 1, 64), (9, 3, 64)]


# one row for itself in the streaming kernel; row tiles, whose cut units are merged by the last CTA (rows of no
# sequence make the call large) or, where few rows see many tokens, by a kernel of its own
@pytest.mark.parametrize("heads,window,sinks,way", [
    (h, *w, way) for h in ROWS for w in WINDOWS for way in ("each", "merged", "joined")
    if (way == "merged") or (way == "each" and (h[1] < 8 or w[0] < 1000)) or (way == "joined" and w[0] >= 1000 and h[1] <= 4)])
def test_rows(heads, window, sinks, way):
    Hq, Hkv, D = heads
    ctx = [1, 290, 40, 18, 0, 299, 256] if way == "each" else [1, 700, 40, 18, 0, 513, 1100]
    ql = [1, 9, 16, 18, 3, 1, 12] if way == "each" else [1, 150, 40, 25, 3, 1, 129]
    g, kc, vc, bt = count_cache(Hq + window % 997, ctx, Hkv, D)
    cu = torch.tensor([0] + torch.tensor(ql).cumsum(0).tolist(), dtype=torch.int32)
    n = int(cu[-1])
    T = max(n + 2, 152 // Hkv + 1)
    if way == "merged":
        seen = min(bt.shape[1] * BS, window + sinks + 2 * BS)
        T = max(T, (60 << 20) // (Hkv * seen * D * 4) + 1, 76 * 2 * (128 // (Hq // Hkv)) // Hkv + 256)
    if way == "joined":
        bt = widened(bt, T, Hkv, D)
    assert row_tiles(T, Hkv, D, bt.shape[1], window, sinks) == (way != "each")
    q = torch.zeros(T, Hq, D, dtype=torch.bfloat16)
    out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    pg.pa_decode_window_multi(out, *dev(q, kc, vc, bt, cu, torch.tensor(ctx, dtype=torch.int32)), window, sinks, 0.1)
    assert bool((out[n:] == 7.0).all())  # rows of no sequence
    want = torch.zeros(n, D).double()
    for b, x in enumerate(ctx):
        for i in range(ql[b]):
            t = ref.seen(x - ql[b] + i + 1, window, sinks)
            want[int(cu[b]) + i] = counts(t, D) / max(len(t), 1)
    check(out[:n], want, way)


@pytest.mark.parametrize("B", [1, 10, 400])  # a piece of a segment per CTA, and a range of segments per warp
@pytest.mark.parametrize("window,sinks", [(1, 0), (15, 2), (16, 16), (100, 4), (257, 33), (1 << 30, 0)])
@pytest.mark.parametrize("heads,kind", [((28, 4, 128), "bf16"), ((32, 4, 64), "bf16"), ((5, 1, 128), "bf16"),
                                        ((28, 4, 128), "fp8"), ((28, 4, 128), "fp8_block"), ((8, 8, 128), "fp8_block")])
def test_window(heads, kind, window, sinks, B):
    Hq, Hkv, D = heads
    lens = CTX if B == 10 else [2500] if B == 1 else [(7 * i) % 331 for i in range(B)]
    g, kc, vc, bt = count_cache(B, lens, Hkv, D)
    want = torch.zeros(len(lens), D).double()
    for b, x in enumerate(lens):
        t = ref.seen(x, window, sinks)
        want[b] = counts(t, D) / max(len(t), 1)
    q, ctx = torch.zeros(len(lens), Hq, D, dtype=torch.bfloat16), torch.tensor(lens, dtype=torch.int32)
    out = torch.full((len(lens), Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    if kind == "bf16":
        pg.pa_decode_window(out, *dev(q, kc, vc, bt, ctx), window, sinks, 0.1)
    else:
        NB = kc.shape[0]
        shape = (NB, Hkv) if kind == "fp8_block" else (Hkv,)
        e = torch.randint(-3, 4, shape, generator=g).float()  # V codes of 2^-e with scales of 2^e stand for 1
        each = torch.exp2(-e)[:, None, :, None] if kind == "fp8_block" else torch.exp2(-e)[None, None, :, None]
        code = lambda x: x.to(torch.float8_e4m3fn).view(torch.uint8)
        k8, v8 = code(kc.float()), code(vc.float() * each)
        inv = torch.tensor([ref.V8_POS.index(i) for i in range(BS)])
        fn = pg.pa_decode_window_fp8_block if kind == "fp8_block" else pg.pa_decode_window_fp8
        fn(out, *dev(q, k8.contiguous(), v8.permute(0, 2, 3, 1)[..., inv].contiguous(), torch.ones(shape),
                     torch.exp2(e), bt, ctx), window, sinks, 0.1)
    check(out, want, kind)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("plens,sizes", [([1, 15, 16, 17], [1, 2, 1, 3]), ([640, 0, 129, 1000], [40, 3, 2, 30]),
                                         ([2500], [70])])
def test_prefix(heads, plens, sizes, wide):
    Hq, Hkv, D = heads
    B = sum(sizes) + 2  # two sequences of no group
    own = [(37 * i * i) % 261 for i in range(B)]
    own[0] = own[-1] = 0
    g, kc, vc, bt = count_cache(Hq + B, plens + own, Hkv, D, own=len(plens))
    pt, bt = bt[:len(plens)].contiguous(), bt[len(plens):].contiguous()
    cu = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32)
    want = torch.zeros(B, D).double()
    for b in range(B):
        grp = next((i for i in range(len(sizes)) if cu[i] <= b < cu[i + 1]), None)
        n = (plens[grp] if grp is not None else 0) + own[b]
        if grp is not None:
            want[b] += counts(torch.arange(plens[grp]), D)
        want[b] = (want[b] + counts(torch.arange(own[b]), D, 0.5)) / max(n, 1)
    out = torch.full((B, Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    pg.pa_decode_prefix(out, *dev(torch.zeros(B, Hq, D, dtype=torch.bfloat16), kc, vc,
                                  widened(pt, B, Hkv, D) if wide else pt, torch.tensor(plens, dtype=torch.int32), cu, bt,
                                  torch.tensor(own, dtype=torch.int32)), 0.1)
    check(out, want, "prefix")


@pytest.mark.parametrize("rows", [0, 8000])  # streamed; on row tiles
@pytest.mark.parametrize("window", [64, 100])
def test_unseen_tokens_that_are_not_finite(window, rows):
    """A token whose K or V is not finite reaches the rows that see it and no other row."""
    Hq, Hkv, D, sinks = 14, 2, 128, 3
    ctx, ql = [400, 300], [30, 120 if rows else 60]
    g, kc, vc, bt, _, _ = pool(41, ctx, Hkv, D)
    for b, ts in {0: [5, 390, 399], 1: [1, 40, 200, 299]}.items():
        for n, t in enumerate(ts):
            blk, o = int(bt[b, t // BS]), t % BS
            vc[blk, o, 0, 5 * n:5 * n + 3] = float("inf") if n % 2 else NAN
            if n == 1:
                kc[blk, o, 1, 7] = NAN
    cu = torch.tensor([0] + torch.tensor(ql).cumsum(0).tolist(), dtype=torch.int32)
    n = int(cu[-1])
    T = max(n, rows)
    assert row_tiles(T, Hkv, D, bt.shape[1], window, sinks) == (rows > 0)
    q = bf16(g, T, Hq, D)
    out = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    pg.pa_decode_window_multi(out, *dev(q, kc, vc, bt, cu, torch.tensor(ctx, dtype=torch.int32)), window, sinks, 0.1)
    got = out.double().cpu()
    assert bool((got[n:] == 7.0).all())
    for b in range(2):
        for i in range(ql[b]):
            t = ref.seen(ctx[b] - ql[b] + i + 1, window, sinks)
            r = int(cu[b]) + i
            want, bound, _, _ = ref.attend(q[r].double(), ref.rows_at(kc, bt[b], t)[0], ref.rows_at(vc, bt[b], t)[0], 0.1)
            fine = torch.isfinite(want)
            assert torch.equal(torch.isfinite(got[r]), fine), f"sequence {b} row {i}"
            assert ((got[r] - want).abs() - bound)[fine].max() <= 0, f"sequence {b} row {i}"


@pytest.mark.parametrize("window,rows", [(50, 12), (50, 8000), (1 << 20, 400)])  # streamed; merged; joined
def test_malformed_offsets_stay_in_bounds(window, rows):
    """Descending and too large row offsets give undefined rows, and no fault; a proper call after them is right."""
    Hq, Hkv, D = 8, 2, 64
    ctx = [100, 100, 100]
    g, kc, vc, bt = count_cache(5, ctx, Hkv, D)
    if window > 50:
        bt = widened(bt, rows, Hkv, D)
    q = torch.zeros(rows, Hq, D, dtype=torch.bfloat16)
    args = dev(q, kc, vc, bt)
    ctx_ = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    out = torch.zeros(rows, Hq, D, dtype=torch.bfloat16, device=DEV)
    for cu in ([0, 90, 4, 12], [5, 3, 2, 1], [-4, 1 << 30, -9, 1 << 20], [0, rows, 3, rows]):
        pg.pa_decode_window_multi(out, *args, i32(cu), ctx_, window, 2, 0.1)
    pg.pa_decode_window_multi(out, *args, i32([0, 4, 8, 12]), ctx_, window, 2, 0.1)
    want = torch.stack([counts(t, D) / len(t) for t in (ref.seen(97 + i % 4, window, 2) for i in range(12))])
    check(out[:12], want, "after malformed offsets")
