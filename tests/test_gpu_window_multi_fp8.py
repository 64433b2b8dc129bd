"""Several query rows per sequence over the 8-bit caches (scales per KV head and
per block): speculative rows, prompt chunks, windows and sinks, against plain
64-bit forms with derived bounds (tests/subset_reference.py): probabilities are
rounded to bf16 or f16 before they meet V (the bound takes bf16's 2^-8), queries
to f16 in small calls (2^-11)."""

import pytest
import torch

import paged_gqa_decode_reshape_gb300 as pg
from tests import subset_reference as ref
from tests.subset_reference import BS, V8_POS
from tests.test_gpu_subset import DEV, NAN, bf16, dev, pool

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import paged_gqa_decode_reshape_gb300.build as b
    b.build()


WIDE = 6250  # blocks of a table that makes a call share reads between rows, where sequences have several


def filler(rows, nseq, Hkv, window, sinks):
    """Rows of a further prompt that make the call share its reads between rows: the call's rule is by the rows, the
    sequences and the most tokens that a row can see (the window, or the width of the tables)."""
    seen = min(WIDE * BS, window + sinks + 2 * BS)
    cost = lambda n, s: 3.9e-5 * n * Hkv * seen - 20 - 1.4e-4 * s * Hkv * seen
    if cost(rows, nseq) > 0:
        return 0
    n = 1
    while cost(rows + n, nseq + 1) <= 0:
        n += 1 + n // 50
    return n


def sharing(ctx, ql, Hkv, window, sinks):
    n = filler(sum(ql), len(ql), Hkv, window, sinks)
    return (ctx + [n], ql + [n]) if n else (ctx, ql)


def wide(bt):
    return torch.nn.functional.pad(bt, (0, WIDE - bt.shape[1]), value=-1)


def codes(kc, vc, per_block, Hkv):
    """8-bit caches, their scales and what they stand for; NaN (slots that hold no token) becomes the code of NaN."""
    k8, v8, ks, vs, k64, v64 = ref.to_fp8(torch.nan_to_num(kc.float(), nan=0.0).to(torch.bfloat16),
                                          torch.nan_to_num(vc.float(), nan=0.0).to(torch.bfloat16), per_block, Hkv)
    k8[torch.isnan(kc.float())] = 0x7F
    bad = torch.isnan(vc.float()).permute(0, 2, 3, 1)  # [NB, Hkv, D, BS]
    inv = torch.tensor([V8_POS.index(i) for i in range(BS)])
    v8[bad[..., inv]] = 0x7F
    k64[torch.isnan(kc.float())], v64[torch.isnan(vc.float())] = NAN, NAN
    return k8, v8, ks, vs, k64, v64


def call(per_block, *args, **more):
    return (pg.pa_decode_window_multi_fp8_block if per_block else pg.pa_decode_window_multi_fp8)(*args, **more)


def attend(q, k64, v64, bt, lim, window, sinks, scale):
    t = ref.seen(lim, window, sinks)
    k, ok = ref.rows_at(k64, bt, t)
    v = ref.rows_at(v64, bt, t)[0]
    return ref.attend(q.double(), k[ok], v[ok], scale, 2.0 ** -8, 2.0 ** -11)


def check_rows(out, q, k64, v64, bt, cu, ctx, ql, window, sinks, scale, every=1):
    for b, x in enumerate(ctx):
        step = max(every, ql[b] // 200)
        for i in list(range(0, ql[b], step)) + ([ql[b] - 1] if ql[b] else []):
            r = int(cu[b]) + i
            want, bound, _, _ = attend(q[r], k64, v64, bt[b], x - ql[b] + i + 1, window, sinks, scale)
            ref.check(out[r], want, bound, f"sequence {b} row {i}")


def offsets(ql):
    return torch.tensor([0] + torch.tensor(ql).cumsum(0).tolist(), dtype=torch.int32)


@pytest.mark.parametrize("share", [False, True])
@pytest.mark.parametrize("per_block", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 0), (100, 4), (257, 130), (1 << 30, 0)])
@pytest.mark.parametrize("heads", [(28, 4), (8, 8), (8, 1), (9, 3)])
def test_rows(heads, window, sinks, per_block, share):
    Hq, Hkv = heads
    ctx = [1, 700, 40, 18, 0, 513, 1100]
    ql = [1, 150, 40, 25, 3, 1, 129]  # a sequence all of whose rows are new; one with more rows than tokens
    if share:
        ctx, ql = sharing(ctx, ql, Hkv, window, sinks)
    g, kc, vc, bt, _, _ = pool(Hq + window % 97, ctx, Hkv, D)
    k8, v8, ks, vs, k64, v64 = codes(kc, vc, per_block, Hkv)
    cu = offsets(ql)
    T = int(cu[-1]) + 2  # two rows of no sequence
    q, scale = bf16(g, T, Hq, D, std=2.0), D ** -0.5
    args = dev(q, k8, v8, ks, vs, wide(bt) if share else bt, cu, torch.tensor(ctx, dtype=torch.int32))
    out = torch.full_like(args[0], 7.0)
    first = None
    for _ in range(2):
        call(per_block, out, *args, window, sinks, scale)
        first = out.clone() if first is None else first
    assert torch.equal(first.view(torch.int16), out.view(torch.int16))
    assert (out[-2:] == 7.0).all()
    check_rows(out, q, k64, v64, bt, cu, ctx, ql, window, sinks, scale)


@pytest.mark.parametrize("share", [False, True])
@pytest.mark.parametrize("per_block", [False, True])
@pytest.mark.parametrize("S,q,x", [(1, 1, 1), (1, 4, 700), (40, 3, 500), (3, 1, 5000), (600, 1, 40), (2, 64, 4000)])
def test_few_rows(S, q, x, per_block, share):
    Hq, Hkv = 28, 4
    ctx, ql = [max(1, x - 7 * b % x) for b in range(S)], [q] * S
    ql = [min(a, b) for a, b in zip(ql, ctx)]
    if share:
        ctx, ql = sharing(ctx, ql, Hkv, 1 << 30, 0)
    g, kc, vc, bt, _, _ = pool(S + x, ctx, Hkv, D)
    k8, v8, ks, vs, k64, v64 = codes(kc, vc, per_block, Hkv)
    cu = offsets(ql)
    rows = bf16(g, int(cu[-1]), Hq, D, std=2.0)
    args = dev(rows, k8, v8, ks, vs, wide(bt) if share else bt, cu, torch.tensor(ctx, dtype=torch.int32))
    out = torch.full_like(args[0], NAN)
    call(per_block, out, *args, 1 << 30, 0, D ** -0.5)
    check_rows(out, rows, k64, v64, bt, cu, ctx, ql, 1 << 30, 0, D ** -0.5, 1 if S < 50 else 2)


@pytest.mark.parametrize("share", [False, True])
@pytest.mark.parametrize("per_block", [False, True])
def test_bad_metadata(per_block, share):
    """Entries outside the pool read as empty, lengths are clamped; malformed offsets give undefined rows, no fault."""
    Hq, Hkv = 8, 2
    g, kc, vc, bt, _, _ = pool(5, [100, 300, 90], Hkv, D)
    bt[1, 3], bt[1, 18], bt[0, 0] = -1, kc.shape[0], 1 << 30
    k8, v8, ks, vs, k64, v64 = codes(kc, vc, per_block, Hkv)
    q = bf16(g, 24, Hq, D)
    table = wide(bt) if share else bt
    out = torch.zeros(24, Hq, D, dtype=torch.bfloat16, device=DEV)
    a = dev(q, k8, v8, ks, vs, table)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    ql, cu = [8, 10, 6], offsets([8, 10, 6])
    call(per_block, out, *a, cu.to(DEV), i32([100, 300, -5]), 1 << 20, 0, 0.1)
    check_rows(out, q, k64, v64, bt, cu, [100, 300, 0], ql, 1 << 20, 0, 0.1)
    assert not share or (not filler(24, 3, Hkv, 1 << 20, 0) and not filler(24, 3, Hkv, WIDE * BS - 34, 2))
    for bad in ([0, 90, 4, 12], [5, 3, 2, 1], [-4, 1 << 30, -9, 1 << 20]):
        call(per_block, out, *a, i32(bad), i32([100, 300, 90]), 50 if not share else WIDE * BS - 34, 2, 0.1)
    torch.cuda.synchronize()


@pytest.mark.parametrize("more", [0, 60])  # cut units: merged by a kernel of their own, or by the last CTA
@pytest.mark.parametrize("per_block", [False, True])
@pytest.mark.parametrize("window,share", [(64, True), (350, True), (64, False), (1 << 20, True)])
def test_nan_codes_of_unseen_tokens_stay_out(window, share, per_block, more):
    """A token with a NaN code reaches the rows that see it and no other row, although rows share its products."""
    Hq, Hkv, sinks = 14, 2, 3
    ctx, ql = [400, 300] + [500] * more, [30, 300] + [2] * more
    if share:
        ctx, ql = sharing(ctx, ql, Hkv, window, sinks)
    g, kc, vc, bt, _, _ = pool(41, ctx, Hkv, D)
    for b, ts in {0: [390, 399], 1: [1, 40, 200, 299]}.items():
        for n, t in enumerate(ts):
            vc[bt[b, t // BS], t % BS, 0, 5 * n:5 * n + 3] = NAN
            if n == 1:
                kc[bt[b, t // BS], t % BS, 1, 7] = NAN
    k8, v8, ks, vs, k64, v64 = codes(kc, vc, per_block, Hkv)
    cu = offsets(ql)
    q = bf16(g, sum(ql), Hq, D)
    out = torch.full((sum(ql), Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    call(per_block, out, *dev(q, k8, v8, ks, vs, wide(bt) if share else bt, cu, torch.tensor(ctx, dtype=torch.int32)),
         window, sinks, 0.1)
    got = out.cpu()
    for b in range(2):
        for i in range(ql[b]):
            want, bound, _, _ = attend(q[int(cu[b]) + i], k64, v64, bt[b], ctx[b] - ql[b] + i + 1, window, sinks, 0.1)
            row, fine = got[int(cu[b]) + i].double(), torch.isfinite(want)
            assert torch.equal(torch.isfinite(row), fine), f"sequence {b} row {i}"
            assert (((row - want).abs() - bound)[fine] <= 0).all(), f"sequence {b} row {i}"


@pytest.mark.parametrize("share", [False, True])
def test_scales_of_every_size(share):
    """Per-block scales from 2^-120 to 2^100 next to each other, subnormal codes, and a block that is still empty."""
    Hq, Hkv = 8, 2
    ctx, ql = [333], [20]
    g, kc, vc, bt, _, _ = pool(12, ctx, Hkv, D)
    NB = kc.shape[0]
    k8 = torch.randint(0, 256, (NB, BS, Hkv, D), generator=g, dtype=torch.uint8)
    v8 = torch.randint(0, 256, (NB, Hkv, D, BS), generator=g, dtype=torch.uint8)
    k8[(k8 & 0x7F) == 0x7F], v8[(v8 & 0x7F) == 0x7F] = 1, 1
    ks = torch.exp2(torch.randint(-12, -6, (NB, Hkv), generator=g).float())
    vs = torch.exp2(torch.randint(-120, 100, (NB, Hkv), generator=g).float())
    vs[bt[0, 2], 0] = 0.0
    ks[bt[0, 2], 0] = 2.0 ** -126
    inv = torch.tensor(V8_POS)
    k64 = k8.view(torch.float8_e4m3fn).double() * ks.double()[:, None, :, None]
    v64 = (v8.view(torch.float8_e4m3fn).double() * vs.double()[:, :, None, None])[..., inv].permute(0, 3, 1, 2)
    cu = offsets(ql)
    assert not filler(20, 1, Hkv, 1 << 20, 0)
    q = bf16(g, 20, Hq, D)
    out = torch.full((20, Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    call(True, out, *dev(q, k8, v8, ks, vs, wide(bt) if share else bt, cu, torch.tensor(ctx, dtype=torch.int32)),
         1 << 20, 0, 0.05)
    check_rows(out, q, k64, v64, bt, cu, ctx, ql, 1 << 20, 0, 0.05)


@pytest.mark.parametrize("per_block", [False, True])
@pytest.mark.parametrize("T,window,sinks", [(5000, 700, 4), (2600, 1 << 30, 0)])
def test_whole_prompt(T, window, sinks, per_block):
    Hq, Hkv = 28, 4
    g, kc, vc, bt, _, _ = pool(T, [T], Hkv, D)
    k8, v8, ks, vs, k64, v64 = codes(kc, vc, per_block, Hkv)
    q = bf16(g, T, Hq, D, std=2.0)
    cu = offsets([T])
    out = torch.full((T, Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    call(per_block, out, *dev(q, k8, v8, ks, vs, bt, cu, torch.tensor([T], dtype=torch.int32)), window, sinks, D ** -0.5)
    check_rows(out, q, k64, v64, bt, cu, [T], [T], window, sinks, D ** -0.5, 173)


@pytest.mark.parametrize("share", [False, True])
@pytest.mark.parametrize("per_block", [False, True])
def test_padded_batch(per_block, share):
    """Sequences without rows, first, last and in long runs between; with lengths of their own and without."""
    Hq, Hkv = 28, 4
    ctx = [0, 300, 50, 0, 700] + [33, 0] * 150 + [129, 16, 0]
    ql = [0, 9, 0, 0, 40] + [0, 0] * 150 + [5, 0, 0]
    if share:  # rows first: the call's rule counts the sequences, too
        n = filler(sum(ql), len(ql), Hkv, 1 << 30, 0)
        ctx, ql = [n] + ctx, [n] + ql
    g, kc, vc, bt, _, _ = pool(19, ctx, Hkv, D)
    k8, v8, ks, vs, k64, v64 = codes(kc, vc, per_block, Hkv)
    cu = offsets(ql)
    q = bf16(g, sum(ql) + 3, Hq, D, std=2.0)
    out = torch.full((len(q), Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    call(per_block, out, *dev(q, k8, v8, ks, vs, wide(bt) if share else bt, cu, torch.tensor(ctx, dtype=torch.int32)),
         1 << 30, 0, D ** -0.5)
    assert (out[-3:] == 7.0).all()
    check_rows(out, q, k64, v64, bt, cu, ctx, ql, 1 << 30, 0, D ** -0.5)


@pytest.mark.parametrize("scale,std", [(0.0884, 12.0), (3.0, 4.0)])
@pytest.mark.parametrize("share", [False, True])
def test_sharp_and_growing_logits(scale, std, share):
    """Maxima that grow from tile to tile by more than what a tile's probabilities hold."""
    Hq, Hkv, ctx, ql = 8, 2, [2000], [9]
    g, kc, vc, bt, _, _ = pool(31, ctx, Hkv, D)
    for j in range(125):
        kc[bt[0, j]] = (kc[bt[0, j]].float() * (0.2 + j / 60)).to(torch.bfloat16)
    k8, v8, ks, vs, k64, v64 = codes(kc, vc, True, Hkv)
    q, cu = bf16(g, 9, Hq, D, std=std), offsets(ql)
    assert not filler(9, 1, Hkv, 1 << 20, 0)
    out = torch.full((9, Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    call(True, out, *dev(q, k8, v8, ks, vs, wide(bt) if share else bt, cu, torch.tensor(ctx, dtype=torch.int32)),
         1 << 20, 0, scale)
    check_rows(out, q, k64, v64, bt, cu, ctx, ql, 1 << 20, 0, scale)


@pytest.mark.parametrize("power", [-60, 0, 60])
def test_queries_of_every_size(power):
    """Shared reads: a query row keeps its values whatever their power of two (as two E4M3 parts and that power), those of
    less than 2^-10 of its largest to within 2^-18 of it; a row that is not finite gives NaN, the ones beside it their own."""
    Hq, Hkv, ctx, ql = 8, 2, [1000], [12]
    assert not filler(12, 1, Hkv, 1 << 20, 0)
    g, kc, vc, bt, _, _ = pool(77, ctx, Hkv, D)
    k8, v8, ks, vs, k64, v64 = codes(kc, vc, False, Hkv)
    q, cu = bf16(g, 12, Hq, D), offsets(ql)
    q[:, :, 1::2] *= 2.0 ** -12  # bf16, a power of two: exact
    q[3, :, 5:9] *= 2.0 ** -30
    q = (q.float() * 2.0 ** power).to(torch.bfloat16)
    q[4, 1, 7], q[9, 6, 0] = NAN, float("inf")
    out = torch.zeros((12, Hq, D), dtype=torch.bfloat16, device=DEV)
    scale = 0.1 * 2.0 ** -power
    call(False, out, *dev(q, k8, v8, ks, vs, wide(bt), cu, torch.tensor(ctx, dtype=torch.int32)), 1 << 20, 0, scale)
    got = out.cpu().double()
    assert torch.isnan(got[4, 1]).all() and torch.isnan(got[9, 6]).all()
    for i in range(12):
        heads = [h for h in range(Hq) if (i, h) not in ((4, 1), (9, 6))]
        rows = torch.nan_to_num(q[i].double(), nan=0.0, posinf=0.0)
        t = torch.arange(1000 - 12 + i + 1)
        k, v = ref.rows_at(k64, bt[0], t)[0], ref.rows_at(v64, bt[0], t)[0]
        # a logit is off by at most e = scale 2^-18 max |q| sum_d |k_d|; weights then change by a factor within e^(+-2 e) in all,
        # and their average of values by at most 2 e max |v| (e is below 0.01 here)
        want, bound, _, _ = ref.attend(rows, k, v, scale, 2.0 ** -8, 2.0 ** -11)
        off = scale * 2.0 ** -18 * rows.abs().amax(1) * k.abs().sum(2).amax(0).repeat_interleave(Hq // Hkv)  # of a logit
        more = 2 * off[:, None] * v.abs().amax(0).repeat_interleave(Hq // Hkv, 0)  # of an average of values
        err = (got[i] - want).abs() - bound - more
        assert (err[heads] <= 0).all(), f"row {i}"


@pytest.mark.parametrize("share", [False, True])
def test_other_stream_and_graph(share):
    """On a stream of its own, then replayed from a graph with other lengths in the same buffers."""
    Hq, Hkv, S = 28, 4, 5
    lens = [[900, 30, 500, 77, 1200], [100, 800, 3, 1100, 640]]
    ql = [40, 3, 100, 1, 9]
    ql2 = [40, 3, 3, 98, 9]
    assert not filler(153, 5, Hkv, 1 << 30, 0)
    runs = []
    for n, (ctx, rows) in enumerate(zip(lens, (ql, ql2))):
        g, kc, vc, bt, _, _ = pool(50 + n, ctx, Hkv, D, extra=220 - sum(-(-x // BS) for x in ctx))
        bt = torch.nn.functional.pad(bt, (0, 80 - bt.shape[1]), value=-1)
        runs.append((ctx, rows, bf16(g, sum(rows), Hq, D), bt, offsets(rows), codes(kc, vc, False, Hkv)))
    bufs = dev(runs[0][2], *runs[0][5][:4], runs[0][3], runs[0][4], torch.tensor(lens[0], dtype=torch.int32))
    out = torch.empty_like(bufs[0])
    if share:
        bufs[5] = wide(bufs[5]).contiguous()
    go = lambda: call(False, out, *bufs, 1 << 30, 0, 0.0884)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        go()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for ctx, rows, q, bt, cu, c in (*runs, runs[0]):
        for buf, new in zip(bufs, (q, *c[:4], wide(bt) if share else bt, cu, torch.tensor(ctx, dtype=torch.int32))):
            buf.copy_(new)
        out.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        check_rows(out, q, c[4], c[5], bt, cu, ctx, rows, 1 << 30, 0, 0.0884, 7)


def test_binding_refuses():
    Hq, Hkv = 8, 2
    g, kc, vc, bt, _, _ = pool(5, [100], Hkv, D)
    k8, v8, ks, vs, _, _ = codes(kc, vc, False, Hkv)
    a = dict(zip("query key_cache value_cache k_scale v_scale block_tables cu_seqlens_q context_lens".split(),
                 dev(bf16(g, 3, Hq, D), k8, v8, ks, vs, bt, offsets([3]), torch.tensor([100], dtype=torch.int32))))
    a.update(out=torch.empty_like(a["query"]), window=50, sinks=0, scale=0.1)
    pg.pa_decode_window_multi_fp8(**a)
    per_block = torch.ones(k8.shape[0], Hkv, device=DEV)
    for over, err in [(dict(k_scale=per_block), ValueError), (dict(v_scale=a["v_scale"][:1]), ValueError),
                      (dict(key_cache=kc.to(DEV)), TypeError), (dict(value_cache=a["key_cache"]), ValueError),
                      (dict(cu_seqlens_q=a["cu_seqlens_q"][:1]), ValueError), (dict(out=a["out"][:2]), ValueError),
                      (dict(window=-1), ValueError), (dict(window=0), pg.PagedDecodeError),
                      (dict(scale=float("nan")), pg.PagedDecodeError)]:
        with pytest.raises(err):
            pg.pa_decode_window_multi_fp8(**{**a, **over})
    with pytest.raises(ValueError):
        b = {**a, "k_bscale": a["k_scale"], "v_bscale": a["v_scale"]}
        del b["k_scale"], b["v_scale"]
        pg.pa_decode_window_multi_fp8_block(**b)
