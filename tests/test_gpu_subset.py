"""The decode operators over a part of the cache -- sliding window with sinks,
shared prefixes, accumulated weights and eviction -- against plain 64-bit
forms (tests/subset_reference.py, with derived bounds), at the sizes and masks
where they can go wrong, and as they are used together."""

import pytest
import torch

import paged_gqa_decode_reshape_gb300 as pg
from tests import subset_reference as ref
from tests.subset_reference import BS

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import paged_gqa_decode_reshape_gb300.build as b
    b.build()


def bf16(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def pool(seed, lens, Hkv, D, extra=2, spoil=True):
    """A cache for these sequences: caches, tables and the permutation, NaN in every slot that holds no token."""
    g = torch.Generator().manual_seed(seed)
    NB = sum(-(-x // BS) for x in lens) + extra
    perm = torch.randperm(NB, generator=g)
    kc, vc = bf16(g, NB, BS, Hkv, D), bf16(g, NB, BS, Hkv, D)
    bt, at = ref.tables(lens, perm)
    if spoil:
        kc[perm[at:]] = NAN
        vc[perm[at:]] = NAN
        for i, x in enumerate(lens):
            if x % BS:
                kc[bt[i, x // BS], x % BS:] = NAN
                vc[bt[i, x // BS], x % BS:] = NAN
    return g, kc, vc, bt, perm, at


def dev(*ts):
    return [t.to(DEV) for t in ts]


# ------------------------------------------------------------------ window

HEADS = [(28, 4, 128), (8, 8, 128), (32, 4, 64), (5, 1, 128), (9, 3, 64)]
WINDOWS = [(1, 0), (16, 0), (17, 1), (100, 4), (128, 16), (333, 63), (1000, 200), (1 << 30, 5)]
CTX = [1, 15, 16, 17, 40, 129, 0, 300, 777, 1203]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("heads", HEADS)
def test_window(heads, window, sinks):
    Hq, Hkv, D = heads
    g, kc, vc, bt, perm, at = pool(Hq + window % 997, CTX, Hkv, D)
    # blocks that hold no visible token are gone: entry -1 (and NaN where they were)
    for b, x in enumerate(CTX):
        vis = set((ref.seen(x, window, sinks) // BS).tolist())
        for j in range(-(-x // BS)):
            if j not in vis:
                kc[bt[b, j]] = NAN
                vc[bt[b, j]] = NAN
                bt[b, j] = -1
    q, scale = bf16(g, len(CTX), Hq, D, std=2.0), D ** -0.5
    ctx = torch.tensor(CTX, dtype=torch.int32)
    q_, kc_, vc_, bt_, ctx_ = dev(q, kc, vc, bt, ctx)
    out = torch.full_like(q_, NAN)
    ws = torch.zeros(pg.pa_decode_window_workspace_size(len(CTX), Hq, Hkv, D), dtype=torch.uint8, device=DEV)
    first = None
    for _ in range(2):  # the second call finds the workspace as the first left it
        pg.pa_decode_window(out, q_, kc_, vc_, bt_, ctx_, window, sinks, scale, workspace=ws)
        first = out.clone() if first is None else first
    assert torch.equal(first.view(torch.int16), out.view(torch.int16))
    assert pg.pa_workspace_status(ws) == 0
    for b, x in enumerate(CTX):
        t = ref.seen(x, window, sinks)
        k, _ = ref.rows_at(kc, bt[b], t)
        v, _ = ref.rows_at(vc, bt[b], t)
        want, bound, _, _ = ref.attend(q[b].double(), k, v, scale)
        ref.check(out[b], want, bound, f"ctx {x}")


@pytest.mark.parametrize("window,sinks", [(1, 0), (31, 3), (128, 16), (700, 100), (5000, 0)])
@pytest.mark.parametrize("per_block", [False, True])
@pytest.mark.parametrize("heads", [(28, 4), (3, 3), (16, 2)])
def test_window_fp8(heads, per_block, window, sinks):
    (Hq, Hkv), D = heads, 128
    g, kc, vc, bt, _, _ = pool(Hq + window, CTX, Hkv, D, spoil=False)
    if per_block:  # blocks of different sizes of values
        kc *= torch.exp2(torch.randint(-3, 3, (kc.shape[0], 1, 1, 1), generator=g).float())
        vc *= torch.exp2(torch.randint(-6, 6, (kc.shape[0], 1, 1, 1), generator=g).float())
    k8, v8, ks, vs, kd, vd = ref.to_fp8(kc, vc, per_block, Hkv)
    for i, x in enumerate(CTX):  # NaN codes past the last token
        if x % BS:
            k8[bt[i, x // BS], x % BS:] = 0x7F
            for o in range(x % BS, BS):
                v8[bt[i, x // BS], :, :, ref.V8_POS[o]] = 0x7F
    q, scale = bf16(g, len(CTX), Hq, D, std=2.0), D ** -0.5
    ctx = torch.tensor(CTX, dtype=torch.int32)
    q_, k_, v_, ks_, vs_, bt_, ctx_ = dev(q, k8, v8, ks, vs, bt, ctx)
    out = torch.full_like(q_, NAN)
    fn = pg.pa_decode_window_fp8_block if per_block else pg.pa_decode_window_fp8
    fn(out, q_, k_, v_, ks_, vs_, bt_, ctx_, window, sinks, scale)
    for b, x in enumerate(CTX):
        t = ref.seen(x, window, sinks)
        k, _ = ref.rows_at(kd, bt[b], t)
        v, _ = ref.rows_at(vd, bt[b], t)
        want, bound, _, _ = ref.attend(q[b].double(), k, v, scale, u_p=2.0 ** -11, u_q=2.0 ** -11)
        ref.check(out[b], want, bound, f"ctx {x}")


def test_window_bad_metadata_reads_as_empty():
    """Entries outside the pool, lengths outside the table: masked, like every decode call."""
    Hq, Hkv, D = 8, 2, 128
    lens = [200, 200, 64]
    g, kc, vc, bt, _, _ = pool(3, lens, Hkv, D)
    bt[0, 11] = kc.shape[0] + 7
    bt[0, 12] = -5
    ctx = torch.tensor([200, -3, 1 << 30], dtype=torch.int32)
    bt[2, 4:] = -1
    q = bf16(g, 3, Hq, D)
    out = torch.full((3, Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    pg.pa_decode_window(out, *dev(q, kc, vc, bt, ctx), 100, 0, 0.1)
    t = ref.seen(200, 100, 0)
    k, ok = ref.rows_at(kc, bt[0], t)
    v, _ = ref.rows_at(vc, bt[0], t)
    want, bound, _, _ = ref.attend(q[0].double(), k[ok], v[ok], 0.1)
    ref.check(out[0], want, bound, "entries outside the pool")
    assert (out[1] == 0).all() and (out[2] == 0).all()  # no tokens; only blocks outside the pool


@pytest.mark.parametrize("B", [1, 700])
def test_window_many_sequences(B):
    """More sequences than SMs, every length from 0 to 76, and one alone."""
    Hq, Hkv, D = 4, 2, 64
    lens = [(7 * i) % 77 for i in range(B)] if B > 1 else [4000]
    window, sinks = (33, 2) if B > 1 else (2500, 7)
    g, kc, vc, bt, _, _ = pool(B, lens, Hkv, D)
    q, ctx = bf16(g, B, Hq, D, std=2.0), torch.tensor(lens, dtype=torch.int32)
    out = torch.full((B, Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    pg.pa_decode_window(out, *dev(q, kc, vc, bt, ctx), window, sinks, 0.125)
    for b, x in enumerate(lens):
        t = ref.seen(x, window, sinks)
        k, v = ref.rows_at(kc, bt[b], t)[0], ref.rows_at(vc, bt[b], t)[0]
        want, bound, _, _ = ref.attend(q[b].double(), k, v, 0.125)
        ref.check(out[b], want, bound, f"sequence {b}")


# ------------------------------------------------------------ window, rows


@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 0), (100, 4), (257, 130), (5000, 1)])
@pytest.mark.parametrize("heads", [(28, 4, 128), (8, 8, 128), (8, 1, 64), (9, 3, 64)])
def test_window_multi(heads, window, sinks):
    Hq, Hkv, D = heads
    ctx = [1, 700, 40, 18, 0, 513, 1100]
    ql = [1, 150, 40, 25, 3, 1, 129]  # a sequence all of whose rows are new; one with more rows than tokens
    g, kc, vc, bt, _, _ = pool(Hq + window, ctx, Hkv, D)
    cu = torch.tensor([0] + torch.tensor(ql).cumsum(0).tolist(), dtype=torch.int32)
    T = int(cu[-1]) + 2  # two rows of no sequence
    q, scale = bf16(g, T, Hq, D, std=2.0), D ** -0.5
    q_, kc_, vc_, bt_, cu_, ctx_ = dev(q, kc, vc, bt, cu, torch.tensor(ctx, dtype=torch.int32))
    out = torch.full_like(q_, 7.0)
    for _ in range(2):
        pg.pa_decode_window_multi(out, q_, kc_, vc_, bt_, cu_, ctx_, window, sinks, scale)
    assert (out[-2:] == 7.0).all()
    for b, x in enumerate(ctx):
        for i in range(ql[b]):
            lim = x - ql[b] + i + 1
            t = ref.seen(lim, window, sinks)
            k, v = ref.rows_at(kc, bt[b], t)[0], ref.rows_at(vc, bt[b], t)[0]
            r = int(cu[b]) + i
            want, bound, _, _ = ref.attend(q[r].double(), k, v, scale)
            ref.check(out[r], want, bound, f"sequence {b} row {i}")


def test_window_multi_malformed_offsets_stay_in_bounds():
    """Descending and too large row offsets give undefined rows, and no fault."""
    Hq, Hkv, D = 8, 2, 64
    g, kc, vc, bt, _, _ = pool(5, [100, 100, 100], Hkv, D)
    q = bf16(g, 12, Hq, D)
    out = torch.zeros(12, Hq, D, dtype=torch.bfloat16, device=DEV)
    for cu in ([0, 90, 4, 12], [5, 3, 2, 1], [-4, 1 << 30, -9, 1 << 20]):
        pg.pa_decode_window_multi(out, *dev(q, kc, vc, bt), torch.tensor(cu, dtype=torch.int32, device=DEV),
                                  torch.tensor([100, 100, 100], dtype=torch.int32, device=DEV), 50, 2, 0.1)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ prefix


def widened(pt, B, Hkv, D):
    """Tables so wide that a call for these shapes (B: query rows) shares its reads, however short the lengths are."""
    return torch.nn.functional.pad(pt, (0, (128 << 20) // (B * Hkv * BS * D * 4) + 1), value=-1)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("heads", [(28, 4, 128), (8, 8, 128), (32, 4, 64), (5, 5, 64), (6, 2, 128)])
@pytest.mark.parametrize("plens,sizes,free", [
    ([1], [3], 0), ([130], [1], 2), ([0, 17, 640], [2, 5, 1], 1), ([1000, 129, 16], [40, 2, 20], 0),
    ([2500], [70], 3),
])
def test_prefix(heads, plens, sizes, free, wide):
    Hq, Hkv, D = heads
    B = sum(sizes) + free
    own = [(37 * i * i) % 261 for i in range(B)]
    own[0] = 0
    g, kc, vc, bt, perm, at = pool(Hq + B, own + plens, Hkv, D)
    bt, pt = bt[:B].contiguous(), bt[B:].contiguous()
    cu = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32)
    q, scale = bf16(g, B, Hq, D, std=2.0), D ** -0.5
    args = dev(q, kc, vc, widened(pt, B, Hkv, D) if wide else pt, torch.tensor(plens, dtype=torch.int32), cu, bt,
               torch.tensor(own, dtype=torch.int32))
    out = torch.full_like(args[0], NAN)
    first = None
    for _ in range(2):
        pg.pa_decode_prefix(out, *args, scale)
        first = out.clone() if first is None else first
    assert torch.equal(first.view(torch.int16), out.view(torch.int16))
    for b in range(B):
        grp = next((i for i in range(len(sizes)) if cu[i] <= b < cu[i + 1]), None)
        t = torch.arange(own[b])
        k, v = ref.rows_at(kc, bt[b], t)[0], ref.rows_at(vc, bt[b], t)[0]
        if grp is not None:
            u = torch.arange(plens[grp])
            k = torch.cat([ref.rows_at(kc, pt[grp], u)[0], k])
            v = torch.cat([ref.rows_at(vc, pt[grp], u)[0], v])
        want, bound, _, _ = ref.attend(q[b].double(), k, v, scale)
        ref.check(out[b], want, bound, f"sequence {b}")


@pytest.mark.parametrize("wide", [False, True])
def test_prefix_bad_metadata(wide):
    """A prefix entry outside the pool reads as empty; malformed offsets and lengths stay in bounds."""
    Hq, Hkv, D = 8, 2, 128
    own, plens = [20, 0, 33], [300, 50]
    g, kc, vc, bt, _, _ = pool(9, own + plens, Hkv, D)
    bt, pt = bt[:3].contiguous(), bt[3:].contiguous()
    pt[0, 3], pt[0, 18] = -1, kc.shape[0]
    q = bf16(g, 3, Hq, D)
    q_, kc_, vc_, pt_, bt_, ctx_ = dev(q, kc, vc, widened(pt, 3, Hkv, D) if wide else pt, bt,
                                       torch.tensor(own, dtype=torch.int32))
    out = torch.full_like(q_, NAN)
    pl = torch.tensor(plens, dtype=torch.int32, device=DEV)
    pg.pa_decode_prefix(out, q_, kc_, vc_, pt_, pl, torch.tensor([0, 3, 3], dtype=torch.int32, device=DEV), bt_,
                        ctx_, 0.1)
    for b in range(3):
        u, t = torch.arange(300), torch.arange(own[b])
        pk, ok = ref.rows_at(kc, pt[0], u)
        pv = ref.rows_at(vc, pt[0], u)[0]
        k = torch.cat([pk[ok], ref.rows_at(kc, bt[b], t)[0]])
        v = torch.cat([pv[ok], ref.rows_at(vc, bt[b], t)[0]])
        want, bound, _, _ = ref.attend(q[b].double(), k, v, 0.1)
        ref.check(out[b], want, bound, f"sequence {b}")
    for cu, lens in (([2, 0, 9], [1 << 30, -4]), ([-7, 1 << 30, -1], [5, 5]), ([0, 1 << 20, 3], [300, 50])):
        pg.pa_decode_prefix(out, q_, kc_, vc_, pt_, torch.tensor(lens, dtype=torch.int32, device=DEV),
                            torch.tensor(cu, dtype=torch.int32, device=DEV), bt_, ctx_, 0.1)
    torch.cuda.synchronize()


# ------------------------------------------------------- weights, eviction


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("ctx", [[1], [0, 5, 16], CTX, [3000, 31], [64] * 300])
def test_weights(heads, ctx):
    Hq, Hkv, D = heads
    g, kc, vc, bt, _, _ = pool(Hq + len(ctx), ctx, Hkv, D)
    B, NB, scale = len(ctx), kc.shape[0], D ** -0.5
    w0 = torch.rand(NB, Hkv, BS, generator=g)
    q = bf16(g, B, Hq, D, std=2.0)
    q_, kc_, vc_, bt_, ctx_, w_ = dev(q, kc, vc, bt, torch.tensor(ctx, dtype=torch.int32), w0)
    out = torch.full_like(q_, NAN)
    pg.pa_decode_weights(out, w_, q_, kc_, vc_, bt_, ctx_, scale)
    want_w, bound_w = w0.double(), w0.double() * 0
    for b, x in enumerate(ctx):
        t = torch.arange(x)
        k, v = ref.rows_at(kc, bt[b], t)[0], ref.rows_at(vc, bt[b], t)[0]
        want, bound, p, rel = ref.attend(q[b].double(), k, v, scale)
        ref.check(out[b], want, bound, f"out, ctx {x}")
        if x:
            blk = bt[b][t // BS].long()
            add = p.reshape(Hkv, -1, x).sum(1).T
            want_w[blk, :, t % BS] += add
            # the probabilities, their sum over the group, and the addition to the weight
            bound_w[blk, :, t % BS] += (rel.max() + 9 * 2.0 ** -24) * add + 2.0 ** -24 * want_w[blk, :, t % BS]
    ref.check(w_, want_w, bound_w, "weights")
    first = w_.clone()
    w_.copy_(w0)
    pg.pa_decode_weights(out, w_, q_, kc_, vc_, bt_, ctx_, scale)
    assert torch.equal(first, w_)  # blocks of one sequence each: the same bits


def test_weights_of_shared_and_bad_blocks():
    """A block of two sequences gets the sum of both; a block listed twice counts twice; bad entries nothing."""
    Hq, Hkv, D = 8, 2, 128
    g, kc, vc, bt, _, _ = pool(4, [64, 64], Hkv, D)
    bt[1, 0] = bt[0, 0]
    bt[1, 2] = bt[1, 1]
    bt[0, 3] = -1
    ctx = torch.tensor([64, 50], dtype=torch.int32)
    q = bf16(g, 2, Hq, D)
    w = torch.zeros(kc.shape[0], Hkv, BS)
    q_, kc_, vc_, bt_, ctx_, w_ = dev(q, kc, vc, bt, ctx, w)
    out = torch.empty_like(q_)
    pg.pa_decode_weights(out, w_, q_, kc_, vc_, bt_, ctx_, 0.1)
    want, worst = w.double(), 0.0
    for b in range(2):
        t = torch.arange(int(ctx[b]))
        k, ok = ref.rows_at(kc, bt[b], t)
        v = ref.rows_at(vc, bt[b], t)[0]
        _, _, p, rel = ref.attend(q[b].double(), k[ok], v[ok], 0.1)
        worst = max(worst, rel.max().item())
        add = p.reshape(Hkv, -1, int(ok.sum())).sum(1).T
        for i, j in enumerate(t[ok].tolist()):
            want[bt[b, j // BS].long(), :, j % BS] += add[i]
    ref.check(w_, want, (worst + 12 * 2.0 ** -24) * want, "weights")


def test_reset_weights():
    w = torch.rand(6, 3, BS) + 1
    slots = torch.tensor([0, 17, -1, 95, 96, 1 << 40, 40, 40], dtype=torch.int64)
    w_ = w.to(DEV)
    pg.pa_reset_weights(w_, slots.to(DEV))
    for s in (0, 17, 95, 40):
        w[s // BS, :, s % BS] = 0
    assert torch.equal(w_.cpu(), w)
    pg.pa_reset_weights(w_, slots[:0].to(DEV))
    assert torch.equal(w_.cpu(), w)


def _evict_case(seed, ctx, budget, recent, Hkv, D, levels=0, mbs=None, dmbs=None):
    new = [min(max(x, 0), budget) for x in ctx]
    g, kc, vc, bt, perm, _ = pool(seed, [max(x, 0) for x in ctx] + new, Hkv, D, spoil=False)
    B = len(ctx)
    need = max(-(-budget // BS), 1)
    dst = torch.full((B, dmbs or need), -1, dtype=torch.int32)
    dst[:, :min(bt.shape[1], dst.shape[1])] = bt[B:, :dst.shape[1]]
    bt = bt[:B].contiguous()
    w = torch.randn(kc.shape[0], Hkv, BS, generator=g)
    if levels:  # many equal weights
        w = torch.floor(torch.rand(kc.shape[0], Hkv, BS, generator=g) * levels)
    return kc, vc, bt, dst, w


def _evict_run(kc, vc, bt, dst, w, ctx, budget, recent):
    B, Hkv = bt.shape[0], kc.shape[2]
    ctx = torch.tensor(ctx, dtype=torch.int32)
    kc_, vc_, w_, bt_, ctx_, dst_ = dev(kc, vc, w, bt, ctx, dst)
    kept = torch.full((B, Hkv, budget), 99, dtype=torch.int32, device=DEV)
    lens = torch.full((B,), 99, dtype=torch.int32, device=DEV)
    pg.pa_evict(kept, lens, kc_, vc_, w_, bt_, ctx_, dst_, recent)
    want = ref.evict(kc, vc, w, bt, ctx, dst, budget, recent)
    for got, exp, what in zip((kept, lens, kc_, vc_, w_), want, ("kept", "new_lens", "key", "value", "weights")):
        got = got.cpu()
        if got.dtype == torch.bfloat16:
            got, exp = got.view(torch.int16), exp.view(torch.int16)
        assert torch.equal(got, exp), what


@pytest.mark.parametrize("ctx,budget,recent", [
    ([0, 1, 50, 333], 50, 7), ([100], 100, 3), ([101], 100, 100), ([101, 7], 100, 0), ([200, 90], 33, 500),
    ([1000, 17, 16, 15], 1, 0), ([1000, 999], 64, 1), ([2500] * 5, 777, 130),
])
@pytest.mark.parametrize("Hkv,D", [(4, 128), (1, 64)])
@pytest.mark.parametrize("levels", [0, 1, 3])
def test_evict(ctx, budget, recent, Hkv, D, levels):
    _evict_run(*_evict_case(budget, ctx, budget, recent, Hkv, D, levels), ctx, budget, recent)


@pytest.mark.parametrize("Hkv,D", [(4, 128), (2, 64)])
def test_evict_many_heads(Hkv, D):
    """More (sequence, KV head) pairs than the GPU has SMs for several CTAs each."""
    ctx = [700, 64, 0, 300, 1, 299] * 13
    _evict_run(*_evict_case(3, ctx, 130, 20, Hkv, D), ctx, 130, 20)


@pytest.mark.parametrize("n,budget", [(6000, 2000), (6000, 3), (60001, 5000)])
@pytest.mark.parametrize("spread", [0.0, 1e-6, 1e-3, 30.0])
def test_evict_clustered_weights(n, budget, spread):
    """Nearly all weights close together (or over many octaves) between one far below and one far above."""
    kc, vc, bt, dst, w = _evict_case(n, [n], budget, 0, 1, 64)
    w = torch.exp(w * spread)
    w[bt[0, 3], 0, 5], w[bt[0, 9], 0, 2] = 3e38, -3e38
    _evict_run(kc, vc, bt, dst, w, [n], budget, 0)


def test_evict_long_row():
    """A row longer than the selection holds in shared memory."""
    ctx = [70001]
    _evict_run(*_evict_case(1, ctx, 300, 40, 1, 64, 500), ctx, 300, 40)


def test_evict_bad_metadata_and_ordering():
    """Entries outside the pool are last and not copied; infinite and negative weights keep their order."""
    ctx, budget, recent = [200, 300], 120, 10
    kc, vc, bt, dst, w = _evict_case(2, ctx, budget, recent, 2, 128)
    bt[0, 2], bt[1, 5], dst[1, 1] = -1, kc.shape[0] + 3, -2
    w[bt[0, 4]] = float("inf")
    w[bt[0, 7], :, ::2] = float("-inf")
    w[bt[1, 0]] = -0.0
    w[bt[1, 1]] = -1e-42
    _evict_run(kc, vc, bt, dst, w, ctx, budget, recent)
    _evict_run(kc, vc, bt, dst, w, [1 << 30, -5], budget, recent)  # clamped to the table, and to nothing


# ------------------------------------------------------------ used together


def test_serving_run():
    """Decode steps that accumulate weights, an eviction, and more steps on the
    destination blocks: Quest metadata rebuilt, a window over what was kept."""
    Hq, Hkv, D, B = 14, 2, 128, 3
    start, steps, budget, recent = [90, 33, 200], 4, 64, 8
    full = [x + steps for x in start]
    g, kc, vc, bt, perm, at = pool(11, [x + 8 for x in full] + [budget + 8] * B, Hkv, D, extra=0, spoil=False)
    dst, bt = bt[B:].contiguous(), bt[:B].contiguous()
    NB, scale = kc.shape[0], D ** -0.5
    w_ = torch.full((NB, Hkv, BS), 5.0, device=DEV)
    kc_, vc_, bt_, dst_ = dev(kc, vc, bt, dst)
    slots = torch.tensor([int(bt[b, t // BS]) * BS + t % BS for b, x in enumerate(start) for t in range(x)])
    pg.pa_reset_weights(w_, slots.to(DEV))
    out = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=DEV)
    total = [torch.zeros(Hkv, x).double() for x in full]
    K, V = kc.clone(), vc.clone()
    worst = 0.0
    for s in range(steps):
        ctx = [x + s + 1 for x in start]
        k, v, q = bf16(g, B, Hkv, D), bf16(g, B, Hkv, D), bf16(g, B, Hq, D, std=2.0)
        slot = torch.tensor([int(bt[b, (x - 1) // BS]) * BS + (x - 1) % BS for b, x in enumerate(ctx)])
        pg.pa_reshape_and_cache(*dev(k, v), kc_, vc_, slot.to(DEV))
        pg.pa_reset_weights(w_, slot.to(DEV))
        pg.pa_decode_weights(out, w_, q.to(DEV), kc_, vc_, bt_, torch.tensor(ctx, dtype=torch.int32, device=DEV),
                             scale)
        for b, x in enumerate(ctx):
            K[slot[b] // BS, slot[b] % BS], V[slot[b] // BS, slot[b] % BS] = k[b], v[b]
            t = torch.arange(x)
            kk, vv = ref.rows_at(K, bt[b], t)[0], ref.rows_at(V, bt[b], t)[0]
            want, bound, p, rel = ref.attend(q[b].double(), kk, vv, scale)
            worst = max(worst, rel.max().item())
            ref.check(out[b], want, bound, f"step {s} sequence {b}")
            total[b][:, :x] += p.reshape(Hkv, -1, x).sum(1)
    for b, x in enumerate(full):
        t = torch.arange(x)
        got = w_.cpu()[bt[b][t // BS].long(), :, t % BS].T
        ref.check(got, total[b], (worst + 20 * 2.0 ** -24) * total[b], "accumulated weights")
    w = w_.cpu()
    kept = torch.empty(B, Hkv, budget, dtype=torch.int32, device=DEV)
    lens = torch.empty(B, dtype=torch.int32, device=DEV)
    pg.pa_evict(kept, lens, kc_, vc_, w_, bt_, torch.tensor(full, dtype=torch.int32, device=DEV), dst_, recent)
    kmin = torch.zeros(NB, Hkv, D, dtype=torch.bfloat16, device=DEV)
    kmax = torch.zeros_like(kmin)
    pg.quest_rebuild_meta(kmin, kmax, kc_, dst_, lens)
    q = bf16(g, B, Hq, D, std=2.0)
    sparse, sel = torch.empty_like(out), torch.empty(B, Hkv, dst.shape[1], dtype=torch.int32, device=DEV)
    pg.quest_decode(sparse, sel, q.to(DEV), kmin, kmax, kc_, vc_, dst_, lens, dst.shape[1], scale)
    pg.pa_decode_window(out, q.to(DEV), kc_, vc_, dst_, lens, 40, 4, scale)
    want = ref.evict(K, V, w, bt, full, dst, budget, recent)
    assert torch.equal(kept.cpu(), want[0]) and torch.equal(lens.cpu(), want[1])
    for b in range(B):
        n = int(want[1][b])
        for t, got, what in ((ref.seen(n, 40, 4), out, "window"), (torch.arange(n), sparse, "every block")):
            k, v = ref.rows_at(want[2], dst[b], t)[0], ref.rows_at(want[3], dst[b], t)[0]
            o, bound, _, _ = ref.attend(q[b].double(), k, v, scale)
            ref.check(got[b], o, bound, f"after eviction, {what}")


def _captured(calls):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        for c in calls:
            c()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for c in calls:
            c()
    return graph


def test_graph_replay_and_other_stream():
    """All operators in one captured graph give the bits of eager calls, also
    with new lengths at the replay; on a stream of their own they do too."""
    Hq, Hkv, D, B = 28, 4, 128, 4
    lens, plens = [400, 33, 900, 64], [500]
    g, kc, vc, tabs, perm, at = pool(21, lens + plens + [128] * B, Hkv, D, spoil=False)
    bt, pt, dst = tabs[:B].contiguous(), tabs[B:B + 1].contiguous(), tabs[B + 1:, :8].contiguous()
    w0 = torch.rand(kc.shape[0], Hkv, BS, generator=g)
    q, qm = bf16(g, B, Hq, D), bf16(g, 40, Hq, D)
    q_, qm_, kc_, vc_, bt_, pt_, dst_, w_ = dev(q, qm, kc, vc, bt, pt, dst, w0)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    ctx, cu, plen, cug = i32(*lens), i32(0, 20, 25, 39, 40), i32(500), i32(0, 3)
    outs = [torch.empty_like(q_) for _ in range(3)] + [torch.empty_like(qm_), torch.empty_like(qm_)]
    wide, wide_rows = widened(pt_, B, Hkv, D), widened(bt_, 40, Hkv, D)
    kept, new = torch.empty(B, Hkv, 128, dtype=torch.int32, device=DEV), i32(0, 0, 0, 0)
    calls = [
        lambda: pg.pa_decode_window(outs[0], q_, kc_, vc_, bt_, ctx, 128, 4, 0.1),
        lambda: pg.pa_decode_prefix(outs[1], q_, kc_, vc_, wide, plen, cug, bt_, ctx, 0.1),
        lambda: pg.pa_decode_weights(outs[2], w_, q_, kc_, vc_, bt_, ctx, 0.1),
        lambda: pg.pa_decode_window_multi(outs[3], qm_, kc_, vc_, bt_, cu, ctx, 100, 8, 0.1),
        lambda: pg.pa_decode_window_multi(outs[4], qm_, kc_, vc_, wide_rows, cu, ctx, 1 << 20, 8, 0.1),
        lambda: pg.pa_evict(kept, new, kc_, vc_, w_, bt_, ctx, dst_, 16),
    ]

    def state():
        return [t.clone() for t in (*outs, kept, new, kc_, vc_, w_)]

    def reset():
        kc_.copy_(kc), vc_.copy_(vc), w_.copy_(w0)
        for t in (*outs, kept, new):
            t.zero_()

    def same(a, b):
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.int16) if x.dtype == torch.bfloat16 else x,
                               y.view(torch.int16) if y.dtype == torch.bfloat16 else y)

    graph = _captured(calls)
    for now in (lens, [1, 17, 899, 0]):
        ctx.copy_(torch.tensor(now, dtype=torch.int32))
        reset()
        for c in calls:
            c()
        want = state()
        reset()
        graph.replay()
        same(want, state())
        reset()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for c in calls:
                c()
        torch.cuda.current_stream().wait_stream(side)
        same(want, state())


def test_two_streams_with_workspaces_of_their_own():
    """Two decode calls in flight at once, each with its own workspace."""
    Hq, Hkv, D = 28, 4, 128
    lens = [3000, 5, 1700, 800]
    g, kc, vc, bt, _, _ = pool(31, lens, Hkv, D)
    q_, kc_, vc_, bt_, ctx_ = dev(bf16(g, 4, Hq, D), kc, vc, bt, torch.tensor(lens, dtype=torch.int32))
    size = pg.pa_decode_window_workspace_size(4, Hq, Hkv, D)
    ws = [torch.zeros(size, dtype=torch.uint8, device=DEV) for _ in range(2)]
    want = pg.pa_decode_window(torch.empty_like(q_), q_, kc_, vc_, bt_, ctx_, 2000, 4, 0.1)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(q_) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                pg.pa_decode_window(outs[i], q_, kc_, vc_, bt_, ctx_, 2000, 4, 0.1, workspace=ws[i])
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))


def test_binding_refuses():
    Hq, Hkv, D = 8, 2, 64
    g, kc, vc, bt, _, _ = pool(1, [40, 40], Hkv, D)
    q_, kc_, vc_, bt_, ctx_ = dev(bf16(g, 2, Hq, D), kc, vc, bt, torch.tensor([40, 40], dtype=torch.int32))
    out = torch.empty_like(q_)
    with pytest.raises(pg.PagedDecodeError):
        pg.pa_decode_window(out, q_, kc_, vc_, bt_, ctx_, 0, 4, 0.1)
    with pytest.raises(ValueError):
        pg.pa_decode_window(out, q_, kc_, vc_, bt_, ctx_, 4, -1, 0.1)
    with pytest.raises(pg.PagedDecodeError):
        pg.pa_decode_window(out, q_, kc_, vc_, bt_, ctx_, 4, 0, float("inf"))
    with pytest.raises(pg.PagedDecodeError):
        pg.pa_decode_window(out, q_, kc_, vc_, bt_, ctx_, 4, 0, 0.1,
                            workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        pg.pa_decode_window(out, q_, kc_, vc_, bt_, ctx_[:1].contiguous(), 4, 0, 0.1)
    with pytest.raises(ValueError):
        pg.pa_decode_window(out.transpose(0, 1), q_, kc_, vc_, bt_, ctx_, 4, 0, 0.1)
    w = torch.zeros(kc.shape[0], Hkv, BS, device=DEV)
    with pytest.raises(ValueError):
        pg.pa_decode_weights(out, w[:, :1].contiguous(), q_, kc_, vc_, bt_, ctx_, 0.1)
    kept = torch.empty(2, Hkv, 33, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):  # new_lens over context_lens
        pg.pa_evict(kept, ctx_, kc_, vc_, w, bt_, ctx_, bt_, 3)
    with pytest.raises(pg.PagedDecodeError):  # 33 tokens do not fit two blocks
        pg.pa_evict(kept, torch.empty_like(ctx_), kc_, vc_, w, bt_, ctx_, bt_[:, :2].contiguous(), 3)


def test_no_workspace_is_allocated_during_capture():
    """A first call that needs a larger workspace than there is is refused inside a capture."""
    import paged_gqa_decode_reshape_gb300 as mod
    Hq, Hkv, D = 8, 2, 64
    g, kc, vc, bt, _, _ = pool(1, [40, 40], Hkv, D)
    q_, kc_, vc_, bt_, ctx_ = dev(bf16(g, 2, Hq, D), kc, vc, bt, torch.tensor([40, 40], dtype=torch.int32))
    out, old = torch.empty_like(q_), mod._subset_ws
    mod._subset_ws = mod._Scratch()
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            with pytest.raises(RuntimeError, match="before the capture"):
                pg.pa_decode_window(out, q_, kc_, vc_, bt_, ctx_, 4, 0, 0.1)
            out.zero_()
    finally:
        mod._subset_ws = old
    graph.replay()
    torch.cuda.synchronize()


# ----------------------------------------------- values, extents, long calls


@pytest.mark.parametrize("more", [0, 60])  # cut units: merged by a kernel of their own, or by the last CTA
@pytest.mark.parametrize("window", [64, 350])
def test_window_multi_keeps_nan_and_inf_of_unseen_tokens_out(window, more):
    """A token whose K or V is not finite reaches the rows that see it and no
    other row, although rows of one tile share its matrix products."""
    Hq, Hkv, D = 14, 2, 128
    ctx, ql, sinks = [400, 300] + [500] * more, [30, 300] + [2] * more, 3
    g, kc, vc, bt, _, _ = pool(41, ctx, Hkv, D)
    bad = {0: [390, 399], 1: [1, 40, 200, 299]}
    for b, ts in bad.items():
        for n, t in enumerate(ts):
            blk, o = int(bt[b, t // BS]), t % BS
            vc[blk, o, 0, 5 * n:5 * n + 3] = float("inf") if n % 2 else NAN
            if n == 1:
                kc[blk, o, 1, 7] = NAN
    cu = torch.tensor([0] + torch.tensor(ql).cumsum(0).tolist(), dtype=torch.int32)
    q = bf16(g, sum(ql), Hq, D)
    out = torch.full((sum(ql), Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    pg.pa_decode_window_multi(out, *dev(q, kc, vc, bt, cu, torch.tensor(ctx, dtype=torch.int32)), window, sinks, 0.1)
    got = out.cpu()
    for b in range(2):
        for i in range(ql[b]):
            t = ref.seen(ctx[b] - ql[b] + i + 1, window, sinks)
            k, v = ref.rows_at(kc, bt[b], t)[0], ref.rows_at(vc, bt[b], t)[0]
            r = int(cu[b]) + i
            want, bound, _, _ = ref.attend(q[r].double(), k, v, 0.1)
            fine = torch.isfinite(want)
            assert torch.equal(torch.isfinite(got[r].double()), fine), f"sequence {b} row {i}"
            over = (got[r].double() - want).abs() - bound
            assert (over[fine] <= 0).all(), f"sequence {b} row {i}"


def test_window_keeps_nan_of_unseen_tokens_out():
    """The tokens between the sinks and the window hold NaN and infinities, in blocks that are partly seen."""
    Hq, Hkv, D = 8, 2, 128
    ctx, window, sinks = [333, 90, 41], 37, 5
    g, kc, vc, bt, _, _ = pool(43, ctx, Hkv, D)
    for b, x in enumerate(ctx):
        vis = set(ref.seen(x, window, sinks).tolist())
        for t in set(range(x)) - vis:
            kc[bt[b, t // BS], t % BS] = NAN
            vc[bt[b, t // BS], t % BS] = float("inf") if t % 2 else NAN
    q = bf16(g, 3, Hq, D)
    out = torch.full((3, Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    pg.pa_decode_window(out, *dev(q, kc, vc, bt, torch.tensor(ctx, dtype=torch.int32)), window, sinks, 0.1)
    for b, x in enumerate(ctx):
        t = ref.seen(x, window, sinks)
        want, bound, _, _ = ref.attend(q[b].double(), ref.rows_at(kc, bt[b], t)[0], ref.rows_at(vc, bt[b], t)[0], 0.1)
        ref.check(out[b], want, bound, f"ctx {x}")


@pytest.mark.parametrize("scale,std", [(0.0884, 12.0), (3.0, 4.0)])
def test_sharp_and_growing_logits(scale, std):
    """Logits of hundreds, with the largest one late: the running maximum grows many times."""
    Hq, Hkv, D = 7, 1, 128
    g, kc, vc, bt, _, _ = pool(47, [1500, 1500], Hkv, D)
    q = bf16(g, 24, Hq, D, std=std)
    for t in range(0, 1500, 90):  # ever larger keys along the first query
        kc[bt[0, t // BS], t % BS, 0] = (q[0, 0].float() * t / 1500 / std).to(torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    cu, ctx = i32(0, 20, 24), i32(1500, 1500)
    out = torch.empty(24, Hq, D, dtype=torch.bfloat16, device=DEV)
    pg.pa_decode_window_multi(out, *dev(q, kc, vc, widened(bt, 24, Hkv, D), cu, ctx), 1 << 30, 0, scale)
    pre = torch.empty(2, Hq, D, dtype=torch.bfloat16, device=DEV)
    pg.pa_decode_prefix(pre, *dev(q[[0, 20]], kc, vc, widened(bt[:1], 2, Hkv, D), ctx[:1], i32(0, 1), bt, ctx), scale)
    one = torch.empty_like(pre)
    pg.pa_decode_window(one, *dev(q[[0, 20]], kc, vc, bt, ctx), 1 << 30, 0, scale)
    rows = lambda b, n: (ref.rows_at(kc, bt[b], torch.arange(n))[0], ref.rows_at(vc, bt[b], torch.arange(n))[0])
    for b, i, r in ((0, 0, 0), (0, 19, 19), (1, 0, 20), (1, 3, 23)):
        k, v = rows(b, 1500 - (20, 4)[b] + i + 1)
        want, bound, _, _ = ref.attend(q[r].double(), k, v, scale)
        ref.check(out[r], want, bound, f"row {r}")
    for b, r in ((0, 0), (1, 20)):
        k, v = rows(b, 1500)
        want, bound, _, _ = ref.attend(q[r].double(), k, v, scale)
        ref.check(one[b], want, bound, f"window {b}")
        if b == 0:
            k, v = torch.cat([k, k]), torch.cat([v, v])
        want, bound, _, _ = ref.attend(q[r].double(), k, v, scale)
        ref.check(pre[b], want, bound, f"prefix {b}")


@pytest.mark.parametrize("T,window,sinks", [(5000, 700, 4), (2600, 1 << 30, 0)])
def test_window_multi_whole_prompt(T, window, sinks):
    """A prompt attended to in one call (every row new), rows sampled."""
    Hq, Hkv, D = 28, 4, 128
    g, kc, vc, bt, _, _ = pool(T, [T], Hkv, D)
    q = bf16(g, T, Hq, D, std=2.0)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    out = torch.full((T, Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    pg.pa_decode_window_multi(out, *dev(q, kc, vc, bt, i32(0, T), i32(T)), window, sinks, 0.0884)
    assert torch.isfinite(out.float()).all()
    for r in list(range(0, T, 131)) + [T - 1]:
        t = ref.seen(r + 1, window, sinks)
        want, bound, _, _ = ref.attend(q[r].double(), ref.rows_at(kc, bt[0], t)[0], ref.rows_at(vc, bt[0], t)[0], 0.0884)
        ref.check(out[r], want, bound, f"row {r}")


def test_blocks_past_32_bit_offsets():
    """A pool of 4.7 GB per cache, the blocks in use at its end: offsets of elements and bytes pass 32 bits."""
    Hq, Hkv, D = 16, 8, 128
    NB = 145_000
    assert NB * BS * Hkv * D > 1 << 31
    lens, plen, n = [100, 37], 150, 30
    g = torch.Generator().manual_seed(5)
    ids = NB - 1 - torch.randperm(n, generator=g)
    sk, sv = bf16(g, n, BS, Hkv, D), bf16(g, n, BS, Hkv, D)
    kc_ = torch.zeros(NB, BS, Hkv, D, dtype=torch.bfloat16, device=DEV)
    vc_ = torch.zeros_like(kc_)
    kc_[ids.to(DEV)], vc_[ids.to(DEV)] = sk.to(DEV), sv.to(DEV)
    w_ = torch.zeros(NB, Hkv, BS, device=DEV)
    small, at = ref.tables(lens + [plen] + [48, 37], torch.arange(n))  # into sk / sv
    big = torch.where(small >= 0, ids[small.clamp(min=0).long()], torch.tensor(-1)).int()
    bt, pt, dst = big[:2].contiguous(), big[2:3].contiguous(), big[3:, :3].contiguous()
    q = bf16(g, 2, Hq, D, std=2.0)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    ctx = i32(*lens)
    q_, bt_, pt_, dst_, ctx_ = dev(q, bt, pt, dst, ctx)
    outs = [torch.empty_like(q_) for _ in range(4)]
    pg.pa_decode_window(outs[0], q_, kc_, vc_, bt_, ctx_, 50, 2, 0.1)
    pg.pa_decode_window_multi(outs[1], q_, kc_, vc_, bt_, i32(0, 1, 2).to(DEV), ctx_, 50, 2, 0.1)
    tiles = torch.empty_like(q_)
    pg.pa_decode_window_multi(tiles, q_, kc_, vc_, widened(bt_, 2, Hkv, D), i32(0, 1, 2).to(DEV), ctx_, 1 << 20, 0, 0.1)
    pg.pa_decode_prefix(outs[2], q_, kc_, vc_, widened(pt_, 2, Hkv, D), i32(plen).to(DEV), i32(0, 2).to(DEV), bt_, ctx_, 0.1)
    pg.pa_decode_weights(outs[3], w_, q_, kc_, vc_, bt_, ctx_, 0.1)
    total = w_.sum().item()
    kept = torch.empty(2, Hkv, 48, dtype=torch.int32, device=DEV)
    new = torch.empty(2, dtype=torch.int32, device=DEV)
    pg.pa_evict(kept, new, kc_, vc_, w_, bt_, ctx_, dst_, 48)
    for b, x in enumerate(lens):
        t = ref.seen(x, 50, 2)
        rows = lambda row, pos: (ref.rows_at(sk, small[row], pos)[0], ref.rows_at(sv, small[row], pos)[0])
        want, bound, _, _ = ref.attend(q[b].double(), *rows(b, t), 0.1)
        ref.check(outs[0][b], want, bound, "window")
        ref.check(outs[1][b], want, bound, "window, rows")
        k, v = rows(b, torch.arange(x))
        want, bound, _, _ = ref.attend(q[b].double(), k, v, 0.1)
        ref.check(outs[3][b], want, bound, "weights")
        ref.check(tiles[b], want, bound, "all tokens, row tiles")
        pk, pv = rows(2, torch.arange(plen))
        want, bound, _, _ = ref.attend(q[b].double(), torch.cat([pk, k]), torch.cat([pv, v]), 0.1)
        ref.check(outs[2][b], want, bound, "prefix")
        m = min(x, 48)  # all of them recent: the last m tokens
        i = torch.arange(m)
        src = small[b][(x - m + i) // BS].long(), (x - m + i) % BS
        got = kc_[big[3 + b][i // BS].long().to(DEV), (i % BS).to(DEV)].cpu()
        assert torch.equal(got.view(torch.int16), sk[src].view(torch.int16))
    assert abs(total - 2 * Hq) < 1e-3  # every head's weights sum to 1


@pytest.mark.parametrize("wide", [False, True])
def test_prefix_with_many_groups_and_no_own_tokens(wide):
    """Groups of one to three sequences, prefixes of every length, own tokens missing."""
    Hq, Hkv, D = 6, 2, 64
    sizes = [1 + i % 3 for i in range(150)]
    plens = [(13 * i) % 300 for i in range(150)]
    B = sum(sizes)
    g, kc, vc, bt, _, _ = pool(61, plens, Hkv, D)
    cu = torch.tensor([0] + torch.tensor(sizes).cumsum(0).tolist(), dtype=torch.int32)
    q = bf16(g, B, Hq, D, std=2.0)
    own, zero = torch.full((B, 1), -1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    out = torch.full((B, Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    pt = widened(bt, B, Hkv, D) if wide else bt
    pg.pa_decode_prefix(out, *dev(q, kc, vc, pt, torch.tensor(plens, dtype=torch.int32), cu, own, zero), 0.125)
    for grp, p in enumerate(plens):
        t = torch.arange(p)
        k, v = ref.rows_at(kc, bt[grp], t)[0], ref.rows_at(vc, bt[grp], t)[0]
        for b in range(int(cu[grp]), int(cu[grp + 1])):
            want, bound, _, _ = ref.attend(q[b].double(), k, v, 0.125)
            ref.check(out[b], want, bound, f"sequence {b}")


@pytest.mark.parametrize("window", [200, 1 << 20])  # each row for itself, or row tiles
def test_calls_after_one_without_rows_see_what_came_before(window):
    """A windowed call whose sequences all have no rows still keeps its place in the stream: the call after it
    reads the result of the call before it."""
    B, Hq, Hkv, D, n = 16, 28, 4, 128, 8192
    g, kc, vc, bt, perm, at = pool(77, [n] * B, Hkv, D, spoil=False)
    q = bf16(g, B, Hq, D)
    q_, kc_, vc_, bt_, ctx_ = dev(q, kc, vc, bt, torch.full((B,), n, dtype=torch.int32))
    cu_ = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    mid, untouched = torch.zeros_like(q_), torch.full_like(q_, 3.0)
    ws = [torch.zeros(pg.pa_decode_workspace_size(B, Hq, Hkv, D), dtype=torch.uint8, device=DEV),
          torch.zeros(pg.pa_decode_window_multi_workspace_size(B, B, Hq, Hkv, D), dtype=torch.uint8, device=DEV),
          torch.zeros(pg.pa_decode_window_workspace_size(B, Hq, Hkv, D), dtype=torch.uint8, device=DEV)]
    scale = D ** -0.5

    def last(out):
        pg.pa_decode_window(out, mid, kc_, vc_, bt_, ctx_, 200, 4, scale, workspace=ws[2])
        return out

    pg.pa_decode(mid, q_, kc_, vc_, bt_, ctx_, scale, workspace=ws[0])
    torch.cuda.synchronize()
    want = last(torch.empty_like(q_))
    for _ in range(20):
        mid.zero_()
        pg.pa_decode(mid, q_, kc_, vc_, bt_, ctx_, scale, workspace=ws[0])
        pg.pa_decode_window_multi(untouched, q_, kc_, vc_, bt_, cu_, ctx_, window, 4, scale, workspace=ws[1])
        got = last(torch.empty_like(q_))
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    assert bool((untouched == 3.0).all())


def test_one_workspace_serves_every_operator_of_the_section():
    """A buffer zeroed once serves the operators in any order, head shape and batch size."""
    calls = []
    for B, Hq, Hkv, D, n in [(2, 28, 4, 128, 900), (40, 16, 4, 64, 300), (150, 8, 2, 128, 65)]:
        g, kc, vc, bt, perm, at = pool(B, [n] * B, Hkv, D, spoil=False)
        q_, kc_, vc_, bt_, ctx_ = dev(bf16(g, B, Hq, D), kc, vc, bt, torch.full((B,), n, dtype=torch.int32))
        cu_, cug_ = dev(torch.arange(B + 1, dtype=torch.int32), torch.tensor([0, B], dtype=torch.int32))
        plen_ = torch.full((1,), n, dtype=torch.int32, device=DEV)
        NB, MBS = kc.shape[0], bt.shape[1]
        calls += [
            (pg.pa_decode_window_workspace_size(B, Hq, Hkv, D),
             lambda o, ws, q=q_, k=kc_, v=vc_, t=bt_, c=ctx_: pg.pa_decode_window(o, q, k, v, t, c, 64, 4, 0.1, workspace=ws), q_),
            (pg.pa_decode_window_multi_workspace_size(B, B, Hq, Hkv, D),
             lambda o, ws, q=q_, k=kc_, v=vc_, t=bt_, c=ctx_, u=cu_, s=(B, Hkv, D): pg.pa_decode_window_multi(
                 o, q, k, v, widened(t, *s), u, c, 1 << 20, 4, 0.1, workspace=ws), q_),
            (pg.pa_decode_window_multi_workspace_size(B, B, Hq, Hkv, D),
             lambda o, ws, q=q_, k=kc_, v=vc_, t=bt_, c=ctx_, u=cu_: pg.pa_decode_window_multi(
                 o, q, k, v, t, u, c, 40, 4, 0.1, workspace=ws), q_),
            (pg.pa_decode_prefix_workspace_size(B, 1, Hq, Hkv, D),
             lambda o, ws, q=q_, k=kc_, v=vc_, t=bt_, c=ctx_, u=cug_, p=plen_, s=(B, Hkv, D): pg.pa_decode_prefix(
                 o, q, k, v, widened(t[:1], *s), p, u, t, c, 0.1, workspace=ws), q_),
            (pg.pa_decode_weights_workspace_size(B, Hq, Hkv, D, MBS),
             lambda o, ws, q=q_, k=kc_, v=vc_, t=bt_, c=ctx_, s=(NB, Hkv, BS): pg.pa_decode_weights(
                 o, torch.zeros(s, device=DEV), q, k, v, t, c, 0.1, workspace=ws), q_),
        ]
    alone = [f(torch.empty_like(q), torch.zeros(n, dtype=torch.uint8, device=DEV)) for n, f, q in calls]
    shared = torch.zeros(max(n for n, _, _ in calls), dtype=torch.uint8, device=DEV)
    order = torch.randperm(3 * len(calls), generator=torch.Generator().manual_seed(5)) % len(calls)
    for i in order.tolist():
        n, f, q = calls[i]
        got = f(torch.empty_like(q), shared)
        assert torch.equal(got.view(torch.int16), alone[i].view(torch.int16)), i


def test_row_counts_that_change_with_every_call():
    """The binding's table of workspace sizes stays bounded, and calls are right before and after it is emptied."""
    Hq, Hkv, D = 8, 2, 64
    g, kc, vc, bt, _, _ = pool(9, [40], Hkv, D, spoil=False)
    q = bf16(g, 5000, Hq, D)
    q_, kc_, vc_, bt_, ctx_ = dev(q, kc, vc, bt, torch.tensor([40], dtype=torch.int32))
    cu_ = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    want = [ref.attend(q[r].double(), *(ref.rows_at(c, bt[0], ref.seen(38 + r, 16, 1))[0] for c in (kc, vc)), 0.1)
            for r in range(3)]
    for T in range(3, 4600):
        out = pg.pa_decode_window_multi(torch.empty_like(q_[:T]), q_[:T], kc_, vc_, bt_, cu_, ctx_, 16, 1, 0.1)
        if T % 500 == 3 or T > 4590:  # the bits may depend on the row count, which decides how the work is cut
            for r in range(3):
                ref.check(out[r], want[r][0], want[r][1], f"{T} rows, row {r}")
    assert len(pg._calls) <= 4096
