"""Block tables, row offsets, positions and slots built on the GPU, and blocks
given back, against the plain rules (tests/step_reference.py): every element
equal, guard elements untouched."""

import random

import pytest
import torch

import paged_gqa_decode_reshape_gb300 as pg
from tests import step_reference as ref
from tests.subset_reference import BS, tables

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
i32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import paged_gqa_decode_reshape_gb300.build as b
    b.build()


def ints(v):
    return torch.tensor(v, dtype=i32)


def stack(seed, lens, spare, mbs=None):
    """Tables of these lengths, a stack with `spare` free blocks and room for the pool, and the pool's size."""
    perm = torch.randperm(sum(-(-max(x, 0) // BS) for x in lens) + spare + 1, generator=torch.Generator().manual_seed(seed))
    bt, at = tables(lens, perm, 0, mbs)
    free = torch.full((len(perm),), -7, dtype=i32)
    free[:spare] = perm[at:at + spare].int()
    return bt, free, len(perm)


def plan(bt, ctx, q, free, nf, NB, T, in_place=False):
    """The seven outputs of the call, on the host."""
    B = bt.shape[0]
    guard = torch.full((B + 3,), 99, dtype=i32, device=DEV)
    bt_, ctx_, q_, free_, nf_ = (x.to(DEV) for x in (bt, ctx, q, free, ints([nf])))
    new_lens = ctx_ if in_place else guard[1:B + 1]
    new_free = nf_ if in_place else torch.full((1,), 99, dtype=i32, device=DEV)
    granted, cu = torch.full((B,), 99, dtype=i32, device=DEV), torch.full((B + 1,), 99, dtype=i32, device=DEV)
    pos, slots = torch.full((T + 1,), 99, dtype=i32, device=DEV), torch.full((T + 1,), 99, dtype=torch.int64, device=DEV)
    pg.pa_plan_step(bt_, ctx_, q_, free_, nf_, NB, new_lens, new_free, granted, cu, pos[:T], slots[:T])
    assert pos[T] == 99 and slots[T] == 99 and guard[0] == 99 and (guard[B + 1:] == 99).all()
    assert torch.equal(free_.cpu(), free) and torch.equal(q_.cpu(), q)
    return [x.cpu() for x in (bt_, new_lens, new_free, granted, cu, pos[:T], slots[:T])]


NAMES = ["block_tables", "new_lens", "new_free", "granted", "cu_seqlens_q", "positions", "slots"]


def same(got, want, names=NAMES):
    for g, w, n in zip(got, want, names):
        assert torch.equal(g, w), f"{n}: {[(i, int(a), int(b)) for i, (a, b) in enumerate(zip(g.view(-1), w.view(-1))) if a != b][:5]}"


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,q,pad", [
    ([0], [1], 0), ([15], [1], 0), ([16], [1], 0), ([17], [0], 1), ([0, 0, 0], [0, 0, 0], 2),
    ([5, 0, 31, 100, 16], [1, 17, 1, 0, 33], 0), ([1, 2, 3], [-4, 2, 5000], 3),
    ([700, 0, 33] * 40, [1, 0, 3] * 40, 17), ([9] * 1025, [1] * 1025, 0), ([0, 16] * 2048, [1, 2] * 2048, 5),
    ([7, 0, 90, 16], [1024] * 4, 0), ([7, 0, 90, 16], [1024] * 4, 1), ([300] * 200, [1] * 199 + [2300], 8),
    ([100, 0, 4], [6000, 9000, 1], 100), ([0] * 3000, [0] * 2999 + [20000], 0),
])
def test_plan(lens, q, pad, in_place):
    need = sum(-(-(x + max(n, 0)) // BS) - -(-x // BS) for x, n in zip(lens, q))
    mbs = max(-(-(x + max(n, 0)) // BS) for x, n in zip(lens, q)) + 1
    bt, free, NB = stack(len(lens) + sum(q), lens, need + 2, mbs)
    ctx, q, T = ints(lens), ints(q), max(1, int(ints(q).clamp(min=0).sum()) + pad)
    same(plan(bt, ctx, q, free, need + 2, NB, T, in_place), ref.plan(bt, ctx, q, free, need + 2, NB, T))


@pytest.mark.parametrize("spare", [0, 1, 2, 5, 6, 40])
def test_plan_without_enough_blocks(spare):
    """The first sequence that does not get its blocks, and the later ones that need some, get nothing; those that
    need none go on."""
    lens, q = [15, 16, 3, 0, 16, 40, 1], [1, 1, 2, 60, 1, 2, 0]
    bt, free, NB = stack(3, lens, spare, 9)
    args = (bt, ints(lens), ints(q), free, spare, NB, 70)
    want = ref.plan(*args)
    assert int(want[3].sum()) < sum(q) or spare >= 6
    same(plan(*args), want)


def test_plan_bad_metadata():
    """Lengths, counts, entries and rows out of range: the documented results, nothing out of bounds."""
    lens = [30, 64, 20, 10, 5]
    bt, free, NB = stack(4, lens, 6, 4)
    free[3], free[4] = -5, NB + 9  # entries outside the pool: their slots are -1
    bt[0, 1] = NB
    big = 2 ** 31 - 1
    for ctx, q, nf, T in [
        ([30, 64, 20, 10, 5], [3, 1, 30, 20, 3], 6, 80),       # past the table's width
        ([30, 64, 20, 10, 5], [3, 0, 13, 20, 3], 6, 38),       # rows past total_q: the last two
        ([-9, big, 20, 10, 5], [3, 1, 13, 20, 40], big, 90),   # clamped lengths, a count past the capacity
        ([30, 64, 20, 10, 5], [big, big, big, 1, big], 6, 4),  # sums past 32 bits
        ([30, 64, 20, 10, 5], [1, 0, 1, 1, 20], -3, 40),       # a negative count
    ]:
        args = (bt, ints(ctx), ints(q), free, nf, NB, T)
        same(plan(*args), ref.plan(*args))


def test_plan_random():
    r = random.Random(1)
    for _ in range(60):
        B = r.choice([1, 2, 31, 33, 200])
        lens = [r.choice([0, r.randrange(40), r.randrange(300)]) for _ in range(B)]
        q = [r.choice([0, 1, 1, r.randrange(50)]) for _ in range(B)]
        need = sum(-(-(x + n) // BS) - -(-x // BS) for x, n in zip(lens, q))
        spare = max(0, need + r.choice([5, 0, -1, -need // 2]))
        bt, free, NB = stack(r.randrange(1000), lens, spare, r.choice([22, 19]))
        T = max(1, sum(q) + r.choice([0, 3, -2]))
        args = (bt, ints(lens), ints(q), free, spare, NB, T)
        same(plan(*args, in_place=r.random() < 0.5), ref.plan(*args))


def release(bt, ctx, keep, free, nf, NB, in_place=False):
    B, F = bt.shape[0], len(free)
    bt_, ctx_, keep_, nf_ = (x.to(DEV) for x in (bt, ctx, keep, ints([nf])))
    buf = torch.cat([free, ints([99])]).to(DEV)
    new_lens = ctx_ if in_place else torch.full((B,), 99, dtype=i32, device=DEV)
    new_free = nf_ if in_place else torch.full((1,), 99, dtype=i32, device=DEV)
    pg.pa_release_blocks(bt_, ctx_, keep_, buf[:F], nf_, NB, new_lens, new_free)
    assert buf[F] == 99 and torch.equal(bt_.cpu(), bt)
    return [x.cpu() for x in (buf[:F], new_lens, new_free)]


RELEASED = ["free_blocks", "new_lens", "new_free"]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,keep", [
    ([1], [0]), ([16], [16]), ([17], [16]), ([17], [17]), ([0], [5]), ([100, 0, 33], [1, 3, -9]),
    ([700, 5, 64] * 50, [0, 5, 33] * 50), ([40000, 1, 30000], [0, 0, 15999]), ([20] * 4096, [0, 16] * 2048),
    ([60000] * 9, [17, 0, 59999] * 3),
])
def test_release(lens, keep, in_place):
    bt, free, NB = stack(len(lens), lens, 4)
    args = (bt, ints(lens), ints(keep), free, 4, NB)
    same(release(*args, in_place), ref.release(*args), RELEASED)


def test_release_bad_metadata():
    """Entries outside the pool are passed over, what has no room is dropped, lengths and counts are clamped."""
    lens = [100, 64, 70, 16 * 700]
    bt, free, NB = stack(8, lens, 5)
    bt[0, 1], bt[0, 3], bt[2, 0], bt[3, 10:650] = -1, NB, -9, -1
    big = 2 ** 31 - 1
    for ctx, keep, nf, F in [(lens, [0, 0, 0, 0], 5, NB), (lens, [0, 20, 33, 100], 5, 12), (lens, [0, 0, 0, 0], 5, 5),
                             ([big, -1, 70, 9], [-1, 5, big, 0], 0, NB), (lens, [0, 0, 0, 0], -4, NB),
                             (lens, [0, 0, 1, 2], big, 40)]:
        args = (bt, ints(ctx), ints(keep), free[:F].clone(), nf, NB)
        same(release(*args), ref.release(*args), RELEASED)


def test_plan_then_release_gives_every_block_back():
    """Steps of a batch, sequences that end and tokens that are taken back, all on the device and in place: at the end
    the stack holds every block once. The second half is replayed from a graph."""
    B, NB, MBS, T = 37, 900, 60, 400
    r = random.Random(5)
    g = lambda x: torch.tensor(x, dtype=i32, device=DEV)
    bt, ctx, free, nf = torch.full((B, MBS), -1, dtype=i32, device=DEV), g([0] * B), g(list(range(NB))), g([NB])
    q, keep, granted, cu = g([0] * B), g([0] * B), g([0] * B), g([0] * (B + 1))
    pos, slots = torch.empty(T, dtype=i32, device=DEV), torch.empty(T, dtype=torch.int64, device=DEV)

    def step():
        pg.pa_plan_step(bt, ctx, q, free, nf, NB, ctx, nf, granted, cu, pos, slots)
        pg.pa_release_blocks(bt, ctx, keep, free, nf, NB, ctx, nf)

    graph = torch.cuda.CUDAGraph()
    lens, owned = [0] * B, set()
    for n in range(60):
        if n == 30:
            with torch.cuda.graph(graph):
                step()
        new = [r.choice([0, 1, 1, r.randrange(30)]) for _ in range(B)]
        kept = [0 if r.random() < 0.1 else max(0, x + y - r.choice([0, 0, 3])) for x, y in zip(lens, new)]
        before = sum(new) <= T
        q.copy_(ints(new))
        keep.copy_(ints(kept))
        step() if n < 30 else graph.replay()
        assert before and granted.tolist() == new
        lens = kept
        assert ctx.tolist() == lens
        table, live = bt.cpu(), []
        for b, x in enumerate(lens):
            live += table[b, :-(-x // BS)].tolist()
        stack_now = free[:int(nf)].tolist()
        assert sorted(live + stack_now) == list(range(NB))


def test_stream_and_two_calls():
    """On a stream that is not the default one, two different calls one after the other."""
    bt, free, NB = stack(6, [10, 40], 8, 6)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        a = plan(bt, ints([10, 40]), ints([7, 30]), free, 8, NB, 40)
        b = plan(bt, ints([10, 33]), ints([1, 0]), free, 8, NB, 3)
    same(a, ref.plan(bt, ints([10, 40]), ints([7, 30]), free, 8, NB, 40))
    same(b, ref.plan(bt, ints([10, 33]), ints([1, 0]), free, 8, NB, 3))


def test_binding_refuses():
    bt, free, NB = stack(6, [10, 40], 8, 6)
    d = lambda x: x.to(DEV)
    args = [d(bt), d(ints([1, 2])), d(ints([1, 2])), d(free), d(ints([8])), NB, d(ints([0, 0])), d(ints([0])), d(ints([0, 0])),
            d(ints([0] * 3)), torch.empty(9, dtype=i32, device=DEV), torch.empty(9, dtype=torch.int64, device=DEV)]
    pg.pa_plan_step(*args)
    for at, bad, err in [(0, bt, ValueError), (1, d(ints([1])), ValueError), (2, d(torch.tensor([1, 2])), TypeError),
                         (4, d(ints([1, 2])), ValueError), (9, d(ints([0, 0])), ValueError), (10, args[10][:8], ValueError),
                         (11, args[11][::2], ValueError), (6, args[2], pg.PagedDecodeError),
                         (5, 0, pg.PagedDecodeError), (0, args[0].t(), ValueError)]:
        with pytest.raises(err):
            pg.pa_plan_step(*[bad if i == at else x for i, x in enumerate(args)])
    with pytest.raises(pg.PagedDecodeError):
        pg.pa_plan_step(*args, block_size=32)
    with pytest.raises(ValueError):
        pg.pa_release_blocks(args[0], args[1], args[2][:1], args[3], args[4], NB, args[6], args[7])
