"""The step operators as they are used together: prompts come in by chunks, sequences decode with speculative rows of which
some are taken back, end, and new ones take their place; tables, slots and lengths stay on the device. Every step is
pa_plan_step, pa_norm_rope_and_cache (or its 8-bit form), attention over the cache, pa_release_blocks. The attention of sampled
rows is compared with the formulas in 64 bits on what the cache holds, which the cache tests compare with the tokens."""

import random

import pytest
import torch

import paged_gqa_decode_reshape_gb300 as pg
from tests import step_reference as sref
from tests import subset_reference as ref
from tests.subset_reference import BS, V8_POS

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
i32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import paged_gqa_decode_reshape_gb300.build as b
    b.build()


class Engine:
    """A layer's cache and the state of B sequences, on the device."""

    def __init__(self, B, NB, MBS, Hq, Hkv, D, fp8, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.shape, self.fp8, self.NB = (B, Hq, Hkv, D), fp8, NB
        z = lambda *s: torch.zeros(s, dtype=i32, device=DEV)
        self.bt, self.ctx, self.nfree = torch.full((B, MBS), -1, dtype=i32, device=DEV), z(B), z(1) + NB
        self.free = torch.randperm(NB, generator=self.g).int().to(DEV)
        if fp8:
            self.kc = torch.zeros(NB, BS, Hkv, D, dtype=torch.uint8, device=DEV)
            self.vc = torch.zeros(NB, Hkv, D, BS, dtype=torch.uint8, device=DEV)
            self.scales = [0.02 + 0.01 * torch.rand(Hkv, generator=self.g) for _ in range(2)]
            self.sc = [s.to(DEV) for s in self.scales]
        else:
            self.kc = torch.zeros(NB, BS, Hkv, D, dtype=torch.bfloat16, device=DEV)
            self.vc = torch.zeros_like(self.kc)
        angle = torch.arange(4096).double()[:, None] * 10000.0 ** (-torch.arange(D // 2).double() * 2 / D)
        self.table = torch.cat([angle.cos(), angle.sin()], 1).float()
        self.qw, self.kw = ((1 + 0.2 * torch.randn(D, generator=self.g)).to(torch.bfloat16) for _ in range(2))
        self.dev = [x.to(DEV) for x in (self.table, self.qw, self.kw)]

    def step(self, q_lens, keep, T):
        """One step with these new tokens; keep(lengths) -> tokens that stay. Returns what the attention saw and gave."""
        B, Hq, Hkv, D = self.shape
        x = torch.randn(T, Hq + 2 * Hkv, D, generator=self.g).to(torch.bfloat16)
        xd, q = x.to(DEV), torch.tensor(q_lens, dtype=i32, device=DEV)
        granted, cu, pos = (torch.empty(n, dtype=i32, device=DEV) for n in (B, B + 1, T))
        slots = torch.empty(T, dtype=torch.int64, device=DEV)
        pg.pa_plan_step(self.bt, self.ctx, q, self.free, self.nfree, self.NB, self.ctx, self.nfree, granted, cu, pos, slots)
        table, qw, kw = self.dev
        qo, out = (torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        parts = xd[:, :Hq], xd[:, Hq:Hq + Hkv], xd[:, Hq + Hkv:]
        if self.fp8:
            pg.pa_norm_rope_and_cache_fp8(qo, *parts, self.kc, self.vc, slots, *self.sc, table, pos, qw, kw)
            pg.pa_decode_window_multi_fp8(out, qo, self.kc, self.vc, *self.sc, self.bt, cu, self.ctx, 1 << 30, 0, D ** -0.5)
        else:
            pg.pa_norm_rope_and_cache(qo, *parts, self.kc, self.vc, slots, table, pos, qw, kw)
            pg.pa_decode_window_multi(out, qo, self.kc, self.vc, self.bt, cu, self.ctx, 1 << 30, 0, D ** -0.5)
        seen = dict(x=x, q=qo.cpu(), out=out, bt=self.bt.cpu(), ctx=self.ctx.tolist(), cu=cu.tolist(), pos=pos.cpu(),
                    granted=granted.tolist())
        left = torch.tensor(keep(seen["ctx"]), dtype=i32, device=DEV)
        pg.pa_release_blocks(self.bt, self.ctx, left, self.free, self.nfree, self.NB, self.ctx, self.nfree)
        return seen

    def cache(self):
        """K and V in fp64, [NB, BS, Hkv, D]."""
        if not self.fp8:
            return self.kc.cpu().double(), self.vc.cpu().double()
        e = torch.float8_e4m3fn
        k, v = self.kc.cpu().view(e).double(), self.vc.cpu().view(e).double()[..., torch.tensor(V8_POS)].permute(0, 3, 1, 2)
        return tuple(c * s.double()[:, None] for c, s in zip((k, v), self.scales))


@pytest.mark.parametrize("fp8", [False, True])
def test_prompts_decode_speculation_and_reuse(fp8):
    B, Hq, Hkv, D, MBS, NB, T = 6, 14, 2, 128, 40, 150, 700
    e = Engine(B, NB, MBS, Hq, Hkv, D, fp8, 3 + fp8)
    r = random.Random(8)
    left = [r.randrange(1, 600) for _ in range(B)]  # of each prompt
    history = [torch.zeros(0, Hkv, D, dtype=torch.bfloat16) for _ in range(B)]  # unrotated keys of what is cached
    for n in range(14):
        q_lens = [min(l, r.choice([33, 100, 250])) if l else r.choice([1, 4]) for l in left]
        grow = list(q_lens)

        def keep(ctx):
            kept = []
            for b, x in enumerate(ctx):
                if not left[b] and r.random() < 0.15:
                    kept.append(0)  # over
                elif not left[b]:
                    kept.append(x - r.randrange(grow[b]))  # the last speculative tokens are rejected
                else:
                    kept.append(x)
            return kept

        s = e.step(q_lens, keep, T)
        assert s["granted"] == q_lens  # there are blocks for all
        k64, v64 = e.cache()
        # no step writes again before the next one, so what the attention read is still there
        for b in range(B):
            first, x = s["cu"][b], s["ctx"][b]
            history[b] = torch.cat([history[b], s["x"][first:first + q_lens[b], Hq:Hq + Hkv]])
            assert len(history[b]) == x
            t = torch.arange(x)
            k, ok = ref.rows_at(k64, s["bt"][b], t)
            v = ref.rows_at(v64, s["bt"][b], t)[0]
            assert ok.all()
            # the cached keys are the tokens', rotated by their positions
            z, S = sref.norm_rope(history[b], e.kw, 1e-6, *sref.angles(e.table, t, None), False)
            if fp8:
                sc = e.scales[0].double()[:, None]
                ref.check(k / sc, (z / sc).clamp(-448, 448), sref.code_bound(z, S, D, sc), f"keys of {b}")
            else:
                ref.check(k, z, sref.bf16_bound(z, S, D), f"keys of {b}")
            for i in sorted({0, q_lens[b] // 2, q_lens[b] - 1}):
                lim = x - q_lens[b] + i + 1
                want, bound, _, _ = ref.attend(s["q"][first + i].double(), k[:lim], v[:lim], D ** -0.5, 2.0 ** -8, 2.0 ** -11)
                ref.check(s["out"][first + i], want, bound, f"step {n}, sequence {b}, row {i}")
        now = e.ctx.tolist()
        for b in range(B):
            history[b] = history[b][:now[b]]
            left[b] = max(0, left[b] - q_lens[b])
            if now[b] == 0:
                left[b] = r.randrange(1, 500)  # a new request in its place
    held = sum(-(-x // BS) for x in e.ctx.tolist())
    assert int(e.nfree) == NB - held


def test_steps_from_a_graph_when_blocks_run_out():
    """A decode step of one token per sequence, captured once and replayed until the pool is empty: sequences that get
    no block keep their length and write nothing; the others go on; freed blocks are taken up again."""
    B, Hq, Hkv, D, MBS, NB = 5, 8, 2, 128, 8, 11
    e = Engine(B, NB, MBS, Hq, Hkv, D, True, 5)
    T = B + 1  # one padded row
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=e.g).to(torch.bfloat16).to(DEV)
    q = torch.ones(B, dtype=i32, device=DEV)
    keep = torch.full((B,), 1 << 20, dtype=i32, device=DEV)
    granted, cu, pos = (torch.empty(n, dtype=i32, device=DEV) for n in (B, B + 1, T))
    slots = torch.empty(T, dtype=torch.int64, device=DEV)
    qo, out = (torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table, qw, kw = e.dev

    def go():
        pg.pa_plan_step(e.bt, e.ctx, q, e.free, e.nfree, NB, e.ctx, e.nfree, granted, cu, pos, slots)
        pg.pa_norm_rope_and_cache_fp8(qo, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], e.kc, e.vc, slots, *e.sc, table, pos,
                                      qw, kw)
        pg.pa_decode_fp8(out[:B], qo[:B], e.kc, e.vc, *e.sc, e.bt, e.ctx, D ** -0.5)
        pg.pa_release_blocks(e.bt, e.ctx, keep, e.free, e.nfree, NB, e.ctx, e.nfree)

    go()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    lens = [1] * B
    for n in range(60):
        if n == 45:  # sequence 0 is over: its blocks go to those that wait
            keep[0], q[0] = 0, 0
            graph.replay()
            keep[0] = 1 << 20
        else:
            graph.replay()
        got = granted.tolist()
        want, bt, s = [a + b for a, b in zip(lens, got)], e.bt.cpu(), slots.tolist()
        now = e.ctx.tolist()
        assert now == ([0] + want[1:] if n == 45 else want)
        for b in range(B):
            full = lens[b] % BS == 0
            assert got[b] == 1 or full or (b == 0 and n >= 45)
            at = lens[b]
            row = cu.tolist()[b]
            if got[b]:
                assert s[row] == int(bt[b, at // BS]) * BS + at % BS
        lens = now
        assert int(e.nfree) == NB - sum(-(-v // BS) for v in lens)
        k64, v64 = e.cache()
        for b in range(B):
            if n == 45 and b == 0:
                continue
            want_o, bound, _, _ = ref.attend(qo[b].cpu().double(), *[ref.rows_at(c, bt[b], torch.arange(lens[b]))[0] for c in (k64, v64)],
                                             D ** -0.5, 2.0 ** -8, 2.0 ** -11)
            if lens[b]:
                ref.check(out[b], want_o, bound, f"replay {n} sequence {b}")
    assert max(lens) > 16 and min(lens[1:]) >= 16
