"""Offsets past 32 bits, the largest steps, and calls beside each other: the step's calls and the chunks over the 8-bit
caches give at the far end of a large cache, or of many rows, what they give at its beginning, bit for bit."""

import pytest
import torch

import paged_gqa_decode_reshape_gb300 as pg
from tests import step_reference as sref
from tests.subset_reference import BS
from tests.test_gpu_subset import DEV, bf16, dev, pool
from tests.test_gpu_window_multi_fp8 import call, check_rows, codes, filler, offsets, wide

pytestmark = pytest.mark.gpu
D = 128
i32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import paged_gqa_decode_reshape_gb300.build as b
    b.build()


@pytest.mark.parametrize("share", [False, True])
@pytest.mark.parametrize("per_block", [False, True])
def test_chunks_at_the_end_of_a_large_cache(per_block, share):
    """The same blocks at the beginning of the pool and past 4 GB of it."""
    Hq, Hkv, ctx, ql = 28, 4, [1000, 77, 300], [20, 9, 30]
    g, kc, vc, bt, _, _ = pool(5, ctx, Hkv, D)
    k8, v8, ks, vs, k64, v64 = codes(kc, vc, per_block, Hkv)
    n, NB = k8.shape[0], (1 << 32) // (BS * Hkv * D) + 1000  # codes of more than 4 GB
    assert not share or not filler(sum(ql), 3, Hkv, 1 << 30, 0)
    q, cu, at = bf16(g, sum(ql), Hq, D, std=2.0), offsets(ql), NB - n
    K, V = torch.empty(NB, BS, Hkv, D, dtype=torch.uint8, device=DEV), torch.empty(NB, Hkv, D, BS, dtype=torch.uint8, device=DEV)
    K[:n], V[:n] = k8.to(DEV), v8.to(DEV)
    K[at:], V[at:] = K[:n], V[:n]
    if per_block:
        S = [torch.empty(NB, Hkv, device=DEV) for _ in range(2)]
        for s, x in zip(S, (ks, vs)):
            s[:n] = x.to(DEV)
            s[at:] = s[:n]
    else:
        S = dev(ks, vs)
    rows, c, lens = dev(q, cu, torch.tensor(ctx, dtype=i32))
    outs = []
    for shift in (0, at):
        table = torch.where(bt < 0, bt, bt + shift)
        out = torch.empty_like(rows)
        call(per_block, out, rows, K, V, *S, (wide(table) if share else table).to(DEV), c, lens, 1 << 30, 0, D ** -0.5)
        outs.append(out.cpu())
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
    check_rows(outs[1], q, k64, v64, bt, cu, ctx, ql, 1 << 30, 0, D ** -0.5, 7)


@pytest.mark.parametrize("fp8", [False, True])
def test_norm_and_rotation_of_rows_past_4_gb(fp8):
    """The last rows of a projection of more than 2^32 bytes, into slots past 4 GB of the cache, as a call of their own."""
    Hq, Hkv, T, last = 2, 1, 300000, 2000
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.empty(T, 64, D, dtype=torch.bfloat16, device=DEV)  # 4.9 GB, of which few heads are used
    x[:last] = 0
    x[T - last:] = torch.randn(last, 64, D, generator=g, device=DEV).to(torch.bfloat16)
    x[last:T - last, :Hq + 2 * Hkv] = 1
    NB = (1 << 32) // (BS * Hkv * D) // (1 if fp8 else 2) + 1000
    table = torch.rand(4000, D, generator=g, device=DEV)
    pos = torch.randint(0, 4000, (T,), generator=g, device=DEV, dtype=i32)
    w = torch.rand(D, generator=g, device=DEV).to(torch.bfloat16)
    slots = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    slots[T - last:] = NB * BS - last + torch.arange(last, device=DEV)
    far = slots[T - last:]
    sc = torch.full((Hkv,), 0.03, device=DEV)

    def run(t0, n, slots, blocks):
        if fp8:
            kc = torch.zeros(blocks, BS, Hkv, D, dtype=torch.uint8, device=DEV)
            vc = torch.zeros(blocks, Hkv, D, BS, dtype=torch.uint8, device=DEV)
        else:
            kc, vc = (torch.zeros(blocks, BS, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        r = x[t0:t0 + n]
        qo = torch.zeros(n, Hq, D, dtype=torch.bfloat16, device=DEV)
        args = qo, r[:, :Hq], r[:, Hq:Hq + Hkv], r[:, Hq + Hkv:Hq + 2 * Hkv], kc, vc, slots
        if fp8:
            pg.pa_norm_rope_and_cache_fp8(*args, sc, sc, table, pos[t0:t0 + n], w, w)
        else:
            pg.pa_norm_rope_and_cache(*args, table, pos[t0:t0 + n], w, w)
        return qo[-last:].clone(), kc[-(last // BS):].clone(), vc[-(last // BS):].clone()

    whole = run(0, T, slots, NB)
    alone = run(T - last, last, far - (NB * BS - last), last // BS)
    for a, b in zip(whole, alone):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)) and bool(b.any())


def test_the_largest_step():
    B, T = 4096, 1 << 20
    g = torch.Generator().manual_seed(1)
    ctx, q = (torch.randint(0, n, (B,), generator=g, dtype=i32) for n in (3000, 500))
    q[7] = 0
    MBS = 220
    need = int(sum(-(-(a + b) // BS) - -(-a // BS) for a, b in zip(ctx.tolist(), q.tolist())))
    used = int(sum(-(-a // BS) for a in ctx.tolist()))
    NB = used + need + 9
    perm = torch.randperm(NB, generator=g).int()
    bt, at = torch.full((B, MBS), -1, dtype=i32), 0
    for b, n in enumerate((-(-ctx // BS)).tolist()):
        bt[b, :n] = perm[at:at + n]
        at += n
    free = torch.cat([perm[at:], torch.full((at,), -5, dtype=i32)])
    nf = need + 9
    want = sref.plan(bt, ctx, q, free, nf, NB, T)
    bt_, ctx_, q_, free_, nf_ = (x.to(DEV) for x in (bt, ctx, q, free, torch.tensor([nf], dtype=i32)))
    granted, cu, pos = (torch.empty(n, dtype=i32, device=DEV) for n in (B, B + 1, T))
    slots = torch.empty(T, dtype=torch.int64, device=DEV)
    pg.pa_plan_step(bt_, ctx_, q_, free_, nf_, NB, ctx_, nf_, granted, cu, pos, slots)
    for a, b in zip((bt_, ctx_, nf_, granted, cu, pos, slots), want):
        assert torch.equal(a.cpu(), b)
    # and all of it back: every block is on the stack again, once
    pg.pa_release_blocks(bt_, ctx_, torch.zeros_like(ctx_), free_, nf_, NB, ctx_, nf_)
    assert int(nf_) == NB and torch.equal(free_[:NB].sort().values.cpu(), torch.arange(NB, dtype=i32))
    assert not ctx_.any()


def test_calls_beside_each_other():
    """Two streams, each with its own chunks, in turn and without waiting: shared reads and each row for itself."""
    Hq, Hkv = 28, 4
    runs = []
    for n, (ctx, ql, share) in enumerate([([2000, 900], [200, 64], True), ([600, 1500, 40], [1, 4, 2], False)]):
        g, kc, vc, bt, _, _ = pool(60 + n, ctx, Hkv, D)
        k8, v8, ks, vs, k64, v64 = codes(kc, vc, False, Hkv)
        q, cu = bf16(g, sum(ql), Hq, D), offsets(ql)
        args = dev(q, k8, v8, ks, vs, wide(bt) if share else bt, cu, torch.tensor(ctx, dtype=i32))
        runs.append((torch.cuda.Stream(), args, [torch.empty_like(args[0]) for _ in range(30)], (q, k64, v64, bt, cu, ctx, ql)))
    torch.cuda.synchronize()
    for i in range(30):
        for st, args, outs, _ in runs:
            with torch.cuda.stream(st):
                call(False, outs[i], *args, 1 << 30, 0, 0.0884)
    torch.cuda.synchronize()
    for _, _, outs, r in runs:
        for o in outs[1:]:
            assert torch.equal(o.view(torch.int16), outs[0].view(torch.int16))
        check_rows(outs[0], *r, 1 << 30, 0, 0.0884, 11)
