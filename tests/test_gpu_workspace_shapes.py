"""One zero-filled workspace serves the dense, sparse, Quest and multi-row decode
calls in any order and of any batch size and head shape: every call gives the
bits that it gives with a fresh workspace."""

import pytest
import torch

import paged_gqa_decode_reshape_gb300 as pg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BS = 16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import paged_gqa_decode_reshape_gb300.build as b
    b.build()


def case(B, n, Hq, Hkv, D, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)
    nb = -(-n // BS)
    kc, vc = rnd(B * nb, BS, Hkv, D), rnd(B * nb, BS, Hkv, D)
    bt = torch.arange(B * nb, dtype=torch.int32, device=DEV).view(B, nb).contiguous()
    return rnd(B, Hq, D), kc, vc, bt, torch.full((B,), n, dtype=torch.int32, device=DEV)


def calls(B, n, Hq, Hkv, D, seed):
    """(workspace bytes, call taking out and workspace, query) of every kind of call on one batch."""
    q, kc, vc, bt, ctx = case(B, n, Hq, Hkv, D, seed)
    NB, MBS, scale = kc.shape[0], bt.shape[1], D ** -0.5
    top = min(MBS, 24)
    sel = torch.arange(top, dtype=torch.int32, device=DEV).expand(B, Hkv, top).contiguous()
    kmin, kmax = torch.empty(NB, Hkv, D, dtype=torch.bfloat16, device=DEV), torch.empty(NB, Hkv, D,
                                                                                        dtype=torch.bfloat16, device=DEV)
    pg.quest_rebuild_meta(kmin, kmax, kc, bt, ctx)
    cu = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    dense = pg.pa_decode_workspace_size(B, Hq, Hkv, D)
    found = [
        (dense, lambda o, ws: pg.pa_decode(o, q, kc, vc, bt, ctx, scale, workspace=ws), q),
        (dense, lambda o, ws: pg.quest_sparse_decode(o, q, kc, vc, bt, ctx, sel, scale, workspace=ws), q),
        (pg.quest_decode_workspace_size(B, Hq, Hkv, D, MBS),
         lambda o, ws: pg.quest_decode(o, torch.empty_like(sel), q, kmin, kmax, kc, vc, bt, ctx, top, scale,
                                       workspace=ws), q),
    ]
    if B <= 2048:
        found.append((pg.pa_decode_multi_workspace_size(B, Hq, Hkv, D),
                      lambda o, ws: pg.pa_decode_multi(o, q, kc, vc, bt, cu, ctx, scale, workspace=ws), q))
    return found


def bits(t):
    return t.view(torch.int16)


def run_in_turn(work, order):
    alone = []
    for n, f, q in work:
        o = torch.full_like(q, 7.0)
        f(o, torch.zeros(n, dtype=torch.uint8, device=DEV))
        alone.append(o)
    shared = torch.zeros(max(n for n, _, _ in work), dtype=torch.uint8, device=DEV)
    for i in order:
        n, f, q = work[i]
        got = torch.full_like(q, 7.0)
        f(got, shared)
        assert torch.equal(bits(got), bits(alone[i])), f"call {i}: {int((got != alone[i]).any(-1).sum())} rows differ"
        assert pg.pa_workspace_status(shared) == 0


def test_batch_sizes_in_turn():
    """A batch of 16 long sequences, then 200 shorter ones, then 16 again."""
    work = calls(16, 3000, 28, 4, 128, 1)[:1] + calls(200, 700, 28, 4, 128, 2)[:1]
    run_in_turn(work, [0, 1, 0, 1, 1, 0])


def test_every_call_and_shape_in_turn():
    work = (calls(2, 4000, 28, 4, 128, 1) + calls(40, 900, 16, 4, 64, 2) + calls(300, 300, 8, 8, 128, 3) +
            calls(700, 130, 6, 3, 64, 4) + calls(1, 9000, 5, 1, 128, 5))
    order = torch.randperm(4 * len(work), generator=torch.Generator().manual_seed(3)) % len(work)
    run_in_turn(work, order.tolist())


def test_more_counters_than_the_fixed_area():
    """4096 sequences of 32 KV heads have more segments than a workspace keeps counters for at its fixed place."""
    work = calls(16, 3000, 28, 4, 128, 1)[:1] + calls(4096, 40, 64, 32, 64, 2)[:1]
    run_in_turn(work, [0, 1, 0, 1])
    multi = calls(16, 3000, 28, 4, 128, 1)[3:] + calls(2048, 40, 64, 32, 64, 2)[3:]
    run_in_turn(multi + work[:1], [0, 1, 0, 2, 1])


def test_the_bindings_own_workspace():
    """Calls without workspace=, of a small batch after a large one and a large one after it."""
    a, b = calls(200, 700, 28, 4, 128, 1)[0], calls(16, 3000, 28, 4, 128, 2)[0]
    want = [f(torch.full_like(q, 7.0), torch.zeros(n, dtype=torch.uint8, device=DEV)) for n, f, q in (a, b)]
    for i in (0, 1, 0, 1, 0):
        n, f, q = (a, b)[i]
        assert torch.equal(bits(f(torch.full_like(q, 7.0), None)), bits(want[i])), i
