"""Values that are not finite in windowed decode calls of several rows, in every
way the row-tile kernel ends a unit: a whole unit in one CTA, a unit cut between
CTAs and merged by a kernel of its own, and one merged by the last CTA."""

import pytest
import torch

import paged_gqa_decode_reshape_gb300 as pg
from tests import subset_reference as ref
from tests.subset_reference import BS
from tests.test_gpu_subset import DEV, NAN, bf16, dev, pool, widened

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import paged_gqa_decode_reshape_gb300.build as b
    b.build()


# further sequences (tokens, rows): few long units are cut and joined by a kernel of their own, many are cut
# and merged by the last CTA, and with units of one tile each most are whole
FILL = {"joined": [], "merged": [(500, 2)] * 60, "whole": [(90, 2)] * 400}


@pytest.mark.parametrize("fill", list(FILL))
def test_infinite_keys_have_weight_zero(fill):
    """A key of infinite size whose logit is -inf has weight 0, also in rows that are computed again because
    another row of their tile sees a token that is not finite."""
    Hq, Hkv, D, scale = 14, 2, 128, 0.1
    ctx, ql = [90, 400] + [c for c, _ in FILL[fill]], [20, 30] + [r for _, r in FILL[fill]]
    g, kc, vc, bt, _, _ = pool(51, ctx, Hkv, D, spoil=False)
    q = bf16(g, sum(ql), Hq, D)
    q[:, :, 3] = -1.0
    gone = {0: [0, 40], 1: [0, 1, 200]}  # tokens with a logit of -inf in every row and head
    for b in range(2):
        for t in gone[b]:
            kc[bt[b, t // BS], t % BS, :, 3] = INF
        t = ctx[b] - 1  # seen by the last row only
        vc[bt[b, t // BS], t % BS, 0, 5:9] = NAN
    cu = torch.tensor([0] + torch.tensor(ql).cumsum(0).tolist(), dtype=torch.int32)
    out = torch.full((sum(ql), Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    pg.pa_decode_window_multi(out, *dev(q, kc, vc, widened(bt, sum(ql), Hkv, D), cu,
                                        torch.tensor(ctx, dtype=torch.int32)), 1 << 20, 0, scale)
    got = out.double().cpu()
    for b in range(2):
        for i in range(ql[b]):
            t = torch.arange(ctx[b] - ql[b] + i + 1)
            t = t[~torch.isin(t, torch.tensor(gone[b]))]
            want, bound, _, _ = ref.attend(q[int(cu[b]) + i].double(), ref.rows_at(kc, bt[b], t)[0],
                                           ref.rows_at(vc, bt[b], t)[0], scale)
            r, fine = got[int(cu[b]) + i], torch.isfinite(want)
            assert fine.all() == (i < ql[b] - 1)
            assert torch.equal(torch.isfinite(r), fine), f"sequence {b} row {i}"
            assert ((r - want).abs() - bound)[fine].max() <= 0, f"sequence {b} row {i}"
