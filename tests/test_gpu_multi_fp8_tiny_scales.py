"""Chunk attention over the 8-bit caches with scales and queries at the lower end of
their ranges, against plain 64-bit forms (tests/subset_reference.py)."""

import pytest
import torch

from tests import subset_reference as ref
from tests.test_gpu_subset import DEV, NAN, bf16, dev, pool
from tests.test_gpu_window_multi_fp8 import D, _cuda, call, codes, filler, offsets, wide  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("share", [False, True])
@pytest.mark.parametrize("per_block,k_power,q_power,scale", [
    (False, -120, -60, 0.0884), (False, -126, -100, 0.0884), (False, -40, -40, 2.0 ** -100), (True, None, -60, 2.0 ** -100)])
def test_logits_too_small_for_fp32(per_block, k_power, q_power, scale, share):
    """Scales and queries whose product is below every fp32 number: all tokens that a row sees weigh the same, and the
    others nothing."""
    Hq, Hkv, ctx, ql = 8, 2, [700, 3], [20, 5]
    assert not filler(25, 2, Hkv, 1 << 20, 0)
    g, kc, vc, bt, _, _ = pool(79, ctx, Hkv, D)
    k8, v8, ks, vs, k64, v64 = codes(kc, vc, per_block, Hkv)
    if k_power is not None:
        k64 = k64 / ks.double()[:, None] * 2.0 ** k_power
        ks = torch.full_like(ks, 2.0 ** k_power)
    q, cu = (bf16(g, 25, Hq, D).float() * 2.0 ** q_power).to(torch.bfloat16), offsets(ql)
    out = torch.full((25, Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    call(per_block, out, *dev(q, k8, v8, ks, vs, wide(bt) if share else bt, cu, torch.tensor(ctx, dtype=torch.int32)),
         1 << 20, 0, scale)
    for b, x in enumerate(ctx):
        for i in range(ql[b]):
            t = torch.arange(max(x - ql[b] + i + 1, 0))
            k, v = ref.rows_at(k64, bt[b], t)[0], ref.rows_at(v64, bt[b], t)[0]
            want, bound, _, _ = ref.attend(q[int(cu[b]) + i].double(), k, v, scale)
            ref.check(out[int(cu[b]) + i], want, bound, f"sequence {b} row {i}")
