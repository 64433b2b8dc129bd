"""What the chunk attention over the 8-bit caches makes of its queries where rows
share reads, against plain 64-bit forms (tests/subset_reference.py)."""

import pytest
import torch

from tests import subset_reference as ref
from tests.test_gpu_subset import DEV, NAN, dev, pool
from tests.test_gpu_window_multi_fp8 import D, _cuda, call, codes, filler, offsets, wide  # noqa: F401
from tests.test_query_parts import parts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [-30, 0, 30])
@pytest.mark.parametrize("per_block", [False, True])
def test_small_queries_beside_a_large_one(per_block, power):
    """Shared reads take a head row as two E4M3 parts: values below 2^-9 of its largest may lose their last bit, and the
    call computes with what the parts stand for. Keys that add up these losses make them visible."""
    Hq, Hkv, ctx, ql = 8, 2, [1000], [12]
    assert not filler(12, 1, Hkv, 1 << 20, 0)
    g, kc, vc, bt, _, _ = pool(78, ctx, Hkv, D)
    # 1, and 127 values in [2^-10, 2^-9) whose last bit of eight is set, of either sign
    m = 129 + 2 * torch.randint(0, 64, (D,), generator=g)
    q = m / 128 * 2.0 ** -10 * (1 - 2 * torch.randint(0, 2, (D,), generator=g))
    q[0] = 1.0
    off = parts(q.double(), torch.tensor(1.0).double()) - q.double()
    assert (off[1:].abs() == 2.0 ** -17).all()
    side = 1.0 - 2 * torch.randint(0, 2, kc.shape[:3], generator=g)[..., None]
    kc = torch.where(torch.isnan(kc), kc, (side * off.sign().float()).to(torch.bfloat16))  # dim 0: 0
    vc = torch.where(torch.isnan(vc), vc, (side * (1 + torch.rand(vc.shape, generator=g))).to(torch.bfloat16))
    k8, v8, ks, vs, k64, v64 = codes(kc, vc, per_block, Hkv)
    rows = (q * 2.0 ** power).expand(12, Hq, D).to(torch.bfloat16)
    out = torch.full((12, Hq, D), NAN, dtype=torch.bfloat16, device=DEV)
    scale = 50 * 2.0 ** -power
    call(per_block, out, *dev(rows.contiguous(), k8, v8, ks, vs, wide(bt), offsets(ql), torch.tensor(ctx, dtype=torch.int32)),
         1 << 20, 0, scale)
    held = (q.double() + off) * 2.0 ** power
    for i in range(12):
        t = torch.arange(1000 - 12 + i + 1)
        k, v = ref.rows_at(k64, bt[0], t)[0], ref.rows_at(v64, bt[0], t)[0]
        want, bound, _, _ = ref.attend(held.expand(Hq, D), k, v, scale)
        ref.check(out[i], want, bound, f"row {i}")
        exact, bound, _, _ = ref.attend(rows[i].double(), k, v, scale)
        assert ((want - exact).abs() > bound).any()  # seen above the other roundings
        # a logit is off by at most e, an average of values by at most (exp(2 e) - 1) times that of their magnitudes
        e = scale * 2.0 ** -17 * rows.double().abs().max() * k.abs().sum(2).max()
        assert ((out[i].double().cpu() - exact).abs() <= bound + torch.expm1(2 * e) * v.abs().amax()).all()
