"""Norm and rotation of queries and keys, with and without the cache write,
against the formulas in 64 bits (tests/step_reference.py, with derived bounds),
at the head shapes, partial rotations, strides and slots where they can go wrong."""

import pytest
import torch

import paged_gqa_decode_reshape_gb300 as pg
from tests import step_reference as ref
from tests.subset_reference import BS, V8_POS, check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import paged_gqa_decode_reshape_gb300.build as b
    b.build()


def make(seed, T, Hq, Hkv, D, R, A=1, P=300, packed=True, norm=(True, True)):
    """Host inputs: q, k, v (parts of one tensor when packed), weights, table, positions, axes."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    if packed:
        x = (n(T, Hq + 2 * Hkv + 1, D) * 2).to(torch.bfloat16)  # one head more than is used
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:Hq + 2 * Hkv]
    else:
        q, k, v = ((n(T, h, D) * 2).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    qw, kw = ((1 + 0.3 * n(D)).to(torch.bfloat16) if w else None for w in norm)
    table = torch.rand(P, R, generator=g) * 2 - 1  # any values: rows are not always cosines and sines
    pos = torch.randint(0, P, (T,) if A == 1 else (A, T), generator=g, dtype=torch.int32)
    axes = None if A == 1 else torch.randint(0, A, (R // 2,), generator=g, dtype=torch.int32)
    return q, k, v, qw, kw, table, pos, axes


def to_dev(*ts):
    """On the device, with the strides they have here (parts of one tensor stay parts of one)."""
    out = []
    for t in ts:
        if t is None:
            out.append(None)
        elif t.is_contiguous():
            out.append(t.to(DEV))
        else:
            whole = torch.empty(0, dtype=t.dtype).set_(t.untyped_storage()).to(DEV)
            out.append(whole.as_strided(t.shape, t.stride(), t.storage_offset()))
    return out


SHAPES = [(28, 4, 128), (8, 8, 128), (1, 1, 128), (5, 1, 64), (32, 4, 64), (9, 3, 64), (40, 8, 128), (3, 2, 128)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,A,packed", [(1, 1, False), (7, 3, True), (130, 1, True), (700, 2, True)])
@pytest.mark.parametrize("heads", SHAPES)
def test_norm_rope(heads, T, A, packed, interleaved):
    Hq, Hkv, D = heads
    for i, R in enumerate(sorted({16, D // 2, D - 16, D})):
        norm = [(True, True), (False, True), (True, False), (False, False)][i]
        q, k, _, qw, kw, table, pos, axes = make(T + R, T, Hq, Hkv, D, R, A, packed=packed, norm=norm)
        q_, k_, qw_, kw_, table_, pos_, axes_ = to_dev(q, k, qw, kw, table, pos, axes)
        qo, ko = (torch.full((T, h, D), 7.0, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv))
        pg.pa_norm_rope(qo, ko, q_, k_, table_, pos_, qw_, kw_, 1e-5, axes_, interleaved)
        cos, sin = ref.angles(table, pos, axes)
        for got, x, w, what in ((qo, q, qw, "q"), (ko, k, kw, "k")):
            z, S = ref.norm_rope(x, w, 1e-5, cos, sin, interleaved)
            check(got, z, ref.bf16_bound(z, S, D), f"{what}, R {R}")


def slots_of(seed, T, NB):
    """Distinct slots: whole blocks, runs that start and end inside blocks, single tokens, and tokens without one."""
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(NB, generator=g)
    s, b = [], 0
    while len(s) < T:
        o = int(torch.randint(0, 16, (1,), generator=g))
        n = [1, 16 - o, 16 + 16 - o, 3][b % 4] if b % 7 else 16
        o = 0 if b % 7 == 0 else o
        run = [int(perm[b + (o + i) // BS]) * BS + (o + i) % BS for i in range(n)]
        s += run if b % 5 != 3 else [-1] * (n % 4)
        b += (o + n - 1) // BS + 1
    out = torch.tensor(s[:T])
    if T > 4:
        out[2], out[T - 1] = -1, NB * BS + 3
    return out


@pytest.mark.parametrize("keep_k", [False, True])
@pytest.mark.parametrize("T", [1, 3, 64, 517])
@pytest.mark.parametrize("heads", [(28, 4, 128), (2, 1, 128), (32, 8, 128), (9, 3, 64)])
def test_cache(heads, T, keep_k):
    Hq, Hkv, D = heads
    NB = T + 12
    q, k, v, qw, kw, table, pos, axes = make(T, T, Hq, Hkv, D, D, 3)
    slots = slots_of(T, T, NB)
    g = torch.Generator().manual_seed(9)
    kc, vc = (torch.randn(NB, BS, Hkv, D, generator=g).to(torch.bfloat16) for _ in range(2))
    q_, k_, v_, qw_, kw_, table_, pos_, axes_, slots_, kc_, vc_ = to_dev(q, k, v, qw, kw, table, pos, axes, slots, kc, vc)
    qo = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV)
    ko = torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=DEV) if keep_k else None
    pg.pa_norm_rope_and_cache(qo, q_, k_, v_, kc_, vc_, slots_, table_, pos_, qw_, kw_, 1e-6, axes_, k_out=ko)
    # the same bits as the two calls
    q2, k2, kc2, vc2 = qo.clone(), torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=DEV), *to_dev(kc, vc)
    pg.pa_norm_rope(q2, k2, q_, k_, table_, pos_, qw_, kw_, 1e-6, axes_)
    pg.pa_reshape_and_cache(k2, v_.contiguous(), kc2, vc2, slots_)
    bits = lambda t: t.view(torch.int16)
    assert torch.equal(bits(qo), bits(q2)) and torch.equal(bits(kc_), bits(kc2)) and torch.equal(bits(vc_), bits(vc2))
    if keep_k:
        assert torch.equal(bits(ko), bits(k2))
    # and what the formulas say, in the slots and nowhere else
    cos, sin = ref.angles(table, pos, axes)
    z, S = ref.norm_rope(k, kw, 1e-6, cos, sin, False)
    ok = (slots >= 0) & (slots < NB * BS)
    want, bound = kc.double().view(-1, Hkv, D), torch.zeros(NB * BS, Hkv, D).double()
    want[slots[ok]], bound[slots[ok]] = z[ok], ref.bf16_bound(z, S, D)[ok]
    check(kc_.view(-1, Hkv, D), want, bound, "key_cache")
    want = vc.clone().view(-1, Hkv, D)
    want[slots[ok]] = v[ok]
    assert torch.equal(bits(vc_.cpu().view(-1, Hkv, D)), bits(want))


@pytest.mark.parametrize("T", [1, 3, 64, 517])
@pytest.mark.parametrize("heads", [(28, 4), (2, 1), (32, 8), (6, 3)])
def test_cache_fp8(heads, T):
    (Hq, Hkv), D, NB = heads, 128, T + 12
    q, k, v, qw, kw, table, pos, _ = make(T + 1, T, Hq, Hkv, D, 64)
    slots = slots_of(T + 5, T, NB)
    g = torch.Generator().manual_seed(9)
    kc = torch.randint(0, 256, (NB, BS, Hkv, D), generator=g, dtype=torch.uint8)
    vc = torch.randint(0, 256, (NB, Hkv, D, BS), generator=g, dtype=torch.uint8)
    ks, vs = 0.01 * (1 + torch.arange(Hkv) / 3), 0.02 * (1 + torch.arange(Hkv) / 5)
    v[0, 0, :4] = torch.tensor([1e6, -1e6, float("inf"), 1e-30]).to(torch.bfloat16)  # saturates, and rounds to 0
    q_, k_, v_, qw_, kw_, table_, pos_, slots_, kc_, vc_, ks_, vs_ = to_dev(q, k, v, qw, kw, table, pos, slots, kc, vc, ks, vs)
    qo = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV)
    ko = torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=DEV)
    pg.pa_norm_rope_and_cache_fp8(qo, q_, k_, v_, kc_, vc_, slots_, ks_, vs_, table_, pos_, qw_, kw_, k_out=ko)
    cos, sin = ref.angles(table, pos, None)
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        z, S = ref.norm_rope(x, w, 1e-6, cos, sin, False)
        check(got, z, ref.bf16_bound(z, S, D), "rotated")
    ok = (slots >= 0) & (slots < NB * BS)
    # values are the codes of the write path that is there already, bit for bit; so is every other byte
    kc2, vc2 = to_dev(kc, vc)
    pg.pa_reshape_and_cache_fp8(ko, v_.contiguous(), kc2, vc2, slots_, ks_, vs_)
    assert torch.equal(vc_, vc2)
    z, S = ref.norm_rope(k, kw, 1e-6, cos, sin, False)
    got = kc_.cpu().view(-1, Hkv, D)
    check(got[slots[ok]].view(E4M3).double(), (z / ks.double()[:, None]).clamp(-448, 448)[ok],
          ref.code_bound(z, S, D, ks.double()[:, None])[ok], "key codes")
    rest = torch.ones(NB * BS, dtype=torch.bool)
    rest[slots[ok]] = False
    assert torch.equal(got[rest], kc.view(-1, Hkv, D)[rest])


@pytest.mark.parametrize("heads,T", [((1, 1, 128), 4096), ((2, 2, 128), 5003), ((5, 1, 64), 4500), ((9, 3, 64), 3001),
                                     ((28, 4, 128), 900), ((3, 2, 128), 2500), ((40, 8, 128), 2600)])
def test_many_tokens(heads, T):
    """From about 4096 steps of heads on, where warps go over ranges of them; tokens of one step and of many."""
    for A, interleaved in ((1, False), (3, True), (4, False), (1, True)):
        test_norm_rope(heads, T, A, True, interleaved)
    test_cache(heads, T, True)
    if heads[2] == 128:
        test_cache_fp8(heads[:2], T)


@pytest.mark.parametrize("T", [300, 1500])
def test_in_place_on_one_projection(T):
    Hq, Hkv, D = 12, 4, 128
    q, k, v, qw, kw, table, pos, _ = make(3, T, Hq, Hkv, D, D)
    whole = torch.empty(0, dtype=q.dtype).set_(q.untyped_storage()).view(T, Hq + 2 * Hkv + 1, D)
    x = whole.to(DEV)
    q_, k_ = x[:, :Hq], x[:, Hq:Hq + Hkv]
    qw_, kw_, table_, pos_ = to_dev(qw, kw, table, pos)
    pg.pa_norm_rope(q_, k_, q_, k_, table_, pos_, qw_, kw_)
    cos, sin = ref.angles(table, pos, None)
    for got, y, w in ((q_, q, qw), (k_, k, kw)):
        z, S = ref.norm_rope(y, w, 1e-6, cos, sin, False)
        check(got, z, ref.bf16_bound(z, S, D), "in place")
    assert torch.equal(x[:, Hq + Hkv:].cpu(), whole[:, Hq + Hkv:])


def test_positions_and_axes_are_clamped():
    T, Hq, Hkv, D = 5, 2, 1, 64
    q, k, _, qw, kw, table, pos, axes = make(4, T, Hq, Hkv, D, 32, 2, P=9)
    pos[0] = torch.tensor([-1, 8, 9, 2 ** 31 - 1, -2 ** 31])
    axes[:4] = torch.tensor([-3, 2, 2 ** 31 - 1, 1])
    q_, k_, qw_, kw_, table_, pos_, axes_ = to_dev(q, k, qw, kw, table, pos, axes)
    qo, ko = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV), torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=DEV)
    pg.pa_norm_rope(qo, ko, q_, k_, table_, pos_, qw_, kw_, axes=axes_)
    z, S = ref.norm_rope(q, qw, 1e-6, *ref.angles(table, pos, axes), False)
    check(qo, z, ref.bf16_bound(z, S, D), "clamped")


def test_odd_values():
    """NaN and infinities stay in their head; a head of zeros is zero; tiny and huge values keep their norm."""
    T, Hq, Hkv, D = 4, 3, 1, 128
    q, k, _, qw, kw, table, pos, _ = make(6, T, Hq, Hkv, D, D, packed=False)
    q[0, 1, 5], q[1, 2, 9] = float("nan"), float("inf")
    q[2, 0] = 0
    q[3, 1] = q[3, 1] * 1e-18
    q[3, 2] = q[3, 2] * 1e17
    q_, k_, qw_, kw_, table_, pos_ = to_dev(q, k, qw, kw, table, pos)
    qo, ko = torch.empty_like(q_), torch.empty_like(k_)
    pg.pa_norm_rope(qo, ko, q_, k_, table_, pos_, qw_, kw_, 0.0)
    got = qo.double().cpu()
    z, S = ref.norm_rope(q, qw, 0.0, *ref.angles(table, pos, None), False)
    odd = torch.zeros(T, Hq, dtype=torch.bool)
    odd[0, 1] = odd[1, 2] = odd[2, 0] = True  # 0 / 0 without an eps: NaN by the formula
    assert torch.isnan(got[0, 1]).all() and not torch.isfinite(got[1, 2]).all()
    check(qo.cpu()[~odd], z[~odd], ref.bf16_bound(z, S, D)[~odd], "the others")
    pg.pa_norm_rope(qo, ko, q_, k_, table_, pos_, qw_, kw_, 1e-6)
    assert (qo[2, 0] == 0).all()


def test_large_strides_and_many_rows():
    """Rows further apart than 32 bits of bytes, and more rows than a grid dimension's 65535."""
    Hq, Hkv, D = 2, 1, 64
    big = torch.empty(3 * (1 << 30) + 1024, dtype=torch.bfloat16, device=DEV)  # 6 GB: rows 2 GB apart
    q, k, _, qw, kw, table, pos, _ = make(7, 3, Hq, Hkv, D, D, packed=False)
    q_ = big.as_strided((3, Hq, D), (1 << 30, D, 1))
    q_.copy_(q)
    k_, qw_, kw_, table_, pos_ = to_dev(k, qw, kw, table, pos)
    ko = torch.empty_like(k_)
    pg.pa_norm_rope(q_, ko, q_, k_, table_, pos_, qw_, kw_)
    z, S = ref.norm_rope(q, qw, 1e-6, *ref.angles(table, pos, None), False)
    check(q_, z, ref.bf16_bound(z, S, D), "far rows")
    del big, q_
    T = 70001
    q, k, _, qw, kw, table, pos, _ = make(8, T, Hq, Hkv, D, 32)
    q_, k_, qw_, kw_, table_, pos_ = to_dev(q, k, qw, kw, table, pos)
    qo, ko = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV), torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=DEV)
    pg.pa_norm_rope(qo, ko, q_, k_, table_, pos_, qw_, kw_)
    z, S = ref.norm_rope(q, qw, 1e-6, *ref.angles(table, pos, None), False)
    check(qo, z, ref.bf16_bound(z, S, D), "many rows")


def test_binding_refuses():
    T, Hq, Hkv, D = 4, 2, 1, 128
    q, k, v, qw, kw, table, pos, _ = make(9, T, Hq, Hkv, D, 64)
    q, k, v, qw, kw, table, pos = to_dev(q, k, v, qw, kw, table, pos)
    qo, ko = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV), torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=DEV)
    args = dict(q_out=qo, k_out=ko, query=q, key=k, cos_sin=table, positions=pos, q_weight=qw, k_weight=kw)
    pg.pa_norm_rope(**args)
    kc = torch.zeros(4, BS, Hkv, D, dtype=torch.bfloat16, device=DEV)
    axes = torch.zeros(32, dtype=torch.int32, device=DEV)
    for over, err in [
        (dict(query=q.float()), TypeError), (dict(query=q.cpu()), ValueError), (dict(query=q[:3]), ValueError),
        (dict(key=k[..., :64]), ValueError), (dict(q_out=ko), ValueError), (dict(k_out=None), TypeError),
        (dict(cos_sin=table.double()), TypeError), (dict(positions=pos.long()), TypeError), (dict(positions=pos[:3]), ValueError),
        (dict(q_weight=qw[:64]), ValueError), (dict(axes=axes), ValueError), (dict(positions=pos[None], axes=axes[:5]), ValueError),
        (dict(cos_sin=table[:, :24].contiguous()), pg.PagedDecodeError), (dict(eps=-1.0), pg.PagedDecodeError),
        (dict(query=q.transpose(0, 1).contiguous().transpose(0, 1)), ValueError),
    ]:
        with pytest.raises(err):
            pg.pa_norm_rope(**{**args, **over})
    slots = torch.arange(T, device=DEV)
    full = dict(q_out=qo, query=q, key=k, value=v, key_cache=kc, value_cache=kc.clone(), slot_mapping=slots, cos_sin=table,
                positions=pos)
    pg.pa_norm_rope_and_cache(**full)
    for over, err in [(dict(value=None), TypeError), (dict(value=q), ValueError), (dict(slot_mapping=slots[:2]), ValueError),
                      (dict(slot_mapping=slots.int()), TypeError), (dict(value_cache=kc[:2]), ValueError),
                      (dict(key_cache=kc.to(torch.uint8)), TypeError)]:
        with pytest.raises(err):
            pg.pa_norm_rope_and_cache(**{**full, **over})
    with pytest.raises(TypeError):
        pg.pa_norm_rope_and_cache_fp8(**full, k_scale=torch.ones(1, device=DEV), v_scale=torch.ones(1, device=DEV))
