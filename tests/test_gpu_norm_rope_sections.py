"""Rotation with several position axes whose frequencies come in contiguous
sections (time, height, width), as models lay them out: where four neighbouring
frequencies share an axis their cosines and sines are read sixteen bytes at a
time. Few tokens and many, against the formulas in 64 bits."""

import pytest
import torch

import paged_gqa_decode_reshape_gb300 as pg
from tests import step_reference as ref
from tests.subset_reference import BS, check
from tests.test_gpu_norm_rope import DEV, E4M3, _cuda, make, slots_of, to_dev  # noqa: F401

pytestmark = pytest.mark.gpu

# sections of the R / 2 frequencies, (axis, how many); frequencies from 32 on of another axis than those below
SECTIONS = [
    ((0, 16), (1, 24), (2, 24)), ((0, 32), (1, 32)), ((3, 16), (2, 16), (1, 16), (0, 16)), ((2, 4), (0, 28), (1, 32)),
    ((0, 8), (1, 12), (2, 12)), ((1, 28), (0, 4)), ((0, 8), (1, 8), (2, 8), (3, 8)),
    ((0, 16), (1, 32)), ((1, 36), (0, 12)), ((0, 4), (1, 4)), ((2, 4), (1, 4), (0, 8)),
]
# heads and tokens of a warp per step, and of a warp per range of steps (4096 steps of four or eight heads and more)
CALLS = [((28, 4, 128), 37), ((28, 4, 128), 700), ((3, 2, 128), 2500), ((9, 3, 64), 5), ((9, 3, 64), 1500)]


def sectioned(seed, T, heads, sections, packed=True):
    Hq, Hkv, D = heads
    R, A = 2 * sum(n for _, n in sections), 1 + max(a for a, _ in sections)
    q, k, v, qw, kw, table, pos, _ = make(seed, T, Hq, Hkv, D, R, A, packed=packed)
    axes = torch.cat([torch.full((n,), a, dtype=torch.int32) for a, n in sections])
    assert (axes.view(-1, 4) == axes.view(-1, 4)[:, :1]).all()
    return q, k, v, qw, kw, table, pos, axes


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,T", CALLS)
@pytest.mark.parametrize("sections", SECTIONS, ids=lambda s: "-".join(f"{a}x{n}" for a, n in s))
def test_sections(sections, heads, T, interleaved):
    D = heads[2]
    if 2 * sum(n for _, n in sections) > D:
        pytest.skip("more frequencies than a head of 64 has")
    q, k, _, qw, kw, table, pos, axes = sectioned(T, T, heads, sections)
    q_, k_, qw_, kw_, table_, pos_, axes_ = to_dev(q, k, qw, kw, table, pos, axes)
    qo, ko = (torch.full((T, h, D), 7.0, dtype=torch.bfloat16, device=DEV) for h in heads[:2])
    pg.pa_norm_rope(qo, ko, q_, k_, table_, pos_, qw_, kw_, 1e-5, axes_, interleaved)
    cos, sin = ref.angles(table, pos, axes)
    for got, x, w, what in ((qo, q, qw, "q"), (ko, k, kw, "k")):
        z, S = ref.norm_rope(x, w, 1e-5, cos, sin, interleaved)
        check(got, z, ref.bf16_bound(z, S, D), what)


@pytest.mark.parametrize("heads,T", [((28, 4, 128), 37), ((28, 4, 128), 1100), ((9, 3, 64), 1500)])
@pytest.mark.parametrize("sections", [SECTIONS[4], SECTIONS[6], SECTIONS[0]], ids=["three", "four", "wide"])
def test_sections_into_the_cache(sections, heads, T):
    """The forms that write a cache: queries and keys as the form without one, keys in their slots and nowhere else."""
    Hq, Hkv, D = heads
    if 2 * sum(n for _, n in sections) > D:
        pytest.skip("more frequencies than a head of 64 has")
    q, k, v, qw, kw, table, pos, axes = sectioned(T, T, heads, sections)
    NB = T + 12
    slots = slots_of(T, T, NB)
    ok = (slots >= 0) & (slots < NB * BS)
    q_, k_, v_, qw_, kw_, table_, pos_, axes_, slots_ = to_dev(q, k, v, qw, kw, table, pos, axes, slots)
    qo, ko, q2, k2 = (torch.full((T, h, D), 7.0, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hq, Hkv))
    kc, vc = (torch.zeros(NB, BS, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pg.pa_norm_rope(qo, ko, q_, k_, table_, pos_, qw_, kw_, 1e-6, axes_)
    pg.pa_norm_rope_and_cache(q2, q_, k_, v_, kc, vc, slots_, table_, pos_, qw_, kw_, 1e-6, axes_, k_out=k2)
    bits = lambda t: t.cpu().view(torch.int16)
    assert torch.equal(bits(qo), bits(q2)) and torch.equal(bits(ko), bits(k2))
    z, S = ref.norm_rope(k, kw, 1e-6, *ref.angles(table, pos, axes), False)
    check(ko, z, ref.bf16_bound(z, S, D), "k")
    want = torch.zeros(NB * BS, Hkv, D, dtype=torch.bfloat16)
    want[slots[ok]] = ko.cpu()[ok]
    assert torch.equal(bits(kc).view(-1, Hkv, D), bits(want))
    if D != 128:
        return
    ks, vs = (0.01 * (1 + torch.arange(Hkv) / n) for n in (3, 5))
    kc8 = torch.zeros(NB, BS, Hkv, D, dtype=torch.uint8, device=DEV)
    vc8 = torch.zeros(NB, Hkv, D, BS, dtype=torch.uint8, device=DEV)
    pg.pa_norm_rope_and_cache_fp8(q2, q_, k_, v_, kc8, vc8, slots_, *to_dev(ks, vs), table_, pos_, qw_, kw_, 1e-6, axes_)
    assert torch.equal(bits(qo), bits(q2))
    got = kc8.cpu().view(-1, Hkv, D)
    check(got[slots[ok]].view(E4M3).double(), (z / ks.double()[:, None]).clamp(-448, 448)[ok],
          ref.code_bound(z, S, D, ks.double()[:, None])[ok], "key codes")
    rest = torch.ones(NB * BS, dtype=torch.bool)
    rest[slots[ok]] = False
    assert (got[rest] == 0).all()
