"""Bad calls of the step operators (planning, releasing, norm and rotation) and
of the chunk attention over 8-bit caches are refused on the host with the
library's status codes, before anything reaches a GPU."""

import ctypes

import pytest

import paged_gqa_decode_reshape_gb300 as pg
import paged_gqa_decode_reshape_gb300.build as pgb

P, P2, P3 = (ctypes.c_void_p(1 << i) for i in (20, 21, 22))  # never dereferenced: the checks fail first
ODD, NEAR = ctypes.c_void_p((1 << 20) + 2), ctypes.c_void_p((1 << 20) + 4)
INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def lib():
    pgb.build()
    return pg.load_library()


STACK = [
    *[({k: None}, INVALID) for k in ("bt", "ctx", "lens", "free", "nfree", "new", "newf")],
    (dict(MBS=0), INVALID), (dict(B=0), INVALID), (dict(BS=0), INVALID), (dict(NB=0), INVALID), (dict(F=0), INVALID),
    (dict(BS=32), UNSUPPORTED), (dict(B=4097), UNSUPPORTED), (dict(MBS=1 << 27), UNSUPPORTED),
    (dict(NB=1 << 31), UNSUPPORTED), (dict(F=1 << 31), UNSUPPORTED),
    (dict(new=NEAR), INVALID),  # overlaps context_lens without being it
    (dict(new=P2), INVALID),    # is the other lengths
]
BASE = dict(bt=P3, MBS=4, ctx=P, lens=P2, B=2, BS=16, NB=64, free=P3, F=64, nfree=P3, new=P, newf=P3, granted=P3, cu=P3,
            pos=P3, slots=P3, T=5, st=None)


@pytest.mark.parametrize("over,status", STACK + [
    *[({k: None}, INVALID) for k in ("granted", "cu", "pos", "slots")], (dict(T=0), INVALID), (dict(T=-3), INVALID),
    (dict(T=(1 << 20) + 1), UNSUPPORTED),
])
def test_plan_refusals(lib, over, status):
    a = {**BASE, **over}
    order = "bt MBS ctx lens B BS NB free F nfree new newf granted cu pos slots T st"
    assert lib.pa_plan_step(*[a[k] for k in order.split()]) == status


@pytest.mark.parametrize("over,status", STACK)
def test_release_refusals(lib, over, status):
    a = {**BASE, **over}
    order = "bt MBS ctx lens B BS NB free F nfree new newf st"
    assert lib.pa_release_blocks(*[a[k] for k in order.split()]) == status


ROPE = dict(qo=P, qos=512, ko=P, kos=256, q=P, qs=512, k=P, ks=256, v=P, vs=256, qw=P, kw=P, eps=1e-6, table=P, P=100,
            R=64, pos=P, axes=P, A=3, inter=0, kc=P, vc=P, ksc=P, vsc=P, slots=P, T=3, Hq=4, Hkv=2, D=128, BS=16, NB=8,
            st=None)
HEAD = "qo qos ko kos q qs k ks"
TAIL = "qw kw eps table P R pos axes A inter"
ORDER = {
    "pa_norm_rope": f"{HEAD} {TAIL} T Hq Hkv D st",
    "pa_norm_rope_and_cache": f"{HEAD} v vs {TAIL} kc vc slots T Hq Hkv D BS NB st",
    "pa_norm_rope_and_cache_fp8": f"{HEAD} v vs {TAIL} kc vc ksc vsc slots T Hq Hkv D BS NB st",
}
EVERY = [
    (dict(qo=None), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(table=None), INVALID),
    (dict(pos=None), INVALID), (dict(axes=None), INVALID), (dict(T=-1), INVALID), (dict(Hq=0), INVALID),
    (dict(Hkv=0), INVALID), (dict(P=0), INVALID), (dict(A=0), INVALID), (dict(R=0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(qs=504), INVALID), (dict(ks=248), INVALID),
    (dict(qos=500), INVALID), (dict(kos=0), INVALID), (dict(qs=516), INVALID), (dict(qos=1 << 32), UNSUPPORTED),
    *[({k: ODD}, INVALID) for k in ("q", "k", "qo", "ko", "qw", "kw", "table")],
    (dict(R=24), UNSUPPORTED), (dict(R=144), UNSUPPORTED), (dict(A=5), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
    (dict(Hq=1 << 16, qs=1 << 23, qos=1 << 23), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED),
]
CACHE = [
    (dict(v=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(slots=None), INVALID),
    (dict(vs=248), INVALID), (dict(v=ODD), INVALID), (dict(kc=ODD), INVALID), (dict(BS=0), INVALID), (dict(NB=0), INVALID),
    (dict(BS=32), UNSUPPORTED), (dict(NB=1 << 31), UNSUPPORTED),
]
SOME = {
    "pa_norm_rope": [(dict(ko=None), INVALID)],
    "pa_norm_rope_and_cache": CACHE,
    "pa_norm_rope_and_cache_fp8": CACHE + [(dict(ksc=None), INVALID), (dict(vsc=None), INVALID),
                                           (dict(D=64), UNSUPPORTED)],
}


@pytest.mark.parametrize("fn", list(ORDER))
def test_rope_refusals(lib, fn):
    for over, status in EVERY + SOME[fn]:
        a = {**ROPE, **over}
        assert getattr(lib, fn)(*[a[k] for k in ORDER[fn].split()]) == status, over
    a = {**ROPE, **{k: None for k in ("qo", "ko", "q", "k", "v", "table", "pos", "kc", "vc", "slots")}, "T": 0}
    assert getattr(lib, fn)(*[a[k] for k in ORDER[fn].split()]) == 0  # no tokens: nothing to do


@pytest.mark.parametrize("fn", ["pa_decode_window_multi_fp8", "pa_decode_window_multi_fp8_block"])
@pytest.mark.parametrize("over,status", [
    *[({k: None}, INVALID) for k in ("out", "q", "kc", "vc", "ks", "vs", "bt", "cu", "ctx", "ws")], (dict(T=0), INVALID),
    (dict(T=(1 << 20) + 1), UNSUPPORTED), (dict(window=0), INVALID), (dict(sinks=-1), INVALID), (dict(D=64), UNSUPPORTED),
    (dict(B=4097), UNSUPPORTED), (dict(Hq=36), UNSUPPORTED), (dict(kc=ODD), INVALID), (dict(scale=0.0), INVALID),
])
def test_chunk_refusals(lib, fn, over, status):
    a = dict(out=P, q=P, kc=P, vc=P, ks=P, vs=P, bt=P, MBS=4, cu=P, ctx=P, B=2, T=5, Hq=28, Hkv=4, D=128, BS=16, NB=64,
             window=8, sinks=2, scale=0.1, ws=P, nb=1 << 40, st=None)
    a.update(over)
    order = "out q kc vc ks vs bt MBS cu ctx B T Hq Hkv D BS NB window sinks scale ws nb st"
    assert getattr(lib, fn)(*[a[k] for k in order.split()]) == status
