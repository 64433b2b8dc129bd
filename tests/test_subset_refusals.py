"""Bad calls of the decode operators over a part of the cache are refused on
the host with the library's status codes, before anything reaches a GPU."""

import ctypes

import pytest

import paged_gqa_decode_reshape_gb300 as pg
import paged_gqa_decode_reshape_gb300.build as pgb

P, P2 = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)  # never dereferenced: the checks fail first
ODD = ctypes.c_void_p((1 << 20) + 2)
INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def lib():
    pgb.build()
    return pg.load_library()


BASE = dict(out=P, q=P, kc=P, vc=P, ks=P, vs=P, pt=P, PMBS=4, plen=P, cug=P, NG=1, bt=P, MBS=4, cu=P, ctx=P, B=2,
            T=5, Hq=28, Hkv=4, D=128, BS=16, NB=64, window=8, sinks=2, scale=0.1, w=P, ws=P, nb=1 << 40, st=None)
ORDER = dict(
    pa_decode_window="out q kc vc bt MBS ctx B Hq Hkv D BS NB window sinks scale ws nb st",
    pa_decode_window_fp8="out q kc vc ks vs bt MBS ctx B Hq Hkv D BS NB window sinks scale ws nb st",
    pa_decode_window_fp8_block="out q kc vc ks vs bt MBS ctx B Hq Hkv D BS NB window sinks scale ws nb st",
    pa_decode_window_multi="out q kc vc bt MBS cu ctx B T Hq Hkv D BS NB window sinks scale ws nb st",
    pa_decode_prefix="out q kc vc pt PMBS plen cug NG bt MBS ctx B Hq Hkv D BS NB scale ws nb st",
    pa_decode_weights="out w q kc vc bt MBS ctx B Hq Hkv D BS NB scale ws nb st",
)
EVERY = [
    (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID),
    (dict(bt=None), INVALID), (dict(ctx=None), INVALID), (dict(ws=None), INVALID), (dict(B=0), INVALID),
    (dict(MBS=0), INVALID), (dict(Hq=30), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q=ODD), INVALID), (dict(kc=ODD), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(BS=32), UNSUPPORTED), (dict(Hq=36), UNSUPPORTED), (dict(B=4097), UNSUPPORTED),
    (dict(MBS=1 << 27), UNSUPPORTED), (dict(NB=1 << 31), UNSUPPORTED), (dict(Hq=70000, Hkv=70000), UNSUPPORTED),
]
SOME = {
    "pa_decode_window": [(dict(window=0), INVALID), (dict(sinks=-1), INVALID)],
    "pa_decode_window_fp8": [(dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(D=64), UNSUPPORTED)],
    "pa_decode_window_fp8_block": [(dict(ks=None), INVALID), (dict(D=64), UNSUPPORTED)],
    "pa_decode_window_multi": [(dict(cu=None), INVALID), (dict(T=0), INVALID), (dict(T=(1 << 20) + 1), UNSUPPORTED),
                               (dict(window=0), INVALID)],
    "pa_decode_prefix": [(dict(pt=None), INVALID), (dict(plen=None), INVALID), (dict(cug=None), INVALID),
                         (dict(NG=0), INVALID), (dict(PMBS=0), INVALID), (dict(NG=4097), UNSUPPORTED),
                         (dict(PMBS=1 << 27), UNSUPPORTED)],
    "pa_decode_weights": [(dict(w=None), INVALID), (dict(w=ODD), INVALID)],
}


@pytest.mark.parametrize("fn", list(ORDER))
def test_decode_refusals(lib, fn):
    for over, status in EVERY + SOME[fn]:
        a = {**BASE, **over}
        assert getattr(lib, fn)(*[a[k] for k in ORDER[fn].split()]) == status, over


EVICT = "kept lens kc vc w bt MBS ctx dst DMBS B Hkv D BS NB budget recent st".split()


@pytest.mark.parametrize("over,status", [
    *[({k: None}, INVALID) for k in ("kept", "lens", "kc", "vc", "w", "bt", "ctx", "dst")],
    (dict(kc=ODD), INVALID), (dict(w=ODD), INVALID), (dict(B=0), INVALID), (dict(budget=0), INVALID),
    (dict(recent=-1), INVALID), (dict(budget=65), INVALID), (dict(D=80), UNSUPPORTED), (dict(BS=8), UNSUPPORTED),
    (dict(B=5000), UNSUPPORTED), (dict(Hkv=1 << 17), UNSUPPORTED), (dict(NB=1 << 33), UNSUPPORTED),
    (dict(budget=(1 << 30) + 1, DMBS=1 << 27), UNSUPPORTED), (dict(B=4096, Hkv=4096, budget=1024, DMBS=64), UNSUPPORTED),
    (dict(lens=P), INVALID), (dict(lens=ctypes.c_void_p((1 << 20) + 4)), INVALID),
])
def test_evict_refusals(lib, over, status):
    a = dict(kept=P, lens=P2, kc=P, vc=P, w=P, bt=P, MBS=9, ctx=P, dst=P, DMBS=4, B=2, Hkv=4, D=128, BS=16, NB=64,
             budget=64, recent=3, st=None)
    a.update(over)
    assert lib.pa_evict(*[a[k] for k in EVICT]) == status


def test_reset_weights_refusals(lib):
    assert lib.pa_reset_weights(None, None, 0, 4, 16, 8, None) == 0
    assert lib.pa_reset_weights(None, P, 3, 4, 16, 8, None) == INVALID
    assert lib.pa_reset_weights(P, None, 3, 4, 16, 8, None) == INVALID
    assert lib.pa_reset_weights(P, P, -1, 4, 16, 8, None) == INVALID
    assert lib.pa_reset_weights(P, P, 3, 4, 8, 8, None) == UNSUPPORTED
    assert lib.pa_reset_weights(P, P, 1 << 32, 4, 16, 8, None) == UNSUPPORTED


def test_workspace_sizes_of_bad_shapes_are_zero(lib):
    assert pg.pa_decode_window_workspace_size(0, 28, 4, 128) == 0
    assert pg.pa_decode_window_workspace_size(2, 28, 4, 100) == 0
    assert pg.pa_decode_window_multi_workspace_size(2, 0, 28, 4, 128) == 0
    assert pg.pa_decode_window_multi_workspace_size(2, (1 << 20) + 1, 28, 4, 128) == 0
    assert pg.pa_decode_prefix_workspace_size(2, 0, 28, 4, 128) == 0
    assert pg.pa_decode_weights_workspace_size(2, 28, 4, 128, 0) == 0
