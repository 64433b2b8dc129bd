"""Plain 64-bit forms of the decode operators over a part of the cache, on
host tensors, with the error bounds their tests use.

Bounds, per output element, from the operations a kernel may round (u = half a
step: 2^-8 for bf16, 2^-11 for f16, 2^-24 for fp32):
* the output is rounded once to bf16:                          2^-8 |o|;
* every probability is rounded once to the matrix products' input type before
  it meets V (bf16 2^-8, f16 for an 8-bit cache 2^-11), in the numerator and
  in the normaliser:                                            2 u_p A,
  with A = sum_t p_t |V_t|;
* a logit is a sum of D products in fp32, z = scale q.k: off by at most
  (D + 4) 2^-24 Z with Z = scale sum_d |q_d k_d|; an 8-bit cache's queries are
  rounded to f16 first: + 2^-11 Z. A probability moves by twice that,
  relatively (numerator and normaliser);
* 2^x is taken with a relative error of at most 2^-21 (twice), and sums over n
  tokens in fp32 add n 2^-24 (twice).
"""

import math

import torch

BS = 16
V8_POS = [4 * ((o % 8) // 2) + 2 * (o // 8) + o % 2 for o in range(BS)]


def tables(lens, perm, at=0, mbs=None):
    """Block tables [n, mbs] int32 for these lengths from perm[at:], and where it stopped."""
    nblk = [-(-x // BS) for x in lens]
    t = torch.full((len(lens), mbs or max(1, max(nblk))), -1, dtype=torch.int32)
    for i, n in enumerate(nblk):
        t[i, :n] = perm[at:at + n].int()
        at += n
    return t, at


def rows_at(cache, table, positions):
    """Cache rows [P, Hkv, D] (fp64) at these positions, and whether their block is in the pool."""
    blk = table[positions // BS].long()
    ok = (blk >= 0) & (blk < cache.shape[0])
    return cache[blk.clamp(0, cache.shape[0] - 1), positions % BS].double(), ok


def seen(lim, window, sinks):
    t = torch.arange(max(lim, 0))
    return t[(t < sinks) | (t >= lim - window)]


def attend(q, k, v, scale, u_p=2.0 ** -8, u_q=0.0):
    """q [Hq, D], k / v [P, Hkv, D] in fp64: out [Hq, D], its bound, p [Hq, P] and p's relative bound [Hq]."""
    Hq, D = q.shape
    P = k.shape[0]
    if P == 0:
        return torch.zeros(Hq, D).double(), torch.zeros(Hq, D).double(), torch.zeros(Hq, 0).double(), torch.zeros(Hq).double()
    r = Hq // k.shape[1]
    k, v = k.repeat_interleave(r, 1), v.repeat_interleave(r, 1)
    p = torch.softmax(torch.einsum("hd,phd->hp", q, k) * scale, -1)
    out, A = torch.einsum("hp,phd->hd", p, v), torch.einsum("hp,phd->hd", p, v.abs())
    Z = (torch.einsum("hd,phd->hp", q.abs(), k.abs()) * scale).amax(-1)
    rel = 2 * ((D + 4) * 2.0 ** -24 + u_q) * Z + 2 * 2.0 ** -21 + 2 * P * 2.0 ** -24
    bound = 2.0 ** -8 * out.abs() + (2 * u_p + rel)[:, None] * A
    return out, bound, p, rel


def check(got, want, bound, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: non-finite outputs"
    over = (got - want).abs() - bound - 1e-30
    worst = over.max().item() if over.numel() else -math.inf
    assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} elements past their bound, by up to {worst:.3e}"


def to_fp8(kc, vc, per_block, Hkv):
    """E4M3 caches of bf16 ones in the library's layouts, their scales, and what they stand for (fp64)."""
    k, v = kc.float(), vc.float()
    if per_block:
        def fit(x):
            a = torch.nan_to_num(x).abs().amax((1, 3)).clamp(min=2.0 ** -100)
            return torch.exp2(torch.ceil(torch.log2(a / 448)))
        ks, vs = fit(k), fit(v)
        kd, vd = ks[:, None, :, None], vs[:, None, :, None]
    else:
        ks = 0.0117 * (1 + torch.arange(Hkv) / 8)
        vs = 0.0127 * (1 + torch.arange(Hkv) / 16)
        kd, vd = ks[None, None, :, None], vs[None, None, :, None]
    k8, v8 = ((x / d).clamp(-448, 448).to(torch.float8_e4m3fn) for x, d in ((k, kd), (v, vd)))
    inv = torch.tensor([V8_POS.index(i) for i in range(BS)])
    return (k8.view(torch.uint8).contiguous(), v8.view(torch.uint8).permute(0, 2, 3, 1)[..., inv].contiguous(),
            ks.contiguous(), vs.contiguous(), k8.float().double() * kd.double(), v8.float().double() * vd.double())


def evict(kc, vc, w, bt, ctx, dst, budget, recent):
    """kept, new_lens and the caches and weights after the call (host copies)."""
    B, Hkv, NB = bt.shape[0], kc.shape[2], kc.shape[0]
    kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32)
    kc2, vc2, w2 = kc.clone(), vc.clone(), w.clone()
    ctx = [min(max(int(x), 0), bt.shape[1] * BS) for x in ctx]
    for b, n in enumerate(ctx):
        t = torch.arange(n)
        blk = bt[b][t // BS].long()
        live = (blk >= 0) & (blk < NB)
        for h in range(Hkv):
            keep = list(range(n))
            if n > budget:
                new = min(recent, budget)
                val = torch.where(live, w[blk.clamp(0, NB - 1), h, t % BS], torch.tensor(-math.inf)).tolist()
                best = sorted(range(n - new), key=lambda j: (-val[j], j))[:budget - new]
                keep = sorted(best) + list(range(n - new, n))
            kept[b, h, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
            for i, j in enumerate(keep):
                d = int(dst[b][i // BS])
                if not live[j] or d < 0 or d >= NB:
                    continue
                kc2[d, i % BS, h] = kc[blk[j], j % BS, h]
                vc2[d, i % BS, h] = vc[blk[j], j % BS, h]
                w2[d, h, i % BS] = w[blk[j], h, j % BS]
    return kept, torch.tensor([min(n, budget) for n in ctx], dtype=torch.int32), kc2, vc2, w2
