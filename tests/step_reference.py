"""Plain forms of what a serving step does around its attention -- block tables
and slots from request lengths, blocks given back, norm and rotation of queries
and keys -- on host tensors, in whole numbers and in 64 bits, with the error
bounds their tests use.

Bounds of a rotated element y' = a cos - b sin (u = 2^-24, half a step of fp32):
* the mean of squares is a sum of D products (at most D + 2 roundings), its root
  and reciprocal take one each at half weight and a full one, the two products by
  it and by the weight two: y is off by at most (D / 2 + 6) u |y|;
* the rotation adds two products and a sum: 3 u (|a cos| + |b sin|);
  together at most (D / 2 + 9) u S with S = |a cos| + |b sin|;
* rounding to bf16 adds 2^-8 of the result (2^-134 at the smallest);
* an E4M3 code: the quotient adds u, the code half a step: 2^-4 of its value, or
  2^-10 below 2^-6.
"""

import torch

from tests.subset_reference import BS


def clamp(x, lo, hi):
    return max(lo, min(int(x), hi))


def plan(bt, ctx, q, free, nf, NB, T):
    """block_tables, new_lens, new_free, granted, cu_seqlens_q, positions, slots after the call."""
    bt = bt.clone()
    B, MBS = bt.shape
    nf = clamp(nf, 0, len(free))
    cu, pos, slots = [0], [0] * T, [-1] * T
    new_lens, granted, rank, taken, total = [], [], 0, 0, 0
    for b in range(B):
        c, n = clamp(ctx[b], 0, MBS * BS), max(int(q[b]), 0)
        total += n
        have, want = -(-c // BS), -(-(c + n) // BS)
        ok = c + n <= MBS * BS and total <= T
        if ok and want > have:
            ok = rank + want - have <= nf
            if ok:
                for j in range(want - have):
                    bt[b, have + j] = int(free[nf - 1 - rank - j])
                taken += want - have
            rank += want - have
        cu.append(min(total, T))
        for r in range(cu[-2], cu[-1]):
            p = c + r - cu[-2]
            pos[r] = p
            if ok and 0 <= int(bt[b, p // BS]) < NB:
                slots[r] = int(bt[b, p // BS]) * BS + p % BS
        granted.append(n if ok else 0)
        new_lens.append(c + granted[-1])
    i32 = torch.int32
    return (bt, torch.tensor(new_lens, dtype=i32), torch.tensor([nf - taken], dtype=i32),
            torch.tensor(granted, dtype=i32), torch.tensor(cu, dtype=i32), torch.tensor(pos, dtype=i32),
            torch.tensor(slots, dtype=torch.int64))


def release(bt, ctx, keep, free, nf, NB):
    """free_blocks, new_lens, new_free after the call."""
    free, F = free.clone(), len(free)
    nf = clamp(nf, 0, F)
    new_lens = []
    for b in range(bt.shape[0]):
        c = clamp(ctx[b], 0, bt.shape[1] * BS)
        k = clamp(keep[b], 0, c)
        new_lens.append(k)
        for j in range(-(-k // BS), -(-c // BS)):
            if 0 <= int(bt[b, j]) < NB:
                if nf < F:
                    free[nf] = bt[b, j]
                nf += 1
    return free, torch.tensor(new_lens, dtype=torch.int32), torch.tensor([min(nf, F)], dtype=torch.int32)


def angles(table, positions, axes):
    """cos and sin [T, R / 2] in fp64; positions [T], or [A, T] with axes [R / 2]."""
    half = table.shape[1] // 2
    p = positions.long().clamp(0, table.shape[0] - 1)
    if axes is None:
        rows = table.double()[p]
        return rows[:, :half], rows[:, half:]
    of = axes.long().clamp(0, positions.shape[0] - 1)
    f = torch.arange(half)
    return table.double()[p[of].T, f], table.double()[p[of].T, half + f]


def norm_rope(x, w, eps, cos, sin, interleaved):
    """x [T, H, D] normed and rotated in fp64, and S (see above) per element."""
    D, half = x.shape[-1], cos.shape[1]
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    z, S = y.clone(), y.abs()
    c, s = cos[:, None], sin[:, None]
    z[..., a] = y[..., a] * c - y[..., b] * s
    z[..., b] = y[..., b] * c + y[..., a] * s
    S[..., a] = (y[..., a] * c).abs() + (y[..., b] * s).abs()
    S[..., b] = (y[..., b] * c).abs() + (y[..., a] * s).abs()
    return z, S


def bf16_bound(z, S, D):
    return 2.0 ** -8 * z.abs() + 2.0 ** -134 + (D / 2 + 9) * 2.0 ** -24 * S


def code_bound(z, S, D, scale):
    """Of a decoded code against z / scale clamped to +-448."""
    v = (z / scale).abs().clamp(max=448)
    return (2.0 ** -4 * v).clamp(min=2.0 ** -10) + (D / 2 + 10) * 2.0 ** -24 * S / scale
