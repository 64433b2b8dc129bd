"""Measured cases of the operators around a serving step's attention:

* ``plan``: block tables, row offsets, positions and slots of a step built on
  the GPU from request lengths and a stack of free blocks;
* ``release``: the blocks behind shortened or finished sequences pushed back
  onto that stack;
* ``rope``: the norm of every query and key head and the rotation by position
  (one axis, or time / height / width) in one pass, with the write of K and V
  into a bf16 or 8-bit paged cache, or without it;
* ``chunk``: attention of several query rows per sequence (speculative tokens,
  prompt chunks) over an 8-bit paged cache, all of it or a window and sinks.

``run`` computes them with elementary torch operations in fp32 (``own`` false)
or through this package's entry points (``own`` true), on the same state.
Lengths are a function of the case alone; values and block tables of the seed.
"""

from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

BS = 16  # tokens per cache block
# the order of a block's 16 tokens in a row of the 8-bit V cache
V8_POS = [4 * ((o % 8) // 2) + 2 * (o // 8) + o % 2 for o in range(BS)]
EPS = 1e-6
FAR = 1 << 30  # a window that hides nothing

# ------------------------------------------------------------------- cases


def listed():
    big = dict(Hq=28, Hkv=4, D=128)  # the head shape of this repository's workloads
    text = dict(R=128, axes=1, inter=False, **big)
    return [
        # a decode step of a small batch: one new token each, nothing but latency
        dict(name="plan_decode", op="plan", B=16, lo=4097, hi=12001, qlo=1, qhi=1, first=0, short=0, pad=0, lens=1),
        # a mixed step: most sequences decode, some bring chunks of their prompts; padded to a captured size
        dict(name="plan_mixed", op="plan", B=256, lo=1, hi=20001, qlo=1, qhi=1, first=9, short=0, pad=77, lens=2),
        # whole prompts of a batch admitted at once
        dict(name="plan_prompts", op="plan", B=64, lo=0, hi=0, qlo=517, qhi=16001, first=0, short=0, pad=0, lens=3),
        # rejected speculative tokens taken back
        dict(name="release_spec", op="release", B=128, lo=33, hi=20011, drop="few", lens=4),
        # long sequences that are over, others that go on
        dict(name="release_done", op="release", B=512, lo=129, hi=20011, drop="many", lens=5),
        # one sequence's next token
        dict(name="rope_one", op="rope", T=1, seqs=1, pad=0, cache="bf16", norm=True, lens=6, **text),
        # a decode batch on the 8-bit cache
        dict(name="rope_fp8_b128", op="rope", T=128, seqs=128, pad=0, cache="fp8", norm=True, lens=7, **text),
        # chunks of a few long prompts, padded
        dict(name="rope_chunks", op="rope", T=8191, seqs=5, pad=55, cache="bf16", norm=True, lens=8, **text),
        # patches of images among text: three axes, small heads, half of each head rotated, no cache
        dict(name="rope_images", op="rope", T=6001, seqs=3, pad=0, cache="none", norm=True, lens=9, Hq=16, Hkv=4, D=64,
             R=32, axes=3, inter=True),
        # a few speculative rows behind a short context
        dict(name="chunk_few", op="chunk", kv="fp8", S=4, qlo=1, qhi=4, lo=300, hi=700, window=FAR, sinks=0, lens=10,
             **big),
        # speculative decoding of a batch: up to six rows per sequence, a window and sinks
        dict(name="chunk_spec", op="chunk", kv="fp8_block", S=32, qlo=1, qhi=6, lo=900, hi=15003, window=4096, sinks=4,
             lens=11, **big),
        # chunks of long prompts, over everything before them
        dict(name="chunk_prompts", op="chunk", kv="fp8", S=3, qlo=517, qhi=2048, lo=9000, hi=16001, window=FAR, sinks=0,
             lens=12, **big),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(max(lo, 1)), math.log(max(hi, 1))))))


_HEADS = [(28, 4, 128), (32, 8, 128), (8, 8, 128), (40, 8, 128), (12, 2, 64), (32, 4, 64), (9, 3, 64), (16, 2, 128)]


def draw(rng):
    op = rng.choice(["plan", "plan", "release", "rope", "rope", "rope", "chunk", "chunk", "chunk"])
    c = dict(op=op, lens=rng.randrange(1 << 30))
    if op == "plan":
        c["B"] = _log(rng, 1, 2048)
        c["hi"] = rng.choice([0, _log(rng, 1, 20000)])
        c["lo"] = min(c["hi"], _log(rng, 1, 20000))
        c["qhi"] = _log(rng, 1, max(1, min(16000, 70_000 // c["B"])))
        c["qlo"] = rng.choice([0, 1, c["qhi"]])
        c["first"] = rng.choice([0, min(c["B"], _log(rng, 1, 12))])
        c["short"] = rng.choice([0, 0, 0, _log(rng, 1, 100)])  # blocks that the free stack lacks
        c["pad"] = rng.choice([0, rng.randrange(500)])
        return c
    if op == "release":
        c["B"] = _log(rng, 1, 1024)
        c["hi"] = _log(rng, 1, min(20000, 1_200_000 // c["B"]))
        c["lo"] = _log(rng, 1, c["hi"])
        c["drop"] = rng.choice(["few", "many"])
        return c
    c["Hq"], c["Hkv"], c["D"] = rng.choice(_HEADS)
    if op == "rope":
        c["T"] = _log(rng, 1, min(7000, 7000 * 36 // (c["Hq"] + 2 * c["Hkv"])))
        c["seqs"] = rng.choice([c["T"], min(c["T"], _log(rng, 1, 40))])
        c["pad"] = rng.choice([0, rng.randrange(1 + c["T"] // 8)])
        c["cache"] = rng.choice(["none", "bf16", "fp8"]) if c["D"] == 128 else rng.choice(["none", "bf16"])
        c["norm"] = rng.random() < 0.75
        c["R"] = rng.choice([c["D"], c["D"], c["D"] // 2, 16])
        c["axes"] = rng.choice([1, 1, 2, 3])
        c["inter"] = rng.random() < 0.3
        return c
    c["Hq"], c["Hkv"], c["D"] = rng.choice([h for h in _HEADS if h[2] == 128])
    c["kv"] = rng.choice(["fp8", "fp8_block"])
    c["window"], c["sinks"] = rng.choice([(FAR, 0), (_log(rng, 1, 8192), rng.choice([0, 1, 4, rng.randrange(200)]))])
    c["qhi"] = _log(rng, 1, 2048)
    c["qlo"] = _log(rng, 1, c["qhi"])
    c["hi"] = _log(rng, c["qhi"], 16000)
    c["lo"] = _log(rng, c["qhi"], c["hi"])
    seen = min(c["hi"], c["window"] + c["sinks"] + c["qhi"])
    c["S"] = min(_log(rng, 1, 48), max(1, 30_000_000 // (seen * c["qhi"])), max(1, 600_000 // seen))
    return c


def _lens(n, lo, hi, seed):
    """n lengths in [lo, hi], evenly spread over their logarithm; the first is hi."""
    r = random.Random(seed)
    return [hi] + [min(hi, _log(r, lo, hi)) for _ in range(n - 1)]


def _lengths(case):
    """The case's lengths: tokens cached per sequence, new or kept ones, rows."""
    op, seed = case["op"], case["lens"]
    r = random.Random(seed + 1)
    if op == "plan":
        ctx = _lens(case["B"], case["lo"], case["hi"], seed) if case["hi"] else [0] * case["B"]
        q = [min(case["qhi"], max(case["qlo"], _log(r, 1, case["qhi"]))) for _ in ctx]
        for i in range(case["first"]):  # sequences that bring a chunk
            q[r.randrange(len(q))] = _log(r, 16, 2048)
        have = [-(-x // BS) for x in ctx]
        need = sum(-(-(x + n) // BS) - h for x, n, h in zip(ctx, q, have))
        return {"ctx": ctx, "q": q, "T": sum(q) + case["pad"], "need": need,
                "free": max(1, need - case["short"]) if case["short"] else need + 5,
                "mbs": max(-(-(x + n) // BS) for x, n in zip(ctx, q)) + 1}
    if op == "release":
        ctx = _lens(case["B"], case["lo"], case["hi"], seed)
        if case["drop"] == "few":
            keep = [max(0, x - r.randrange(8)) for x in ctx]
        else:
            keep = [r.choice([0, 0, x, r.randrange(x + 1)]) for x in ctx]
        return {"ctx": ctx, "keep": keep}
    if op == "rope":
        n, s = case["T"], case["seqs"]
        cuts = sorted(r.sample(range(1, n), s - 1)) if s > 1 else []
        rows = [b - a for a, b in zip([0] + cuts, cuts + [n])]
        return {"rows": rows, "start": [r.randrange(32000) for _ in rows]}
    ctx = _lens(case["S"], case["lo"], case["hi"], seed)
    return {"ctx": ctx, "q": [min(x, y) for x, y in zip(_lens(case["S"], case["qlo"], case["qhi"], seed + 1), ctx)]}


# ------------------------------------------------------------------ inputs


def _tables(lens, perm, mbs=0):
    """Block tables [n, mbs] for these lengths from perm, -1 past each sequence's blocks, and the blocks used."""
    nblk = [-(-x // BS) for x in lens]
    t = np.full((len(lens), max(1, mbs, max(nblk))), -1, np.int32)
    at = 0
    for i, n in enumerate(nblk):
        t[i, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(t).to("cuda"), at


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _prepare_plan(case, seed):
    L = _lengths(case)
    used = sum(-(-x // BS) for x in L["ctx"])
    NB = used + (L["free"] if case["op"] == "plan" else 7)
    perm = np.random.RandomState(seed % (1 << 32)).permutation(NB).astype(np.int32)
    s = dict(case=case, NB=NB, ctx=_ints(L["ctx"]))
    s["bt"], at = _tables(L["ctx"], perm, L.get("mbs", 0))
    free = np.full(NB, -1, np.int32)  # room for every block of the pool
    free[:NB - at] = perm[at:]
    s["free"], s["nfree"] = torch.from_numpy(free).to("cuda"), _ints([NB - at])
    B = len(L["ctx"])
    s["new_lens"], s["new_free"] = _ints([0] * B), _ints([0])
    if case["op"] == "plan":
        s["q"], s["granted"], s["cu"] = _ints(L["q"]), _ints([0] * B), _ints([0] * (B + 1))
        s["pos"] = torch.empty(L["T"], dtype=torch.int32, device="cuda")
        s["slots"] = torch.empty(L["T"], dtype=torch.int64, device="cuda")
    else:
        s["keep"] = _ints(L["keep"])
    return s


def _prepare_rope(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    L = _lengths(case)
    T, pad, Hq, Hkv, D, R = case["T"], case["pad"], case["Hq"], case["Hkv"], case["D"], case["R"]
    A = T + pad

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(torch.bfloat16)

    # one projection's output: the heads of q, k and v side by side, of uneven sizes
    qkv = normal(A, Hq + 2 * Hkv, D, std=1.7)
    s = dict(case=case, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], n=T)
    s["q_out"] = torch.empty((A, Hq, D), dtype=torch.bfloat16, device=dev)
    s["k_out"] = torch.empty((A, Hkv, D), dtype=torch.bfloat16, device=dev) if case["cache"] == "none" else None
    s["qw"], s["kw"] = ((1 + 0.2 * normal(D).float()).to(torch.bfloat16) for _ in range(2)) if case["norm"] else (None, None)
    P = 32000 + max(L["rows"]) + 1
    inv = 10000.0 ** (-torch.arange(R // 2, device=dev, dtype=torch.float64) * 2 / R)
    angle = torch.arange(P, device=dev, dtype=torch.float64)[:, None] * inv
    s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
    pos = np.concatenate([np.arange(n) + a for n, a in zip(L["rows"], L["start"])] + [np.zeros(pad, np.int64)])
    if case["axes"] == 1:
        s["pos"], s["axes"] = torch.from_numpy(pos.astype(np.int32)).to(dev), None
    else:  # time, and a raster of 57 patches per row for the others
        other = [pos, pos // 57, pos % 57][:case["axes"]]
        s["pos"] = torch.from_numpy(np.stack(other).astype(np.int32)).to(dev)
        s["axes"] = _ints([i * case["axes"] // (R // 2) for i in range(R // 2)])
    if case["cache"] != "none":
        nblk = [-(-(a % BS + n) // BS) for n, a in zip(L["rows"], L["start"])]
        NB = sum(nblk) + 3
        perm = np.random.RandomState(seed % (1 << 32)).permutation(NB)
        slots, at = [], 0
        for n, a, b in zip(L["rows"], L["start"], nblk):
            o = a % BS + np.arange(n)
            slots.append(perm[at + o // BS] * BS + o % BS)
            at += b
        slots.append(np.full(pad, -1))
        s["slots"] = torch.from_numpy(np.concatenate(slots).astype(np.int64)).to(dev)
        if case["cache"] == "bf16":
            s["kc"], s["vc"] = normal(NB, BS, Hkv, D), normal(NB, BS, Hkv, D)
        else:
            s["kc"], s["vc"] = (torch.randint(0, 120, sh, generator=g, device=dev, dtype=torch.uint8)
                                for sh in ((NB, BS, Hkv, D), (NB, Hkv, D, BS)))
            s["ks"] = torch.full((Hkv,), 0.0117, device=dev) * (1 + torch.arange(Hkv, device=dev) / 8)
            s["vs"] = torch.full((Hkv,), 0.0127, device=dev) * (1 + torch.arange(Hkv, device=dev) / 16)
    return s


def _prepare_chunk(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    L = _lengths(case)
    NB = sum(-(-x // BS) for x in L["ctx"]) + 3
    perm = np.random.RandomState(seed % (1 << 32)).permutation(NB)
    s = dict(case=case, scale=D ** -0.5, lens=L)
    s["bt"], _ = _tables(L["ctx"], perm)
    s["ctx"] = _ints(L["ctx"])
    s["cu"] = _ints([0] + [int(x) for x in np.cumsum(L["q"])])
    # twice the usual spread of queries: logits with a standard deviation of 2
    s["q"] = (torch.randn(sum(L["q"]), Hq, D, generator=g, device=dev) * 2).to(torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    k, v = torch.randn(2, NB, BS, Hkv, D, generator=g, device=dev)
    if case["kv"] == "fp8":  # a scale per KV head
        s["ks"] = torch.full((Hkv,), 0.0117, device=dev) * (1 + torch.arange(Hkv, device=dev) / 8)
        s["vs"] = torch.full((Hkv,), 0.0127, device=dev) * (1 + torch.arange(Hkv, device=dev) / 16)
        kd, vd = s["ks"][None, None, :, None], s["vs"][None, None, :, None]
    else:  # a power of two per block and KV head that fits its largest value
        def fit(x):
            return torch.exp2(torch.ceil(torch.log2(x.abs().amax((1, 3)) / 448))).contiguous()
        s["ks"], s["vs"] = fit(k), fit(v)
        kd, vd = s["ks"][:, None, :, None], s["vs"][:, None, :, None]
    k8, v8 = ((x / d).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x, d in ((k, kd), (v, vd)))
    # the code of NaN in the unused slots of every sequence's last block: nothing may read them
    seq = [i for i, x in enumerate(L["ctx"]) for _ in range(-x % BS)]
    pos = [x + j for x in L["ctx"] for j in range(-x % BS)]
    if seq:
        seq, pos = torch.tensor(seq, device=dev), torch.tensor(pos, device=dev)
        k8[s["bt"][seq, pos // BS].long(), pos % BS] = 127
        v8[s["bt"][seq, pos // BS].long(), pos % BS] = 127
    inv = torch.tensor([V8_POS.index(i) for i in range(BS)], device=dev)
    s["kc"], s["vc"] = k8.contiguous(), v8.permute(0, 2, 3, 1)[..., inv].contiguous()
    return s


def prepare(case, seed):
    make = {"plan": _prepare_plan, "release": _prepare_plan, "rope": _prepare_rope, "chunk": _prepare_chunk}
    return make[case["op"]](case, seed)


# -------------------------------------------------------- the plain forms


def _plan_out(s):
    return {k: s[k] for k in ("bt", "new_lens", "new_free", "granted", "cu", "pos", "slots")}


def _plain_plan(s):
    bt, T = s["bt"], s["pos"].shape[0]
    B, MBS = bt.shape
    dev = bt.device
    F, NB = s["free"].shape[0], s["NB"]
    nf = s["nfree"].long().clamp(0, F)
    c, q = s["ctx"].long().clamp(0, MBS * BS), s["q"].long().clamp(min=0)
    end = q.cumsum(0)
    have, want = (c + BS - 1) // BS, (c + q + BS - 1) // BS
    fits = (c + q <= MBS * BS) & (end <= T)
    need = torch.where(fits, want - have, 0)
    upto = need.cumsum(0)
    ok = fits & ((need == 0) | (upto <= nf))
    granted = torch.where(ok, q, 0)
    j = torch.arange(MBS, device=dev)[None]
    i = j - have[:, None]
    new = (i >= 0) & (i < need[:, None]) & ok[:, None]
    at = (nf - 1 - (upto - need)[:, None] - i).clamp(0, F - 1)
    bt.copy_(torch.where(new, s["free"][at], bt))
    s["new_lens"].copy_(c + granted)
    s["new_free"].copy_(nf - torch.where(ok, need, 0).sum())
    s["granted"].copy_(granted)
    s["cu"][1:] = end.clamp(max=T)
    s["cu"][:1] = 0
    r = torch.arange(T, device=dev)
    cu = s["cu"].long()
    seq = torch.zeros(T + 1, dtype=torch.long, device=dev).index_add_(0, cu[1:], torch.ones_like(cu[1:])).cumsum(0)[:T]
    live, seq = seq < B, seq.clamp(max=B - 1)
    pos = c[seq] + r - cu[seq]
    phys = bt[seq, (pos // BS).clamp(max=MBS - 1)].long()
    s["pos"].copy_(torch.where(live, pos, 0))
    s["slots"].copy_(torch.where(live & ok[seq] & (phys >= 0) & (phys < NB), phys * BS + pos % BS, -1))
    return _plan_out(s)


def _release_out(s):
    return {"free": s["free"], "new_lens": s["new_lens"], "new_free": s["new_free"]}


def _plain_release(s):
    bt, free = s["bt"], s["free"]
    MBS, F = bt.shape[1], free.shape[0]
    nf = s["nfree"].long().clamp(0, F)
    c = s["ctx"].long().clamp(0, MBS * BS)
    k = torch.minimum(s["keep"].long().clamp(min=0), c)
    j = torch.arange(MBS, device=bt.device)[None]
    out = (j >= ((k + BS - 1) // BS)[:, None]) & (j < ((c + BS - 1) // BS)[:, None]) & (bt >= 0) & (bt < s["NB"])
    out = out.reshape(-1)
    at = nf + out.long().cumsum(0) - 1
    # what is not released, or has no room, goes to a place behind the stack
    put = torch.cat([free, free.new_zeros(1)])
    put[torch.where(out & (at < F), at, F)] = bt.reshape(-1)
    free.copy_(put[:F])
    s["new_lens"].copy_(k)
    s["new_free"].copy_((nf + out.sum()).clamp(max=F))
    return _release_out(s)


def _rope_out(s):
    if s["case"]["cache"] == "none":
        return {"q": s["q_out"], "k": s["k_out"]}
    if s["case"]["cache"] == "bf16":
        return {"q": s["q_out"], "key_cache": s["kc"], "value_cache": s["vc"]}
    e4m3 = torch.float8_e4m3fn
    return {"q": s["q_out"], "key_cache": s["kc"].view(e4m3), "value_cache": s["vc"].view(e4m3)}


def _plain_rope(s):
    c = s["case"]
    R, half, n = c["R"], c["R"] // 2, s["n"]
    pos = s["pos"].long()
    if c["axes"] == 1:
        cs = s["table"][pos]
        cos, sin = cs[:, :half], cs[:, half:]
    else:
        f = torch.arange(half, device=pos.device)
        p = pos[s["axes"].long()].T  # [T, half]
        cos, sin = s["table"][p, f], s["table"][p, half + f]
    cos, sin = cos[:, None], sin[:, None]

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        r = x[..., :R]
        if c["inter"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).reshape(r.shape)
        else:
            a, b = r[..., :half], r[..., half:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, x[..., R:]], -1)

    s["q_out"].copy_(turned(s["q"], s["qw"]))
    k = turned(s["k"], s["kw"])
    if c["cache"] == "none":
        s["k_out"].copy_(k)
        return _rope_out(s)
    blk, off = s["slots"][:n] // BS, s["slots"][:n] % BS
    if c["cache"] == "bf16":
        s["kc"][blk, off] = k[:n].to(torch.bfloat16)
        s["vc"][blk, off] = s["v"][:n]
        return _rope_out(s)
    e4m3 = torch.float8_e4m3fn
    s["kc"][blk, off] = (k[:n] / s["ks"][:, None]).clamp(-448, 448).to(e4m3).view(torch.uint8)
    at = 4 * ((off % 8) // 2) + 2 * (off // 8) + off % 2
    s["vc"][blk, :, :, at] = (s["v"][:n].float() / s["vs"][:, None]).clamp(-448, 448).to(e4m3).view(torch.uint8)
    return _rope_out(s)


def _plain_chunk(s):
    c, L = s["case"], s["lens"]
    dev = s["q"].device
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G = Hq // Hkv
    at8 = torch.tensor(V8_POS, device=dev)
    out = s["out"]
    S = len(L["q"])
    i0 = r0 = 0
    while i0 < S:  # as many sequences at a time as a few GB of logits hold
        i1, Q, P = i0, 0, 0
        while i1 < S:
            q2 = max(Q, L["q"][i1])
            p2 = max(P, min(L["ctx"][i1], c["sinks"] + c["window"] + L["q"][i1]))
            if i1 > i0 and (i1 + 1 - i0) * q2 * p2 * Hq > 1 << 30:
                break
            i1, Q, P = i1 + 1, q2, p2
        ctx, cu = s["ctx"][i0:i1].long(), s["cu"][i0:i1 + 1].long()
        ql = cu[1:] - cu[:-1]
        n, rows = i1 - i0, sum(L["q"][i0:i1])
        r = torch.arange(Q, device=dev)
        lim = (ctx - ql)[:, None] + r[None] + 1  # [n, Q]: row r sees positions below it
        window = min(c["window"], max(L["ctx"]))
        if c["sinks"] + window + Q >= max(L["ctx"][i0:i1]):
            p = torch.arange(max(L["ctx"][i0:i1]), device=dev)[None].expand(n, -1)
            f = p < c["sinks"]
        else:
            i = torch.arange(c["sinks"] + window + Q - 1, device=dev)[None]
            f = (i < c["sinks"]).expand(n, -1)
            p = torch.where(f, i, (ctx - ql - window + 1)[:, None] + i - c["sinks"])
        e, fe = p[:, None], f[:, None]
        ok = (e >= 0) & (e < lim[..., None]) & (fe | ((e >= c["sinks"]) & (e >= lim[..., None] - window)))
        ok &= (r[None] < ql[:, None])[..., None]
        pc = p.clamp(min=0).clamp(max=s["bt"].shape[1] * BS - 1)
        blk = s["bt"][i0:i1].gather(1, pc // BS).long().clamp(min=0)
        k = s["kc"].view(torch.float8_e4m3fn)[blk, pc % BS].float()
        # advanced indices apart from each other: the result is [n, P, Hkv, D]
        v = s["vc"].view(torch.float8_e4m3fn)[blk, :, :, at8[pc % BS]].float()
        ks, vs = (s["ks"][blk], s["vs"][blk]) if c["kv"] == "fp8_block" else (s["ks"], s["vs"])
        any_row = ok.any(1)[:, :, None, None]
        k, v = torch.where(any_row, k * ks[..., :, None], 0.0), torch.where(any_row, v * vs[..., :, None], 0.0)
        q = s["q"][(cu[:-1, None] + r[None]).clamp(max=s["q"].shape[0] - 1)].float()
        q = q.reshape(n, Q, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(n, Hkv, G * Q, D)
        z = (q @ k.permute(0, 2, 3, 1)).reshape(n, Hkv, G, Q, -1) * s["scale"]
        z = torch.where(ok[:, None, None], z, -math.inf)
        m = z.amax(-1, keepdim=True)
        z = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
        z = z / z.sum(-1, keepdim=True).clamp(min=1e-37)
        o = z.reshape(n, Hkv, G * Q, -1) @ v.permute(0, 2, 1, 3)
        o = o.reshape(n, Hkv, G, Q, D).permute(0, 3, 1, 2, 4).reshape(n, Q, Hq, D)
        seq = torch.repeat_interleave(torch.arange(n, device=dev), ql, output_size=rows)
        out[r0:r0 + rows] = o[seq, torch.arange(rows, device=dev) - (cu[seq] - cu[0])].to(torch.bfloat16)
        i0, r0 = i1, r0 + rows
    return out


# --------------------------------------------------------------- one pass


def _calls(s):
    import paged_gqa_decode_reshape_gb300 as pg

    c = s["case"]
    if c["op"] == "plan":
        pg.pa_plan_step(s["bt"], s["ctx"], s["q"], s["free"], s["nfree"], s["NB"], s["new_lens"], s["new_free"],
                        s["granted"], s["cu"], s["pos"], s["slots"])
        return _plan_out(s)
    if c["op"] == "release":
        pg.pa_release_blocks(s["bt"], s["ctx"], s["keep"], s["free"], s["nfree"], s["NB"], s["new_lens"],
                             s["new_free"])
        return _release_out(s)
    if c["op"] == "rope":
        more = dict(q_weight=s["qw"], k_weight=s["kw"], eps=EPS, axes=s["axes"], interleaved=c["inter"])
        if c["cache"] == "none":
            pg.pa_norm_rope(s["q_out"], s["k_out"], s["q"], s["k"], s["table"], s["pos"], **more)
        elif c["cache"] == "bf16":
            pg.pa_norm_rope_and_cache(s["q_out"], s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["table"],
                                      s["pos"], **more)
        else:
            pg.pa_norm_rope_and_cache_fp8(s["q_out"], s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["ks"],
                                          s["vs"], s["table"], s["pos"], **more)
        return _rope_out(s)
    fn = pg.pa_decode_window_multi_fp8 if c["kv"] == "fp8" else pg.pa_decode_window_multi_fp8_block
    return fn(s["out"], s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["bt"], s["cu"], s["ctx"], c["window"], c["sinks"],
              s["scale"])


def run(state):
    if own:
        return _calls(state)
    plain = {"plan": _plain_plan, "release": _plain_release, "rope": _plain_rope, "chunk": _plain_chunk}
    return plain[state["case"]["op"]](state)


# -------------------------------------------------------- the least work


def work(case):
    L, op = _lengths(case), case["op"]
    if op == "plan":
        blocks, B = min(L["need"], L["free"]), case["B"]
        return {"bytes": 20 * B + 8 * blocks + 12 * L["T"] + 12, "flops": 0}
    if op == "release":
        blocks = sum(-(-x // BS) - -(-k // BS) for x, k in zip(L["ctx"], L["keep"]))
        return {"bytes": 12 * case["B"] + 8 * blocks + 8, "flops": 0}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if op == "rope":
        T, A, R = case["T"], case["T"] + case["pad"], case["R"]
        angles = 4 * R * min(T, 32000) + 4 * A * case["axes"]
        q, kv = 4 * Hq * D * A, {"none": 4 * A, "bf16": 8 * T, "fp8": 6 * T}[case["cache"]] * Hkv * D
        slots = 8 * A if case["cache"] != "none" else 0
        return {"bytes": q + kv + angles + slots + (4 * D if case["norm"] else 0),
                "flops": A * (Hq + Hkv) * ((4 * D if case["norm"] else 0) + 3 * R)}
    kv = pairs = blocks = 0
    for x, q in zip(L["ctx"], L["q"]):
        w, first = case["window"], case["sinks"]
        tokens = min(x, w + first + q - 1)
        kv += tokens
        blocks += -(-tokens // BS)
        lim = np.arange(x - q + 1, x + 1)
        pairs += int(np.minimum(lim, w + np.minimum(first, np.maximum(lim - w, 0))).sum())
    scales = 8 * Hkv * (blocks if case["kv"] == "fp8_block" else 1)
    return {"bytes": kv * 2 * Hkv * D + sum(L["q"]) * 4 * Hq * D + 8 * case["S"] + 4 * blocks + scales,
            "flops": 4 * D * Hq * pairs}


# ------------------------------------------------- the definition in 64 bits


def _exact_plan(s, L):
    bt = s["bt"].cpu().numpy().copy()
    free, nf = s["free"].cpu().numpy(), int(s["nfree"][0])
    B, MBS = bt.shape
    T = L["T"]
    cu, pos, slots = np.zeros(B + 1, np.int32), np.zeros(T, np.int32), np.full(T, -1, np.int64)
    new_lens, granted = np.zeros(B, np.int32), np.zeros(B, np.int32)
    row, asked, taken = 0, 0, 0
    for b, (x, n) in enumerate(zip(L["ctx"], L["q"])):
        have, want = -(-x // BS), -(-(x + n) // BS)
        ok = x + n <= MBS * BS and row + n <= T
        if ok and want > have:
            if asked + want - have <= nf:
                bt[b, have:want] = [free[nf - 1 - asked - i] for i in range(want - have)]
                taken += want - have
            else:
                ok = False
            asked += want - have
        p = x + np.arange(min(n, T - row))
        pos[row:row + len(p)] = p
        if ok:
            slots[row:row + n] = bt[b, p // BS].astype(np.int64) * BS + p % BS
            granted[b] = n
        new_lens[b] = x + granted[b]
        row += len(p)
        cu[b + 1] = row
    got = {"bt": bt, "new_lens": new_lens, "new_free": np.array([nf - taken], np.int32), "granted": granted, "cu": cu,
           "pos": pos, "slots": slots}
    return {k: torch.from_numpy(v) for k, v in got.items()}


def _exact_release(s, L):
    bt, free, nf = s["bt"].cpu().numpy(), s["free"].cpu().numpy().copy(), int(s["nfree"][0])
    for b, (x, k) in enumerate(zip(L["ctx"], L["keep"])):
        gone = bt[b, -(-k // BS):-(-x // BS)]
        free[nf:nf + len(gone)] = gone
        nf += len(gone)
    return {"free": torch.from_numpy(free), "new_lens": torch.tensor(L["keep"], dtype=torch.int32),
            "new_free": torch.tensor([nf], dtype=torch.int32)}


def _exact_rope(s, case):
    R, D, n = case["R"], case["D"], s["n"]
    pos = s["pos"].long() if case["axes"] > 1 else s["pos"].long()[None]
    of = s["axes"].tolist() if case["axes"] > 1 else [0] * (R // 2)
    table = s["table"].double()

    def turned(x, w):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / D + EPS) * w.double()
        z = y.clone()
        for i in range(R // 2):
            a, b = (2 * i, 2 * i + 1) if case["inter"] else (i, i + R // 2)
            at = pos[of[i]]
            co, si = table[at, i][:, None], table[at, R // 2 + i][:, None]
            z[..., a] = y[..., a] * co - y[..., b] * si
            z[..., b] = y[..., a] * si + y[..., b] * co
        return z

    q, k = turned(s["q"], s["qw"]), turned(s["k"], s["kw"])
    if case["cache"] == "none":
        return {"q": q, "k": k}
    slots = s["slots"][:n]
    if case["cache"] == "bf16":
        kc, vc = s["kc"].double(), s["vc"].double()
        kc.view(-1, *kc.shape[2:])[slots] = k[:n]
        vc.view(-1, *vc.shape[2:])[slots] = s["v"][:n].double()
        return {"q": q, "key_cache": kc, "value_cache": vc}
    kc, vc = (s[x].view(torch.float8_e4m3fn).double() for x in ("kc", "vc"))
    kc.view(-1, *kc.shape[2:])[slots] = (k[:n] / s["ks"].double()[:, None]).clamp(-448, 448)
    where = torch.tensor(V8_POS, device=slots.device)[slots % BS]
    vc.permute(0, 3, 1, 2)[slots // BS, where] = (s["v"][:n].double() / s["vs"].double()[:, None]).clamp(-448, 448)
    return {"q": q, "key_cache": kc, "value_cache": vc}


def _exact_chunk(s, case):
    L = s["lens"]
    q = s["q"].double()
    out = torch.zeros_like(q)
    Hq, Hkv = case["Hq"], case["Hkv"]
    where = torch.tensor(V8_POS, device=q.device)
    r = 0
    for b, (x, n) in enumerate(zip(L["ctx"], L["q"])):
        t = torch.arange(x, device=q.device)
        t = t[(t < case["sinks"]) | (t >= x - n + 1 - case["window"])]
        blk = s["bt"][b].long()[t // BS]
        last = x - n + torch.arange(n, device=q.device)[:, None]
        seen = (t[None] <= last) & ((t[None] < case["sinks"]) | (t[None] > last - case["window"]))
        for g in range(Hkv):
            ks, vs = (s[c].double()[blk, g][:, None] if case["kv"] == "fp8_block" else s[c].double()[g] for c in ("ks", "vs"))
            k = s["kc"][:, :, g][blk, t % BS].view(torch.float8_e4m3fn).double() * ks
            v = s["vc"][:, g].permute(0, 2, 1)[blk, where[t % BS]].view(torch.float8_e4m3fn).double() * vs
            for h in range(g * (Hq // Hkv), (g + 1) * (Hq // Hkv)):
                z = (q[r:r + n, h] @ k.T) * s["scale"]
                out[r:r + n, h] = torch.softmax(z.masked_fill(~seen, -math.inf), -1) @ v
        r += n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s, _lengths(case))
    if case["op"] == "release":
        return _exact_release(s, _lengths(case))
    if case["op"] == "rope":
        return _exact_rope(s, case)
    return _exact_chunk(s, case)
