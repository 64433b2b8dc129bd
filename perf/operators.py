"""Measured cases of the decode operators that work on a part of the paged cache:

* ``window``: attention over the last tokens and a few first ones (sinks), one
  query token per sequence, bf16 or 8-bit cache;
* ``window_multi``: the same for several query rows per sequence (speculative
  tokens, prefill chunks);
* ``prefix``: a batch whose sequences share long prefixes, each prefix's KV
  read once for its whole group;
* ``weights``: decode attention that also adds up, per cached token, the
  attention weight it received;
* ``evict``: the tokens with the largest weights (and the newest ones) moved
  to fresh blocks, the rest dropped.

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

# ------------------------------------------------------------------- cases


def listed():
    big = dict(Hq=28, Hkv=4, D=128)  # the head shape of this repository's workloads
    return [
        # one short chat turn: nothing but latency
        dict(name="window_one", op="window", kv="bf16", B=1, lo=700, hi=700, window=256, sinks=4, lens=1, **big),
        # a serving batch at 8K context, half of it inside the window
        dict(name="window_8k", op="window", kv="bf16", B=16, lo=4097, hi=12001, window=4096, sinks=4, lens=2, **big),
        # a large ragged batch on the 8-bit cache, some contexts shorter than the window
        dict(name="window_fp8_b128", op="window", kv="fp8", B=128, lo=33, hi=20011, window=2048, sinks=16, lens=3,
             **big),
        # speculative decoding: up to six rows per sequence
        dict(name="multi_spec", op="window_multi", S=32, qlo=1, qhi=6, lo=900, hi=15003, window=4096, sinks=4,
             lens=4, **big),
        # prefill chunks of long prompts next to shorter ones
        dict(name="multi_chunk", op="window_multi", S=3, qlo=517, qhi=2048, lo=9000, hi=16001, window=4096, sinks=64,
             lens=5, **big),
        # a few requests behind one system prompt
        dict(name="prefix_few", op="prefix", B=8, groups=1, plo=2001, phi=2001, lo=1, hi=301, lens=6, **big),
        # a batch of agents on one 8K context
        dict(name="prefix_8k", op="prefix", B=64, groups=1, plo=8192, phi=8192, lo=100, hi=1023, lens=7, **big),
        # several tenants, each with its own prefix, small heads
        dict(name="prefix_tenants", op="prefix", B=128, groups=5, plo=129, phi=16000, lo=1, hi=2049, lens=8, Hq=16,
             Hkv=4, D=64),
        # weights of a small batch of short sequences
        dict(name="weights_few", op="weights", B=3, lo=17, hi=600, lens=9, **big),
        # weights at 8K context
        dict(name="weights_8k", op="weights", B=16, lo=4097, hi=12001, lens=10, **big),
        # one sequence brought back under its budget
        dict(name="evict_one", op="evict", B=1, lo=1500, hi=1500, budget=1024, recent=128, lens=11, **big),
        # a batch at 8K context brought down to 4K
        dict(name="evict_8k", op="evict", B=16, lo=3001, hi=12001, budget=4096, recent=512, lens=12, **big),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_HEADS = [(28, 4, 128), (32, 8, 128), (8, 8, 128), (40, 8, 128), (12, 2, 64), (32, 4, 64), (9, 3, 64), (16, 2, 128)]


def draw(rng):
    op = rng.choice(["window", "window", "window_multi", "prefix", "prefix", "weights", "evict"])
    Hq, Hkv, D = rng.choice(_HEADS)
    c = dict(op=op, Hq=Hq, Hkv=Hkv, D=D, lens=rng.randrange(1 << 30))
    if op == "window":
        c["kv"] = rng.choice(["bf16", "fp8", "fp8_block"]) if D == 128 else "bf16"
        c["window"], c["sinks"] = _log(rng, 1, 8192), rng.choice([0, 1, 4, rng.randrange(200)])
        c["hi"] = _log(rng, 1, 20000)
        c["lo"] = _log(rng, 1, c["hi"])
        c["B"] = min(_log(rng, 1, 200), max(1, 600_000 // min(c["hi"], c["window"] + c["sinks"])),
                     max(1, 800_000 // c["hi"]))
    elif op == "window_multi":
        c["window"], c["sinks"] = _log(rng, 1, 8192), rng.choice([0, 1, 4, rng.randrange(200)])
        c["qhi"] = _log(rng, 1, 2048)
        c["qlo"] = _log(rng, 1, c["qhi"])
        c["hi"] = _log(rng, c["qhi"], 20000)
        c["lo"] = _log(rng, c["qhi"], c["hi"])
        seen = min(c["hi"], c["window"] + c["sinks"] + c["qhi"])
        c["S"] = min(_log(rng, 1, 48), max(1, 20_000_000 // (seen * c["qhi"])), max(1, 600_000 // seen))
    elif op == "prefix":
        c["phi"] = _log(rng, 16, 16000)
        c["plo"] = _log(rng, 1, c["phi"])
        c["hi"] = _log(rng, 1, 2049)
        c["lo"] = _log(rng, 1, c["hi"])
        c["B"] = min(_log(rng, 1, 160), max(1, 1_000_000 // (c["phi"] + c["hi"])))
        c["groups"] = min(c["B"], _log(rng, 1, 12))
    elif op == "weights":
        c["hi"] = _log(rng, 1, 30000)
        c["lo"] = _log(rng, 1, c["hi"])
        c["B"] = min(_log(rng, 1, 128), max(1, 100_000 // c["hi"]))
    else:
        c["hi"] = _log(rng, 64, 30000)
        c["lo"] = _log(rng, 32, c["hi"])
        c["budget"] = _log(rng, 16, min(8192, c["hi"]))
        c["recent"] = rng.randrange(c["budget"] + 1)
        c["B"] = min(_log(rng, 1, 64), max(1, 200_000 // (c["hi"] + c["budget"])))
    return c


def _lens(n, lo, hi, seed):
    """n lengths in [lo, hi], evenly spread over their logarithm; the first is hi."""
    r = random.Random(seed)
    return [hi] + [_log(r, max(lo, 1), hi) for _ in range(n - 1)]


def _lengths(case):
    """The case's lengths: tokens per sequence, and what else its operator has."""
    op, seed = case["op"], case["lens"]
    n = case["S"] if op == "window_multi" else case["B"]
    got = {"ctx": _lens(n, case["lo"], case["hi"], seed)}
    if op == "window_multi":
        got["q"] = _lens(n, case["qlo"], case["qhi"], seed + 1)
    if op == "prefix":
        got["prefix"] = _lens(case["groups"], case["plo"], case["phi"], seed + 2)
        r = random.Random(seed + 3)
        cuts = sorted(r.sample(range(1, n), case["groups"] - 1)) if case["groups"] > 1 else []
        got["cu"] = [0] + cuts + [n]
    return got


# ------------------------------------------------------------------ inputs


def _tables(lens, perm, at, device):
    """Block tables [n, max] for these lengths from perm[at:], -1 past each sequence's blocks."""
    nblk = [-(-x // BS) for x in lens]
    t = np.full((len(lens), max(1, max(nblk))), -1, np.int32)
    for i, n in enumerate(nblk):
        t[i, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(t).to(device), at


def _spoil(cache, tables, lens):
    """NaN in the unused slots of every sequence's last block: nothing may read them."""
    seq = [i for i, x in enumerate(lens) for _ in range(-x % BS)]
    pos = [x + k for x in lens for k in range(-x % BS)]
    if seq:
        seq, pos = torch.tensor(seq, device=cache.device), torch.tensor(pos, device=cache.device)
        cache[tables[seq, pos // BS].long(), pos % BS] = float("nan")


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    L = _lengths(case)
    ctx = L["ctx"]
    n = len(ctx)
    extra = L.get("prefix", []) + ([min(x, case["budget"]) for x in ctx] if case["op"] == "evict" else [])
    NB = sum(-(-x // BS) for x in ctx + extra) + 3
    perm = np.random.RandomState(seed % (1 << 32)).permutation(NB)
    s = dict(case=case, scale=D ** -0.5, lens=L)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(torch.bfloat16)

    s["kc"], s["vc"] = normal(NB, BS, Hkv, D), normal(NB, BS, Hkv, D)
    s["bt"], at = _tables(ctx, perm, 0, dev)
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    rows = sum(L["q"]) if "q" in L else n
    if case["op"] != "evict":
        # twice the usual spread of queries: logits with a standard deviation of 2
        s["q"] = normal(rows, Hq, D, std=2.0)
        s["out"] = torch.empty_like(s["q"])
        if case.get("kv", "bf16") == "bf16":
            _spoil(s["kc"], s["bt"], ctx)
            _spoil(s["vc"], s["bt"], ctx)
    if case["op"] == "window_multi":
        s["cu"] = torch.tensor([0] + list(np.cumsum(L["q"])), dtype=torch.int32, device=dev)
    if case["op"] == "prefix":
        s["pt"], at = _tables(L["prefix"], perm, at, dev)
        s["plen"] = torch.tensor(L["prefix"], dtype=torch.int32, device=dev)
        s["cu"] = torch.tensor(L["cu"], dtype=torch.int32, device=dev)
        _spoil(s["kc"], s["pt"], L["prefix"])
        _spoil(s["vc"], s["pt"], L["prefix"])
    if case["op"] in ("weights", "evict"):
        w = torch.rand(NB, Hkv, BS, generator=g, device=dev)
        # accumulated weights are mostly small and often equal (many exactly 0)
        s["weights"] = (torch.floor(w.pow(6) * 4096) / 256).contiguous()
    if case["op"] == "evict":
        s["dst"], at = _tables([min(x, case["budget"]) for x in ctx], perm, at, dev)
        want = max(1, -(-case["budget"] // BS))
        if s["dst"].shape[1] < want:
            s["dst"] = torch.nn.functional.pad(s["dst"], (0, want - s["dst"].shape[1]), value=-1).contiguous()
        s["kept"] = torch.empty((n, Hkv, case["budget"]), dtype=torch.int32, device=dev)
        s["new_lens"] = torch.empty((n,), dtype=torch.int32, device=dev)
    kv = case.get("kv", "bf16")
    if kv != "bf16":
        k, v = s["kc"].float(), s["vc"].float()
        if kv == "fp8":  # a scale per KV head
            s["ks"] = torch.full((Hkv,), 0.0117, device=dev) * (1 + torch.arange(Hkv, device=dev) / 8)
            s["vs"] = torch.full((Hkv,), 0.0127, device=dev) * (1 + torch.arange(Hkv, device=dev) / 16)
            kd, vd = s["ks"][None, None, :, None], s["vs"][None, None, :, None]
        else:  # a power of two per block and KV head that fits its largest value
            def fit(x):
                return torch.exp2(torch.ceil(torch.log2(x.abs().amax((1, 3)) / 448))).contiguous()
            s["ks"], s["vs"] = fit(k), fit(v)
            kd, vd = s["ks"][:, None, :, None], s["vs"][:, None, :, None]
        k8, v8 = ((x / d).clamp(-448, 448).to(torch.float8_e4m3fn) for x, d in ((k, kd), (v, vd)))
        s["kc"] = k8.view(torch.uint8).contiguous()
        inv = torch.tensor([V8_POS.index(i) for i in range(BS)], device=dev)
        s["vc"] = v8.view(torch.uint8).permute(0, 2, 3, 1)[..., inv].contiguous()
    return s


# -------------------------------------------------------- the plain forms


def _rows(cache, tables, pos):
    """[n, P, Hkv, D] fp32: the cache rows at positions pos [n, P] of each sequence (any row where pos is not one)."""
    p = pos.clamp(min=0).clamp(max=tables.shape[1] * BS - 1)
    blk = tables.gather(1, p // BS).long().clamp(min=0)
    return cache[blk, p % BS].float(), blk, p


def _kv(s, pos):
    """K and V at positions pos [n, P] of the state's sequences, decoded to fp32."""
    kv = s["case"].get("kv", "bf16")
    if kv == "bf16":
        return _rows(s["kc"], s["bt"], pos)[0], _rows(s["vc"], s["bt"], pos)[0]
    p = pos.clamp(min=0).clamp(max=s["bt"].shape[1] * BS - 1)
    blk = s["bt"].gather(1, p // BS).long().clamp(min=0)
    off = torch.tensor(V8_POS, device=pos.device)[p % BS]
    k = s["kc"].view(torch.float8_e4m3fn)[blk, p % BS].float()
    # advanced indices apart from each other: the result is [n, P, Hkv, D]
    v = s["vc"].view(torch.float8_e4m3fn)[blk, :, :, off].float()
    ks, vs = (s["ks"][blk], s["vs"][blk]) if kv == "fp8_block" else (s["ks"], s["vs"])
    return k * ks[..., :, None], v * vs[..., :, None]


def _attend(q, k, v, ok, scale):
    """out [n, R, Hq, D] and the probabilities [n, Hkv, G, R, P] for queries
    q [n, R, Hq, D] over k / v [n, P, Hkv, D], where ok [n, R, P] (or [n, 1, P])."""
    n, R, Hq, D = q.shape
    Hkv = k.shape[2]
    qf = q.float().reshape(n, R, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(n, Hkv, -1, D)
    any_row = ok.any(1)[:, :, None, None]
    k, v = torch.where(any_row, k, 0.0), torch.where(any_row, v, 0.0)
    z = (qf @ k.permute(0, 2, 3, 1)).reshape(n, Hkv, Hq // Hkv, R, -1) * scale
    z = torch.where(ok[:, None, None], z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-37)
    o = p.reshape(n, Hkv, -1, p.shape[-1]) @ v.permute(0, 2, 1, 3)
    return o.reshape(n, Hkv, Hq // Hkv, R, D).permute(0, 3, 1, 2, 4).reshape(n, R, Hq, D), p


def _plain_window(s):
    c = s["case"]
    sinks, window = c["sinks"], min(c["window"], max(s["lens"]["ctx"]))
    i = torch.arange(sinks + window, device=s["q"].device)[None]
    ctx = s["ctx"].long()[:, None]
    first = i < sinks
    pos = torch.where(first, i, ctx - window + i - sinks)
    ok = torch.where(first, pos < ctx, pos >= sinks)
    k, v = _kv(s, pos)
    return _attend(s["q"][:, None], k, v, ok[:, None], s["scale"])[0][:, 0].to(torch.bfloat16)


def _plain_window_multi(s):
    c, L = s["case"], s["lens"]
    dev = s["q"].device
    Q = max(L["q"])
    sinks, window = c["sinks"], min(c["window"], max(L["ctx"]))
    ctx, cu = s["ctx"].long(), s["cu"].long()
    ql = cu[1:] - cu[:-1]
    r = torch.arange(Q, device=dev)
    lim = (ctx - ql)[:, None] + r[None] + 1  # [S, Q]: row r sees positions below it
    i = torch.arange(sinks + window + Q - 1, device=dev)[None]
    first = i < sinks
    pos = torch.where(first, i, (ctx - ql - window + 1)[:, None] + i - sinks)
    k, v = _kv(s, pos)
    p, f = pos[:, None], first[:, None]
    ok = (p < lim[..., None]) & (f | ((p >= sinks) & (p >= lim[..., None] - window))) & (r[None] < ql[:, None])[..., None]
    q = s["q"][(cu[:-1, None] + r[None]).clamp(max=s["q"].shape[0] - 1)]
    o = _attend(q, k, v, ok, s["scale"])[0]
    seq = torch.repeat_interleave(torch.arange(len(L["q"]), device=dev), ql, output_size=s["q"].shape[0])
    return o[seq, torch.arange(s["q"].shape[0], device=dev) - cu[seq]].to(torch.bfloat16)


def _plain_prefix(s):
    L = s["lens"]
    dev = s["q"].device
    n = len(L["ctx"])
    cu = s["cu"].long()
    group = torch.repeat_interleave(torch.arange(len(L["prefix"]), device=dev), cu[1:] - cu[:-1], output_size=n)
    i = torch.arange(max(L["prefix"]), device=dev)[None].expand(len(L["prefix"]), -1)
    j = torch.arange(max(L["ctx"]), device=dev)[None].expand(n, -1)
    ok = torch.cat([(i < s["plen"][:, None])[group], j < s["ctx"][:, None]], 1)
    k = torch.cat([_rows(s["kc"], s["pt"], i)[0][group], _rows(s["kc"], s["bt"], j)[0]], 1)
    v = torch.cat([_rows(s["vc"], s["pt"], i)[0][group], _rows(s["vc"], s["bt"], j)[0]], 1)
    return _attend(s["q"][:, None], k, v, ok[:, None], s["scale"])[0][:, 0].to(torch.bfloat16)


def _plain_weights(s):
    j = torch.arange(max(s["lens"]["ctx"]), device=s["q"].device)[None].expand(len(s["lens"]["ctx"]), -1)
    ok = j < s["ctx"][:, None]
    k, blk, pos = _rows(s["kc"], s["bt"], j)
    o, p = _attend(s["q"][:, None], k, _rows(s["vc"], s["bt"], j)[0], ok[:, None], s["scale"])
    add = p[:, :, :, 0].sum(2)  # [n, Hkv, P]
    n, Hkv, P = add.shape
    h = torch.arange(Hkv, device=add.device)[None, :, None]
    w = s["weights"]
    at = ((blk[:, None] * Hkv + h) * BS + pos[:, None] % BS).reshape(-1)
    # what lies past a sequence adds 0
    w.view(-1).index_add_(0, at, add.reshape(-1))
    return {"out": o[:, 0].to(torch.bfloat16), "weights": w}


def _plain_evict(s):
    c, L = s["case"], s["lens"]
    w, ctx = s["weights"], s["ctx"].long()
    n, Hkv, budget = s["kept"].shape
    P = max(L["ctx"])
    j = torch.arange(P, device=w.device)[None].expand(n, -1)
    blk = s["bt"].gather(1, j // BS).long().clamp(min=0)
    old = w[blk, :, j % BS].permute(0, 2, 1)  # [n, Hkv, P]
    new = j >= ctx[:, None] - min(c["recent"], budget)
    key = torch.where(new[:, None], math.inf, old)
    key = torch.where((j >= ctx[:, None])[:, None], -math.inf, key)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    m = min(budget, P)
    live = torch.arange(m, device=w.device)[None] < ctx[:, None]  # [n, m]
    kept = torch.where(live[:, None], order[..., :m], P).sort(-1).values
    at = kept.clamp(max=P - 1)
    h = torch.arange(Hkv, device=w.device)[None, :, None]
    src = s["bt"].long()[torch.arange(n, device=w.device)[:, None, None], at // BS].clamp(min=0)
    i = torch.arange(m, device=w.device)[None, None].expand(n, Hkv, -1)
    dst = s["dst"].long()[torch.arange(n, device=w.device)[:, None, None], i // BS]
    take = live[:, None].expand(-1, Hkv, -1)
    hh = h.expand(n, -1, m)
    d, o, x, y, z = dst[take], (i % BS)[take], src[take], (at % BS)[take], hh[take]
    kc, vc = s["kc"], s["vc"]
    kc[d, o, z], vc[d, o, z], w[d, z, o] = kc[x, y, z], vc[x, y, z], w[x, z, y]
    s["kept"].fill_(-1)
    s["kept"][..., :m] = torch.where(take, kept, -1).int()
    s["new_lens"].copy_(ctx.clamp(max=budget))
    return {"kept": s["kept"], "new_lens": s["new_lens"], "key_cache": kc, "value_cache": vc, "weights": w}


# --------------------------------------------------------------- one pass


def _calls(s):
    import paged_gqa_decode_reshape_gb300 as pg

    c = s["case"]
    if c["op"] == "window":
        if c["kv"] == "bf16":
            return pg.pa_decode_window(s["out"], s["q"], s["kc"], s["vc"], s["bt"], s["ctx"], c["window"], c["sinks"],
                                       s["scale"])
        fn = pg.pa_decode_window_fp8 if c["kv"] == "fp8" else pg.pa_decode_window_fp8_block
        return fn(s["out"], s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["bt"], s["ctx"], c["window"], c["sinks"],
                  s["scale"])
    if c["op"] == "window_multi":
        return pg.pa_decode_window_multi(s["out"], s["q"], s["kc"], s["vc"], s["bt"], s["cu"], s["ctx"], c["window"],
                                         c["sinks"], s["scale"])
    if c["op"] == "prefix":
        return pg.pa_decode_prefix(s["out"], s["q"], s["kc"], s["vc"], s["pt"], s["plen"], s["cu"], s["bt"],
                                   s["ctx"], s["scale"])
    if c["op"] == "weights":
        pg.pa_decode_weights(s["out"], s["weights"], s["q"], s["kc"], s["vc"], s["bt"], s["ctx"], s["scale"])
        return {"out": s["out"], "weights": s["weights"]}
    pg.pa_evict(s["kept"], s["new_lens"], s["kc"], s["vc"], s["weights"], s["bt"], s["ctx"], s["dst"], c["recent"])
    return {"kept": s["kept"], "new_lens": s["new_lens"], "key_cache": s["kc"], "value_cache": s["vc"],
            "weights": s["weights"]}


def run(state):
    if own:
        return _calls(state)
    op = state["case"]["op"]
    if op == "window":
        return _plain_window(state)
    if op == "window_multi":
        return _plain_window_multi(state)
    if op == "prefix":
        return _plain_prefix(state)
    if op == "weights":
        return _plain_weights(state)
    return _plain_evict(state)


# -------------------------------------------------------- the least work


def work(case):
    L = _lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    eb = 2 if case.get("kv", "bf16") == "bf16" else 1
    row = 2 * Hkv * D * eb  # K and V of one token
    ctx = L["ctx"]
    io = 2 * 2 * Hq * D  # a query row and its output

    def tables(tokens):
        return 4 * -(-tokens // BS)

    if case["op"] == "window":
        seen = [min(x, case["window"] + case["sinks"]) for x in ctx]
        t = sum(seen)
        scales = 8 * Hkv * sum(-(-x // BS) for x in seen) if case["kv"] == "fp8_block" else 0
        return {"bytes": t * row + len(ctx) * (io + 4) + sum(map(tables, seen)) + scales, "flops": 4 * D * Hq * t}
    if case["op"] == "window_multi":
        kv = pairs = 0
        for x, q in zip(ctx, L["q"]):
            kv += min(x, case["window"] + case["sinks"] + q - 1)
            lim = np.arange(x - q + 1, x + 1)
            pairs += int(np.minimum(lim, case["window"] + np.minimum(case["sinks"], np.maximum(lim - case["window"], 0))).sum())
        return {"bytes": kv * row + sum(L["q"]) * io + len(ctx) * 8 + tables(kv), "flops": 4 * D * Hq * pairs}
    if case["op"] == "prefix":
        once = sum(L["prefix"]) + sum(ctx)
        pairs = sum(p * (b - a) for p, a, b in zip(L["prefix"], L["cu"], L["cu"][1:])) + sum(ctx)
        return {"bytes": once * row + len(ctx) * (io + 4) + tables(once) + 8 * len(L["prefix"]),
                "flops": 4 * D * Hq * pairs}
    if case["op"] == "weights":
        t = sum(ctx)
        return {"bytes": t * (row + 8 * Hkv) + len(ctx) * (io + 4) + tables(t), "flops": 4 * D * Hq * t}
    kept = sum(min(x, case["budget"]) for x in ctx)
    return {"bytes": sum(ctx) * Hkv * 4 + kept * (2 * row + 8 * Hkv) + 4 * len(ctx) * (Hkv * case["budget"] + 2) +
            tables(sum(ctx)) + tables(kept), "flops": sum(ctx) * Hkv}


# ------------------------------------------------- the definition in 64 bits


def _one(q, k, v, scale):
    """Softmax attention of q [Hq, D] over k / v [P, Hkv, D] in fp64, one sequence: out and weights [Hq, P]."""
    Hq, D = q.shape
    if k.shape[0] == 0:
        return torch.zeros_like(q), q.new_zeros(Hq, 0)
    k, v = (x.repeat_interleave(Hq // x.shape[1], 1) for x in (k, v))
    p = torch.softmax(torch.einsum("hd,phd->hp", q, k) * scale, -1)
    return torch.einsum("hp,phd->hd", p, v), p


def _cached(s, row, positions, what, tables="bt"):
    """Rows of the K or V cache [P, Hkv, D] in fp64 at these positions of one sequence."""
    blk = s[tables][row].long()[positions // BS]
    kv = s["case"].get("kv", "bf16")
    c = s[what]
    if kv == "bf16":
        return c[blk, positions % BS].double()
    scale = (s["ks"] if what == "kc" else s["vs"]).double()
    scale = scale[blk][:, :, None] if kv == "fp8_block" else scale[None, :, None]
    if what == "kc":
        return c[blk, positions % BS].view(torch.float8_e4m3fn).double() * scale
    o = positions % BS
    at = 4 * ((o % 8) // 2) + 2 * (o // 8) + o % 2
    whole = c[blk].view(torch.float8_e4m3fn).double()  # [P, Hkv, D, 16]
    return whole.gather(3, at[:, None, None, None].expand(-1, *whole.shape[1:3], 1))[..., 0] * scale


def exact(case, seed):
    s = prepare(case, seed)
    L, op, scale = s["lens"], case["op"], s["scale"]
    dev = s["kc"].device
    if op == "evict":
        Hkv, budget = case["Hkv"], case["budget"]
        kept = np.full((len(L["ctx"]), Hkv, budget), -1, np.int32)
        kc, vc, w = s["kc"].clone(), s["vc"].clone(), s["weights"].clone()
        for b, x in enumerate(L["ctx"]):
            m, tab, dst = min(x, budget), s["bt"][b].long(), s["dst"][b].long()
            j = torch.arange(x, device=dev)
            for h in range(Hkv):
                row = s["weights"][tab[j // BS], h, j % BS].double().cpu().numpy()
                keep = np.arange(x)
                if x > budget:
                    new = min(case["recent"], budget)
                    best = np.lexsort((np.arange(x - new), -row[:x - new]))[:budget - new]
                    keep = np.concatenate([np.sort(best), np.arange(x - new, x)])
                kept[b, h, :m] = keep
                a, i = torch.from_numpy(keep).to(dev), torch.arange(m, device=dev)
                kc[dst[i // BS], i % BS, h] = s["kc"][tab[a // BS], a % BS, h]
                vc[dst[i // BS], i % BS, h] = s["vc"][tab[a // BS], a % BS, h]
                w[dst[i // BS], h, i % BS] = s["weights"][tab[a // BS], h, a % BS]
        return {"kept": torch.from_numpy(kept), "new_lens": torch.tensor([min(x, budget) for x in L["ctx"]]).int(),
                "key_cache": kc.double(), "value_cache": vc.double(), "weights": w.double()}
    q = s["q"].double()
    out = torch.zeros(q.shape, dtype=torch.float64, device=dev)
    if op == "window":
        for b, x in enumerate(L["ctx"]):
            t = torch.arange(x, device=dev)
            t = t[(t < case["sinks"]) | (t >= x - case["window"])]
            out[b] = _one(q[b], _cached(s, b, t, "kc"), _cached(s, b, t, "vc"), scale)[0]
        return out
    if op == "window_multi":
        r = 0
        Hq, Hkv = case["Hq"], case["Hkv"]
        for b, (x, ql) in enumerate(zip(L["ctx"], L["q"])):
            t = torch.arange(x, device=dev)
            t = t[(t < case["sinks"]) | (t >= x - ql + 1 - case["window"])]
            k, v = _cached(s, b, t, "kc"), _cached(s, b, t, "vc")
            last = x - ql + torch.arange(ql, device=dev)[:, None]
            seen = (t[None] <= last) & ((t[None] < case["sinks"]) | (t[None] > last - case["window"]))
            for h in range(Hq):
                z = (q[r:r + ql, h] @ k[:, h * Hkv // Hq].T) * scale
                out[r:r + ql, h] = torch.softmax(z.masked_fill(~seen, -math.inf), -1) @ v[:, h * Hkv // Hq]
            r += ql
        return out
    if op == "prefix":
        for a, b, (grp, pl) in zip(L["cu"], L["cu"][1:], enumerate(L["prefix"])):
            t = torch.arange(pl, device=dev)
            pk, pv = _cached(s, grp, t, "kc", "pt"), _cached(s, grp, t, "vc", "pt")
            for i in range(a, b):
                u = torch.arange(L["ctx"][i], device=dev)
                k, v = torch.cat([pk, _cached(s, i, u, "kc")]), torch.cat([pv, _cached(s, i, u, "vc")])
                out[i] = _one(q[i], k, v, scale)[0]
        return out
    w = s["weights"].double()
    for b, x in enumerate(L["ctx"]):
        t = torch.arange(x, device=dev)
        out[b], p = _one(q[b], _cached(s, b, t, "kc"), _cached(s, b, t, "vc"), scale)
        blk = s["bt"][b].long()[t // BS]
        w[blk, :, t % BS] += p.reshape(case["Hkv"], -1, x).sum(1).T
    return {"out": out, "weights": w}
