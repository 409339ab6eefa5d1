"""The serving-step operators around a 4-bit context pool, as measured cases.

    plan      block tables and slot maps from the request lengths
    release   the blocks of finished requests back to the free list
    rope      rotary positions with several axes (time, height, width)
    append    the step's new K/V rows quantised into the 4-bit pool
    attend    the relay decode step over a 4-bit context pool

`own` selects the framework's calls; otherwise every operator is computed in
elementary torch operations.  Cases are dicts of plain values; inputs are made
from the seed alone, and the multiset of request lengths from the case alone.
"""
import random

import numpy as np
import torch

own = False

BLOCK = 16
LEFT = 2.0 ** -6     # what output rows that no request owns hold before (and after) the call


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one chat request early in its answer, grouped heads: nothing but latency
        dict(name="attend: one request", op="attend", B=1, Lq=1, H=32, Hkv=8, D=128, group=128, Ls=512, lo=37, hi=37,
             chunks=0),
        # the Llama-2-7B shape of the repository's benchmark (multi-head, 32 chats over one prompt)
        dict(name="attend: llama2_7b", op="attend", B=32, Lq=1, H=32, Hkv=32, D=128, group=128, Ls=2048, lo=64, hi=1024,
             chunks=0),
        # the Llama-2-70B grouped shape with long documents as contexts
        dict(name="attend: 70b, long contexts", op="attend", B=32, Lq=1, H=64, Hkv=8, D=128, group=64, Ls=2048, lo=1000,
             hi=16384, chunks=0),
        # decode requests mixed with prompt chunks of the Llama-2-13B shape, fine groups
        dict(name="attend: 13b, mixed with chunks", op="attend", B=16, Lq=128, H=40, Hkv=40, D=128, group=32, Ls=1024,
             lo=1, hi=4096, chunks=4),
        # one decode step of 32 requests, grouped heads
        dict(name="append: decode step", op="append", B=32, Lq=1, Hkv=8, D=128, group=128, lo=64, hi=1024),
        # prompt chunks of four requests, ragged, multi-head
        dict(name="append: prompt chunks", op="append", B=4, Lq=2048, Hkv=32, D=128, group=64, lo=1500, hi=2048),
        # one decode step of 32 requests behind images
        dict(name="rope: decode step", op="rope", B=32, Lq=1, H=32, Hkv=8, D=128, Ls=2048, a0=16, a1=24, a2=24,
             interleaved=False, ragged=False, inverse=False),
        # image and video prompts, ragged, the axes dealt to the pairs in turn
        dict(name="rope: image prompts", op="rope", B=4, Lq=2048, H=64, Hkv=8, D=128, Ls=512, a0=24, a1=20, a2=20,
             interleaved=True, ragged=True, inverse=False),
        # the bookkeeping of a decode step
        dict(name="plan: decode step", op="plan", B=32, Lq=1, lo=64, hi=1024, max_blocks=64),
        # many prompts admitted at once
        dict(name="plan: admission", op="plan", B=512, Lq=1024, lo=1, hi=1024, max_blocks=128),
        # a few requests of a batch end
        dict(name="release: a few", op="release", B=32, done=3, lo=64, hi=1024, max_blocks=64),
        # a large batch of long requests is taken down
        dict(name="release: many", op="release", B=512, done=400, lo=1000, hi=16384, max_blocks=1024),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "rope", "plan", "release"])
    if op == "attend":
        while True:
            D = rng.choice([64, 128, 128])
            Hkv = rng.choice([1, 2, 4, 5, 8, 20, 32])
            G = rng.choice([1, 1, 2, 4, 5, 8, 12])
            B = _log_int(rng, 1, 64)
            hi = _log_int(rng, 1, 16384)
            lo = _log_int(rng, 1, hi)
            Lq = rng.choice([1, 1, 2, 5, 33, 128])
            chunks = 0 if Lq == 1 else (B if Lq <= 5 else _log_int(rng, 1, min(B, 4)))
            c = dict(op="attend", B=B, Lq=Lq, H=Hkv * G, Hkv=Hkv, D=D,
                     group=rng.choice([g for g in (32, 64, 128) if g <= D]), Ls=rng.choice([0, _log_int(rng, 16, 4096)]),
                     lo=lo, hi=hi, chunks=chunks)
            w, most = work(c), [work(x) for x in listed() if x["op"] == "attend"]
            if c["H"] <= 96 and w["bytes"] <= max(x["bytes"] for x in most) and \
                    w["flops"] <= max(x["flops"] for x in most) and \
                    B * Lq * c["H"] * (c["Ls"] + hi) <= 16 * 128 * 40 * 5120 and B * hi * Hkv * D <= 32 * 16384 * 8 * 128:
                return c
    if op == "append":
        while True:
            Lq = rng.choice([1, 1, _log_int(rng, 2, 2048)])
            D = rng.choice([64, 128])
            c = dict(op="append", B=_log_int(rng, 1, 256), Lq=Lq, Hkv=rng.choice([1, 2, 5, 8, 32]), D=D,
                     group=rng.choice([g for g in (32, 64, 128) if g <= D]), lo=max(1, Lq // 2), hi=max(Lq, 1024))
            if work(c)["bytes"] <= work(listed()[5])["bytes"]:
                return c
    if op == "rope":
        while True:
            D = rng.choice([64, 128])
            Lq = rng.choice([1, 1, _log_int(rng, 2, 4096)])
            Hkv = rng.choice([1, 2, 5, 8, 32])
            a1 = rng.choice([D // 8, D // 6, 3 * D // 16, 1])
            a2 = rng.choice([0, a1])
            c = dict(op="rope", B=_log_int(rng, 1, 256), Lq=Lq, H=Hkv * rng.choice([1, 4, 7]), Hkv=Hkv, D=D,
                     Ls=rng.choice([0, _log_int(rng, 16, 32768)]), a0=D // 2 - a1 - a2, a1=a1, a2=a2,
                     interleaved=rng.random() < 0.5 and 6 * a1 <= D, ragged=Lq > 1, inverse=rng.random() < 0.25)
            if work(c)["bytes"] <= work(listed()[7])["bytes"]:
                return c
    if op == "plan":
        Lq = rng.choice([1, 1, _log_int(rng, 2, 1024)])
        hi = max(Lq, _log_int(rng, 16, 2000))
        return dict(op="plan", B=_log_int(rng, 1, 512), Lq=Lq, lo=_log_int(rng, 1, hi), hi=hi,
                    max_blocks=(hi + 15) // 16 + rng.randrange(0, 9))
    B = _log_int(rng, 1, 512)
    hi = _log_int(rng, 16, 16000)
    return dict(op="release", B=B, done=rng.randint(1, B), lo=_log_int(rng, 1, hi), hi=hi,
                max_blocks=(hi + 15) // 16 + rng.randrange(0, 9))


def _lens(case):
    """The request lengths of a case: evenly spread over [lo, hi], both ends included."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [hi] if B == 1 else [lo + (hi - lo) * b // (B - 1) for b in range(B)]


def _rows(case, lens):
    """(context length, query rows) of every request: `chunks` of them bring up to Lq rows, the others one."""
    B, Lq = case["B"], case["Lq"]
    got = []
    for b in range(B):
        ql = max(1, Lq - 5 * (B - 1 - b)) if Lq > 5 and b >= B - case["chunks"] else (Lq if case["chunks"] == B else 1)
        got.append((max(lens[b], ql), ql))
    return got


def work(case):
    op = case["op"]
    if op == "attend":
        D, H, Hkv = case["D"], case["H"], case["Hkv"]
        rows = _rows(case, _lens(case))
        kv = 2 * (D // 2 + 4 * (D // case["group"]))
        nbytes = sum(n for n, _ in rows) * Hkv * kv + case["Ls"] * Hkv * D * 4 + sum(q for _, q in rows) * H * (4 * D + 4)
        seen = sum(q * (case["Ls"] + n - q) + q * (q + 1) // 2 for n, q in rows)
        return {"bytes": nbytes, "flops": 4 * D * H * seen}
    if op == "append":
        rows = sum(q for _, q in _append_rows(case, _lens(case)))
        D = case["D"]
        return {"bytes": rows * case["Hkv"] * 2 * (2 * D + D // 2 + 4 * (D // case["group"])),
                "flops": rows * case["Hkv"] * 2 * D * 6}
    if op == "rope":
        tokens = sum(_rope_rows(case))
        n = tokens * (case["H"] + case["Hkv"]) * case["D"]
        return {"bytes": 4 * n + 12 * tokens, "flops": 3 * n}
    lens = _lens(case)
    if op == "plan":
        rows = _plan_rows(case, lens)
        new = sum((n + 15) // 16 - (n - q + 15) // 16 for n, q in rows)
        return {"bytes": 4 * (2 * len(rows) + 2 * new + case["B"] * case["Lq"] + len(rows) + 2), "flops": 2 * case["B"] * case["Lq"]}
    ids = sum((n + 15) // 16 for n in lens[-case["done"]:])
    return {"bytes": 4 * (2 * ids + 2 * case["B"] + 2), "flops": ids}


def _append_rows(case, lens):
    """Decode: one row behind each context; chunks: the whole length is new, up to Lq rows."""
    return [(n, min(n, case["Lq"])) for n in lens]


def _plan_rows(case, lens):
    return [(n, min(n, case["Lq"])) for n in lens]


def _rope_rows(case):
    B, Lq = case["B"], case["Lq"]
    return [max(1, Lq - (b * Lq) // (3 * B)) if case["ragged"] else Lq for b in range(B)]


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).half()


def _quantise(x, group):
    """[..., D] fp16 -> codes [..., D / 2] uint8 and [..., D / group, 2] fp16 (scale, lowest value), in 32 bits."""
    v = x.float().unflatten(-1, (-1, group))
    lo, hi = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
    fifteen = torch.full_like(hi, 15.0)          # a tensor: a division, not a product with a rounded reciprocal
    scale = ((hi - lo) / fifteen).half()
    s = scale.float()
    c = torch.where(s > 0, (v - lo) / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(v))
    c = c.round().clamp(0, 15).to(torch.uint8).flatten(-2)
    sz = torch.cat([scale, lo.half()], -1)
    return c[..., 0::2] | (c[..., 1::2] << 4), sz


def _tables(lens, max_blocks, g, spare=0.1):
    """Block tables over a shuffled pool; unused entries are -1."""
    need = [(n + BLOCK - 1) // BLOCK for n in lens]
    total = sum(need)
    num_blocks = total + max(2, int(total * spare))
    order = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
    n = torch.tensor(need, device="cuda")
    first = torch.cumsum(n, 0) - n
    j = torch.arange(max_blocks, device="cuda")
    at = (first[:, None] + j).clamp(max=num_blocks - 1)
    bt = torch.where(j < n[:, None], order[at], torch.full_like(order[at], -1))
    return bt.to(torch.int32).contiguous(), num_blocks, order[total:].contiguous()


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    shuffled = random.Random(int(seed))
    s = dict(case)
    op = case["op"]
    if op == "attend":
        lens = _lens(case)
        rows = _rows(case, lens)
        shuffled.shuffle(rows)
        ctx, ql = [n for n, _ in rows], [q for _, q in rows]
        max_blocks = (max(ctx) + BLOCK - 1) // BLOCK + 1
        bt, num_blocks, spare = _tables(ctx, max_blocks, g)
        B, Lq, H, Hkv, D = (case[k] for k in ("B", "Lq", "H", "Hkv", "D"))
        s["block_tables"], s["ctx_lens"] = bt, _int(ctx)
        s["q_lens"] = None if all(q == Lq for q in ql) else _int(ql)
        s["q_total"] = sum(ql)
        s["q"] = _normal(g, B, Lq, H, D)
        s["sys_k"], s["sys_v"] = _normal(g, case["Ls"], Hkv, D), _normal(g, case["Ls"], Hkv, D)
        for name in ("k", "v"):
            codes, sz = _quantise(_normal(g, num_blocks, Hkv, BLOCK, D), case["group"])
            sz[spare.long()] = float("nan")        # blocks that no request holds
            s[name + "_codes"], s[name + "_sz"] = codes.contiguous(), sz.contiguous()
        s["out"] = torch.full((B, Lq, H, D), LEFT, dtype=torch.float16, device="cuda")
        s["lse"] = torch.full((B, Lq, H), LEFT, dtype=torch.float32, device="cuda")
    elif op == "append":
        rows = _append_rows(case, _lens(case))
        shuffled.shuffle(rows)
        ctx, ql = [n for n, _ in rows], [q for _, q in rows]
        B, Lq, Hkv, D = (case[k] for k in ("B", "Lq", "Hkv", "D"))
        bt, num_blocks, _ = _tables(ctx, (max(ctx) + BLOCK - 1) // BLOCK, g)
        s["block_tables"], s["ctx_lens"] = bt, _int(ctx)
        s["q_lens"] = None if all(q == Lq for q in ql) else _int(ql)
        # channels of keys differ in offset and spread
        spread = torch.exp(0.5 * torch.randn(Hkv, D, generator=g, device="cuda"))
        s["k_new"] = (_normal(g, B, Lq, Hkv, D).float() * spread + torch.randn(Hkv, D, generator=g, device="cuda")).half()
        s["v_new"] = _normal(g, B, Lq, Hkv, D)
        for name in ("k", "v"):
            codes = torch.randint(0, 256, (num_blocks, Hkv, BLOCK, D // 2), generator=g, device="cuda", dtype=torch.uint8)
            sz = torch.rand(num_blocks, Hkv, BLOCK, D // case["group"], 2, generator=g, device="cuda").half()
            s[name + "_codes"], s[name + "_sz"] = codes, sz
    elif op == "rope":
        B, Lq, H, Hkv, D = (case[k] for k in ("B", "Lq", "H", "Hkv", "D"))
        ql = _rope_rows(case)
        shuffled.shuffle(ql)
        s["q_lens"] = None if all(q == Lq for q in ql) else _int(ql)
        s["q"], s["k_new"] = _normal(g, B, Lq, H, D), _normal(g, B, Lq, Hkv, D)
        # a prompt's frames, rows and columns behind the tokens before them
        start = torch.randint(0, 8192, (B, 1), generator=g, device="cuda")
        i = torch.arange(Lq, device="cuda")
        s["positions"] = torch.stack([start + i // 1024, start + (i % 1024) // 32, start + i % 32]).to(torch.int32).contiguous()
        s["sections"] = (case["a0"], case["a1"], case["a2"])
        s["base"] = 10000.0
        s["q_out"], s["k_out"] = torch.full_like(s["q"], LEFT), torch.full_like(s["k_new"], LEFT)
    else:
        lens = _lens(case)
        if op == "plan":
            rows = _plan_rows(case, lens)
            shuffled.shuffle(rows)
            lens, ql = [n for n, _ in rows], [q for _, q in rows]
            s["q_lens"] = None if all(q == case["Lq"] for q in ql) else _int(ql)
            held = [n - q for n, q in rows]
        else:
            flags = [0] * (case["B"] - case["done"]) + [1] * case["done"]
            pairs = list(zip(lens, flags))
            shuffled.shuffle(pairs)
            lens, flags = [n for n, _ in pairs], [f for _, f in pairs]
            s["done"] = _int(flags)
            held = lens
        bt, _, _ = _tables(held, case["max_blocks"], g)
        # the pool holds every request at its length and a tenth more; the free list is what no table names
        total = sum((n + BLOCK - 1) // BLOCK for n in lens)
        num_blocks = total + total // 10 + 8
        ids = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
        taken = bt >= 0
        n_taken = int(taken.sum())
        bt[taken] = ids[:n_taken]
        s["free_blocks"] = torch.full((num_blocks,), -1, dtype=torch.int32, device="cuda")
        s["free_blocks"][: num_blocks - n_taken] = ids[n_taken:]
        s["n_free"] = _int([num_blocks - n_taken])
        s["n_free_out"] = _int([0])
        s["block_tables"], s["ctx_lens"], s["num_blocks"] = bt, _int(lens), num_blocks
        if op == "plan":
            s["slot_map"] = torch.full((case["B"], case["Lq"]), -2, dtype=torch.int32, device="cuda")
    return s


# ----------------------------------------------------------------------------- one pass
def run(state):
    return {"attend": _attend, "append": _append, "rope": _rope, "plan": _plan, "release": _release}[state["op"]](state)


def _cache(relay, s):
    if "cache" not in s:      # a view of the pool's four tensors, which the program keeps beside them
        s["cache"] = relay.Q4Cache(s["k_codes"], s["k_sz"], s["v_codes"], s["v_sz"])
    return s["cache"]


def _small_workspace(s):
    if "ws" not in s:
        s["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    return s["ws"]


def _dequantise(codes, sz):
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    sz = sz.float()
    return (c.unflatten(-1, (sz.shape[-2], -1)) * sz[..., :1] + sz[..., 1:]).flatten(-2)


def _attend(s):
    if own:
        import shared_prompt_decode_gb300 as relay
        cache = _cache(relay, s)
        if "ws" not in s:
            s["dims"] = relay.make_dims(s["q"], s["Ls"], s["k_codes"].shape[0], s["block_tables"].shape[1],
                                        max_q_total=0 if s["q_lens"] is None else s["q_total"], Hkv=s["Hkv"])
            s["ws"] = relay.make_workspace_q4(s["dims"])
        relay.relay_attention_decode_q4(s["q"], s["sys_k"], s["sys_v"], cache, s["block_tables"], s["ctx_lens"],
                                        s["q_lens"], out=s["out"], lse_out=s["lse"], workspace=s["ws"], dims=s["dims"])
        return {"out": s["out"], "lse": s["lse"]}
    B, Lq, H, Hkv, D, Ls = (s[k] for k in ("B", "Lq", "H", "Hkv", "D", "Ls"))
    bt, ctx = s["block_tables"].clamp(min=0).long(), s["ctx_lens"].long()
    ql = torch.full_like(ctx, Lq) if s["q_lens"] is None else s["q_lens"].long()
    N = bt.shape[1] * BLOCK
    t = torch.arange(N, device="cuda")
    i = torch.arange(Lq, device="cuda")
    held = (t < ctx[:, None])[:, None, :, None]
    # the contexts as [B, Hkv, N, D], nothing where a request holds no token
    k = _dequantise(s["k_codes"][bt], s["k_sz"][bt]).transpose(1, 2).reshape(B, Hkv, N, D)
    k = torch.where(held, k, 0.0)
    q = s["q"].float().view(B, Lq, Hkv, H // Hkv, D)
    scale = D ** -0.5
    sc = torch.einsum("blkgd,bknd->blkgn", q, k) * scale
    del k
    seen = t < (ctx - ql + 1)[:, None, None] + i[:, None]                       # [B, Lq, N]
    sc = torch.where((seen & (t < ctx[:, None, None]))[:, :, None, None], sc, float("-inf"))
    sy = torch.einsum("blkgd,skd->blkgs", q, s["sys_k"].float()) * scale
    sc = torch.cat([sy, sc], -1)
    m = sc.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(sc - m)
    total = p.sum(-1, keepdim=True)
    v = _dequantise(s["v_codes"][bt], s["v_sz"][bt]).transpose(1, 2).reshape(B, Hkv, N, D)
    v = torch.where(held, v, 0.0)
    o = torch.einsum("blkgn,bknd->blkgd", p[..., Ls:], v) + torch.einsum("blkgs,skd->blkgd", p[..., :Ls], s["sys_v"].float())
    o = (o / total.clamp(min=1e-38)).reshape(B, Lq, H, D).half()
    lse = (m + torch.log(total)).reshape(B, Lq, H)
    valid = i < ql[:, None]
    return {"out": torch.where(valid[..., None, None], o, s["out"]), "lse": torch.where(valid[..., None], lse, s["lse"])}


def _append(s):
    pool = {k: s[k] for k in ("k_codes", "k_sz", "v_codes", "v_sz")}
    if own:
        import shared_prompt_decode_gb300 as relay
        relay.relay_kv_append_q4(s["k_new"], s["v_new"], s["block_tables"], s["ctx_lens"], _cache(relay, s), s["q_lens"],
                                 workspace=_small_workspace(s))
        return pool
    Lq, ctx = s["Lq"], s["ctx_lens"].long()
    ql = torch.full_like(ctx, Lq) if s["q_lens"] is None else s["q_lens"].long()
    i = torch.arange(Lq, device="cuda")
    b, row = torch.nonzero(i < ql[:, None], as_tuple=True)
    pos = ctx[b] - ql[b] + row
    blk, at = s["block_tables"][b, pos // BLOCK].long(), pos % BLOCK
    for name in ("k", "v"):
        codes, sz = _quantise(s[name + "_new"][b, row], s["group"])
        pool[name + "_codes"][blk, :, at] = codes
        pool[name + "_sz"][blk, :, at] = sz
    return pool


def _rope(s):
    if own:
        import shared_prompt_decode_gb300 as relay
        relay.relay_rope_axes(s["q"], s["positions"], s["Ls"], s["sections"], k_new=s["k_new"], q_lens=s["q_lens"],
                              base=s["base"], interleaved=s["interleaved"], inverse=s["inverse"], q_out=s["q_out"],
                              k_out=s["k_out"], workspace=_small_workspace(s))
        return {"q": s["q_out"], "k": s["k_out"]}
    Lq, half = s["Lq"], s["D"] // 2
    a0, a1, a2 = s["sections"]
    j = torch.arange(half, device="cuda")
    if s["interleaved"]:      # the axes in turn, for as long as a further axis has pairs left
        axis = torch.where((j % 3 == 1) & (j < 3 * a1), 1, torch.where((j % 3 == 2) & (j < 3 * a2), 2, 0))
    else:
        axis = (j >= a0).long() + (j >= a0 + a1).long()
    pos = (s["positions"].double() + s["Ls"])[axis].permute(1, 2, 0)                # [B, Lq, D / 2]
    ang = pos * s["base"] ** (-2.0 * j.double() / s["D"])
    cos, sin = ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]
    if s["inverse"]:
        sin = -sin
    rows = torch.full((s["B"],), Lq, device="cuda") if s["q_lens"] is None else s["q_lens"]
    valid = (torch.arange(Lq, device="cuda") < rows[:, None])[..., None, None]

    def turn(x, left):
        x0, x1 = x[..., :half].float(), x[..., half:].float()
        return torch.where(valid, torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).half(), left)
    return {"q": turn(s["q"], s["q_out"]), "k": turn(s["k_new"], s["k_out"])}


def _plan(s):
    if own:
        import shared_prompt_decode_gb300 as relay
        relay.relay_block_plan(s["ctx_lens"], s["block_tables"], s["free_blocks"], s["n_free"], q_lens=s["q_lens"],
                               Lq=s["Lq"], slot_map=s["slot_map"], n_free_out=s["n_free_out"], workspace=_small_workspace(s))
        return {"block_tables": s["block_tables"], "slot_map": s["slot_map"], "n_free": s["n_free_out"]}
    Lq, ctx, bt = s["Lq"], s["ctx_lens"].long(), s["block_tables"]
    ql = torch.full_like(ctx, Lq) if s["q_lens"] is None else s["q_lens"].long()
    held = (ctx - ql + BLOCK - 1) // BLOCK
    need = (ctx + BLOCK - 1) // BLOCK - held
    base = torch.cumsum(need, 0) - need
    granted = (need == 0) | (base + need <= s["n_free"])
    need = torch.where(granted, need, 0)
    j = torch.arange(bt.shape[1], device="cuda") - held[:, None]
    new = (j >= 0) & (j < need[:, None])
    at = (s["n_free"] - 1 - base[:, None] - j).clamp(0, s["free_blocks"].shape[0] - 1)
    bt = torch.where(new, s["free_blocks"][at], bt)
    i = torch.arange(Lq, device="cuda")
    pos = (ctx - ql)[:, None] + i
    page = torch.gather(bt, 1, (pos // BLOCK).clamp(max=bt.shape[1] - 1))
    slot = torch.where((i < ql[:, None]) & granted[:, None], page * BLOCK + pos % BLOCK, -1)
    return {"block_tables": bt, "slot_map": slot.to(torch.int32), "n_free": (s["n_free"] - need.sum()).to(torch.int32)}


def _release(s):
    if own:
        import shared_prompt_decode_gb300 as relay
        relay.relay_block_release(s["done"], s["ctx_lens"], s["block_tables"], s["free_blocks"], s["n_free"],
                                  n_free_out=s["n_free_out"], workspace=_small_workspace(s))
        return {"free_blocks": s["free_blocks"], "n_free": s["n_free_out"]}
    bt, ctx = s["block_tables"], s["ctx_lens"].long()
    n = torch.where(s["done"] != 0, (ctx + BLOCK - 1) // BLOCK, 0)
    first = s["n_free"] + torch.cumsum(n, 0) - n
    j = torch.arange(bt.shape[1], device="cuda")
    mine = j < n[:, None]
    free = s["free_blocks"].clone()
    free[(first[:, None] + j)[mine]] = bt[mine]
    return {"free_blocks": free, "n_free": (s["n_free"] + n.sum()).to(torch.int32)}


# ----------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("plan", "release"):
        return None
    if op == "attend":
        return _exact_attend(s)
    if op == "rope":
        return _exact_rope(s)
    # the scales and lowest values that the append writes; the codes are whole numbers
    got = {"k_codes": None, "v_codes": None}
    ctx, bt = s["ctx_lens"].tolist(), s["block_tables"].cpu().numpy()
    ql = [s["Lq"]] * s["B"] if s["q_lens"] is None else s["q_lens"].tolist()
    for name in ("k", "v"):
        sz = s[name + "_sz"].double().cpu().numpy()
        new = s[name + "_new"].double().cpu().numpy()
        for b in range(s["B"]):
            x = new[b, : ql[b]].reshape(ql[b], s["Hkv"], -1, s["group"])
            at = np.arange(ctx[b] - ql[b], ctx[b])
            val = np.stack([(x.max(-1) - x.min(-1)) / 15.0, x.min(-1)], -1)
            sz[bt[b, at // BLOCK], :, at % BLOCK] = val
        got[name + "_sz"] = sz
    return got


def _exact_attend(s):
    B, Lq, H, Hkv, D, Ls = (s[k] for k in ("B", "Lq", "H", "Hkv", "D", "Ls"))
    out, lse = s["out"].double(), s["lse"].double()
    ctx = s["ctx_lens"].tolist()
    ql = [Lq] * B if s["q_lens"] is None else s["q_lens"].tolist()
    sys_k, sys_v = s["sys_k"].double(), s["sys_v"].double()

    def values(name, ids, n):
        codes, sz = s[name + "_codes"][ids], s[name + "_sz"][ids].double()
        x = torch.empty(*codes.shape[:-1], D, dtype=torch.float64, device="cuda")
        x[..., 0::2] = codes.bitwise_and(15).double()
        x[..., 1::2] = codes.bitwise_right_shift(4).double()
        per = D // sz.shape[-2]
        x = x * sz[..., 0].repeat_interleave(per, -1) + sz[..., 1].repeat_interleave(per, -1)
        return x.transpose(1, 2).reshape(-1, Hkv, D)[:n]
    for b in range(B):
        n, rows = ctx[b], ql[b]
        ids = s["block_tables"][b, : (n + BLOCK - 1) // BLOCK].long()
        keys = torch.cat([sys_k, values("k", ids, n)])
        vals = torch.cat([sys_v, values("v", ids, n)])
        last = Ls + n - rows + 1 + torch.arange(rows, device="cuda")
        hidden = torch.arange(Ls + n, device="cuda") >= last[:, None]
        for hk in range(Hkv):
            heads = slice(hk * (H // Hkv), (hk + 1) * (H // Hkv))
            x = s["q"][b, :rows, heads].double().transpose(0, 1) @ keys[:, hk].T / D ** 0.5
            x = x.masked_fill(hidden, float("-inf"))
            lse[b, :rows, heads] = torch.logsumexp(x, -1).T
            out[b, :rows, heads] = (torch.softmax(x, -1) @ vals[:, hk]).transpose(0, 1)
    return {"out": out, "lse": lse}


def _exact_rope(s):
    D, Lq = s["D"], s["Lq"]
    axis = np.zeros(D // 2, dtype=np.int64)
    if s["interleaved"]:
        for a in (1, 2):
            axis[a: 3 * s["sections"][a]: 3] = a
    else:
        axis = np.repeat(np.arange(3), s["sections"])
    freq = s["base"] ** (-np.arange(0, D, 2, dtype=np.float64) / D)
    pos = s["positions"].cpu().numpy().astype(np.float64) + s["Ls"]
    ang = np.moveaxis(pos[axis], 0, -1) * freq * (-1.0 if s["inverse"] else 1.0)
    c = torch.from_numpy(np.cos(ang)).cuda()[:, :, None]
    d = torch.from_numpy(np.sin(ang)).cuda()[:, :, None]
    ql = [Lq] * s["B"] if s["q_lens"] is None else s["q_lens"].tolist()
    got = {}
    for key, src in (("q", "q"), ("k", "k_new")):
        x, y = s[src].double().chunk(2, -1)
        full = torch.cat([x * c - y * d, y * c + x * d], -1)
        for b, n in enumerate(ql):
            full[b, n:] = s[key + "_out"][b, n:].double()
        got[key] = full
    return got
