"""The 4-bit context pool on the GPU: the quantising append bit for bit, and
the attention over the pool against its definition in 64 bits.

Tolerance of the attention, per element, from the roundings that the kernels
make: the output is rounded to fp16 (2^-11 of it, or 2^-25), the weights to
fp16 before the product with the values: sum_j d_j w_j x_j / sum_j w_j with
|d_j| <= 2^-11 is at most 2^-11 max |x|, x the fp16 system values or s (c - 8)
of the 4-bit ones (prompt chunks on the tensor cores round the values s c + z
instead, by 2^-11 of them, and keep the weights); weights below fp16's normal numbers are off by 2^-25 of the
common scale at most, which counts only through n keys.  fp32 sums add 2e-5 of
the largest value."""
import ctypes

import numpy as np
import pytest
import torch

import shared_prompt_decode_gb300 as relay
from shared_prompt_decode_gb300 import build

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
GROUPS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


# ----------------------------------------------------------------------------- append
def quantise_ref(x, group):
    """[..., D] fp16 numpy -> codes [..., D] and (s, z) [..., D / group, 2], the definition in fp32."""
    v = x.astype(np.float32).reshape(*x.shape[:-1], -1, group)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], np.float32(0), v)
    lo, hi = v.min(-1), v.max(-1)
    s16 = ((hi - lo) / np.float32(15)).astype(np.float16)
    s = s16.astype(np.float32)
    safe = np.where(s > 0, s, np.float32(1))
    c = np.where((s > 0)[..., None], np.minimum(np.rint((v - lo[..., None]) / safe[..., None]), 15), 0).astype(np.uint8)
    sz = np.stack([s16, lo.astype(np.float16)], -1)
    sz[bad] = np.nan
    return c.reshape(x.shape), sz


def pack(c):
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def append_case(B, Lq, Hkv, D, group, seed):
    r = np.random.default_rng(seed)
    max_blocks = -(-(Lq + 40) // 16)
    n = r.integers(Lq, 16 * max_blocks + 1, B)
    q = r.integers(0, Lq + 1, B)
    if B > 1:
        q[0], q[-1] = Lq, min(1, Lq)
    num = B * max_blocks + 3
    table = r.permutation(num)[:B * max_blocks].reshape(B, max_blocks)
    k, v = (r.standard_normal((B, Lq, Hkv, D)).astype(np.float16) for _ in range(2))
    return n, q, num, table, k, v


def filled_pool(num, Hkv, D, group, seed=0):
    g = torch.Generator().manual_seed(seed)
    codes = lambda: torch.randint(0, 256, (num, Hkv, 16, D // 2), generator=g, dtype=torch.uint8).to(DEV)
    sz = lambda: torch.randn(num, Hkv, 16, D // group, 2, generator=g).half().to(DEV)
    return relay.Q4Cache(codes(), sz(), codes(), sz())


def same_bits(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def expect_append(cache, n, q, table, k, v, group):
    want = [t.cpu().numpy().copy() for t in (cache.k_codes, cache.k_sz, cache.v_codes, cache.v_sz)]
    for b in range(len(n)):
        for i in range(q[b]):
            pos = n[b] - q[b] + i
            for at, x in ((0, k), (2, v)):
                c, sz = quantise_ref(x[b, i], group)
                want[at][table[b, pos // 16], :, pos % 16] = pack(c)
                want[at + 1][table[b, pos // 16], :, pos % 16] = sz
    return want


def check_pool(cache, want):
    for t, w in zip((cache.k_codes, cache.k_sz, cache.v_codes, cache.v_sz), want):
        got = t.cpu().numpy()
        assert np.array_equal(got, w, equal_nan=got.dtype == np.float16)


@pytest.mark.parametrize("D,group", GROUPS)
@pytest.mark.parametrize("B,Lq,Hkv", [(1, 1, 1), (3, 1, 8), (2, 33, 5), (40, 4, 2)])
def test_append(D, group, B, Lq, Hkv):
    n, q, num, table, k, v = append_case(B, Lq, Hkv, D, group, B * D + group)
    cache = filled_pool(num, Hkv, D, group)
    want = expect_append(cache, n, q, table, k, v, group)
    w = relay.relay_kv_append_q4(torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV), i32(table), i32(n), cache, i32(q))
    assert relay.device_status(w) == 0
    check_pool(cache, want)
    # the same rows through a slot map
    slots = np.full((B, Lq), -1)
    for b in range(B):
        for i in range(q[b]):
            pos = n[b] - q[b] + i
            slots[b, i] = table[b, pos // 16] * 16 + pos % 16
    for ql in (None, i32(q)):
        c2 = filled_pool(num, Hkv, D, group)
        w = relay.relay_kv_append_q4(torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV), None, None, c2, ql,
                                     slot_map=i32(slots))
        assert relay.device_status(w) == 0
        check_pool(c2, want)


@pytest.mark.parametrize("D,group", [(64, 32), (128, 128)])
def test_append_values(D, group):
    """Constant groups, ranges that overflow or underflow the scale, ties, signed zeros, NaN and infinities."""
    rows = np.random.default_rng(5).standard_normal((12, 1, 1, D)).astype(np.float16)
    rows[0] = 1.5
    rows[1] = 0
    rows[1, ..., 1::2] = -0.0
    rows[2, ..., 0], rows[2, ..., 1] = 65504, -65504
    rows[3] = 0
    rows[3, ..., 3] = 6e-8                         # the smallest subnormal: the scale rounds to zero
    rows[4] *= np.float16(6e-5)                    # subnormal values
    rows[5] = (np.arange(D) % 31 / 2).astype(np.float16)      # s = 1: ties at every half
    rows[6, ..., 5] = np.nan
    rows[7, ..., D - 1] = np.inf
    rows[8, ..., 0] = -np.inf
    rows[9] = np.float16(1000) + rows[9]           # far from zero
    rows[10] = (np.arange(D) % 16).astype(np.float16)         # codes 0..15 themselves
    B = len(rows)
    n, q, table = np.full(B, 16), np.ones(B, int), np.arange(B)[:, None]
    cache = filled_pool(B, 1, D, group)
    want = expect_append(cache, n, q, table, rows, -rows, group)
    relay.relay_kv_append_q4(torch.from_numpy(rows).to(DEV), torch.from_numpy(-rows).to(DEV), i32(table), i32(n), cache)
    check_pool(cache, want)


def test_append_flags():
    D, group, B, Lq = 128, 64, 5, 3
    n, q, num, table, k, v = append_case(B, Lq, 2, D, group, 1)
    q[:] = (3, 4, 2, 1, 3)
    n[:] = (20, 20, 1, 20, 10 ** 6)
    table[3, 1] = num
    cache, before = filled_pool(num, 2, D, group), filled_pool(num, 2, D, group)
    ok = q.copy()
    ok[1:] = 0
    want = expect_append(before, n, ok, table, k, v, group)
    w = relay.relay_kv_append_q4(torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV), i32(table), i32(n), cache, i32(q))
    assert relay.device_status(w) == relay.FLAG_BAD_Q_LEN | relay.FLAG_BAD_CTX_LEN | relay.FLAG_BAD_BLOCK
    check_pool(cache, want)
    slots = np.full((B, Lq), 16 * num)
    w = relay.relay_kv_append_q4(torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV), None, None, cache,
                                 slot_map=i32(slots))
    assert relay.device_status(w) == relay.FLAG_BAD_BLOCK
    check_pool(cache, want)


# ----------------------------------------------------------------------------- attention
class Case:
    """A batch over a 4-bit pool: quantised normal keys and values, NaN scales in every slot that no request holds."""

    def __init__(self, ctx, q_lens, H, Hkv, D, group, Ls, seed=0, vscale=1.0, spare=3):
        r = np.random.default_rng(seed)
        self.ctx, self.H, self.Hkv, self.D, self.group, self.Ls = list(ctx), H, Hkv, D, group, Ls
        self.B, self.Lq = len(ctx), max(list(q_lens) + [1])
        self.q_lens = list(q_lens)
        self.max_blocks = max(1, max(-(-n // 16) for n in ctx) + 1)
        need = [-(-n // 16) for n in ctx]
        self.num = sum(need) + spare
        ids = r.permutation(self.num)
        self.table = np.full((self.B, self.max_blocks), -1)
        k = 0
        for b, m in enumerate(need):
            self.table[b, :m] = ids[k:k + m]
            k += m
        self.q = r.standard_normal((self.B, self.Lq, H, D)).astype(np.float16)
        self.sys_k = r.standard_normal((Ls, Hkv, D)).astype(np.float16)
        self.sys_v = (vscale * r.standard_normal((Ls, Hkv, D))).astype(np.float16)
        self.codes, self.sz = {}, {}
        for name, scale in (("k", 1.0), ("v", vscale)):
            x = (scale * (r.standard_normal((self.num, Hkv, 16, D)) + 0.3 * r.standard_normal((1, Hkv, 1, D)))).astype(np.float16)
            c, sz = quantise_ref(x, group)
            held = np.zeros((self.num, 16), bool)
            for b, n in enumerate(ctx):
                for t in range(n):
                    held[self.table[b, t // 16], t % 16] = True
            sz = np.where(held[:, None, :, None, None], sz, np.float16(np.nan))
            self.codes[name], self.sz[name] = c, sz

    def pool(self):
        f = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
        return relay.Q4Cache(f(pack(self.codes["k"])), f(self.sz["k"]), f(pack(self.codes["v"])), f(self.sz["v"]))

    def values(self, name, b, n):
        ids = self.table[b, :-(-n // 16)]
        s = np.repeat(self.sz[name][ids].astype(np.float64), self.group, axis=3)
        x = self.codes[name][ids] * s[..., 0] + s[..., 1]
        return x.transpose(0, 2, 1, 3).reshape(-1, self.Hkv, self.D)[:n]

    def reference(self, part="full"):
        """Output, log-sum-exp and the element tolerances, in fp64."""
        G = self.H // self.Hkv
        out = np.zeros((self.B, self.Lq, self.H, self.D))
        lse = np.full((self.B, self.Lq, self.H), -np.inf)
        tol, ltol = np.zeros_like(out), np.zeros_like(lse)
        for b in range(self.B):
            n, rows = self.ctx[b], self.q_lens[b]
            kc, vc = self.values("k", b, n), self.values("v", b, n)
            for i in range(rows):
                seen = max(0, min(n, n - rows + 1 + i))
                keys, vals = kc[:seen], vc[:seen]
                if part == "full":
                    keys = np.concatenate([self.sys_k.astype(np.float64), keys])
                    vals = np.concatenate([self.sys_v.astype(np.float64), vals])
                if len(keys) == 0:
                    continue
                for h in range(self.H):
                    k = keys[:, h // G]
                    q = self.q[b, i, h].astype(np.float64)
                    x = k @ q / np.sqrt(self.D)
                    m = x.max()
                    p = np.exp(x - m)
                    out[b, i, h] = p @ vals[:, h // G] / p.sum()
                    lse[b, i, h] = m + np.log(p.sum())
                    ids = self.table[b, :-(-seen // 16)]
                    top = 0.0 if seen == 0 else 8 * np.nanmax(self.sz["v"][ids, h // G, :, :, 0].astype(np.float64))
                    big = max(top, np.abs(vals[:, h // G]).max())
                    o = out[b, i, h]
                    tol[b, i, h] = 2.0 ** -11 * np.abs(o) + 2.0 ** -25 + (2.0 ** -11 + 2.0 ** -25 * len(keys) + 2e-5) * big
                    # the scores' fp32 sums: D terms of |q||k|, and the parts s q.c and z sum(q) of the same size
                    ltol[b, i, h] = 2e-6 + 2.0 ** -22 * (np.abs(k) @ np.abs(q)).max() * 4 / np.sqrt(self.D)
        return out, lse, tol, ltol


def run(c, part="full", **kw):
    f = lambda a: torch.from_numpy(a).to(DEV)
    ql = None if all(x == c.Lq for x in c.q_lens) else i32(c.q_lens)
    mq = 0 if ql is None else max(1, sum(c.q_lens))
    pool = kw.pop("pool", None) or c.pool()
    dims = relay.make_dims(f(c.q), c.Ls if part == "full" else 0, c.num, c.max_blocks, max_q_total=mq, Hkv=c.Hkv,
                           ctx_split=kw.pop("ctx_split", 0), sys_range=kw.pop("sys_range", 0))
    w = relay.make_workspace_q4(dims)
    lse = torch.full((c.B, c.Lq, c.H), 7.0, device=DEV)
    if part == "full":
        out = torch.full(c.q.shape, 7.0, dtype=torch.float16, device=DEV)
        for _ in range(2):      # the second call finds the workspace as the first one left it
            relay.relay_attention_decode_q4(f(c.q), f(c.sys_k), f(c.sys_v), pool, i32(c.table), i32(c.ctx), ql, out=out,
                                            lse_out=lse, workspace=w, dims=dims)
    else:
        out = torch.full(c.q.shape, 7.0, device=DEV)
        relay.relay_ctx_attn_q4(f(c.q), pool, i32(c.table), i32(c.ctx), ql, o_ctx=out, lse_ctx=lse, workspace=w, dims=dims)
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), relay.device_status(w)


def within(got, want, tol, what):
    err = np.abs(got - want)
    ok = bool((err <= tol).all())      # (a NaN is not)
    assert ok, f"{what}: off by {np.nanmax(err):.3e}, {np.nanmax(err - tol):.3e} more than allowed"


def check(c, got, part="full"):
    out, lse, flags = got
    assert flags == 0
    ref, ref_lse, tol, ltol = c.reference(part)
    for b in range(c.B):
        r = c.q_lens[b]
        within(out[b, :r], ref[b, :r], tol[b, :r], f"out of request {b}")
        empty = np.isinf(ref_lse[b, :r])
        assert np.array_equal(lse[b, :r][empty], ref_lse[b, :r][empty])
        within(lse[b, :r][~empty], ref_lse[b, :r][~empty], ltol[b, :r][~empty], f"lse of request {b}")
        assert (out[b, r:] == 7.0).all() and (lse[b, r:] == 7.0).all()      # rows behind the last one


LENS = [0, 1, 15, 16, 17, 33, 100, 255, 600]


@pytest.mark.parametrize("D,group", GROUPS)
@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2), (12, 1), (16, 2)])
def test_decode(D, group, H, Hkv):
    c = Case(LENS, [1] * len(LENS), H, Hkv, D, group, 70, seed=D + group + H)
    check(c, run(c))


@pytest.mark.parametrize("D,group", GROUPS)
@pytest.mark.parametrize("H,Hkv,rows", [(4, 4, (3, 1, 0, 20, 2, 1, 7)), (10, 2, (1, 2, 5, 3, 40, 0, 1)), (5, 1, (1, 1, 90, 1, 4, 2, 70))])
def test_several_rows(D, group, H, Hkv, rows):
    """Requests of many rows beside decode requests and requests of none; one has more rows than tokens, and its first
    rows see the prompt alone."""
    c = Case([40, 17, 64, 9, 300, 5, 129], rows, H, Hkv, D, group, 33, seed=group + H)
    check(c, run(c))


@pytest.mark.parametrize("Ls", [0, 1, 64, 300])
def test_prompt_lengths_and_empty_rows(Ls):
    c = Case([0, 3, 0, 50], [1] * 4, 8, 2, 128, 128, Ls, seed=Ls)
    check(c, run(c))
    c = Case([2, 40, 0], [5, 5, 5], 4, 4, 64, 32, Ls, seed=Ls + 1)
    check(c, run(c))


@pytest.mark.parametrize("part", ["full", "ctx"])
@pytest.mark.parametrize("ctx_split", [64, 128, 1024])
def test_forced_splits(part, ctx_split):
    c = Case([1, 63, 64, 65, 700, 300], [1, 3, 1, 2, 1, 40], 6, 3, 128, 64, 40, seed=ctx_split)
    got = run(c, part, ctx_split=ctx_split)
    if part == "full":
        check(c, got)
    else:
        check(c, got, part)


def test_long_contexts_of_one_request():
    c = Case([9001], [1], 8, 2, 128, 128, 0, seed=3)
    check(c, run(c))
    c = Case([5000], [3], 4, 4, 64, 64, 17, seed=4)
    check(c, run(c))


@pytest.mark.parametrize("D,group,G", [(128, 128, 1), (128, 64, 8), (128, 32, 4), (64, 32, 2)])
def test_long_shares(D, group, G):
    """So many keys that a warp goes through far more pages of one head than in the other tests: the sums' last bits.  The
    reference is formed on the device, in 64 bits."""
    torch.manual_seed(41)
    B, Hkv, n = 4, 16, 24000
    blocks = n // 16
    codes = [torch.randint(0, 256, (B * blocks, Hkv, 16, D // 2), dtype=torch.uint8, device=DEV) for _ in "kv"]
    sz = [torch.stack([0.2 + 0.05 * torch.rand(B * blocks, Hkv, 16, D // group, device=DEV),
                       -1.7 + 0.1 * torch.randn(B * blocks, Hkv, 16, D // group, device=DEV)], -1).half() for _ in "kv"]
    pool = relay.Q4Cache(codes[0], sz[0], codes[1], sz[1])
    table = torch.randperm(B * blocks, device=DEV).int().view(B, blocks)
    q = torch.randn(B, 1, Hkv * G, D, device=DEV).half()
    out, lse = relay.relay_ctx_attn_q4(q, pool, table, i32([n] * B))
    for b in range(B):
        for h in range(0, Hkv, 5):
            x = []
            for c, s in zip(codes, sz):
                ids = table[b].long()
                w = torch.stack([c[ids, h] & 15, c[ids, h] >> 4], -1).flatten(-2).double().unflatten(-1, (-1, group))
                x.append((w * s[ids, h, :, :, :1].double() + s[ids, h, :, :, 1:].double()).flatten(-2).flatten(0, 1))
            p = q[b, 0, h * G:(h + 1) * G].double() @ x[0].T / D ** 0.5
            ref = torch.softmax(p, -1) @ x[1]
            got = out[b, 0, h * G:(h + 1) * G].double()
            # weights rounded by 2^-11 at random, sqrt(sum w^2) of them: their error, and that of n fp32 sums as large
            # as the values (5 sigma of D G elements' rms)
            w2 = torch.softmax(p, -1).square().sum(-1, keepdim=True).sqrt()
            rms = float(((got - ref) / (2.0 ** -11 * w2 * x[1].square().mean().sqrt())).square().mean().sqrt())
            assert rms < 1.0, f"request {b}, head {h}: {rms:.2f} of the weights' rounding"
            assert torch.allclose(lse[b, 0, h * G:(h + 1) * G].double(), torch.logsumexp(p, -1), atol=2e-5)


@pytest.mark.parametrize("D,group", [(128, 32), (128, 128), (64, 64)])
@pytest.mark.parametrize("ctx,q_lens,H,Hkv", [
    ([10, 300, 0], [40, 1, 64], 4, 4),              # rows that see no key; a chunk without a context
    ([100, 700, 0, 1], [1, 1, 1, 1], 64, 1),        # single rows of 64 heads a group
    ([500, 130, 64], [60, 0, 33], 10, 2),           # tiles that end inside a row's heads; no rows at all
    ([63, 64, 65, 128, 129], [63, 64, 65, 33, 34], 2, 2),
    ([40] * 40, [40] * 40, 1, 1),                   # more requests than columns of one
    ([2000], [1], 200, 1),
])
def test_prompt_chunk_edges(ctx, q_lens, H, Hkv, D, group):
    c = Case(ctx, q_lens, H, Hkv, D, group, 17, seed=50)
    check(c, run(c))
    check(c, run(c, "ctx"), "ctx")


def test_two_graphs_of_prompt_chunks_share_a_workspace():
    """Captured one after the other over one workspace and replayed in turn, with lengths changed in between."""
    cs = [Case([300, 50], [64, 1], 4, 2, 128, 64, 33, seed=51), Case([80, 400], [1, 64], 4, 2, 128, 64, 33, seed=52)]
    f = lambda a: torch.from_numpy(a).to(DEV)
    blocks, num = max(c.max_blocks for c in cs), max(c.num for c in cs)
    for c in cs:
        c.table = np.pad(c.table, ((0, 0), (0, blocks - c.max_blocks)), constant_values=-1)
        c.max_blocks = blocks
    dims = [relay.make_dims(f(c.q), c.Ls, c.num, blocks, max_q_total=80, Hkv=c.Hkv) for c in cs]
    w = relay.make_workspace_q4(dims[0])
    ins = [(f(c.q), f(c.sys_k), f(c.sys_v), c.pool(), i32(c.table), i32(c.ctx), i32(c.q_lens)) for c in cs]
    outs = [torch.full(c.q.shape, 7.0, dtype=torch.float16, device=DEV) for c in cs]
    graphs = []
    s = torch.cuda.Stream()
    for d, x, o in zip(dims, ins, outs):
        with torch.cuda.stream(s):
            relay.relay_attention_decode_q4(*x, out=o, workspace=w, dims=d)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            relay.relay_attention_decode_q4(*x, out=o, workspace=w, dims=d)
        graphs.append(g)
    for turn in range(3):
        if turn == 2:      # the chunks one row shorter
            for c, x in zip(cs, ins):
                c.q_lens = [max(1, n - 1) for n in c.q_lens]
                x[6].copy_(i32(c.q_lens))
        for c, g, o in zip(cs, graphs, outs):
            o.fill_(7.0)
            g.replay()
        for c, o in zip(cs, outs):
            ref, _, tol, _ = c.reference()
            for b, n in enumerate(c.q_lens):
                within(o[b, :n].double().cpu().numpy(), ref[b, :n], tol[b, :n], f"turn {turn}, request {b}")
                assert (o[b, n:] == 7.0).all()
    assert relay.device_status(w) == 0


@pytest.mark.parametrize("scale", [0.01, 0.6])
@pytest.mark.parametrize("rows", [1, 5, 40])
def test_given_scale(scale, rows):
    c = Case([200, 90], [rows, 1], 4, 2, 128, 64, 30, seed=60)
    f = lambda a: torch.from_numpy(a).to(DEV)
    out, lse = relay.relay_ctx_attn_q4(f(c.q), c.pool(), i32(c.table), i32(c.ctx), i32(c.q_lens), scale=scale)
    c.q = c.q.astype(np.float64) * (scale * np.sqrt(128))      # (the reference takes 1 / sqrt(D))
    ref, ref_lse, tol, ltol = c.reference("ctx")
    for b, n in enumerate(c.q_lens):
        within(out[b, :n].double().cpu().numpy(), ref[b, :n], tol[b, :n], f"out of request {b}")
        seen = ~np.isinf(ref_lse[b, :n])
        within(lse[b, :n].double().cpu().numpy()[seen], ref_lse[b, :n][seen], ltol[b, :n][seen], f"lse of request {b}")


def test_prompt_chunks_with_room_for_more():
    """Contexts far shorter than the block tables allow: their splits follow the contexts."""
    c = Case([1500, 20, 900], [130, 1, 40], 2, 1, 128, 128, 10, seed=7)
    c.max_blocks = 3000
    c.table = np.pad(c.table, ((0, 0), (0, 3000 - c.table.shape[1])), constant_values=-1)
    check(c, run(c))


def test_prompt_chunks_over_long_contexts():
    """Prompt chunks whose contexts go to several splits, of a length that is no multiple of the kernel's stage."""
    c = Case([4400, 700, 2100], [40, 1, 140], 2, 2, 128, 128, 20, seed=5)
    check(c, run(c))
    c = Case([2500, 4337], [50, 33], 6, 3, 64, 32, 0, seed=6)
    check(c, run(c, "ctx"), "ctx")


@pytest.mark.parametrize("D,group", [(128, 128), (128, 32), (64, 64), (64, 32)])
@pytest.mark.parametrize("what", ["s", "z"])
@pytest.mark.parametrize("rows", [1, 5, 12, 40])
def test_large_keys(D, group, what, rows):
    """Keys of one group that are 2^10 times the others, against queries 2^-10 of the usual: their products with a scale
    leave fp16's range as the tiles would hold them.  Two neighbouring keys of a page, and a page."""
    c = Case([130, 90], [rows, 1], 4, 2, D, group, 30, seed=30)
    c.q = (c.q.astype(np.float32) * 2.0 ** -10).astype(np.float16)
    for blk, t in ((c.table[0, 2], slice(5, 7)), (c.table[0, 5], slice(0, 16)), (c.table[1, 1], slice(15, 16))):
        x = c.sz["k"][blk, :, t, -1, 0 if what == "s" else 1]
        c.sz["k"][blk, :, t, -1, 0 if what == "s" else 1] = x.astype(np.float32) * 2.0 ** 10
    check(c, run(c))


@pytest.mark.parametrize("D,group", [(128, 128), (128, 64), (64, 32)])
def test_prompt_chunks_over_values_behind_fp16(D, group):
    """Values s * 15 + z of up to 95,000, of some keys and of one of their groups: fp32 results."""
    c = Case([150, 90], [48, 1], 2, 2, D, group, 0, seed=31)
    for t in (3, 64, 65, 149):
        c.sz["v"][c.table[0, t // 16], :, t % 16, 0] = [6000.0, 5000.0]
        c.sz["v"][c.table[0, t // 16], :, t % 16, -1, 1] = -60000.0
    check(c, run(c, "ctx"), "ctx")


@pytest.mark.parametrize("D,group", [(128, 128), (128, 32), (64, 32)])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_one_group_of_a_seen_value_is_no_number(D, group, bad):
    """The group's dimensions are NaN in the rows that see the key; its other dimensions, and the rows before, are what
    they were."""
    c = Case([100], [40], 2, 2, D, group, 20, seed=32)
    t = 80      # seen by rows 20 and up
    clean = c.reference()
    at = D // group - 1
    c.sz["v"][c.table[0, t // 16], 1, t % 16, at, 1] = bad
    out, lse, flags = run(c)
    assert flags == 0
    hit = np.zeros(out.shape, bool)
    hit[0, 20:, 1, at * group:] = True
    assert np.isnan(out[hit]).all()
    keep = ~hit
    within(out[keep], clean[0][keep], clean[2][keep], "out")
    within(lse, clean[1], clean[3], "lse")


def test_many_requests():
    r = np.random.default_rng(8)
    c = Case(list(r.integers(0, 60, 512)), [1] * 512, 2, 1, 64, 32, 40, seed=9)
    check(c, run(c))


def test_large_batch_takes_the_tensor_cores():
    """More than 256 rows per KV head: the prompt's part runs on the tensor-core kernel in front."""
    r = np.random.default_rng(10)
    c = Case(list(r.integers(1, 50, 70)), [1] * 70, 8, 2, 128, 64, 300, seed=11)
    check(c, run(c))


@pytest.mark.parametrize("vscale", [2.0 ** -12, 2.0 ** 12])
@pytest.mark.parametrize("D,group", [(128, 128), (64, 32)])
def test_value_scales(vscale, D, group):
    """Values far from 1: the weights' common power of two keeps them in fp16's normal range.  A key in the middle
    whose values are 2^8 larger moves the power while the item runs."""
    c = Case([200, 90], [1, 1], 4, 2, D, group, 0, seed=12, vscale=vscale)
    blk = c.table[0, 6]
    c.sz["v"][blk] = (c.sz["v"][blk].astype(np.float32) * min(256.0, 2.0 ** 15 / vscale / 8)).astype(np.float16)
    check(c, run(c))


def test_hidden_keys_may_be_nan():
    """A request of several rows whose last tokens are NaN: the rows before them are not touched by it."""
    c = Case([50, 30], [20, 1], 6, 2, 128, 64, 21, seed=13)
    clean = c.reference()
    for t in (45, 46, 47, 48, 49):
        blk = c.table[0, t // 16]
        c.sz["k"][blk, :, t % 16] = np.nan
        c.sz["v"][blk, :, t % 16] = np.nan
    out, lse, flags = run(c)
    assert flags == 0
    for b, r in ((0, 15), (1, 1)):
        within(out[b, :r], clean[0][b, :r], clean[2][b, :r], "out")
        within(lse[b, :r], clean[1][b, :r], clean[3][b, :r], "lse")


def test_device_checks():
    c = Case([40, 20], [1, 1], 4, 2, 128, 128, 16, seed=14)
    c.table[0, 1] = c.num
    assert run(c)[2] == relay.FLAG_BAD_BLOCK
    c = Case([40, 20], [1, 1], 4, 2, 128, 128, 16, seed=14)
    c.ctx[1] = 16 * c.max_blocks + 1
    out, lse, flags = run(c)
    assert flags == relay.FLAG_BAD_CTX_LEN and (out == 7.0).all()
    c = Case([40, 20], [2, 1], 4, 2, 128, 128, 16, seed=14)
    c.q_lens[1] = 3
    out, lse, flags = run(c)
    assert flags & relay.FLAG_BAD_Q_LEN and (out == 7.0).all()


# ----------------------------------------------------------------------------- the step as it is used
@pytest.mark.parametrize("D,group,H,Hkv", [(128, 128, 8, 2), (64, 32, 4, 4)])
def test_serving_loop(D, group, H, Hkv):
    """Admission, decode steps, a request that ends and one that takes its place: blocks planned on the device, rows
    turned, quantised and attended to; every step's output against fp64 over what the pool holds, decode steps from one
    captured graph."""
    r = np.random.default_rng(20)
    B, Ls, num, max_blocks, Lq = 4, 50, 30, 8, 40
    sections = (D // 2 - 2 * (D // 8), D // 8, D // 8)
    cache = relay.make_q4_cache(num, Hkv, D, group)
    sysk, sysv = (torch.randn(Ls, Hkv, D, device=DEV).half() for _ in range(2))
    free = i32(r.permutation(num))
    n_free, table = i32([num]), torch.full((B, max_blocks), -1, dtype=torch.int32, device=DEV)
    ctx, ws = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(256, dtype=torch.uint8, device=DEV)
    values = {}

    def buffers(L):
        f = lambda h, t=torch.float16: torch.empty(B, L, h, D, dtype=t, device=DEV)
        dims = relay.make_dims(f(H), Ls, num, max_blocks, max_q_total=B * L, Hkv=Hkv)
        return dict(q=f(H), k=f(Hkv), v=f(Hkv), out=f(H), pos=torch.empty(3, B, L, dtype=torch.int32, device=DEV),
                    ql=torch.empty(B, dtype=torch.int32, device=DEV), dims=dims, ws=relay.make_workspace_q4(dims),
                    slots=torch.empty(B, L, dtype=torch.int32, device=DEV))

    def step(s):
        ctx.add_(s["ql"])
        relay.relay_block_plan(ctx, table, free, n_free, q_lens=s["ql"], Lq=s["q"].shape[1], slot_map=s["slots"], workspace=ws)
        relay.relay_rope_axes(s["q"], s["pos"], Ls, sections, k_new=s["k"], q_lens=s["ql"], workspace=ws)
        relay.relay_kv_append_q4(s["k"], s["v"], None, None, cache, s["ql"], slot_map=s["slots"], workspace=ws)
        relay.relay_attention_decode_q4(s["q"], sysk, sysv, cache, table, ctx, s["ql"], out=s["out"], workspace=s["ws"],
                                        dims=s["dims"])

    def fill(s, ql):
        for name in ("q", "k", "v"):
            s[name].copy_(torch.from_numpy(r.standard_normal(tuple(s[name].shape)).astype(np.float16)))
        s["pos"].copy_(torch.from_numpy(r.integers(0, 500, tuple(s["pos"].shape))))
        s["ql"].copy_(torch.tensor(ql, dtype=torch.int32))
        s["out"].fill_(7.0)

    def verify(s, ql, ctx_before):
        torch.cuda.synchronize()
        assert relay.device_status(ws) == 0 and relay.device_status(s["ws"]) == 0
        L = s["q"].shape[1]
        lens = [a + b for a, b in zip(ctx_before, ql)]
        assert ctx.tolist() == lens
        t = table.cpu().numpy()
        held = [int(x) for b in range(B) for x in t[b, :-(-lens[b] // 16)]]
        rest = free.cpu().tolist()[:int(n_free)]
        assert sorted(held + rest) == list(range(num))      # no block lost, none twice
        c = Case([max(n, 1) for n in lens], ql, H, Hkv, D, group, Ls)
        c.ctx, c.Lq, c.table = lens, L, t
        c.q = s["q"].cpu().numpy()
        c.sys_k, c.sys_v = sysk.cpu().numpy(), sysv.cpu().numpy()
        unpack = lambda x: np.stack([x & 15, x >> 4], -1).reshape(*x.shape[:-1], -1)
        c.codes = {"k": unpack(cache.k_codes.cpu().numpy()), "v": unpack(cache.v_codes.cpu().numpy())}
        c.sz = {"k": cache.k_sz.cpu().numpy(), "v": cache.v_sz.cpu().numpy()}
        ref, _, tol, _ = c.reference()
        out = s["out"].double().cpu().numpy()
        for b in range(B):
            within(out[b, :ql[b]], ref[b, :ql[b]], tol[b, :ql[b]], f"out of request {b}")
            assert (out[b, ql[b]:] == 7.0).all()
            # what was appended stands for the rows within half a step, the scale's rounding and the clamp
            for i in range(ql[b]):
                pos = lens[b] - ql[b] + i
                for name in ("k", "v"):
                    sz = c.sz[name][t[b, pos // 16], :, pos % 16].astype(np.float64)
                    sz = np.repeat(sz, group, axis=1)
                    x = c.codes[name][t[b, pos // 16], :, pos % 16] * sz[..., 0] + sz[..., 1]
                    got = s[name][b, i].double().cpu().numpy()
                    within(x, got, sz[..., 0] * (0.5 + 15 * 2.0 ** -11 + 1e-5), "stored row")

    chunk, one = buffers(Lq), buffers(1)
    ql, before = [40, 17, 0, 1], [0] * B
    fill(chunk, ql)
    step(chunk)
    verify(chunk, ql, before)
    # decode steps, the first one eager, the others one graph
    graph = None
    for k in range(4):
        before, ql = ctx.tolist(), [1, 1, 0, 1]
        fill(one, ql)
        if k == 0:
            step(one)
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step(one)
                # capture ran nothing
                assert ctx.tolist() == before
            graph.replay()
        verify(one, ql, before)
    # request 0 ends, its row is given to a new prompt
    done = i32([1, 0, 0, 0])
    n0 = int(n_free)
    relay.relay_block_release(done, ctx, table, free, n_free, workspace=ws)
    assert int(n_free) == n0 + 3
    ctx[0] = 0
    before, ql = ctx.tolist(), [33, 1, 20, 5]
    fill(chunk, ql)
    step(chunk)
    verify(chunk, ql, before)


def test_wait_that_gives_up_is_reported():
    """Prompt chunks run on a pipeline whose waits are bounded in time.  In a build whose limit is zero the first wait that
    is not met at once gives up: the call ends, reports it, and leaves the context and the workspace usable."""
    path = build.build(variant="wait0", defines=["RELAY_WAIT_LIMIT_NS=0ull"])
    short = ctypes.CDLL(path).relay_ctx_attn_q4
    full = relay.lib().relay_ctx_attn_q4
    short.restype, short.argtypes = full.restype, full.argtypes
    c = Case([900, 700, 350], [128, 1, 60], 4, 4, 128, 64, 0, seed=40)
    q, pool, table, ctx, ql = torch.from_numpy(c.q).to(DEV), c.pool(), i32(c.table), i32(c.ctx), i32(c.q_lens)
    dims = relay.make_dims(q, 0, c.num, c.max_blocks, max_q_total=sum(c.q_lens), Hkv=c.Hkv)
    w = relay.make_workspace_q4(dims)
    out, lse = torch.zeros(c.q.shape, device=DEV), torch.zeros(c.q.shape[:3], device=DEV)
    seen = 0
    for _ in range(3):
        rc = short(ctypes.byref(dims), q.data_ptr(), ctypes.byref(pool._struct), table.data_ptr(), ctx.data_ptr(), ql.data_ptr(),
                   out.data_ptr(), lse.data_ptr(), w.data_ptr(), w.numel(), torch.cuda.current_stream().cuda_stream)
        assert rc == relay.OK
        torch.cuda.synchronize()
        seen |= relay.device_status(w)
    assert seen == relay.FLAG_WAIT_TIMEOUT
    out, lse = relay.relay_ctx_attn_q4(q, pool, table, ctx, ql, workspace=w, dims=dims)
    ref, ref_lse, tol, ltol = c.reference("ctx")
    for b, r in enumerate(c.q_lens):
        within(out[b, :r].double().cpu().numpy(), ref[b, :r], tol[b, :r], f"out of request {b}")
