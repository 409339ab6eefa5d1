"""The steps around the cache on the GPU: block tables and slot maps from the
request lengths, the return of blocks, rotary positions with several axes.
Whole numbers are compared exactly with a loop over requests; rotations with
fp64 under one rounding to fp16 plus the fp32 arithmetic."""
import numpy as np
import pytest
import torch

import shared_prompt_decode_gb300 as relay

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from shared_prompt_decode_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype).to(DEV)


def ws():
    return torch.zeros(256, dtype=torch.uint8, device=DEV)


# ----------------------------------------------------------------------------- block plan
def plan_ref(n, q, Lq, table, free, nf, num_blocks):
    """The definition, a request at a time."""
    table, slots = table.copy(), np.full((len(n), Lq), -1, dtype=np.int64)
    flags, base, left = 0, 0, nf
    if not 0 <= nf <= num_blocks:
        flags, nf, left = relay.FLAG_POOL, 0, 0
    for b in range(len(n)):
        if not 0 <= q[b] <= Lq:
            flags |= relay.FLAG_BAD_Q_LEN
            continue
        if not q[b] <= n[b] <= 16 * table.shape[1]:
            flags |= relay.FLAG_BAD_CTX_LEN
            continue
        held = -(-(n[b] - q[b]) // 16)
        need = -(-n[b] // 16) - held
        if need and base + need > nf:
            flags |= relay.FLAG_POOL
            base += need
            continue
        for j in range(need):
            table[b, held + j] = free[nf - 1 - (base + j)]
        base += need
        left -= need
        for i in range(q[b]):
            pos = n[b] - q[b] + i
            blk = table[b, pos // 16]
            if 0 <= blk < num_blocks:
                slots[b, i] = blk * 16 + pos % 16
            else:
                flags |= relay.FLAG_BAD_BLOCK
    return table, slots, left, flags


def plan_case(B, Lq, max_blocks, seed, free_blocks=None, ragged=True):
    r = np.random.default_rng(seed)
    n = r.integers(0, 16 * max_blocks + 1, B)
    q = np.minimum(r.integers(0, Lq + 1, B) if ragged else np.full(B, Lq), n)
    held = -(-(n - q) // 16)
    num_blocks = int((-(-n // 16)).sum()) + 5
    ids = r.permutation(num_blocks)
    table = np.full((B, max_blocks), -7)
    k = 0
    for b in range(B):
        table[b, :held[b]] = ids[k:k + held[b]]
        k += held[b]
    free = np.full(num_blocks, -9)
    nf = num_blocks - k if free_blocks is None else free_blocks
    free[:num_blocks - k] = ids[k:]
    return n, q, table, free, nf, num_blocks


def run_plan(n, q, Lq, table, free, nf, in_place=False, q_lens=True):
    t, f, c, w = dev(table), dev(free), dev([nf]), ws()
    out = c if in_place else dev([-1])
    slots = relay.relay_block_plan(dev(n), t, f, c, q_lens=dev(q) if q_lens else None, Lq=Lq, n_free_out=None if in_place else out,
                                   workspace=w)
    assert np.array_equal(f.cpu().numpy(), free)
    return t.cpu().numpy(), slots.cpu().numpy(), int(out), relay.device_status(w)


@pytest.mark.parametrize("B,Lq,max_blocks", [(1, 1, 1), (1, 17, 3), (3, 40, 5), (31, 1, 9), (33, 5, 4), (512, 1, 17),
                                             (512, 300, 40), (200, 1000, 63)])
@pytest.mark.parametrize("in_place", [False, True])
def test_block_plan(B, Lq, max_blocks, in_place):
    n, q, table, free, nf, num = plan_case(B, Lq, max_blocks, B + Lq)
    want = plan_ref(n, q, Lq, table, free, nf, num)
    got = run_plan(n, q, Lq, table, free, nf, in_place)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert got[2:] == want[2:] and want[3] == 0


@pytest.mark.parametrize("nf", [0, 1, 7, 40, -3, 10 ** 6])
def test_block_plan_short_or_broken_list(nf):
    n, q, table, free, _, num = plan_case(40, 60, 8, 3)
    want = plan_ref(n, q, 60, table, free, nf, num)
    got = run_plan(n, q, 60, table, free, nf)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert got[3] == want[3] == relay.FLAG_POOL
    if 0 <= nf <= num:
        assert got[2] == want[2]


def test_block_plan_bad_lengths_and_ids():
    n, q, table, free, nf, num = plan_case(20, 30, 6, 4)
    n[3], q[3] = 10 ** 6, 2
    q[5] = -1
    q[7] = 31
    n[9], q[9] = 4, 9
    free[nf - 2] = num            # handed out second
    n[0], q[0] = 40, 40           # a request from nothing: draws first
    n[11], q[11] = 20, 3
    table[11, :2] = (1, -1)       # its last held block
    want = plan_ref(n, q, 30, table, free, nf, num)
    got = run_plan(n, q, 30, table, free, nf)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2:] == want[2:]
    assert got[3] == relay.FLAG_BAD_CTX_LEN | relay.FLAG_BAD_Q_LEN | relay.FLAG_BAD_BLOCK


def test_block_plan_every_request_lq_rows_and_one_workspace_for_many_calls():
    w = ws()
    for Lq in (1, 64, 700):
        n, q, table, free, nf, num = plan_case(64, Lq, 80, Lq, ragged=False)
        n = np.maximum(n, Lq)
        n, q, table, free, nf, num = n, np.full(64, Lq), np.full((64, 80), -7), np.arange(64 * 80), 64 * 80, 64 * 80
        table[:, :] = np.arange(64 * 80).reshape(64, 80)
        free = free[::-1].copy()
        want = plan_ref(n, q, Lq, table, free, nf, num)
        t, c = dev(table), dev([nf])
        for _ in range(3):      # the counter in the workspace is back at zero
            c.fill_(nf)
            slots = relay.relay_block_plan(dev(n), t, dev(free), c, Lq=Lq, workspace=w)
            assert np.array_equal(slots.cpu().numpy(), want[1]) and int(c) == want[2]
    assert relay.device_status(w) == 0 and int(w.sum()) == 0


# ----------------------------------------------------------------------------- block release
@pytest.mark.parametrize("B,max_blocks", [(1, 1), (5, 300), (32, 64), (512, 40), (300, 1000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_block_release(B, max_blocks, in_place):
    r = np.random.default_rng(B)
    n = r.integers(0, 16 * max_blocks + 1, B)
    done = r.integers(0, 3, B)            # any value but 0 is done
    blocks = -(-n // 16)
    num = int(blocks.sum()) + 7
    ids = r.permutation(num)
    table = np.full((B, max_blocks), -1)
    k = 0
    for b in range(B):
        table[b, :blocks[b]] = ids[k:k + blocks[b]]
        k += blocks[b]
    free = np.full(num, -9)
    nf = num - k
    free[:nf] = ids[k:]
    want, m = free.copy(), nf
    for b in range(B):
        if done[b]:
            want[m:m + blocks[b]] = table[b, :blocks[b]]
            m += blocks[b]
    f, c, w = dev(free), dev([nf]), ws()
    out = relay.relay_block_release(dev(done), dev(n), dev(table), f, c, None if in_place else dev([0]), workspace=w)
    assert np.array_equal(f.cpu().numpy(), want) and int(out) == m and relay.device_status(w) == 0
    if not in_place:
        assert int(c) == nf


def test_block_release_twice_and_bad_rows():
    n, done = np.array([33, 64, 16, 5, 200]), np.array([1, 1, 1, 0, 1])
    table = np.arange(20).reshape(5, 4)
    table[1, 2] = 99
    free, num = np.full(12, -9), 12
    w, f, c = ws(), dev(free), dev([5])
    relay.relay_block_release(dev(done), dev(n), dev(table), f, c, workspace=w)
    # 3 fit; 4 more come to 12; the third's block is one too many; the last length is out of range
    assert f.cpu().tolist() == [-9] * 5 + [0, 1, 2, 4, 5, -1, 7] and int(c) == 12
    assert relay.device_status(w) == relay.FLAG_POOL | relay.FLAG_BAD_BLOCK | relay.FLAG_BAD_CTX_LEN
    for bad in (-1, 13):
        f2, c2 = dev(free), dev([bad])
        out = relay.relay_block_release(dev(done), dev(n), dev(table), f2, c2, dev([3]), workspace=w)
        assert np.array_equal(f2.cpu().numpy(), free) and relay.device_status(w) & relay.FLAG_POOL and int(out) == bad


# ----------------------------------------------------------------------------- rotary positions
def rope_ref(x, pos, Ls, axis, base, inverse):
    D = x.shape[-1]
    x = x.double().cpu().numpy()
    ang = (pos.astype(np.float64)[axis].transpose(1, 2, 0) + Ls) * base ** (-2.0 * np.arange(D // 2) / D)
    c, s = np.cos(ang)[:, :, None], np.sin(ang)[:, :, None] * (-1 if inverse else 1)
    x0, x1 = x[..., :D // 2], x[..., D // 2:]
    return np.concatenate([x0 * c - x1 * s, x1 * c + x0 * s], -1)


def rope_tol(want, x):
    """Half a step of fp16, or half its smallest step, and the fp32 part: sine and cosine of an angle that is off by
    2^-24 turns at most (pi 2^-24 < 2e-7 rad from the fraction, as much from sincospi) and two roundings."""
    x = np.abs(x.double().cpu().numpy())
    half = x.shape[-1] // 2
    r = x[..., :half] + x[..., half:]
    return 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 8e-7 * np.concatenate([r, r], -1)


ROPE = [  # B, Lq, H, Hkv, D, sections, interleaved
    (1, 1, 1, 1, 64, (32,), False), (3, 1, 32, 8, 128, (16, 24, 24), False), (2, 7, 5, 5, 64, (8, 12, 12), False),
    (2, 5, 9, 3, 128, (24, 20, 20), True), (1, 33, 64, 1, 128, (22, 21, 21), True), (2, 3, 4, 2, 64, (14, 9, 9), True),
    (5, 2, 7, 7, 128, (1, 60, 2, 1), False), (2, 300, 12, 4, 128, (64, 0, 0), False),
]


@pytest.mark.parametrize("case", ROPE)
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_axes(case, inverse, in_place):
    B, Lq, H, Hkv, D, sections, inter = case
    g = torch.Generator().manual_seed(B * Lq + H)
    q = torch.randn(B, Lq, H, D, generator=g).half().to(DEV)
    k = torch.randn(B, Lq, Hkv, D, generator=g).half().to(DEV)
    pos = torch.randint(-50, 40000, (len(sections), B, Lq), generator=g, dtype=torch.int32)
    pos[0, 0, 0] = 2 ** 31 - 1
    pos[-1, -1, -1] = -2 ** 31
    ql = [Lq - (b * Lq) // (2 * B) for b in range(B)]
    axis = np.frombuffer(relay.rope_axis_map(sections, D, inter), dtype=np.uint8)
    assert [int((axis == a).sum()) for a in range(len(sections))] == list(sections)
    Ls, base, w = 2048, 10000.0, ws()
    x, y = q.clone(), k.clone()
    qo, ko = (x, y) if in_place else (torch.full_like(q, 3.0), torch.full_like(k, 3.0))
    relay.relay_rope_axes(x, pos.to(DEV), Ls, sections, k_new=y, q_lens=dev(ql), base=base, interleaved=inter,
                          inverse=inverse, q_out=None if in_place else qo, k_out=None if in_place else ko, workspace=w)
    assert relay.device_status(w) == 0
    for got, src in ((qo, q), (ko, k)):
        want = rope_ref(src, pos.numpy(), Ls, axis, base, inverse)
        got_n = got.double().cpu().numpy()
        for b in range(B):
            err = np.abs(got_n[b, :ql[b]] - want[b, :ql[b]])
            assert (err <= rope_tol(want[b, :ql[b]], src[b, :ql[b]])).all(), err.max()
            left = src[b, ql[b]:] if in_place else torch.full_like(src[b, ql[b]:], 3.0)
            assert torch.equal(got[b, ql[b]:], left)


def test_rope_axes_equal_positions_are_relay_rope():
    """Text: one position on every axis gives the same angles as relay_rope, both within one fp16 rounding of them."""
    B, H, Hkv, D, Ls = 6, 8, 2, 128, 700
    n = torch.tensor([1, 5, 1000, 30000, 8, 77], dtype=torch.int32, device=DEV)
    q, k = torch.randn(B, 1, H, D, device=DEV).half(), torch.randn(B, 1, Hkv, D, device=DEV).half()
    q2, k2 = q.clone(), k.clone()
    relay.relay_rope(q2, n, Ls, k_new=k2)
    relay.relay_rope_axes(q, (n - 1).view(1, B, 1).expand(3, B, 1).contiguous(), Ls, (16, 24, 24), k_new=k)
    for a, b in ((q, q2), (k, k2)):
        assert (a.float() - b.float()).abs().max() <= 2.0 ** -10 * 6      # a step apart at most, values below 6


def test_rope_axes_inverse_is_the_gradient():
    """The rotation is linear: the gradient of <R x, g> is R^T g, which `inverse` gives, and differences agree.  All
    values are dyadic, so the only roundings are the results' own: each entry within 2^-11 of its size (<= 4)."""
    B, H, D = 2, 3, 64
    gen = torch.Generator().manual_seed(0)
    x = (torch.randint(-8, 9, (B, 1, H, D), generator=gen) / 8).half().to(DEV)
    g = (torch.randint(-8, 9, (B, 1, H, D), generator=gen) / 8).half().to(DEV)
    pos = torch.randint(0, 5000, (3, B, 1), generator=gen, dtype=torch.int32).to(DEV)
    turn = lambda v, inv=False: relay.relay_rope_axes(v, pos, 5, (8, 12, 12), inverse=inv, q_out=torch.empty_like(v))[0]
    grad = turn(g, True)
    base = turn(x).double()
    step = 2.0
    for j in range(0, D, 7):
        e = x.clone()
        e[..., j] += step
        diff = ((turn(e).double() - base) * g.double()).sum(-1) / step
        # two rotated rows of 2 entries moved by the step, rounded to 2^-11 of at most 4 each, times |g| <= 1
        assert (diff - grad[..., j].double()).abs().max() <= 2 * D * 4 * 2.0 ** -11 / step
    # and turning back gives x again: two roundings of entries of at most 2
    back = turn(turn(x), True)
    assert (back.float() - x.float()).abs().max() <= 3 * 2 * 2.0 ** -11


def test_rope_axes_bad_q_len():
    q = torch.ones(3, 2, 4, 64, device=DEV).half()
    w = ws()
    relay.relay_rope_axes(q, torch.full((3, 3, 2), 9, dtype=torch.int32, device=DEV), 0, (8, 12, 12), q_lens=dev([2, 3, -1]),
                          workspace=w)
    assert relay.device_status(w) == relay.FLAG_BAD_Q_LEN
    assert (q[1:] == 1).all() and not (q[0] == 1).all()
