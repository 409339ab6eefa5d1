"""Refusals of the 4-bit pool's calls and of the steps around the cache, without a GPU: host-side validation comes
before any CUDA call, and the binding's shape checks before any pointer reaches the library."""
import ctypes

import pytest
import torch

FAKE = 0x7f0000000000      # never dereferenced: validation fails first
f16, i32, u8 = torch.float16, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def relay():
    from shared_prompt_decode_gb300 import build
    build.build()
    import shared_prompt_decode_gb300 as r
    r.lib()
    return r


def dims(relay, **kw):
    base = dict(B=32, Lq=1, H=32, D=128, Ls=2048, block_size=16, num_blocks=1200, max_blocks_per_seq=64,
                max_q_total=0, ctx_split=0, sys_range=0, scale=0.0, Hkv=0)
    return relay.Dims(**{**base, **kw})


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


def pool(relay, group=128, **kw):
    at = {k: kw.get(k, FAKE) for k in ("k_codes", "k_sz", "v_codes", "v_sz")}
    return relay.Q4Struct(at["k_codes"], at["k_sz"], at["v_codes"], at["v_sz"], group)


def test_layouts_and_exports(relay, tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "relay.h"\n'
                    'int main(void){printf("%zu %zu %zu %zu %d %d\\n", sizeof(relay_q4_cache_t), offsetof(relay_q4_cache_t, k_sz),'
                    ' offsetof(relay_q4_cache_t, v_codes), offsetof(relay_q4_cache_t, group), (int)RELAY_FLAG_POOL,'
                    ' RELAY_MAX_ROPE_AXES);return 0;}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(prog), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    S = relay.Q4Struct
    assert got == [ctypes.sizeof(S), S.k_sz.offset, S.v_codes.offset, S.group.offset, relay.FLAG_POOL, relay.MAX_ROPE_AXES]
    for name in ("relay_attention_decode_q4", "relay_ctx_attn_q4", "relay_kv_append_q4", "relay_workspace_size_q4",
                 "relay_block_plan", "relay_block_release", "relay_rope_axes"):
        assert hasattr(relay.lib(), name)


def test_workspace_size_q4(relay):
    n = relay.workspace_size_q4(dims(relay))
    assert n > 0 and n % 256 == 0
    assert relay.workspace_size_q4(dims(relay, B=64)) > n
    for bad in (dict(D=96), dict(block_size=32), dict(B=513), dict(H=0), dict(Hkv=3), dict(ctx_split=8)):
        assert relay.workspace_size_q4(dims(relay, **bad)) == 0


@pytest.mark.parametrize("which", ["decode", "ctx"])
def test_attention_refusals(relay, which):
    lib = relay.lib()

    def call(d=None, c=None, ws_bytes=1 << 32, no_cache=False, **o):
        d = dims(relay) if d is None else d
        c = None if no_cache else ctypes.byref(pool(relay) if c is None else c)
        p = lambda k, v=FAKE: vp(o.get(k, v))
        if which == "decode":
            return lib.relay_attention_decode_q4(ctypes.byref(d), p("q"), p("sys_k"), p("sys_v"), c, p("bt"), p("cl"),
                                                 p("ql", None), p("out"), p("lse", None), p("ws"), ws_bytes, None)
        return lib.relay_ctx_attn_q4(ctypes.byref(d), p("q"), c, p("bt"), p("cl"), p("ql", None), p("out"),
                                     p("lse"), p("ws"), ws_bytes, None)
    assert call(no_cache=True) == relay.ERR_INVALID_ARG
    for group in (0, 16, 48, 256, -32):
        assert call(c=pool(relay, group)) == relay.ERR_UNSUPPORTED
    assert call(d=dims(relay, D=64)) == relay.ERR_UNSUPPORTED                  # a group of 128 in heads of 64
    assert call(d=dims(relay, D=96)) == relay.ERR_UNSUPPORTED
    assert call(d=dims(relay, Hkv=5)) == relay.ERR_INVALID_ARG
    for k in ("k_codes", "k_sz", "v_codes", "v_sz"):
        assert call(c=pool(relay, **{k: None})) == relay.ERR_INVALID_ARG
        assert call(c=pool(relay, **{k: FAKE + 8})) == relay.ERR_INVALID_ARG   # not 16-byte aligned
    for k in ("q", "cl", "bt", "out", "ws"):
        assert call(**{k: None}) == (relay.ERR_WORKSPACE if k == "ws" else relay.ERR_INVALID_ARG), k
        assert call(**{k: FAKE + 2}) == relay.ERR_INVALID_ARG, k
    assert call(ws_bytes=1024) == relay.ERR_WORKSPACE
    assert call(d=dims(relay, Lq=2, max_q_total=3)) == relay.ERR_INVALID_ARG   # no q_lens: 64 rows
    assert call(d=dims(relay, B=0)) == relay.OK
    if which == "decode":
        assert call(sys_k=None) == relay.ERR_INVALID_ARG
        assert call(sys_v=FAKE + 8) == relay.ERR_INVALID_ARG


def test_append_refusals(relay):
    lib = relay.lib()

    def call(d=None, c=None, ws_bytes=256, **o):
        d = dims(relay, Lq=2) if d is None else d
        p = lambda k, v=FAKE: vp(o.get(k, v))
        return lib.relay_kv_append_q4(ctypes.byref(d), p("kn"), p("vn"), p("bt"), p("cl"), p("ql", None), p("sm", None),
                                      ctypes.byref(pool(relay) if c is None else c), p("ws"), ws_bytes, None)
    assert call(c=pool(relay, 24)) == relay.ERR_UNSUPPORTED
    assert call(c=pool(relay, v_sz=None)) == relay.ERR_INVALID_ARG
    assert call(ws=None) == relay.ERR_WORKSPACE
    assert call(ws_bytes=255) == relay.ERR_WORKSPACE
    assert call(ws=FAKE + 16) == relay.ERR_INVALID_ARG
    for k in ("kn", "vn", "bt", "cl"):
        assert call(**{k: None}) == relay.ERR_INVALID_ARG, k
        assert call(**{k: FAKE + 2}) == relay.ERR_INVALID_ARG, k
    assert call(sm=FAKE + 2, bt=None, cl=None) == relay.ERR_INVALID_ARG
    assert call(d=dims(relay, num_blocks=0)) == relay.ERR_INVALID_ARG
    assert call(d=dims(relay, num_blocks=1 << 27)) == relay.ERR_UNSUPPORTED        # 32-bit slots
    assert call(d=dims(relay, B=0)) == relay.OK


def test_step_refusals(relay):
    lib = relay.lib()

    def plan(d=None, ws_bytes=256, **o):
        d = dims(relay) if d is None else d
        args = [vp(o.get(k, FAKE)) for k in ("cl", "ql", "free", "nf", "bt", "sm", "nfo", "ws")]
        return lib.relay_block_plan(ctypes.byref(d), *args, ws_bytes, None)

    def release(d=None, ws_bytes=256, **o):
        d = dims(relay) if d is None else d
        args = [vp(o.get(k, FAKE)) for k in ("done", "cl", "bt", "free", "nf", "nfo", "ws")]
        return lib.relay_block_release(ctypes.byref(d), *args, ws_bytes, None)
    for call in (plan, release):
        assert call(ws=None) == relay.ERR_WORKSPACE and call(ws_bytes=8) == relay.ERR_WORKSPACE
        assert call(d=dims(relay, B=513)) == relay.ERR_UNSUPPORTED
        assert call(d=dims(relay, B=0)) == relay.OK
        for k in ("cl", "free", "nf", "bt", "nfo"):
            assert call(**{k: None}) == relay.ERR_INVALID_ARG, k
            assert call(**{k: FAKE + 2}) == relay.ERR_INVALID_ARG, k
    assert plan(d=dims(relay, num_blocks=1 << 27)) == relay.ERR_UNSUPPORTED
    assert release(done=None) == relay.ERR_INVALID_ARG

    def rope(d=None, n=3, axis=bytes(64), base=1e4, ws_bytes=256, **o):
        d = dims(relay, Hkv=8) if d is None else d
        p = lambda k: vp(o.get(k, FAKE))
        return lib.relay_rope_axes(ctypes.byref(d), p("q"), p("k"), p("pos"), n, axis, p("ql"), base, 0, p("qo"), p("ko"),
                                   p("ws"), ws_bytes, None)
    assert rope(ws=None) == relay.ERR_WORKSPACE
    assert rope(n=0) == rope(n=5) == rope(axis=None) == relay.ERR_INVALID_ARG
    assert rope(axis=bytes(63) + b"\3") == relay.ERR_INVALID_ARG                # axis 3 of three
    assert rope(base=1.0) == rope(base=float("nan")) == relay.ERR_INVALID_ARG
    for k in ("q", "qo", "pos", "k", "ko"):                                     # k without k_out and the other way too
        assert rope(**{k: None}) == relay.ERR_INVALID_ARG, k
        assert rope(**{k: FAKE + 2}) == relay.ERR_INVALID_ARG, k
    assert rope(d=dims(relay, B=0)) == relay.OK


def test_axis_map(relay):
    assert relay.rope_axis_map((2, 1, 29), 64) == b"\0\0\1" + b"\2" * 29
    assert relay.rope_axis_map((14, 9, 9), 64, True) == b"\0\1\2" * 9 + b"\0" * 5
    assert relay.rope_axis_map((64,), 128, True) == bytes(64)
    for sections, D, inter in (((20, 22, 22), 128, True), ((31,), 64, False), ((8, 8, 8, 4, 4), 64, False),
                               ((40, -8), 64, False), ((), 64, False), ((1, 31), 64, True)):
        with pytest.raises(ValueError):
            relay.rope_axis_map(sections, D, inter)


class FakePool:
    """The shape of a pool, for checks that come before its tensors are used."""
    def __init__(self, num=8, Hkv=4, D=64):
        self.num_blocks, self.Hkv, self.D, self.group, self.device = num, Hkv, D, 32, torch.device("cpu")
        self.k_codes = torch.zeros(num, Hkv, 16, D // 2, dtype=u8)


def test_binding_checks(relay):
    z = torch.zeros
    q, kn = z(2, 1, 4, 64, dtype=f16), z(2, 1, 4, 64, dtype=f16)
    bt, cl = z(2, 4, dtype=i32), z(2, dtype=i32)
    sysk = z(32, 4, 64, dtype=f16)
    codes, sz = z(8, 4, 16, 32, dtype=u8), z(8, 4, 16, 2, 2, dtype=f16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        relay.Q4Cache(codes, sz, codes, sz)
    for c, s in ((codes[:, :, :8], sz), (codes, sz[..., 0]), (codes, sz[:7]), (codes, z(8, 4, 16, 3, 2, dtype=f16))):
        with pytest.raises(ValueError):
            relay.Q4Cache(c, s, c, s)
    with pytest.raises(ValueError, match="k_codes"):
        relay.Q4Cache(codes, sz, codes[:4], sz)
    for group in (16, 128):
        with pytest.raises(ValueError, match="group"):
            relay.make_q4_cache(4, 2, 64, group)
    p = FakePool()
    bad = [dict(out=z(2, 1, 4, 32, dtype=f16)), dict(lse_out=z(2, 1, 3)), dict(q_lens=z(3, dtype=i32)),
           dict(ctx_lens=z(1, dtype=i32)), dict(block_tables=z(3, 4, dtype=i32)), dict(sys_v=sysk[:31]),
           dict(sys_k=z(32, 2, 64, dtype=f16), sys_v=z(32, 2, 64, dtype=f16)), dict(cache=FakePool(D=128)),
           dict(cache=FakePool(Hkv=3))]
    good = dict(q=q, sys_k=sysk, sys_v=sysk, cache=p, block_tables=bt, ctx_lens=cl)
    for over in bad:
        with pytest.raises(ValueError) as e:
            relay.relay_attention_decode_q4(**{**good, **over})
        assert "must be a CUDA tensor" not in str(e.value), over.keys()
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        relay.relay_attention_decode_q4(**good)
    with pytest.raises(ValueError, match="lse_ctx"):
        relay.relay_ctx_attn_q4(q, p, bt, cl, lse_ctx=z(2, 4))
    for over, what in ((dict(v_new=kn[:1]), "v_new"), (dict(slot_map=z(2, 2, dtype=i32)), "slot_map"),
                       (dict(cache=FakePool(Hkv=2)), "KV heads"), (dict(q_lens=cl[:1]), "q_lens")):
        with pytest.raises(ValueError, match=what):
            relay.relay_kv_append_q4(**{**dict(k_new=kn, v_new=kn, block_tables=bt, ctx_lens=cl, cache=p), **over})
    pos = z(3, 2, 1, dtype=i32)
    for over, what in ((dict(positions=pos[:2]), "positions"), (dict(sections=(8, 12, 11)), "sections"),
                       (dict(k_new=kn[:1]), "k_new"), (dict(k_out=kn), "k_out"), (dict(q_out=q[:1]), "q_out"),
                       (dict(q_lens=cl[:1]), "q_lens")):
        with pytest.raises(ValueError, match=what):
            relay.relay_rope_axes(**{**dict(q=q, positions=pos, Ls=0, sections=(8, 12, 12)), **over})
    one = z(1, dtype=i32)
    with pytest.raises(ValueError, match="slot_map"):
        relay.relay_block_plan(cl, bt, z(8, dtype=i32), one, slot_map=z(2, 3, dtype=i32))
    with pytest.raises(ValueError, match="block_tables"):
        relay.relay_block_plan(cl, bt[:1], z(8, dtype=i32), one)
    with pytest.raises(ValueError, match="CUDA tensor"):
        relay.relay_block_plan(cl, bt, z(8, dtype=i32), one)
    with pytest.raises(ValueError, match="CUDA tensor"):
        relay.relay_block_release(cl, cl, bt, z(8, dtype=i32), one)
