"""Refusals on the host of rope, rope_table, plan_step and of the mxfp4 cache in every entry that takes a format: through
the C ABI with pointers that are never read (each call fails its checks or has size zero), and through the binding."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(1 << 20)
FAR = ctypes.c_void_p(1 << 40)
ODD = ctypes.c_void_p((1 << 20) + 1)
HALF = ctypes.c_void_p((1 << 20) + 2)
EIGHT = ctypes.c_void_p((1 << 20) + 8)
NULL = None
OK, INVALID, UNSUPPORTED = 0, -1, -2
MXFP4 = 3


@pytest.fixture(scope="module")
def m():
    from mla_latent_cache_attention_gb300 import build
    build.build()
    import mla_latent_cache_attention_gb300 as mod
    mod.lib()
    return mod


@pytest.fixture(scope="module")
def L(m):
    return m.lib()


def rope(L, **kw):
    a = dict(type=0, q=FAKE, q_s0=4 * 64, q_s1=64, qo=FAR, qo_s0=4 * 64, qo_s1=64, H=4, D=64, q_at=0, k=NULL, k_s0=0, k_s1=0, ko=NULL,
             ko_s0=0, ko_s1=0, Hk=0, Dk=0, k_at=0, pos=FAKE, cs=FAKE, mp=8, R=64, half=0, inverse=0, T=2, stream=NULL)
    a.update(kw)
    return L.mla_rope(*a.values())


KEYS = dict(k=ctypes.c_void_p(1 << 30), k_s0=64, k_s1=64, ko=ctypes.c_void_p(1 << 41), ko_s0=64, ko_s1=64, Hk=1, Dk=64)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(T=0)), (INVALID, dict(T=-1)), (INVALID, dict(type=3)), (INVALID, dict(type=-1)), (INVALID, dict(R=0)), (INVALID, dict(R=63)),
    (UNSUPPORTED, dict(R=514)), (UNSUPPORTED, dict(D=1032, q_s1=1032, q_s0=4128, qo_s1=1032, qo_s0=4128)), (INVALID, dict(H=0)),
    (INVALID, dict(D=62)), (INVALID, dict(q_at=-2)), (INVALID, dict(q_at=2)), (INVALID, dict(q=NULL)), (INVALID, dict(qo=NULL)),
    (INVALID, dict(pos=NULL)), (INVALID, dict(cs=NULL)), (INVALID, dict(mp=0)), (INVALID, dict(q=ODD)), (INVALID, dict(type=2, q=HALF)),
    (INVALID, dict(cs=HALF)), (INVALID, dict(pos=HALF)), (INVALID, dict(q_s1=63)), (INVALID, dict(q_s0=255)), (INVALID, dict(qo_s1=63)),
    (INVALID, dict(qo_s0=255)), (INVALID, dict(qo=EIGHT)), (INVALID, dict(qo=FAKE, qo_s0=512)), (INVALID, {**KEYS, "ko": NULL}),
    (INVALID, {**KEYS, "k": NULL}), (INVALID, {**KEYS, "Hk": 0}), (INVALID, {**KEYS, "Dk": 63}), (INVALID, {**KEYS, "k_at": 2}),
    (INVALID, {**KEYS, "ko": KEYS["k"]}), (INVALID, {**KEYS, "k_s0": 63}),
])
def test_rope(L, want, kw):
    assert rope(L, **kw) == want


def table(L, **kw):
    a = dict(out=FAKE, n=8, R=64, base=10000.0, scaling=0, factor=1.0, original=0, fast=32.0, slow=1.0, attn=1.0, stream=NULL)
    a.update(kw)
    return L.mla_rope_table(*a.values())


@pytest.mark.parametrize("want,kw", [
    (OK, dict(n=0)), (INVALID, dict(n=-1)), (UNSUPPORTED, dict(n=1 << 40)), (INVALID, dict(R=0)), (INVALID, dict(R=7)), (UNSUPPORTED, dict(R=514)),
    (INVALID, dict(base=1.0)), (INVALID, dict(base=float("inf"))), (INVALID, dict(base=float("nan"))), (INVALID, dict(scaling=4)),
    (INVALID, dict(scaling=-1)), (INVALID, dict(scaling=1, factor=0.0)), (INVALID, dict(scaling=2, factor=float("nan"))),
    (INVALID, dict(scaling=2, factor=2.0, R=2)), (INVALID, dict(scaling=3, factor=2.0)), (INVALID, dict(scaling=3, factor=2.0, original=9, fast=0.0)),
    (INVALID, dict(scaling=3, factor=2.0, original=9, slow=-1.0)), (INVALID, dict(attn=float("inf"))), (INVALID, dict(out=NULL)), (INVALID, dict(out=HALF)),
])
def test_rope_table(L, want, kw):
    assert table(L, **kw) == want


def plan(L, **kw):
    a = dict(seq=FAKE, new=FAKE, fin=NULL, bt=FAKE, bts=4, cols=4, free=FAKE, cap=16, nf=FAKE, so=FAKE, nfo=FAKE, served=FAKE, cu=FAKE, slots=FAKE,
             pos=FAKE, B=2, T=4, bs=64, stream=NULL)
    a.update(kw)
    return L.mla_plan_step(*a.values())


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(B=0)), (INVALID, dict(B=-1)), (INVALID, dict(T=-1)), (INVALID, dict(bs=0)), (INVALID, dict(cols=0)), (INVALID, dict(bts=3)),
    (INVALID, dict(cap=-1)), (INVALID, dict(cap=1 << 31)), (INVALID, dict(seq=NULL)), (INVALID, dict(new=NULL)), (INVALID, dict(bt=NULL)),
    (INVALID, dict(free=NULL)), (INVALID, dict(nf=NULL)), (INVALID, dict(so=NULL)), (INVALID, dict(nfo=NULL)), (INVALID, dict(served=NULL, B=1025)),
    (INVALID, dict(cu=NULL)), (INVALID, dict(slots=NULL)), (INVALID, dict(pos=NULL)), (INVALID, dict(seq=HALF)), (INVALID, dict(bt=HALF)),
    (INVALID, dict(slots=HALF)), (INVALID, dict(pos=HALF)), (INVALID, dict(cu=HALF)), (INVALID, dict(free=HALF)),
])
def test_plan(L, want, kw):
    assert plan(L, **kw) == want


def decode(L, **kw):
    a = dict(q=FAKE, q_s0=16 * 576, q_s1=576, kv=FAKE, fmt=MXFP4, nb=10, bstride=64 * 400, estride=400, bs=64, bt=FAKE, bts=4, seq=FAKE, B=2, ql=1,
             H=16, mc=4096, sm=0.1, qs=1.0, ks=1.0, out=FAKE, o0=16 * 512, o1=512, lse=NULL, ws=FAKE, wsn=1 << 30, stream=NULL)
    a.update(kw)
    return L.mla_paged_decode(*a.values())


@pytest.mark.parametrize("want,kw", [
    (OK, dict(B=0)), (INVALID, dict(fmt=4)), (INVALID, dict(fmt=-1)), (INVALID, dict(estride=384)), (INVALID, dict(estride=408, bstride=64 * 408)),
    (INVALID, dict(bstride=63 * 400)), (INVALID, dict(bstride=64 * 400 + 8)), (INVALID, dict(kv=EIGHT)), (INVALID, dict(q=EIGHT)),
    (INVALID, dict(q_s1=568)), (INVALID, dict(q_s1=580)), (UNSUPPORTED, dict(H=129)), (INVALID, dict(bs=0)), (INVALID, dict(ql=0)),
    (INVALID, dict(mc=0)), (INVALID, dict(seq=NULL)), (INVALID, dict(o1=511)),
])
def test_decode(L, want, kw):
    assert decode(L, **kw) == want


def test_inserts_and_gathers(L):
    def insert(**kw):
        a = dict(ql=FAKE, s0=16 * 512, s1=512, qpe=FAKE, p0=16 * 64, p1=64, kv=FAKE, kv0=512, kp=FAKE, kp0=64, q=FAKE, cache=FAKE, fmt=MXFP4,
                 nb=10, bstride=64 * 400, estride=400, bs=64, slots=FAKE, qinv=NULL, cinv=NULL, pos=NULL, cs=NULL, mp=100, B=2, H=16, stream=NULL)
        a.update(kw)
        return L.mla_q_concat_cache_insert(*a.values())
    assert insert(B=0) == OK
    for kw in (dict(fmt=4), dict(estride=396), dict(estride=402, bstride=64 * 402), dict(bstride=64 * 400 - 4), dict(cache=HALF),
               dict(qinv=FAKE, cinv=FAKE), dict(pos=FAKE)):
        assert insert(**kw) == INVALID, kw

    def gather(**kw):
        a = dict(cache=FAKE, fmt=MXFP4, nb=10, bstride=64 * 400, estride=400, bs=64, slots=FAKE, n=3, out=FAKE, stream=NULL)
        a.update(kw)
        return L.mla_gather_dequant(*a.values())
    for kw in (dict(fmt=4), dict(estride=396), dict(estride=402, bstride=64 * 402), dict(bstride=64 * 400 - 4), dict(cache=HALF)):
        assert gather(**kw) == INVALID, kw
    # the index cache has no 4-bit form
    assert L.mla_index_gather(FAKE, MXFP4, 4, 64 * 128, 128, FAKE, 64, 64, FAKE, 3, 3, FAKE, NULL, 2, 10, FAKE, 128, NULL) == INVALID


def test_the_fp8_prefill_epilogue_stays_fp8(L):
    # key concat takes mxfp4; the raw E4M3 cache has its own epilogue
    a = [FAKE, 4 * 192, 192, FAKE, 4 * 128, 128, FAKE, 64, FAKE, 512, FAKE, FAKE, MXFP4, 10, 64 * 400, 400, 64, FAKE, NULL, NULL, 0, 2, 4, 128, NULL]
    a[15] = 396
    assert L.mla_key_concat_cache_insert(*a) == INVALID
    a[15], a[12] = 400, 1
    assert L.mla_key_concat_cache_insert(*a) == INVALID


def test_the_decode_s_workspace(m, L):
    n = lambda fmt, B, q, H, ctx=131072, sms=152: L.mla_paged_decode_workspace_size_for(fmt, B, q, H, ctx, sms)
    for fmt in (0, 1, 2):
        assert n(fmt, 64, 4, 16) == L.mla_paged_decode_workspace_size(64, 4, 16, 131072, 152) > 0
    # two partials of 512 values and a log-sum-exp a run and column; runs x groups of columns fill the SMs
    up = lambda x: -(-x // 256) * 256
    for q, H, runs in ((1, 16, 152), (1, 17, 152), (1, 32, 152), (1, 33, 152), (4, 16, 152), (1, 65, 76), (1, 128, 76), (7, 128, 10), (64, 128, 1)):
        cols = q * H
        assert n(MXFP4, 9, q, H) == up(2 * runs * cols * 2048) + up(2 * runs * cols * 4) + up(runs * 8)
    assert n(MXFP4, 1, 1, 16) == n(MXFP4, 500, 1, 16) == n(MXFP4, 1, 1, 16, 64)     # neither requests nor lengths
    assert m.paged_decode_workspace_size(4, 1, 16, 4096, 152, fmt="mxfp4") == n(MXFP4, 4, 1, 16)
    assert m.paged_decode_workspace_size(64, 4, 16, 131072, 152) == n(0, 64, 4, 16)


def test_binding_refuses_host_tensors_and_wrong_arguments(m):
    z = torch.zeros
    bf, u8, i32, i64 = torch.bfloat16, torch.uint8, torch.int32, torch.int64
    cache = z(4, 16, 400, dtype=u8)
    with pytest.raises(ValueError, match="CUDA"):
        m.rope(z(2, 4, 64, dtype=bf), z(2, dtype=i64), z(8, 64))
    with pytest.raises(ValueError, match="layout"):
        m.rope(z(2, 4, 64, dtype=bf), z(2, dtype=i64), z(8, 64), layout="other")
    with pytest.raises(ValueError, match="CUDA"):
        m.plan_step(z(2, dtype=i32), z(2, dtype=i32), z(2, 3, dtype=i32), z(4, dtype=i32), z(1, dtype=i32), block_size=16, num_tokens=4)
    with pytest.raises(ValueError, match="CUDA"):
        m.paged_decode(z(2, 16, 576, dtype=bf), cache, z(2, 3, dtype=i32), z(2, dtype=i32), fmt="mxfp4", max_context=32, softmax_scale=1.0)
    with pytest.raises(ValueError, match="CUDA"):
        m.gather_context(cache, z(2, 3, dtype=i32), z(3, dtype=i32), fmt="mxfp4", num_tokens=4)
    with pytest.raises(ValueError, match="CUDA"):
        m.q_concat_cache_insert(z(2, 4, 512, dtype=bf), z(2, 4, 64, dtype=bf), z(2, 512, dtype=bf), z(2, 64, dtype=bf), cache, z(2, dtype=i64), fmt="mxfp4")
    with pytest.raises(ValueError, match="bf16 or fp8"):
        m.index_gather(None, None, None, None, fmt="mxfp4", num_tokens=4)
    with pytest.raises(ValueError, match="CUDA device"):
        m.rope_table(8, 64, device="cpu")
    for kw in (dict(dim=63), dict(dim=0), dict(dim=514), dict(max_position=-1), dict(scaling="cubic")):
        with pytest.raises(ValueError):
            m.rope_table(**{**dict(max_position=8, dim=64, device="cpu"), **kw})
