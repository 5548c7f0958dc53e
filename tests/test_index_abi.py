"""Refusals of the selector's entry points on the host: through the C ABI with pointers that are never
read (every call fails its checks or has size zero), and through the binding."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)
NULL = None
OK, INVALID, UNSUPPORTED = 0, -1, -2


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


def insert(L, **kw):
    a = dict(q=FAKE, q_s0=4 * 128, q_s1=128, k=FAKE, k_s0=128, w=FAKE, w_s0=4, ws=1.0, qo=FAKE, wo=FAKE, c=FAKE, fmt=1, nb=4,
             bstride=64 * 128, estride=128, sc=FAKE, ss=64, bs=64, slots=FAKE, pos=NULL, cs=NULL, mp=0, T=2, Hi=4, st=NULL)
    a.update(kw)
    return L.mla_index_q_cache_insert(*a.values())


@pytest.mark.parametrize("want,kw", [
    (OK, dict(T=0)), (INVALID, dict(T=-1)), (INVALID, dict(fmt=2)), (INVALID, dict(fmt=7)), (UNSUPPORTED, dict(Hi=0)),
    (UNSUPPORTED, dict(Hi=65, q_s0=65 * 128, w_s0=65)), (INVALID, dict(q=NULL)), (INVALID, dict(w=NULL)), (INVALID, dict(slots=NULL)),
    (INVALID, dict(q_s1=127)), (INVALID, dict(q_s0=511)), (INVALID, dict(k_s0=100)), (INVALID, dict(w_s0=3)), (INVALID, dict(qo=ODD)),
    (INVALID, dict(sc=NULL)), (INVALID, dict(fmt=0, bstride=64 * 256, estride=256)), (INVALID, dict(estride=120)),
    (INVALID, dict(estride=136)), (INVALID, dict(bstride=63 * 128)), (INVALID, dict(ss=63)), (INVALID, dict(ss=66)), (INVALID, dict(c=ODD)),
    (INVALID, dict(sc=ODD)), (INVALID, dict(bs=0)), (INVALID, dict(nb=0)), (INVALID, dict(pos=FAKE)), (INVALID, dict(cs=FAKE)),
    (INVALID, dict(pos=FAKE, cs=FAKE, mp=0)), (INVALID, dict(pos=FAKE, cs=ODD, mp=8)), (UNSUPPORTED, dict(nb=1 << 31)),
])
def test_insert(L, want, kw):
    assert insert(L, **kw) == want


def gather(L, **kw):
    a = dict(c=FAKE, fmt=1, nb=4, bstride=64 * 128, estride=128, sc=FAKE, ss=64, bs=64, bt=FAKE, bts=3, cols=3, cu=FAKE, st=NULL,
             batch=2, n=10, dst=FAKE, row=128, stream=NULL)
    a.update(kw)
    return L.mla_index_gather(*a.values())


@pytest.mark.parametrize("want,kw", [
    (OK, dict(n=0)), (OK, dict(batch=0)), (INVALID, dict(n=-1)), (INVALID, dict(batch=-1)), (UNSUPPORTED, dict(n=1 << 31)),
    (INVALID, dict(fmt=2)), (INVALID, dict(c=NULL)), (INVALID, dict(bt=NULL)), (INVALID, dict(cols=0)), (INVALID, dict(bts=2)),
    (INVALID, dict(cu=NULL)), (INVALID, dict(dst=NULL)), (INVALID, dict(row=127)), (INVALID, dict(sc=NULL)),
])
def test_gather(L, want, kw):
    assert gather(L, **kw) == want


def scores(L, **kw):
    a = dict(q=FAKE, q_s0=4 * 128, q_s1=128, w=FAKE, w_s0=4, c=FAKE, fmt=1, nb=4, bstride=64 * 128, estride=128, sc=FAKE, ss=64, bs=64,
             bt=FAKE, bts=3, cols=3, seq=FAKE, cu=FAKE, B=2, T=3, Hi=4, tok=1, out=FAKE, os=100, width=100, stream=NULL)
    a.update(kw)
    return L.mla_index_scores(*a.values())


@pytest.mark.parametrize("want,kw", [
    (OK, dict(T=0)), (OK, dict(B=0)), (OK, dict(width=0)), (INVALID, dict(T=-1)), (INVALID, dict(B=-1)), (INVALID, dict(width=-1)),
    (INVALID, dict(cu=NULL)), (UNSUPPORTED, dict(Hi=0)), (UNSUPPORTED, dict(Hi=65)), (UNSUPPORTED, dict(tok=0)), (UNSUPPORTED, dict(tok=8)),
    (UNSUPPORTED, dict(tok=256)), (UNSUPPORTED, dict(bs=48, bstride=48 * 128, ss=48)), (UNSUPPORTED, dict(bs=8, bstride=8 * 128, ss=8)),
    (INVALID, dict(q=NULL)), (INVALID, dict(w=NULL)), (INVALID, dict(seq=NULL)), (INVALID, dict(out=NULL)), (INVALID, dict(q=ODD)),
    (INVALID, dict(q_s1=136)), (INVALID, dict(q_s1=64)), (INVALID, dict(q_s0=256)), (INVALID, dict(w_s0=3)), (INVALID, dict(os=99)),
    (INVALID, dict(sc=NULL)), (INVALID, dict(fmt=2)), (INVALID, dict(bt=NULL)),
])
def test_scores(L, want, kw):
    assert scores(L, **kw) == want


def select(L, **kw):
    a = dict(x=FAKE, xs=100, width=100, seq=FAKE, cu=FAKE, B=2, T=3, tok=1, k=8, first=0, last=0, blocks=FAKE, bs=8, slots=NULL, ss=0,
             bt=NULL, bts=0, cols=0, page=0, nb=0, stream=NULL)
    a.update(kw)
    return L.mla_index_select(*a.values())


SLOTS = dict(slots=FAKE, ss=8, bt=FAKE, bts=3, cols=3, page=64, nb=10)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(T=0)), (OK, dict(B=0)), (INVALID, dict(T=-1)), (INVALID, dict(cu=NULL)), (INVALID, dict(k=0)), (UNSUPPORTED, dict(k=8193, bs=8193)),
    (INVALID, dict(tok=0)), (INVALID, dict(first=-1)), (INVALID, dict(last=-1)), (INVALID, dict(first=5, last=4)), (INVALID, dict(width=-1) | dict(x=NULL)),
    (UNSUPPORTED, dict(width=1 << 30, xs=1 << 30)), (INVALID, dict(x=NULL)), (INVALID, dict(seq=NULL)), (INVALID, dict(blocks=NULL)),
    (INVALID, dict(xs=99)), (INVALID, dict(bs=7)), (INVALID, {**SLOTS, "ss": 7}), (INVALID, {**SLOTS, "bt": NULL}), (INVALID, {**SLOTS, "page": 0}),
    (INVALID, {**SLOTS, "nb": 0}), (UNSUPPORTED, {**SLOTS, "nb": 1 << 25}), (UNSUPPORTED, {**SLOTS, "tok": 1 << 28, "ss": 1 << 31}),
])
def test_select(L, want, kw):
    got = select(L, **kw)
    assert got == want or (kw.get("width") == -1 and got in (INVALID, UNSUPPORTED))


def selected(L, **kw):
    a = dict(q=FAKE, q_s0=16 * 576, q_s1=576, kv=FAKE, fmt=0, nb=10, bstride=64 * 1152, estride=1152, bs=64, bt=FAKE, bts=4, cols=4,
             seq=FAKE, cu=FAKE, blocks=FAKE, b_s=3, topk=3, B=2, T=2, H=16, sm=0.1, qs=1.0, ks=1.0, out=FAKE, o0=16 * 512, o1=512,
             lse=NULL, ws=FAKE, wsn=1 << 30, stream=NULL)
    a.update(kw)
    return L.mla_selected_decode(*a.values())


@pytest.mark.parametrize("want,kw", [
    (OK, dict(T=0)), (OK, dict(B=0)), (INVALID, dict(T=-1)), (INVALID, dict(cu=NULL, T=3)), (INVALID, dict(topk=0)), (INVALID, dict(bs=0)),
    (UNSUPPORTED, dict(topk=1 << 24, b_s=1 << 24)), (INVALID, dict(seq=NULL)), (INVALID, dict(blocks=NULL)), (INVALID, dict(b_s=2)),
    (UNSUPPORTED, dict(H=129)), (UNSUPPORTED, dict(H=0)), (INVALID, dict(bt=NULL)),
])
def test_selected(L, want, kw):
    assert selected(L, **kw) == want


def test_binding_refuses_host_tensors_and_wrong_types(m):
    z = torch.zeros
    bf, u8, i32, i64 = torch.bfloat16, torch.uint8, torch.int32, torch.int64
    with pytest.raises(ValueError, match="CUDA"):
        m.index_q_cache_insert(z(2, 4, 128, dtype=bf), z(2, 128, dtype=bf), z(2, 4), z(2, 16, 128, dtype=u8), z(2, 16), z(2, dtype=i64), fmt="fp8")
    with pytest.raises(ValueError, match="CUDA"):
        m.index_scores(z(2, 4, 128, dtype=u8), z(2, 4), z(2, 16, 128, dtype=u8), z(2, 16), z(2, 3, dtype=i32), z(2, dtype=i32), fmt="fp8", max_context=8)
    with pytest.raises(ValueError, match="CUDA"):
        m.index_select(z(2, 8), z(2, dtype=i32), 4)
    with pytest.raises(ValueError, match="CUDA"):
        m.index_gather(z(2, 16, 128, dtype=u8), z(2, 16), z(2, 3, dtype=i32), z(3, dtype=i32), fmt="fp8", num_tokens=4)
    with pytest.raises(ValueError, match="CUDA"):
        m.selected_decode(z(2, 16, 576, dtype=bf), z(4, 64, 576, dtype=bf), z(2, 3, dtype=i32), z(2, dtype=i32), z(2, 3, dtype=i32), fmt="bf16", softmax_scale=1.0)
    with pytest.raises(ValueError, match="bf16 or fp8"):
        m.index_gather(None, None, None, None, fmt="fp8_ds_mla", num_tokens=4)


def test_selected_workspace_holds_the_lists_and_the_partials(L):
    # lists alone for one split: lengths and tables, each on a 256-byte boundary
    n = lambda fmt, T, k, bs, H, sms=152: L.mla_selected_decode_workspace_size(fmt, T, k, bs, H, sms)
    assert n(0, 0, 4, 64, 16) == 0 and n(0, 4, 0, 64, 16) == 0
    assert n(0, 3, 2, 64, 16) == 256 + 256
    # 126 rows of 96 heads are five waves of whole rows; of 128 the last two are cut, by themselves
    assert n(2, 126, 32, 64, 96) == 512 + 126 * 32 * 4
    assert 512 + 128 * 32 * 4 + 2 * 2 * 96 * 2048 <= n(2, 128, 32, 64, 96) < 512 + 128 * 32 * 4 + 2 * 17 * 96 * 2048
    # the rows beyond a whole wave
    lists = lambda T, k: -(-T * 4 // 256) * 256 + -(-T * k * 4 // 256) * 256
    for fmt, T, H, rows in ((2, 26, 96, 25), (0, 40, 128, 38), (1, 78, 128, 76)):
        assert n(fmt, rows, 16, 64, H) == lists(rows, 16)
        assert n(fmt, T, 16, 64, H) >= lists(T, 16) + (T - rows) * 2 * H * 2048
    # a single row of a long list is cut into many
    assert n(0, 1, 256, 64, 16) > 256 + 1024 + 16 * 512 * 4 * 8
