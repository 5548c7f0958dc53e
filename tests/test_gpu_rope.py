"""Rotary positions on the GPU against plain 64-bit references."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
LEAST = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


@pytest.fixture(scope="module")
def m():
    import mla_latent_cache_attention_gb300 as mod
    mod.lib()
    return mod


def table(n, R, seed=0):
    ang = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def turned(x, pos, tab, layout, at, inverse=False):
    """x [T, H, D] in 64 bits."""
    R = tab.shape[1]
    i = torch.arange(R // 2)
    a, b = (at + i, at + i + R // 2) if layout == "half" else (at + 2 * i, at + 2 * i + 1)
    y = x.double().clone()
    c, s = tab[pos].double()[:, None, :R // 2], tab[pos].double()[:, None, R // 2:]
    if inverse:
        s = -s
    y[..., a], y[..., b] = x[..., a].double() * c - x[..., b].double() * s, x[..., b].double() * c + x[..., a].double() * s
    return y


def near(got, want, x, layout, at, R):
    """Two fp32 roundings (2^-24 of the products' magnitudes each), then one to the type."""
    dt = got.dtype
    mag = x.double().abs()
    i = torch.arange(R // 2)
    a, b = (at + i, at + i + R // 2) if layout == "half" else (at + 2 * i, at + 2 * i + 1)
    both = torch.zeros_like(mag)
    both[..., a] = both[..., b] = mag[..., a] + mag[..., b]
    g = got.double().cpu()
    tol = HALF_STEP[dt] * want.abs() + 2.0 ** -23 * both + LEAST[dt]
    assert bool(((g - want).abs() <= tol).all()), ((g - want).abs() / tol).max()
    rest = torch.ones(x.shape[-1], dtype=torch.bool)
    rest[a], rest[b] = False, False
    assert torch.equal(got.cpu()[..., rest], x[..., rest])


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,H,D,R,at", [(1, 1, 2, 2, 0), (3, 5, 64, 64, 0), (33, 16, 192, 64, 128), (7, 9, 192, 64, 40), (5, 3, 100, 30, 7),
                                        (2, 64, 128, 128, 0), (4, 2, 1024, 512, 256), (6, 7, 96, 32, 64), (9, 1, 80, 16, 8), (130, 33, 128, 64, 0)])
@pytest.mark.parametrize("inverse", [False, True])
def test_shapes(m, dt, layout, T, H, D, R, at, inverse):
    g = torch.Generator().manual_seed(T * 1000 + D)
    q, k = torch.randn((T, H, D), generator=g).to(dt), torch.randn((T, 1, R + 8), generator=g).to(dt)
    pos, tab = torch.randint(0, 5000, (T,), generator=g), table(5000, R)
    p, c = pos.cuda(), tab.cuda()
    qo, ko = m.rope(q.cuda(), p, c, k.cuda(), layout=layout, inverse=inverse, q_at=at)
    near(qo, turned(q, pos, tab, layout, at, inverse), q, layout, at, R)
    near(ko, turned(k, pos, tab, layout, 8, inverse), k, layout, 8, R)
    # alone and in place: the same bits
    alone = m.rope(q.cuda(), p, c, layout=layout, inverse=inverse, q_at=at)
    q1, k1 = q.cuda(), k.cuda()
    r = m.rope(q1, p, c, k1, layout=layout, inverse=inverse, q_at=at, q_out=q1, k_out=k1)
    assert r[0] is q1 and torch.equal(alone, qo) and torch.equal(q1, qo) and torch.equal(k1, ko)
    assert m.read_device_errors() == 0


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,H,Hk,D,R,at", [(1, 1, 1, 64, 64, 0), (5, 3, 2, 96, 64, 32), (2, 64, 64, 128, 128, 0), (3, 1, 7, 1024, 512, 256), (4, 90, 1, 1024, 8, 1016),
                                           (4099, 56, 8, 128, 128, 0), (4099, 60, 4, 136, 64, 8)])
def test_keys_of_the_queries_shape(m, dt, layout, T, H, Hk, D, R, at):
    """Up to tensors larger than the L2."""
    g = torch.Generator(device="cuda").manual_seed(T + H)
    q, k = torch.randn((T, H, D), generator=g, device="cuda").to(dt), torch.randn((T, Hk, D), generator=g, device="cuda").to(dt)
    pos, tab = torch.randint(0, 5000, (T,), generator=g, device="cuda"), table(5000, R).cuda()
    qo, ko = m.rope(q, pos, tab, k, layout=layout, q_at=at, k_at=at)
    some = torch.randint(0, T, (min(T, 64),), generator=g, device="cuda") if T > 64 else torch.arange(T, device="cuda")
    some[-1] = T - 1
    for got, x in ((qo, q), (ko, k)):
        xs, ps = x[some].cpu(), pos[some].cpu()
        near(got[some], turned(xs, ps, tab.cpu(), layout, at), xs, layout, at, R)
    # each alone, in place, and from a table that is not aligned to pieces: the same bits
    odd = torch.empty(tab.numel() + 1, device="cuda")[1:].view_as(tab).copy_(tab)
    assert torch.equal(m.rope(q, pos, tab, layout=layout, q_at=at), qo) and torch.equal(m.rope(k, pos, odd, layout=layout, q_at=at), ko)
    assert torch.equal(m.rope(q, pos, odd, layout=layout, q_at=at), qo)
    m.rope(q, pos, tab, k, layout=layout, q_at=at, k_at=at, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and m.read_device_errors() == 0


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_slices_of_one_buffer(m, layout):
    """q and k as strided slices of a fused projection, in place; what lies between stays."""
    T, H, Hk, D = 21, 6, 2, 128
    buf = torch.randn((T, (H + 2 * Hk) * D + 8)).bfloat16()
    pos, tab = torch.randint(0, 999, (T,)), table(999, 64)
    d = buf.cuda()
    view = lambda b: (b[:, :H * D].unflatten(1, (H, D)), b[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D)))
    q, k = view(d)
    m.rope(q, pos.cuda(), tab.cuda(), k, layout=layout, q_out=q, k_out=k)
    for got, x in zip(view(d), view(buf)):
        near(got, turned(x, pos, tab, layout, 64), x, layout, 64, 64)
    assert torch.equal(d[:, (H + Hk) * D:].cpu(), buf[:, (H + Hk) * D:])


def test_inverse_is_the_gradient(m):
    """d/dx of <w, rope(x)> is the inverse of w: against differences of the rotation itself, in fp32."""
    T, H, D, R = 4, 2, 24, 16
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn((T, H, D), generator=g), torch.randn((T, H, D), generator=g)
    pos, tab = torch.randint(0, 77, (T,), generator=g).cuda(), table(77, R).cuda()
    for layout in ("interleaved", "half"):
        grad = m.rope(w.cuda(), pos, tab, layout=layout, inverse=True).cpu().double()
        f = lambda v: m.rope(v.cuda(), pos, tab, layout=layout).cpu().double()
        for _ in range(20):
            t, h, d = (int(torch.randint(0, n, (), generator=g)) for n in (T, H, D))
            e = torch.zeros_like(x)
            e[t, h, d] = 0.5
            slope = ((f(x + e) - f(x - e)) * w.double()).sum()          # linear: the step may be large
            assert abs(float(slope - grad[t, h, d])) <= 1e-5 * float(w.abs().max() * 4)
        # and back again: the rotation's inverse, up to the rounding of either
        assert torch.allclose(m.rope(f(x).float().cuda(), pos, tab, layout=layout, inverse=True).cpu(), x, atol=4 * 2.0 ** -22)


def test_positions_out_of_range_are_clamped(m):
    x, tab = torch.randn((4, 1, 64)), table(10, 64)
    got = m.rope(x.cuda(), torch.tensor([-1, 10, 2 ** 40, 3]).cuda(), tab.cuda())
    near(got, turned(x, torch.tensor([0, 9, 9, 3]), tab, "interleaved", 0), x, "interleaved", 0, 64)
    assert m.read_device_errors() == 8


def test_no_tokens_and_rows_past_32_bits(m):
    c = table(16, 64).cuda()
    assert m.rope(torch.empty((0, 4, 64), device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), c).shape == (0, 4, 64)
    big = torch.empty((70000, 1, 65536), dtype=torch.bfloat16, device="cuda")      # 9 GB: rows of 64 values far apart
    q = big[:, :, :64]
    q.copy_(torch.randn((70000, 1, 64), device="cuda"))
    before = q.cpu().clone()
    pos = torch.arange(70000, device="cuda") % 16
    m.rope(q, pos, c, q_out=q)
    near(q, turned(before, pos.cpu(), c.cpu(), "interleaved", 0), before, "interleaved", 0, 64)


def test_captured_on_another_stream(m):
    x, pos, tab = torch.randn((5, 3, 64), device="cuda"), torch.arange(5, device="cuda"), table(9, 64).cuda()
    out = torch.empty_like(x)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        m.rope(x, pos, tab, q_out=out)
    for _ in range(2):
        x.normal_()
        g.replay()
        assert torch.equal(out, m.rope(x, pos, tab))


# ------------------------------------------------------------------------------------------ the table

def frequencies(R, base, scaling, factor, original, fast, slow):
    i = np.arange(R // 2)
    g = base ** (-2.0 * i / R)
    if scaling == "linear":
        return g / factor
    if scaling == "ntk":
        return (base * factor ** (R / (R - 2))) ** (-2.0 * i / R)
    if scaling == "yarn":
        turns = lambda beta: R * math.log(original / (2 * math.pi * beta)) / (2 * math.log(base))
        lo, hi = max(math.floor(turns(fast)), 0), min(math.ceil(turns(slow)), R - 1)
        r = np.clip((i - lo) / (hi - lo if hi > lo else 0.001), 0, 1)
        return g * (1 - r) + g / factor * r
    return g


@pytest.mark.parametrize("scaling,kw", [(None, {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)), ("yarn", dict(factor=32.0, original=4096)),
                                        ("yarn", dict(factor=2.0, original=7, beta_fast=1.0, beta_slow=1.0, attn_scale=1.5))])
@pytest.mark.parametrize("n,R,base", [(1, 2, 10000.0), (3001, 64, 10000.0), (257, 512, 5e5), (700, 30, 1e6)])
def test_table(m, scaling, kw, n, R, base):
    if scaling == "ntk" and R == 2:
        pytest.skip("refused")
    got = m.rope_table(n, R, base=base, scaling=scaling, **kw).cpu().numpy()
    f = frequencies(R, base, scaling, kw.get("factor", 1.0), kw.get("original", 0), kw.get("beta_fast", 32.0), kw.get("beta_slow", 1.0))
    scale = kw.get("attn_scale", 0.1 * math.log(kw["factor"]) + 1 if scaling == "yarn" else 1.0)
    ang = np.arange(n)[:, None] * f
    want = np.concatenate([np.cos(ang), np.sin(ang)], 1) * scale
    # rounded once to fp32; the angle is off by a few roundings in 64 bits of up to n
    assert np.all(np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -149 + scale * n * 2.0 ** -48)


def test_far_positions(m):
    """Angles of positions past 2^20, where fp32 angles are off by more than a hundredth."""
    n = (1 << 20) + 5
    got = m.rope_table(n, 64)[-5:].cpu().numpy()
    ang = np.arange(n - 5, n)[:, None] * frequencies(64, 10000.0, None, 1, 0, 0, 0)
    assert np.all(np.abs(got - np.concatenate([np.cos(ang), np.sin(ang)], 1)) <= 2.0 ** -24 + n * 2.0 ** -48)


def test_both_marshallings_give_the_same(m, monkeypatch):
    q, k = torch.randn((9, 4, 96), device="cuda").half(), torch.randn((9, 2, 64), device="cuda").half()
    pos, tab = torch.arange(9, device="cuda"), table(9, 64).cuda()
    kw = dict(layout="half", inverse=True, q_at=16)
    real, served = m._plain_step(), []

    class Counted:
        def rope(self, *a):
            r = real.rope(*a)
            served.append(r is not None)
            return r

    monkeypatch.setattr(m, "_step", Counted())
    a = (*m.rope(q, pos, tab, k, **kw), m.rope(q, pos, tab, **kw))
    assert served == [True, True]
    monkeypatch.setattr(m, "_step", m._DeclinedStep)
    b = (*m.rope(q, pos, tab, k, **kw), m.rope(q, pos, tab, **kw))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_arguments_of_keys_need_keys(m):
    x, pos, tab = torch.randn((2, 3, 64), device="cuda"), torch.arange(2, device="cuda"), table(9, 64).cuda()
    for kw in (dict(k_at=0), dict(k_out=torch.empty_like(x))):
        with pytest.raises(ValueError, match="need k"):
            m.rope(x, pos, tab, **kw)
    with pytest.raises(ValueError, match="fit"):
        m.rope(x, pos, tab, q_at=1)
    with pytest.raises(m.MLAError):        # in place one, not the other
        m.rope(x, pos, tab, x.clone(), q_out=x)
