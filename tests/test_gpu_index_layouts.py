"""Layouts of the selector's tensors on the GPU, through both forms of the binding: refused on the host, or
served as the packed ones."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, U8, F32, I32, I64 = torch.bfloat16, torch.uint8, torch.float32, torch.int32, torch.int64


class Declined:
    """A marshalling that serves nothing: every call takes its Python form."""
    insert = gather = scores = select = selected = staticmethod(lambda *a: None)


@pytest.fixture(params=["C form", "Python form"])
def m(request, monkeypatch):
    import mla_latent_cache_attention_gb300 as mod
    mod.lib()
    mod._plain()
    if request.param == "Python form":
        monkeypatch.setattr(mod, "_marshal", Declined())
    return mod


def z(*s, dt):
    return torch.zeros(s, dtype=dt, device="cuda")


def test_rows_that_overlap_are_refused(m):
    """Expanded tensors and others whose rows are closer than they are long."""
    T, k, cols, W = 4, 8, 5, 40
    one = lambda n, dt: z(1, n, dt=dt).expand(T, -1)
    q, w, c, s = z(T, 2, 128, dt=U8), z(T, 2, dt=F32), z(3, 16, 128, dt=U8), z(3, 16, dt=F32)
    lens, cu, good = z(T, dt=I32), z(T + 1, dt=I32), z(T, cols, dt=I32)
    refused = lambda what: pytest.raises(m.MLAError, match=what)
    with refused("block_table"):
        m.index_gather(c, s, one(cols, I32), cu, fmt="fp8", num_tokens=3)
    with refused("block_table"):
        m.index_scores(q, w, c, s, one(cols, I32), lens, fmt="fp8", max_context=W)
    for out in (one(W, F32), torch.as_strided(z(500, dt=F32), (T, W), (W - 1, 1))):
        with refused("scores rows"):
            m.index_scores(q, w, c, s, good, lens, fmt="fp8", max_context=W, scores=out)
        with refused("scores rows"):
            m.index_select(out, lens, k)
    x = z(T, W, dt=F32)
    with refused("blocks rows"):
        m.index_select(x, lens, k, blocks=one(k, I32))
    with refused("slots rows"):
        m.index_select(x, lens, k, block_table=good, page_size=16, num_blocks=3, slots=one(k, I32))
    with refused("block_table"):
        m.index_select(x, lens, k, block_table=one(cols, I32), page_size=16, num_blocks=3)
    dec = lambda t, b: m.selected_decode(z(T, 2, 576, dt=BF), z(3, 16, 576, dt=BF), t, lens, b, fmt="bf16", softmax_scale=1.0)
    with refused("blocks rows"):
        dec(good, one(k, I32))
    with refused("block_table"):
        dec(one(cols, I32), torch.full((T, k), -1, dtype=I32, device="cuda"))
    assert m.read_device_errors() == 0


def test_rows_further_apart_than_they_are_long(m):
    """Every row tensor as a part of a wider one."""
    g = torch.Generator(device="cuda").manual_seed(3)
    T, k, cols, W, ps = 5, 6, 4, 40, 16
    wide = lambda t, by: torch.nn.functional.pad(t, (0, by), value=7)[:, :t.shape[1]]
    x = torch.randn((T, W), generator=g, device="cuda")
    table = torch.randint(0, 20, (T, cols), generator=g, device="cuda", dtype=I32)
    lens = torch.tensor([40, 1, 17, 33, 0], dtype=I32, device="cuda")
    a = m.index_select(x, lens, k, block_table=table, page_size=ps, num_blocks=20)
    b = m.index_select(wide(x, 3), lens, k, block_table=wide(table, 2), page_size=ps, num_blocks=20, blocks=wide(a[0] * 0, 5),
                       slots=wide(a[1] * 0, 1))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    q, w = torch.randn((T, 3, 128), generator=g, device="cuda").to(BF), torch.rand((T, 3), generator=g, device="cuda")
    c = torch.randn((20, ps, 128), generator=g, device="cuda").to(BF)
    s = z(T, W, dt=F32)
    m.index_scores(q, w, c, None, table, lens, fmt="bf16", max_context=W, scores=s)
    t = wide(z(T, W, dt=F32), 9)
    m.index_scores(q, wide(w, 1), c, None, wide(table, 3), lens, fmt="bf16", max_context=W, scores=t)
    assert torch.equal(s, t)
    pages = a[0] // ps
    pages = torch.where(a[0] >= 0, pages, -1)[:, :1].contiguous()
    kv, mq = torch.randn((20, ps, 576), generator=g, device="cuda").to(BF), torch.randn((T, 2, 576), generator=g, device="cuda").to(BF)
    o = m.selected_decode(mq, kv, table, lens, pages, fmt="bf16", softmax_scale=0.1)[0]
    p = m.selected_decode(mq, kv, wide(table, 2), lens, wide(pages, 4), fmt="bf16", softmax_scale=0.1)[0]
    assert torch.equal(o, p)
    cu = torch.tensor([0, 3, 4, 8, 8, 8], dtype=I32, device="cuda")
    assert torch.equal(m.index_gather(c, None, table, cu, fmt="bf16", num_tokens=8),
                       m.index_gather(c, None, wide(table, 2), cu, fmt="bf16", num_tokens=8, dst=wide(z(8, 128, dt=BF), 4)))
    assert m.read_device_errors() == 0


@pytest.mark.parametrize("fmt,H", [("bf16", 16), ("fp8", 64), ("fp8_ds_mla", 96)])
def test_one_workspace_for_a_batch_that_shrinks(m, fmt, H):
    """A workspace for 160 rows serves every smaller batch, with the results of a workspace of its own."""
    g = torch.Generator(device="cuda").manual_seed(H)
    ps, k, nb, most = 64, 16, 40, 160
    if fmt == "bf16":
        kv = torch.randn((nb, ps, 576), generator=g, device="cuda").to(BF)
    else:
        kv = torch.randint(0, 0x60, (nb, ps, 576), generator=g, device="cuda", dtype=torch.int32).to(U8)
        if fmt == "fp8_ds_mla":
            sc = torch.full((nb, ps, 4), 0.01, device="cuda").view(U8)
            kv = torch.cat([kv[..., :512], sc, torch.randn((nb, ps, 64), generator=g, device="cuda").to(BF).view(U8)], -1).contiguous()
    q = torch.randn((most, H, 576), generator=g, device="cuda").to(BF)
    if fmt == "fp8":
        q = torch.randint(0, 0x40, (most, H, 576), generator=g, device="cuda", dtype=torch.int32).to(U8)
    table = torch.randint(0, nb, (most, 20), generator=g, device="cuda", dtype=I32)
    lens = torch.randint(1, 20 * ps, (most,), generator=g, device="cuda", dtype=I32)
    pages = torch.arange(k, device="cuda", dtype=I32).expand(most, k)
    pages = torch.where(pages * ps < lens[:, None], pages, -1)
    ws = torch.empty(m.selected_decode_workspace_bound(fmt, most, k, ps, H), dtype=U8, device="cuda")
    for T in (160, 153, 152, 100, 64, 33, 32, 17, 8, 3, 1):
        run = lambda **kw: m.selected_decode(q[:T], kv, table[:T], lens[:T], pages[:T], fmt=fmt, softmax_scale=0.01, return_lse=True, **kw)
        (a, la), (b, lb) = run(workspace=ws), run()
        assert torch.equal(a, b) and torch.equal(la, lb), T
    assert m.read_device_errors() == 0


def test_scores_without_columns_select_nothing(m):
    """A step of which no request has a context yet: scores of width 0, rows of -1."""
    T, k = 3, 4
    cu = torch.tensor([0, 2, 3], dtype=I32, device="cuda")
    lens = z(2, dt=I32)
    sc = m.index_scores(z(T, 4, 128, dt=U8), z(T, 4, dt=F32), z(2, 16, 128, dt=U8), z(2, 16, dt=F32), z(2, 3, dt=I32), lens, cu,
                        fmt="fp8", max_context=0)
    assert sc.shape == (T, 0)
    for bt in (1, 16):
        for table in (z(2, 3, dt=I32), z(2, 0, dt=I32)):
            blocks, slots = m.index_select(sc, lens, k, cu, block_tokens=bt, first=1, last=1, block_table=table, page_size=16, num_blocks=2)
            assert blocks.tolist() == [[-1] * k] * T and slots.tolist() == [[-1] * (k * bt)] * T
    blocks, none = m.index_select(sc, lens, k, cu)
    assert blocks.tolist() == [[-1] * k] * T and none is None
    # keys that the width leaves out
    blocks, _ = m.index_select(sc, lens + 40, k, cu)
    assert blocks.tolist() == [[-1] * k] * T
    out, lse = m.selected_decode(z(T, 2, 576, dt=BF), z(2, 16, 576, dt=BF), z(2, 3, dt=I32), lens, blocks, cu, fmt="bf16",
                                 softmax_scale=1.0, return_lse=True)
    assert not out.any() and torch.isneginf(lse).all()
    assert m.read_device_errors() == 0


def test_caches_of_another_format_are_refused(m):
    q, t, n, b = z(2, 4, 576, dt=BF), z(2, 5, dt=I32), z(2, dt=I32), torch.full((2, 2), -1, dtype=I32, device="cuda")
    run = lambda fmt, kv: m.selected_decode(z(2, 4, 576, dt=U8) if fmt == "fp8" else q, kv, t, n, b, fmt=fmt, softmax_scale=1.0)
    for fmt, dt, w in (("fp8", BF, 576), ("fp8_ds_mla", BF, 576), ("fp8_ds_mla", U8, 576), ("bf16", U8, 576), ("bf16", BF, 512), ("fp8", U8, 512)):
        with pytest.raises((ValueError, TypeError), match="kv_cache"):
            run(fmt, z(3, 16, 1200, dt=dt)[..., :w])
    for fmt, dt, w in (("fp8", U8, 576), ("fp8_ds_mla", U8, 656), ("bf16", U8, 1152), ("bf16", BF, 576)):
        assert not run(fmt, z(3, 16, 1200, dt=dt)[..., :w])[0].any()
    assert m.read_device_errors() == 0


def test_single_rows_of_transposed_tensors(m):
    """One row and one index head as transposes of columns give: the stride of the row is 1."""
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    thin = lambda t: t.reshape(-1, 1).contiguous().t()           # [1, n], strides (1, 1)
    x, w, k = thin(r(40)), thin(r(3)), thin(r(128).to(BF))
    assert x.stride() == (1, 1)
    lens, table = torch.tensor([40], dtype=I32, device="cuda"), thin(torch.tensor([2, 0, 1], dtype=I32, device="cuda"))
    a = m.index_select(x, lens, 6, block_table=table, page_size=16, num_blocks=3)
    b = m.index_select(x.clone(memory_format=torch.contiguous_format).reshape(1, 40), lens, 6, block_table=table.reshape(1, 3),
                       page_size=16, num_blocks=3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    q = r(1, 3, 128).to(BF)
    res = []
    for kk, ww in ((k, w), (k.reshape(1, 128).clone(), w.reshape(1, 3).clone())):
        c, s = z(3, 16, 128, dt=U8), z(3, 16, dt=F32)
        slot = torch.tensor([37], dtype=I64, device="cuda")
        qo, wo = m.index_q_cache_insert(q, kk, ww, c, s, slot, fmt="fp8")
        sc = m.index_scores(qo, wo if ww is not w else thin(wo[0]), c, s, table, lens, fmt="fp8", max_context=40)
        res.append([qo, wo, c, s, sc])
    assert all(torch.equal(i, j) for i, j in zip(*res))
    assert m.read_device_errors() == 0


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("Hi,bt", [(5, 1), (21, 1), (33, 16), (5, 64)])
def test_scores_do_not_depend_on_what_lies_beside_a_key(m, fmt, Hi, bt):
    """The same keys with NaN or zeros in the unwritten rest of their page, and with a NaN key among them: every other
    key has the same bits."""
    g = torch.Generator(device="cuda").manual_seed(Hi)
    n, ps = 200, 64
    table, lens = torch.tensor([[3, 1, 0, 2]], dtype=I32, device="cuda"), torch.tensor([n], dtype=I32, device="cuda")
    w = torch.randn((1, Hi), generator=g, device="cuda")
    if fmt == "bf16":
        c, s, nan = torch.randn((4, ps, 128), generator=g, device="cuda").to(BF), None, float("nan")
        q = torch.randn((1, Hi, 128), generator=g, device="cuda").to(BF)
    else:
        code = lambda *shape: (torch.randint(0, 0x50, shape, generator=g, device="cuda", dtype=I32)
                               + 128 * torch.randint(0, 2, shape, generator=g, device="cuda", dtype=I32)).to(U8)
        c, s, nan = code(4, ps, 128), torch.rand((4, ps), generator=g, device="cuda"), 0x7F
        q = code(1, Hi, 128)
    c[2, n - 192:] = 0
    run = lambda c: m.index_scores(q, w, c, s, table, lens, fmt=fmt, block_tokens=bt, max_context=n)
    want = run(c)
    tail = c.clone()
    tail[2, n - 192:] = nan
    assert torch.equal(run(tail), want)
    tail[1, 5] = nan            # position 69
    got = run(tail)
    at = 69 // bt
    assert torch.isnan(got[0, at]) and torch.equal(torch.cat([got[0, :at], got[0, at + 1:]]), torch.cat([want[0, :at], want[0, at + 1:]]))
    assert m.read_device_errors() == 0


@pytest.mark.parametrize("fmt,H", [("bf16", 16), ("bf16", 40), ("fp8", 16), ("fp8", 32), ("fp8", 64), ("fp8_ds_mla", 96)])
@pytest.mark.parametrize("ps", [64, 48])
def test_selected_rows_do_not_depend_on_what_lies_beside_them(m, fmt, H, ps):
    """The same bits with NaN or zeros in the unwritten rest of a page, and beside rows of other lengths."""
    g = torch.Generator(device="cuda").manual_seed(H)
    n, T = 11 * ps + 5, 6
    if fmt == "bf16":
        kv, nan = torch.randn((20, ps, 576), generator=g, device="cuda").to(BF), float("nan")
    else:
        code = torch.randint(0, 0x50, (20, ps, 576), generator=g, device="cuda", dtype=I32)
        kv, nan = (code + 128 * torch.randint(0, 2, (20, ps, 576), generator=g, device="cuda", dtype=I32)).to(U8), 0x7F
        if fmt == "fp8_ds_mla":
            sc = torch.rand((20, ps, 4), generator=g, device="cuda").view(U8)
            kv, nan = torch.cat([kv[..., :512], sc, torch.randn((20, ps, 64), generator=g, device="cuda").to(BF).view(U8)], -1).contiguous(), 0xFF
    q = torch.randn((T, H, 576), generator=g, device="cuda").to(BF)
    if fmt == "fp8":
        q = torch.randint(0, 0x40, (T, H, 576), generator=g, device="cuda", dtype=I32).to(U8)
    table = torch.randperm(20, generator=g, device="cuda").to(I32)[:12].expand(T, 12).contiguous()
    lens = torch.tensor([n, n, 1, n, 3 * ps, n], dtype=I32, device="cuda")
    pages = torch.tensor([[0, 3, 4, 11]] * 2 + [[0, -1, -1, -1]] + [[11, 0, 7, 9], [2, 1, -1, -1], [11, -1, -1, -1]], dtype=I32, device="cuda")
    run = lambda kv, lens=lens, pages=pages: m.selected_decode(q, kv, table, lens, pages, fmt=fmt, softmax_scale=0.02, return_lse=True)
    out, lse = run(kv)
    assert bool(torch.isfinite(out).all() and torch.isfinite(lse).all())
    for v in (nan, 0):
        stale = kv.clone()
        last = int(table[0, 11])
        stale[last, 5:] = v             # past the contexts' end
        o, l = run(stale)
        assert torch.equal(o, out) and torch.equal(l, lse)
    # other rows of other lengths, and none: the first row's bits stay
    o, l = run(kv, lens=torch.tensor([n, 0, 5, 2, 0, 1], dtype=I32, device="cuda"),
               pages=torch.tensor([[0, 3, 4, 11], [-1] * 4, [0, -1, -1, -1], [0, -1, -1, -1], [-1] * 4, [0, -1, -1, -1]], dtype=I32, device="cuda"))
    assert torch.equal(o[0], out[0]) and torch.equal(l[0], lse[0])
    assert m.read_device_errors() == 0


def test_rows_before_and_after_the_requests(m):
    """Rows ahead of cu_q_lens[0] and behind its last entry: left as they are (zeros and -inf from the attention)."""
    g = torch.Generator(device="cuda").manual_seed(9)
    T, ps = 7, 16
    cu, lens = torch.tensor([2, 4, 5], dtype=I32, device="cuda"), torch.tensor([20, 9], dtype=I32, device="cuda")
    table = torch.tensor([[2, 0], [1, 3]], dtype=I32, device="cuda")
    cache = torch.randn((4, ps, 128), generator=g, device="cuda").to(BF)
    q, w = torch.randn((T, 3, 128), generator=g, device="cuda").to(BF), torch.rand((T, 3), generator=g, device="cuda")
    sc = torch.full((T, 20), 5.0, device="cuda")
    m.index_scores(q, w, cache, None, table, lens, cu, fmt="bf16", max_context=20, scores=sc)
    want = m.index_scores(q[2:5].contiguous(), w[2:5], cache, None, table, lens, cu - 2, fmt="bf16", max_context=20, scores=sc[2:5].clone())
    outside = [0, 1, 5, 6]
    assert torch.equal(sc[2:5], want) and bool((sc[outside] == 5).all())
    blocks, slots = torch.full((T, 4), 77, dtype=I32, device="cuda"), torch.full((T, 4), 78, dtype=I32, device="cuda")
    m.index_select(sc, lens, 4, cu, block_table=table, page_size=ps, num_blocks=4, blocks=blocks, slots=slots)
    b, s = m.index_select(sc[2:5], lens, 4, cu - 2, block_table=table, page_size=ps, num_blocks=4)
    assert torch.equal(blocks[2:5], b) and torch.equal(slots[2:5], s)
    assert bool((blocks[outside] == 77).all()) and bool((slots[outside] == 78).all())
    kv, mq = torch.randn((4, ps, 576), generator=g, device="cuda").to(BF), torch.randn((T, 2, 576), generator=g, device="cuda").to(BF)
    pages = torch.zeros((T, 1), dtype=I32, device="cuda")
    o, l = m.selected_decode(mq, kv, table, lens, pages, cu, fmt="bf16", softmax_scale=0.1, return_lse=True)
    p, k = m.selected_decode(mq[2:5].contiguous(), kv, table, lens, pages[2:5], cu - 2, fmt="bf16", softmax_scale=0.1, return_lse=True)
    assert torch.equal(o[2:5], p) and torch.equal(l[2:5], k)
    assert not o[outside].any() and bool(torch.isneginf(l[outside]).all())
    dst = torch.full((9, 128), 3.0, device="cuda").to(BF)
    m.index_gather(cache, None, table, cu, fmt="bf16", num_tokens=9, dst=dst)
    assert torch.equal(dst[2:5], torch.stack([cache[2, 0], cache[2, 1], cache[1, 0]]))
    assert bool((dst[:2] == 3).all() and (dst[5:] == 3).all())
    assert m.read_device_errors() == 0
