"""The selector's kernels where offsets pass 32 bits, and attention over the selected pages of prompt rows: sampled rows
against the 64-bit forms."""
import numpy as np
import pytest
import torch

from tests import index_ref as ref
from tests.gpu_helpers import assert_attn_close, assert_lse_close, t_bf16, t_i32, t_u8
from tests.test_gpu_index import FMTS, SCORE_TOL, latent_cache, rand_bf16, table_for

pytestmark = pytest.mark.gpu

BF, U8, I32, I64 = torch.bfloat16, torch.uint8, torch.int32, torch.int64


@pytest.fixture(scope="module")
def m():
    import mla_latent_cache_attention_gb300 as mod
    mod.lib()
    yield mod
    torch.cuda.empty_cache()


def queries(rng, T, H, fmt):
    """(q on the GPU, its values)"""
    if fmt == "fp8":
        codes = ref.to_e4m3(rng.standard_normal((T, H, 576)) * 20)
        return t_u8(codes), ref.E4M3[codes] * 0.05
    bits = rand_bf16(rng, (T, H, 576))
    return t_bf16(bits), ref.bf16_to_f64(bits)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H,rows,k", [(16, [1100, 0, 301], 6), (96, [200, 1], 9)])
def test_selected_pages_of_prompt_rows(m, fmt, H, rows, k):
    """Hundreds of rows of a request, each with its own pages and its newest, partly visible one."""
    rng = np.random.default_rng(H)
    ps, lens = 64, [n + 700 if n != 1 else 65 for n in rows]
    tab, nb = table_for(rng, lens, ps)
    kv, vals = latent_cache(rng, nb, ps, fmt, 0.05)
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    T = int(cu[-1])
    q, qv = queries(rng, T, H, fmt)
    seen = ref.visible(lens, cu, T)
    blocks = np.full((T, k), -1, dtype=np.int32)
    for t, (b, vis) in enumerate(seen):
        pages = -(-vis // ps)
        old = rng.permutation(pages - 1)[:k - 1] if pages > 1 else []
        pick = np.sort(np.concatenate([old, [pages - 1]])).astype(np.int32)
        blocks[t, :len(pick)] = pick
    m.read_device_errors()
    out, lse = m.selected_decode(q, kv, t_i32(tab), t_i32(lens), t_i32(blocks), t_i32(cu), fmt=fmt, softmax_scale=192 ** -0.5,
                                 q_scale=0.05, k_scale=0.05, return_lse=True)
    assert m.read_device_errors() == 0 and bool(torch.isfinite(lse).all())
    pick = sorted({0, 1, rows[0] - 1, T - 1} | set(rng.integers(0, T, 24).tolist()))
    want_o, want_l = [], []
    for t in pick:
        b, vis = seen[t]
        ent = np.array([vals[tab[b, c], j] for c in blocks[t] if c >= 0 for j in range(min(ps, vis - c * ps))])
        o, l = ref.attend(qv[t], ent.reshape(-1, 576), 192 ** -0.5)
        want_o.append(o)
        want_l.append(l)
    assert_attn_close(out[pick], np.array(want_o), f"{fmt} H={H}")
    assert_lse_close(lse[pick], np.array(want_l), f"{fmt} H={H}")


@pytest.mark.parametrize("fmt", FMTS)
def test_selected_outputs_and_queries_past_32_bits(m, fmt):
    """33000 rows of 128 heads: 2^31 and more elements of q and out."""
    rng = np.random.default_rng(1)
    T, H, ps, n = 33000, 128, 16, 16
    tab, nb = table_for(rng, [n], ps)
    kv, vals = latent_cache(rng, nb, ps, fmt, 0.05)
    few, qv = queries(rng, 8, H, fmt)
    q = few[torch.arange(T, device="cuda") % 8]
    assert T * H * 512 > 2 ** 31
    zero = torch.zeros((T, 1), dtype=I32, device="cuda")
    m.read_device_errors()
    out, lse = m.selected_decode(q, kv, t_i32(tab), torch.tensor([n + T - 1], dtype=I32, device="cuda"), zero,
                                 torch.tensor([0, T], dtype=I32, device="cuda"), fmt=fmt, softmax_scale=192 ** -0.5, q_scale=0.05, k_scale=0.05,
                                 return_lse=True)
    assert m.read_device_errors() == 0
    ent = vals[tab[0, 0]].reshape(-1, 576)
    for t in (0, 5, 16383, 32767, 32768, T - 1):
        o, l = ref.attend(qv[t % 8], ent, 192 ** -0.5)
        assert_attn_close(out[t], o, f"row {t}")
        assert_lse_close(lse[t], l, f"row {t}")
    # equal queries and pages have equal results, in every row
    o = out.view(-1, 8, H * 512)[:, :, ::37]
    assert bool((o == o[:1]).all())


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
def test_index_cache_past_32_bits(m, fmt):
    """Insert, scores, selection and gather in pages whose byte offsets pass 2^32."""
    g = torch.Generator(device="cuda").manual_seed(2)
    ps, n, Hi = 64, 300, 7
    per = -(-n // ps)
    e = 2 if fmt == "bf16" else 1
    nb = (1 << 32) // (ps * 128 * e) + 3 * per
    cache = torch.empty((nb, ps, 128), dtype=BF if e == 2 else U8, device="cuda")
    scales = None if e == 2 else torch.empty((nb, ps), device="cuda")
    pages = torch.randperm(2 * per, generator=g, device="cuda")[:per] + (nb - 2 * per)
    table = pages.to(I32).reshape(1, per)
    pos = torch.arange(n, device="cuda")
    slots = pages[pos // ps] * ps + pos % ps
    assert int(slots.min()) * 128 * e > 2 ** 32
    q, k = torch.randn((n, Hi, 128), generator=g, device="cuda").to(BF), torch.randn((n, 128), generator=g, device="cuda").to(BF)
    w = torch.rand((n, Hi), generator=g, device="cuda")
    m.read_device_errors()
    qo, wo = m.index_q_cache_insert(q, k, w, cache, scales, slots, fmt=fmt)
    lens, cu = torch.tensor([n], dtype=I32, device="cuda"), torch.tensor([0, 1], dtype=I32, device="cuda")
    back = m.index_gather(cache, scales, table, cu * n, fmt=fmt, num_tokens=n)
    keys, qk = back.cpu().double(), qo[-1:].cpu()
    if e == 2:
        assert torch.equal(back, k)
        qv = qk.double()
    else:
        # a code is off by at most 2^-4 of its value or half the smallest step, 2^-10 of a scale below amax / 224
        err = (keys - k.cpu().double()).abs()
        assert (err <= 2 ** -4 * k.cpu().double().abs() + 2 ** -10 / 224 * k.cpu().double().abs().amax(1, keepdim=True)
                + 2 ** -8 * k.cpu().double().abs()).all()
        qv = torch.from_numpy(ref.E4M3[qk.numpy()])
        codes = cache[pages].cpu().numpy()
        sc = scales[pages].cpu().numpy().astype(np.float64)
        keys = torch.from_numpy((ref.E4M3[codes] * sc[:, :, None]).reshape(-1, 128)[:n])
    got = m.index_scores(qo[-1:], wo[-1:], cache, scales, table, lens, fmt=fmt, max_context=n)[0].cpu().double()
    dot = qv[0] @ keys.t()
    ww = wo[-1].cpu().double()
    want, mag = (ww[:, None] * dot.clamp(min=0)).sum(0), (ww[:, None] * (qv[0].abs() @ keys.t().abs())).sum(0)
    assert ((got - want).abs() <= SCORE_TOL * mag).all()
    x = torch.randn((1, n), generator=g, device="cuda")
    blocks, s = m.index_select(x, lens, 20, block_table=table, page_size=ps, num_blocks=nb)
    top = x[0].topk(20).indices.sort().values
    assert torch.equal(blocks[0].long(), top) and torch.equal(s[0].long(), slots[top])
    assert m.read_device_errors() == 0


def test_scores_of_more_than_2_31_columns_in_all(m):
    """4096 rows of 560000 scores: row offsets past 2^31 elements, scored and selected."""
    g = torch.Generator(device="cuda").manual_seed(5)
    T, ps, Hi = 4096, 128, 2
    n = 560000
    assert T * n > 2 ** 31
    per = n // ps
    cache = torch.randn((per, ps, 128), generator=g, device="cuda").to(BF)
    table = torch.randperm(per, generator=g, device="cuda").to(I32).reshape(1, per)
    q, w = torch.randn((T, Hi, 128), generator=g, device="cuda").to(BF), torch.rand((T, Hi), generator=g, device="cuda")
    lens, cu = torch.tensor([n], dtype=I32, device="cuda"), torch.tensor([0, T], dtype=I32, device="cuda")
    m.read_device_errors()
    sc = m.index_scores(q, w, cache, None, table, lens, cu, fmt="bf16", max_context=n)
    keys = cache[table[0].long()].reshape(n, 128).double()
    blocks, slots = m.index_select(sc, lens, 64, cu, block_table=table, page_size=ps, num_blocks=per)
    for t in (0, 1, 3000, 3834, 3835, T - 1):
        vis = n - T + t + 1
        dot = q[t].double() @ keys[:vis].t()
        want, mag = (w[t].double()[:, None] * dot.clamp(min=0)).sum(0), (w[t].double()[:, None] * (q[t].double().abs() @ keys[:vis].abs().t())).sum(0)
        assert bool(((sc[t, :vis].double() - want).abs() <= SCORE_TOL * mag).all()), t
        val, idx = sc[t, :vis].sort(descending=True, stable=True)
        top = idx[:64].sort().values
        assert torch.equal(blocks[t].long(), top), t
        assert torch.equal(slots[t].long(), table[0].long()[top // ps] * ps + top % ps), t
    assert m.read_device_errors() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_selected_pages_of_a_cache_past_32_bits(m, fmt):
    rng = np.random.default_rng(6)
    ps, n = 64, 500
    per = -(-n // ps)
    small, vals = latent_cache(rng, per, ps, fmt, 0.05)
    width = small.shape[2]
    nb = (1 << 32) // (ps * width * small.element_size()) + per + 5
    kv = torch.empty((nb, ps, width), dtype=small.dtype, device="cuda")
    kv[nb - per:] = small
    order = rng.permutation(per)
    q, qv = queries(rng, 1, 32, fmt)
    m.read_device_errors()
    out, lse = m.selected_decode(q, kv, t_i32((order + nb - per).reshape(1, -1)), t_i32([n]), t_i32([[0, 3, per - 1]]), fmt=fmt,
                                 softmax_scale=192 ** -0.5, q_scale=0.05, k_scale=0.05, return_lse=True)
    assert m.read_device_errors() == 0
    ent = np.array([vals[order[c], j] for c in (0, 3, per - 1) for j in range(min(ps, n - c * ps))])
    o, l = ref.attend(qv[0], ent, 192 ** -0.5)
    assert_attn_close(out[0], o)
    assert_lse_close(lse[0], l)
