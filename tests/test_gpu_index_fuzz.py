"""Seeded random shapes of the selector's kernels against the plain 64-bit forms: ragged requests,
odd head counts, page sizes, block sizes, narrow tables and widths, ties, empty rows."""
import numpy as np
import pytest
import torch

from tests import test_gpu_index as base

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import mla_latent_cache_attention_gb300 as mod
    mod.lib()
    return mod


def ragged(rng, B, hi, most_rows):
    lens = [int(x) for x in rng.integers(0, hi + 1, B)]
    lens[int(rng.integers(0, B))] = hi
    rows = [int(rng.integers(0, min(most_rows, n + 2) + 1)) for n in lens]
    if sum(rows) == 0:
        rows[0] = 1
    return lens, rows


@pytest.mark.parametrize("seed", range(40))
def test_scores(m, seed):
    rng = np.random.default_rng(9000 + seed)
    B = int(rng.integers(1, 7))
    lens, rows = ragged(rng, B, int(rng.choice([1, 17, 130, 700, 1500])), int(rng.choice([1, 4, 40])))
    bt = int(rng.choice([1, 1, 16, 32, 64, 128]))
    width = None
    if rng.random() < 0.3:
        width = max(1, int(-(-max(lens) // bt) * rng.uniform(0.3, 1.0)))
    base.check_scores(m, str(rng.choice(["fp8", "bf16"])), int(rng.integers(1, 65)), rows, lens,
                      int(rng.choice([16, 32, 64, 128, 256, 384])), bt, seed=seed, width=width, pad_rows=int(rng.integers(0, 3)))
    assert m.read_device_errors() == 0


@pytest.mark.parametrize("seed", range(40))
def test_select(m, seed):
    rng = np.random.default_rng(9100 + seed)
    B = int(rng.integers(1, 6))
    bt = int(rng.choice([1, 1, 3, 16, 64]))
    lens, rows = ragged(rng, B, int(rng.choice([1, 40, 3000, 30000])) * bt, int(rng.choice([1, 3])))
    T = sum(rows) + int(rng.integers(0, 3))
    W = max(1, -(-max(lens) // bt) + int(rng.integers(-2, 5)))
    x = rng.standard_normal((T, W)).astype(np.float32)
    kind = rng.integers(0, 5)
    if kind == 1:
        x = np.round(x * 2)
    elif kind == 2:
        x[rng.random((T, W)) < 0.9] = -np.inf
    elif kind == 3:
        x = np.cumsum(np.abs(x), 1).astype(np.float32)
    elif kind == 4:
        x[rng.random((T, W)) < 0.3] = np.nan
    k = int(rng.choice([1, 5, 64, 700, 2048]))
    first = int(rng.integers(0, min(k, 4)))
    last = int(rng.integers(0, min(k - first, 4) + 1))
    slots = bool(rng.random() < 0.5) and k * bt <= 4096
    base.check_select(m, x.astype(np.float32), lens, rows, bt, k, first, last, ps=int(rng.choice([1, 16, 48, 64])), slots=slots, seed=seed)
    assert m.read_device_errors() == 0


@pytest.mark.parametrize("seed", range(24))
def test_selected(m, seed):
    rng = np.random.default_rng(9200 + seed)
    B = int(rng.integers(1, 4))
    ps = int(rng.choice([16, 32, 64, 128, 40]))
    lens, rows = ragged(rng, B, int(rng.choice([1, 100, 900])), 3)
    cu = np.concatenate([[0], np.cumsum(rows)])
    lists = []
    for b, vis in base.ref.visible(lens, cu, sum(rows)):
        pages = -(-vis // ps)
        pick = rng.permutation(pages)[: int(rng.integers(0, pages + 1))] if pages else []
        lists.append([int(p) for p in pick])
    base.check_selected(m, str(rng.choice(base.FMTS)), int(rng.choice([1, 8, 16, 24, 32, 96])), rows, lens, ps, lists, seed=seed,
                        stale_nan=True)


def test_tables_narrower_than_the_contexts(m):
    """Tokens whose page is not in the table: -inf scores, -1 slots, zero keys, and the flag."""
    rng = np.random.default_rng(1)
    lens = [200, 90]
    cache, vals, scales, sc = base.index_cache(rng, 9, 64, "fp8")
    tab = base.t_i32([[3, 5], [1, 7]])
    q = base.t_u8(rng.integers(0, 127, (2, 8, 128), dtype=np.uint8))
    w = torch.ones((2, 8), device="cuda")
    m.read_device_errors()
    out = m.index_scores(q, w, cache, scales, tab, base.t_i32(lens), fmt="fp8", max_context=200)
    assert m.read_device_errors() == 2
    assert torch.isneginf(out[0, 128:200]).all() and torch.isfinite(out[0, :128]).all() and torch.isfinite(out[1, :90]).all()
    _, slots = m.index_select(torch.arange(200.0, device="cuda").repeat(2, 1), base.t_i32(lens), 100, block_table=tab, page_size=64, num_blocks=9)
    assert m.read_device_errors() == 2
    assert (slots[0, 28:] == -1).all() and (slots[0, :28] >= 0).all() and (slots[1, :90] >= 0).all()
    got = m.index_gather(cache, scales, tab, base.t_i32([0, 140]), fmt="fp8", num_tokens=140)
    assert m.read_device_errors() == 2 and (got[128:] == 0).all() and (got[:128] != 0).any()


def test_outputs_that_are_views_and_single_rows(m):
    """Strided outputs, one row, one column."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((1, 300)).astype(np.float32)
    big = torch.full((4, 50), -9, dtype=torch.int32, device="cuda")
    m.index_select(base.f32(x), base.t_i32([300]), 7, blocks=big[1:2, 3:10])
    want = np.sort(np.argsort(-x[0], kind="stable")[:7])
    assert np.array_equal(big[1, 3:10].cpu().numpy(), want) and (big[0] == -9).all() and (big[1, 10:] == -9).all()
    one = torch.full((3, 1), 5, dtype=torch.int32, device="cuda")
    m.index_select(base.f32(rng.standard_normal((3, 9))), base.t_i32([1, 0, 1]), 1, blocks=one)
    assert one.cpu().tolist() == [[0], [-1], [0]]
    cache, vals, scales, sc = base.index_cache(rng, 3, 16, "fp8")
    q = base.t_u8(rng.integers(0, 127, (2, 3, 128), dtype=np.uint8))
    wide = torch.full((5, 64), 7.0, device="cuda")
    a = m.index_scores(q, torch.ones((2, 3), device="cuda"), cache, scales, base.t_i32([[0], [2]]), base.t_i32([16, 5]), fmt="fp8",
                       max_context=16, scores=wide[1:3, 10:26])
    b = m.index_scores(q, torch.ones((2, 3), device="cuda"), cache, scales, base.t_i32([[0], [2]]), base.t_i32([16, 5]), fmt="fp8", max_context=16)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1, :5], b[1, :5])
    assert (wide[1:3, :10] == 7).all() and (wide[1:3, 26:] == 7).all() and (wide[2, 15:26] == 7).all() and (wide[0] == 7).all()


def test_select_of_many_long_rows_with_ties_and_a_stride_period(m):
    """More rows than SMs hold at once; rows that repeat with a period of the sample's stride, rows of one
    value, ascending rows: the ordered way."""
    rng = np.random.default_rng(3)
    T, n, k = 500, 20000, 700
    x = rng.standard_normal((T, n)).astype(np.float32)
    x[::7] = np.tile(rng.standard_normal(20).astype(np.float32), n // 20)[:n]
    x[1::7] = 1.5
    x[2::7] = np.sort(x[2::7], 1)
    x[3::7] = np.round(x[3::7])
    t = base.f32(x)
    got = m.index_select(t, base.t_i32([n] * T), k)[0].cpu().numpy()
    order = np.argsort(-x, axis=1, kind="stable")[:, :k]
    assert np.array_equal(got, np.sort(order, 1))
