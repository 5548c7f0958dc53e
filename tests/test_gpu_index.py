"""GPU parity of the selector in front of sparse attention against plain 64-bit forms: the index
insert and gather bit for bit, the selection index for index, the scores within the bound of their
fp32 sums, the decode over selected pages within the attention tolerance; then a run of them
together, on other streams and in captured graphs."""
import numpy as np
import pytest
import torch

from mla_latent_cache_attention_gb300 import synth
from tests import index_ref as ref
from tests.gpu_helpers import assert_attn_close, assert_lse_close, bf16_bits, t_bf16, t_i32, t_i64, t_u8

pytestmark = pytest.mark.gpu

# fp32 sums: 128 products of a head (each step may truncate, 2^-23), then 64 weighted terms and the
# key's scale (2^-24 each), relative to the sum of the absolute terms
SCORE_TOL = 128 * 2.0 ** -23 + 66 * 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    import mla_latent_cache_attention_gb300 as mod
    mod.lib()
    return mod


def f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def rand_bf16(rng, shape, scale=1.0):
    return ref.to_bf16_bits(rng.standard_normal(shape) * scale)


def index_cache(rng, nb, ps, fmt):
    """(stored cache, values, scales or None, scale per key)"""
    if fmt == "bf16":
        bits = rand_bf16(rng, (nb, ps, 128))
        return t_bf16(bits), ref.bf16_to_f64(bits), None, np.ones((nb, ps))
    codes = rng.integers(0, 256, (nb, ps, 128), dtype=np.uint8)
    codes[(codes & 127) == 127] = 0x30
    sc = np.exp2(rng.integers(-6, 4, (nb, ps))).astype(np.float32)
    return t_u8(codes), ref.E4M3[codes], f32(sc), sc.astype(np.float64)


def table_for(rng, lens, ps, extra=2):
    per = [-(-int(n) // ps) for n in lens]
    nb = sum(per) + extra
    ids = rng.permutation(nb)
    w = max(1, max(per))
    tab = np.zeros((len(lens), w), dtype=np.int32)
    at = 0
    for b, n in enumerate(per):
        tab[b, :n] = ids[at:at + n]
        at += n
    return tab, nb


# ------------------------------------------------------------------------------------------ insert

def insert_case(rng, T, Hi, pad=0):
    q = rand_bf16(rng, (T, Hi, 128), 3.0)
    k = rand_bf16(rng, (T, 128), 0.2)
    w = rng.standard_normal((T, Hi)).astype(np.float32)
    if T > 2:
        q[1, 0] = 0                                            # a zero vector: scale 1
        k[2] = 0
        q[0, Hi - 1] = ref.to_bf16_bits(rng.standard_normal(128) * 1e-30)
    return q, k, w


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("T,Hi,ps", [(1, 1, 16), (3, 5, 64), (33, 64, 64), (7, 31, 48), (130, 16, 128)])
@pytest.mark.parametrize("rope", [True, False])
def test_insert_bit_exact(m, fmt, T, Hi, ps, rope):
    rng = np.random.default_rng(T * 100 + Hi + rope)
    q, k, w = insert_case(rng, T, Hi)
    nb = -(-T // ps) + 2
    slots = rng.permutation(nb * ps)[:T].astype(np.int64)
    if T > 3:
        slots[3] = -1                                          # not inserted
    pos = rng.integers(0, 500, T).astype(np.int64)
    cs = synth.cos_sin_table(512).astype(np.float32)
    cache, vals, scales, _ = index_cache(rng, nb, ps, fmt)
    before = cache.clone()
    qo, wo = m.index_q_cache_insert(t_bf16(q), t_bf16(k), f32(w), cache, scales, t_i64(slots), fmt=fmt, weight_scale=0.37,
                                    positions=t_i64(pos) if rope else None, cos_sin_cache=f32(cs) if rope else None)
    row = cs[pos] if rope else None
    yq = ref.rotate(ref.bf16_to_f64(q), None if row is None else row[:, None])
    yk = ref.rotate(ref.bf16_to_f64(k), row)
    ws = w * np.float32(0.37)
    flat = cache.reshape(nb * ps, 128)
    keep = np.ones(nb * ps, dtype=bool)
    for t in range(T):
        if slots[t] >= 0:
            keep[slots[t]] = False
    keep_t = torch.from_numpy(np.flatnonzero(keep)).cuda()
    assert torch.equal(flat[keep_t].view(torch.uint8), before.reshape(nb * ps, 128)[keep_t].view(torch.uint8))
    live = slots >= 0
    at = t_i64(slots[live])
    if fmt == "bf16":
        assert np.array_equal(bf16_bits(qo), ref.to_bf16_bits(yq))
        assert np.array_equal(bf16_bits(flat[at]), ref.to_bf16_bits(yk[live]))
        assert np.array_equal(wo.cpu().numpy(), ws)
    else:
        cq, sq = ref.quantise(yq)
        ck, sk = ref.quantise(yk)
        assert np.array_equal(qo.cpu().numpy(), cq)
        assert np.array_equal(flat[at].cpu().numpy(), ck[live])
        assert np.array_equal(scales.reshape(-1)[at].cpu().numpy(), sk[live].astype(np.float32))
        assert np.array_equal(wo.cpu().numpy(), ws * sq.astype(np.float32))
    assert m.read_device_errors() == 0


def test_insert_strided_inputs_and_padded_cache(m):
    """Rows that are slices of wider tensors (also off the 16-byte grid) and a cache with padded keys."""
    rng = np.random.default_rng(5)
    T, Hi, ps, nb = 9, 7, 16, 3
    q, k, w = insert_case(rng, T, Hi)
    slots = rng.permutation(nb * ps)[:T].astype(np.int64)
    wide_q, wide_k = np.zeros((T, Hi, 131), np.uint16), np.zeros((T, 200), np.uint16)
    wide_q[:, :, 3:], wide_k[:, 5:133] = q, k
    wide_w = np.zeros((T, Hi + 4), np.float32)
    wide_w[:, :Hi] = w
    big = torch.full((nb, ps, 144), 9, dtype=torch.uint8, device="cuda")
    sc = torch.full((nb, ps + 4), -1.0, device="cuda")
    qo, wo = m.index_q_cache_insert(t_bf16(wide_q)[:, :, 3:], t_bf16(wide_k)[:, 5:133], f32(wide_w)[:, :Hi], big[:, :, :128],
                                    sc[:, :ps], t_i64(slots), fmt="fp8")
    cq, sq = ref.quantise(ref.bf16_to_f64(q).astype(np.float32))
    ck, sk = ref.quantise(ref.bf16_to_f64(k).astype(np.float32))
    assert np.array_equal(qo.cpu().numpy(), cq) and np.array_equal(wo.cpu().numpy(), w * sq.astype(np.float32))
    got, gs = big.cpu().numpy().reshape(nb * ps, 144), sc.cpu().numpy()
    assert np.array_equal(got[slots, :128], ck) and (got[:, 128:] == 9).all()
    assert np.array_equal(gs[:, :ps].reshape(-1)[slots], sk.astype(np.float32)) and (gs[:, ps:] == -1).all()


def test_insert_bad_slot_and_position_are_reported(m):
    rng = np.random.default_rng(6)
    q, k, w = insert_case(rng, 2, 3)
    cache, _, scales, _ = index_cache(rng, 2, 16, "fp8")
    before, cs = cache.clone(), f32(synth.cos_sin_table(32))
    m.read_device_errors()
    m.index_q_cache_insert(t_bf16(q), t_bf16(k), f32(w), cache, scales, t_i64([2 * 16, 10 ** 12]), fmt="fp8")
    assert m.read_device_errors() == 4 and torch.equal(cache, before)
    q1, _ = m.index_q_cache_insert(t_bf16(q), t_bf16(k), f32(w), cache, scales, t_i64([-1, -1]), fmt="fp8",
                                   positions=t_i64([-5, 99]), cos_sin_cache=cs)
    assert m.read_device_errors() == 8
    q2, _ = m.index_q_cache_insert(t_bf16(q), t_bf16(k), f32(w), cache, scales, t_i64([-1, -1]), fmt="fp8",
                                   positions=t_i64([0, 31]), cos_sin_cache=cs)
    assert torch.equal(q1, q2) and m.read_device_errors() == 0


# ------------------------------------------------------------------------------------------ gather

@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("ps", [16, 64, 100])
def test_gather_bit_exact(m, fmt, ps):
    rng = np.random.default_rng(ps)
    lens = [130, 0, 1, 700, 64]
    tab, nb = table_for(rng, lens, ps)
    cache, vals, scales, sc = index_cache(rng, nb, ps, fmt)
    starts = np.array([3, 0, 0, 250, 63], dtype=np.int32)
    take = [127, 0, 1, 450, 1]
    cu = np.concatenate([[0], np.cumsum(take)]).astype(np.int32)
    n = int(cu[-1])
    dst = torch.full((n + 3, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    m.index_gather(cache, scales, t_i32(tab), t_i32(cu), t_i32(starts), fmt=fmt, num_tokens=n + 3, dst=dst)
    want = []
    for b in range(len(lens)):
        for i in range(take[b]):
            p = int(starts[b]) + i
            want.append((vals * sc[:, :, None])[tab[b, p // ps], p % ps])
    assert np.array_equal(bf16_bits(dst[:n]), ref.to_bf16_bits(np.array(want)))
    assert torch.all(dst[n:] == 7.0) and m.read_device_errors() == 0
    odd = torch.zeros((n, 131), dtype=torch.bfloat16, device="cuda")
    m.index_gather(cache, scales, t_i32(tab), t_i32(cu), t_i32(starts), fmt=fmt, num_tokens=n, dst=odd[:, 1:129])
    assert torch.equal(odd[:, 1:129], dst[:n]) and torch.all(odd[:, 0] == 0) and torch.all(odd[:, 129:] == 0)


def test_gather_scales_that_are_not_powers_of_two_round_once(m):
    rng = np.random.default_rng(8)
    cache, vals, _, _ = index_cache(rng, 2, 16, "fp8")
    sc = rng.uniform(0.01, 0.1, (2, 16)).astype(np.float32)
    got = m.index_gather(cache, f32(sc), t_i32([[1, 0]]), t_i32([0, 32]), fmt="fp8", num_tokens=32)
    want = (vals.astype(np.float32) * sc[:, :, None]).astype(np.float32)[[1, 0]].reshape(32, 128)
    assert np.array_equal(bf16_bits(got), ref.to_bf16_bits(want))


def test_gather_bad_pages_give_zeros_and_a_flag(m):
    rng = np.random.default_rng(9)
    cache, vals, scales, sc = index_cache(rng, 3, 16, "fp8")
    m.read_device_errors()
    got = m.index_gather(cache, scales, t_i32([[0, 3, -1]]), t_i32([0, 64]), fmt="fp8", num_tokens=64)
    assert m.read_device_errors() == 2
    assert torch.all(got[16:] == 0)
    assert np.array_equal(bf16_bits(got[:16]), ref.to_bf16_bits(vals[0] * sc[0][:, None]))


# ------------------------------------------------------------------------------------------ scores

def check_scores(m, fmt, Hi, rows, lens, ps, bt, *, seed, width=None, mangle=None, pad_rows=0, stale_nan=True):
    rng = np.random.default_rng(seed)
    tab, nb = table_for(rng, lens, ps)
    cache, vals, scales, sc = index_cache(rng, nb, ps, fmt)
    T = sum(rows) + pad_rows
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    if fmt == "bf16":
        bits = rand_bf16(rng, (T, Hi, 128))
        q, qv = t_bf16(bits), ref.bf16_to_f64(bits)
    else:
        codes = rng.integers(0, 256, (T, Hi, 128), dtype=np.uint8)
        codes[(codes & 127) == 127] = 0x31
        q, qv = t_u8(codes), ref.E4M3[codes]
    w = (rng.standard_normal((T, Hi)) * 0.1).astype(np.float32)
    if stale_nan:      # slots behind the sequences hold NaN: no visible score may see them
        seen = np.zeros((nb, ps), dtype=bool)
        for b, n in enumerate(lens):
            for j in range(int(n)):
                seen[tab[b, j // ps], j % ps] = True
        hide = torch.from_numpy(~seen).cuda()
        if fmt == "bf16":
            cache[hide] = float("nan")
        else:
            cache[hide] = 0x7F
            scales[hide] = float("nan")
    if mangle:
        mangle(tab, nb)
    width = -(-max(lens) // bt) if width is None else width
    out = torch.full((T, width + 5), 123.0, device="cuda")
    m.index_scores(q, f32(w), cache, scales, t_i32(tab), t_i32(lens), t_i32(cu), fmt=fmt, block_tokens=bt,
                   max_context=width * bt, scores=out)
    want, mag, written = ref.scores(qv, w.astype(np.float64), vals, sc, tab, lens, cu, width, bt, nb)
    got = out.cpu().numpy().astype(np.float64)
    assert (got[:, width:] == 123.0).all(), "columns past the width were written"
    got = got[:, :width]
    assert (got[~written] == 123.0).all(), "hidden columns were written"
    fin = written & np.isfinite(want)
    assert np.array_equal(got[written & ~fin], want[written & ~fin])
    err = np.abs(got[fin] - want[fin])
    assert (err <= SCORE_TOL * mag[fin] + 1e-30).all(), f"max error / bound {(err / (SCORE_TOL * mag[fin] + 1e-30)).max()}"
    return got, want


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("Hi", [1, 5, 8, 16, 31, 32, 64])
def test_scores_decode_rows(m, fmt, Hi):
    check_scores(m, fmt, Hi, [1, 1, 1, 1], [1, 129, 700, 64], 64, 1, seed=Hi)
    assert m.read_device_errors() == 0


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("bt", [1, 16, 32, 64, 128])
def test_scores_pages_and_blocks(m, fmt, ps, bt):
    check_scores(m, fmt, 32, [4, 2, 1], [517, 128, 1000], ps, bt, seed=ps + bt)
    assert m.read_device_errors() == 0


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("Hi,bt", [(64, 1), (64, 64), (24, 1), (8, 128), (3, 16)])
def test_scores_causal_chunks(m, fmt, Hi, bt):
    """Ragged prefill chunks: query tiles that end inside a request, rows with few keys, a whole prefill
    from the first token, an empty request."""
    check_scores(m, fmt, Hi, [70, 0, 33, 5], [400, 0, 33, 260], 64, bt, seed=Hi * 7 + bt)
    assert m.read_device_errors() == 0


def test_scores_rows_without_keys_and_padding_rows(m):
    """More rows than keys (the first rows see nothing), an empty request, rows of no request."""
    check_scores(m, "fp8", 16, [9, 3, 1], [4, 0, 20], 16, 1, seed=3, pad_rows=6)
    check_scores(m, "bf16", 64, [9, 3, 1], [4, 0, 20], 16, 64, seed=4, pad_rows=3)
    assert m.read_device_errors() == 0


def test_scores_are_cut_at_the_width(m):
    check_scores(m, "fp8", 64, [6, 1], [1000, 300], 64, 1, seed=11, width=333)
    check_scores(m, "bf16", 32, [6, 1], [1000, 300], 64, 64, seed=12, width=7)


def test_scores_bad_pages_are_minus_infinity(m):
    def mangle(tab, nb):
        tab[0, 1], tab[1, 0], tab[1, 4] = nb + 3, -7, nb
    for bt in (1, 64):
        m.read_device_errors()
        got, want = check_scores(m, "fp8", 32, [3, 2], [300, 333], 64, bt, seed=21 + bt, mangle=mangle)
        assert m.read_device_errors() == 2 and np.isneginf(want[np.isinf(want)]).all()


def test_scores_many_requests_and_a_long_one(m):
    rng = np.random.default_rng(31)
    lens = rng.integers(0, 300, 1300).tolist()
    check_scores(m, "fp8", 4, [1 if n else 0 for n in lens], lens, 64, 16, seed=31, stale_nan=False)
    check_scores(m, "fp8", 64, [2], [40007], 64, 1, seed=32, stale_nan=False)
    assert m.read_device_errors() == 0


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("Hi", [5, 64])
def test_scores_keep_nan_and_only_the_keys_that_hold_it(m, fmt, Hi):
    rng = np.random.default_rng(41)
    cache, vals, scales, sc = index_cache(rng, 2, 64, fmt)
    if fmt == "bf16":
        cache[0, 3, 7] = float("nan")
        q = t_bf16(rand_bf16(rng, (1, Hi, 128)))
    else:
        cache[0, 3, 7] = 0x7F
        q = t_u8(rng.integers(0, 127, (1, Hi, 128), dtype=np.uint8))
    out = m.index_scores(q, torch.ones((1, Hi), device="cuda"), cache, scales, t_i32([[0, 1]]), t_i32([100]), fmt=fmt,
                         max_context=100)
    bad = torch.isnan(out[0])
    assert bad[3] and bad.sum() == 1


def test_scores_infinite_key_with_padded_heads(m):
    """An infinite key value meets the zero rows that pad the heads: the heads alone count."""
    q = torch.ones((1, 5, 128), dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros((1, 16, 128), dtype=torch.bfloat16, device="cuda")
    cache[0, 2, 9], cache[0, 4, 9] = float("inf"), float("-inf")
    out = m.index_scores(q, torch.ones((1, 5), device="cuda"), cache, None, t_i32([[0]]), t_i32([16]), fmt="bf16", max_context=16)
    want = torch.zeros(16)
    want[2] = float("inf")
    assert torch.equal(out[0].cpu(), want)


# ------------------------------------------------------------------------------------------ select

def check_select(m, x, lens, rows, bt, k, first=0, last=0, ps=0, slots=False, seed=0, pad_rows=0):
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    tab, nb = table_for(rng, lens, ps) if slots else (None, 0)
    T = x.shape[0]
    blocks = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    sl = torch.full((T, k * bt), -9, dtype=torch.int32, device="cuda") if slots else None
    m.index_select(f32(x), t_i32(lens), k, t_i32(cu), block_tokens=bt, first=first, last=last,
                   block_table=None if tab is None else t_i32(tab), page_size=ps, num_blocks=nb, blocks=blocks, slots=sl)
    wb, ws, req = ref.select(x, lens, cu, bt, k, first, last, tab, ps, nb)
    live = np.array(req) >= 0
    got = blocks.cpu().numpy()
    assert np.array_equal(got[live], wb[live]) and (got[~live] == -9).all()
    if slots:
        gs = sl.cpu().numpy()
        assert np.array_equal(gs[live], ws[live]) and (gs[~live] == -9).all()


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 1000, 1024, 1025, 5000, 40000, 140001])
@pytest.mark.parametrize("k", [1, 7, 64, 2048])
def test_select_exact(m, n, k):
    rng = np.random.default_rng(n + k)
    x = rng.standard_normal((2, n)).astype(np.float32)
    check_select(m, x, [n, max(1, n - 3)], [1, 1], 1, k, slots=(k <= 64), ps=64, seed=n)
    assert m.read_device_errors() == 0


@pytest.mark.parametrize("kind", ["equal", "few", "signs", "inf", "nan", "tiny", "huge", "close", "zeros"])
@pytest.mark.parametrize("n,k", [(700, 64), (3000, 2048), (70000, 513)])
def test_select_ties_and_special_values(m, kind, n, k):
    rng = np.random.default_rng(n)
    x = rng.standard_normal((1, n)).astype(np.float32)
    if kind == "equal":
        x[:] = -2.5
    elif kind == "few":
        x = np.round(x).astype(np.float32)
    elif kind == "signs":
        x = np.where(rng.random((1, n)) < 0.5, np.float32(0.0), np.float32(-0.0)).astype(np.float32)
    elif kind == "inf":
        x[0, rng.integers(0, n, n // 2)] = -np.inf
        x[0, rng.integers(0, n, 5)] = np.inf
    elif kind == "nan":
        x[0, rng.permutation(n)[: n - k // 2]] = np.nan
    elif kind == "tiny":
        x *= np.float32(1e-42)
    elif kind == "huge":
        x *= np.float32(1e38)
    elif kind == "close":
        x = (1.0 + rng.integers(0, 40, (1, n)) * 2.0 ** -23).astype(np.float32)
    else:
        x[0, : n - 3] = 0
    check_select(m, x, [n], [1], 1, k, slots=True, ps=16, seed=1)


@pytest.mark.parametrize("bt,ps", [(16, 64), (64, 64), (128, 32), (1, 100), (64, 16)])
@pytest.mark.parametrize("first,last", [(0, 0), (1, 2), (3, 0), (0, 5), (4, 4)])
def test_select_blocks_forced_and_slots(m, bt, ps, first, last):
    rng = np.random.default_rng(bt + ps)
    rows, lens = [3, 0, 1, 4], [1000, 0, 5, 2 * bt + 3]
    T = sum(rows) + 2
    x = rng.standard_normal((T, -(-max(lens) // bt) + 4)).astype(np.float32)
    x[:, 0] = -np.inf
    check_select(m, x, lens, rows, bt, 8, first, last, ps=ps, slots=True, seed=bt)
    assert m.read_device_errors() == 0


def test_select_many_rows_of_a_prefill(m):
    rng = np.random.default_rng(3)
    x = np.round(rng.standard_normal((260, 2300)) * 50).astype(np.float32)
    check_select(m, x, [2300, 100], [160, 100], 1, 300, seed=2)


def test_select_ignores_what_lies_behind_a_row_and_a_narrow_width(m):
    x = np.full((2, 50), np.float32(1e30))
    x[0, :20] = np.arange(20)
    x[1, :33] = -np.arange(33)
    check_select(m, x, [20, 33], [1, 1], 1, 4)
    check_select(m, x[:, :10].copy(), [20, 33], [1, 1], 1, 4)      # scores narrower than the context


def test_select_bad_pages_are_reported(m):
    m.read_device_errors()
    _, slots = m.index_select(f32([[5, 4, 3, 2]]), t_i32([4]), 4, block_table=t_i32([[9, 1]]), page_size=2, num_blocks=4)
    assert slots.cpu().tolist() == [[-1, -1, 2, 3]] and m.read_device_errors() == 2


# ------------------------------------------------------------------------------------------ selected pages

def latent_cache(rng, nb, ps, fmt, k_scale):
    """(stored cache on the GPU, entry values [nb, ps, 576])"""
    if fmt == "bf16":
        bits = rand_bf16(rng, (nb, ps, 576))
        return t_bf16(bits), ref.bf16_to_f64(bits)
    if fmt == "fp8":
        codes = ref.to_e4m3(np.clip(rng.standard_normal((nb, ps, 576)) * 20, -400, 400))
        return t_u8(codes), ref.E4M3[codes] * k_scale
    codes = ref.to_e4m3(np.clip(rng.standard_normal((nb, ps, 512)) * 20, -400, 400))
    sc = rng.uniform(0.01, 0.1, (nb, ps, 4)).astype(np.float32)
    rope = rand_bf16(rng, (nb, ps, 64))
    rec = np.concatenate([codes, sc.view(np.uint8).reshape(nb, ps, 16), rope.view(np.uint8).reshape(nb, ps, 128)], -1)
    return t_u8(rec), np.concatenate([ref.E4M3[codes] * np.repeat(sc, 128, -1), ref.bf16_to_f64(rope)], -1)


def check_selected(m, fmt, H, rows, lens, ps, lists, *, seed, order=None, stale_nan=False, expect_err=0, pad_rows=0):
    """lists[t]: page indices of row t (ragged; padded with -1 here)."""
    rng = np.random.default_rng(seed)
    qs = ks = 0.05
    tab, nb = table_for(rng, lens, ps)
    kv, vals = latent_cache(rng, nb, ps, fmt, ks)
    T = sum(rows) + pad_rows
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    if fmt == "fp8":
        codes = ref.to_e4m3(rng.standard_normal((T, H, 576)) * 20)
        q, qv = t_u8(codes), ref.E4M3[codes] * qs
    else:
        bits = rand_bf16(rng, (T, H, 576))
        q, qv = t_bf16(bits), ref.bf16_to_f64(bits)
    if stale_nan:
        seen = np.zeros((nb, ps), dtype=bool)
        for b, n in enumerate(lens):
            for j in range(int(n)):
                seen[tab[b, j // ps], j % ps] = True
        hide = torch.from_numpy(~seen).cuda()
        if fmt == "bf16":
            kv[hide] = float("nan")
        else:
            kv[hide] = 0x7F
    k = max(1, max(len(l) for l in lists))
    blocks = np.full((T, k), -1, dtype=np.int32)
    for t, l in enumerate(lists):
        blocks[t, :len(l)] = l
    m.read_device_errors()
    out, lse = m.selected_decode(q, kv, t_i32(tab), t_i32(lens), t_i32(blocks), t_i32(cu), fmt=fmt, softmax_scale=192 ** -0.5,
                                 q_scale=qs, k_scale=ks, return_lse=True)
    assert m.read_device_errors() == expect_err
    want_o, want_l = np.zeros((T, H, 512)), np.full((T, H), -np.inf)
    for t, (b, vis) in enumerate(ref.visible(lens, cu, T)):
        ent, part = [], False
        for c in (blocks[t] if b >= 0 else []):
            if c < 0 or c * ps >= vis:
                continue
            if (c + 1) * ps > vis:
                if part:
                    continue
                part = True
            ent += [vals[tab[b, c], j] for j in range(min(ps, vis - c * ps))]
        want_o[t], want_l[t] = ref.attend(qv[t], np.array(ent).reshape(-1, 576), 192 ** -0.5)
    assert_attn_close(out, want_o, f"{fmt} H={H} ps={ps}")
    assert_lse_close(lse, want_l, f"{fmt} H={H} ps={ps}")


FMTS = ["bf16", "fp8", "fp8_ds_mla"]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H", [1, 16, 17, 96, 128])
def test_selected_heads(m, fmt, H):
    check_selected(m, fmt, H, [1, 1, 1], [500, 64, 63], 64, [[0, 3, 7], [0], [0]], seed=H)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256, 48])
def test_selected_page_sizes_causal_rows(m, fmt, ps):
    """Rows of one request end in the middle of a page, each at its own token; the second request's
    first row lists a page that only its second row sees, which is reported."""
    lens = [5 * ps + 3, 2 * ps + 1]
    lists = [[0, 2, 4], [4, 1, 0], [5, 3], [0, 1, 2, 3, 4, 5], [2], [0, 1]]
    check_selected(m, fmt, 16, [4, 2], lens, ps, lists, seed=ps, stale_nan=True, expect_err=1)


@pytest.mark.parametrize("fmt", FMTS)
def test_selected_order_duplicates_and_empty_rows(m, fmt):
    lens = [300, 300, 10]
    lists = [[4, 2, -1, 0], [-1, -1], [1, 1, 3], [], [0]]
    check_selected(m, fmt, 16, [2, 2, 1], lens, 64, lists, seed=77)


def test_selected_bad_lists_are_reported(m):
    check_selected(m, "bf16", 16, [1, 1], [100, 100], 64, [[0, 2], [1]], seed=1, expect_err=1)         # past the context
    check_selected(m, "bf16", 16, [1, 1], [100, 100], 64, [[1, 0, 1], [1]], seed=2, expect_err=1)      # the part twice
    check_selected(m, "bf16", 16, [2, 0], [1, 50], 64, [[0], [0]], seed=3, expect_err=1)               # a row without keys


def test_selected_rows_of_no_request_are_zero(m):
    check_selected(m, "fp8", 16, [1, 2], [100, 200], 64, [[0, 1], [2], [0, 3]], seed=5, pad_rows=3)


def test_selected_without_requests_is_zero(m):
    """Three rows and no request at all (a padded batch): zeros and -inf, with buffers handed in too."""
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.zeros((3, 16, 576), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((2, 64, 576), dtype=torch.bfloat16, device="cuda")
    out = torch.full((3, 16, 520), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, 16), 7.0, device="cuda")
    got, l = m.selected_decode(q, kv, torch.zeros((0, 2), **i32), torch.zeros(0, **i32), torch.zeros((3, 2), **i32),
                               torch.zeros(1, **i32), fmt="bf16", softmax_scale=0.1, out=out, lse=lse)
    assert got is out and l is lse
    assert bool((out[..., :512] == 0).all()) and bool((out[..., 512:] == 7).all()) and bool((lse == -float("inf")).all())


def test_sizes_past_32_bits_are_refused(m):
    """Sizes that would wrap in the call's 32-bit arguments."""
    x = torch.zeros((2, 8), device="cuda")
    seq = torch.full((2,), 8, dtype=torch.int32, device="cuda")
    for kw in (dict(block_tokens=2 ** 32 + 1), dict(first=2 ** 32), dict(last=2 ** 32), dict(page_size=2 ** 32 + 64)):
        with pytest.raises(ValueError, match="32-bit"):
            m.index_select(x, seq, 4, **kw)
    with pytest.raises(ValueError, match="32-bit"):
        m.index_select(x, seq, 2 ** 32 + 4)
    q, w = torch.zeros((2, 8, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 8), device="cuda")
    cache, table = torch.zeros((2, 64, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    for kw in (dict(block_tokens=0), dict(block_tokens=2 ** 32 + 16), dict(max_context=-1)):
        with pytest.raises(ValueError, match="block_tokens"):
            m.index_scores(q, w, cache, None, table, seq, **{"fmt": "bf16", "max_context": 8, **kw})


@pytest.mark.parametrize("fmt,T,H", [("fp8_ds_mla", 26, 96), ("bf16", 40, 128), ("fp8", 78, 128), ("fp8", 156, 16)])
def test_selected_rows_beyond_a_whole_wave(m, fmt, T, H):
    """A batch whose last rows take a launch of their own; empty, short and unowned rows among them."""
    rng = np.random.default_rng(T)
    lens = rng.integers(900, 1100, T)
    lens[-1] = 37
    lists = [sorted(rng.permutation(-(-int(n) // 64))[:16].tolist()) for n in lens]
    lists[0] = lists[T - 2] = []
    check_selected(m, fmt, H, [1] * T, lens.astype(np.int32), 64, lists, seed=T)
    check_selected(m, fmt, H, [1] * (T - 3), lens[:T - 3].astype(np.int32), 64, lists, seed=T, pad_rows=3)


@pytest.mark.parametrize("fmt", FMTS)
def test_selected_split_over_a_long_list(m, fmt):
    check_selected(m, fmt, 16, [1], [64 * 90 + 5], 64, [list(range(0, 91, 2))], seed=6)


# ------------------------------------------------------------------------------------------ together

class Chain:
    """One decode step over index keys and fp8_ds_mla records: insert, scores, selection, attention."""

    def __init__(self, seed=0, B=5, Hi=32, H=16, ps=64, steps=3):
        rng = np.random.default_rng(seed)
        self.B, self.Hi, self.H, self.ps = B, Hi, H, ps
        self.lens = rng.integers(1, 900, B).astype(np.int32)
        self.tab, self.nb = table_for(rng, self.lens + steps, ps)
        self.cache, _, self.scales, _ = index_cache(rng, self.nb, ps, "fp8")
        self.rec, self.vals = latent_cache(rng, self.nb, ps, "fp8_ds_mla", 1.0)
        self.table, self.seq = t_i32(self.tab), t_i32(self.lens)
        self.cs = f32(synth.cos_sin_table(1024))
        self.q = t_bf16(rand_bf16(rng, (B, Hi, 128)))
        self.k = t_bf16(rand_bf16(rng, (B, 128)))
        self.w = f32(rng.random((B, Hi)))
        self.mq = t_bf16(rand_bf16(rng, (B, H, 576)))
        self.pos = t_i64(self.lens - 1)
        self.slots = t_i64([self.tab[b, (n - 1) // ps] * ps + (n - 1) % ps for b, n in enumerate(self.lens)])

    def step(self, m, topk=64, bt=1):
        qi, wi = m.index_q_cache_insert(self.q, self.k, self.w, self.cache, self.scales, self.slots, fmt="fp8",
                                        weight_scale=0.05, positions=self.pos, cos_sin_cache=self.cs)
        sc = m.index_scores(qi, wi, self.cache, self.scales, self.table, self.seq, fmt="fp8", block_tokens=bt, max_context=1024)
        if bt == 1:
            blocks, slots = m.index_select(sc, self.seq, topk, block_table=self.table, page_size=self.ps, num_blocks=self.nb)
            indptr = torch.arange(0, (self.B + 1) * topk, topk, dtype=torch.int32, device="cuda")
            out, lse = m.sparse_fwd(self.mq, self.rec.reshape(-1, 656), indptr, slots.reshape(-1), 192 ** -0.5,
                                    has_invalid=True, return_lse=True)
        else:
            blocks, _ = m.index_select(sc, self.seq, topk, block_tokens=bt, first=1, last=1)
            out, lse = m.selected_decode(self.mq, self.rec, self.table, self.seq, blocks, fmt="fp8_ds_mla",
                                         softmax_scale=192 ** -0.5, return_lse=True)
        return sc, blocks, out, lse

    def check(self, got, topk, bt):
        sc, blocks, out, lse = got
        keys = ref.E4M3[self.cache.cpu().numpy()] * self.scales.cpu().numpy()[:, :, None].astype(np.float64)
        cs = self.cs.cpu().numpy()[self.lens - 1]
        yq = ref.rotate(ref.bf16_to_f64(bf16_bits(self.q)), cs[:, None])
        cq, sq = ref.quantise(yq)
        w = self.w.cpu().numpy() * np.float32(0.05) * sq.astype(np.float32)
        s = sc.cpu().numpy()
        cu = np.arange(self.B + 1)
        want, mag, written = ref.scores(ref.E4M3[cq], w.astype(np.float64), keys, np.ones(keys.shape[:2]), self.tab, self.lens, cu,
                                        s.shape[1], bt, self.nb)
        assert (np.abs(s - want)[written] <= SCORE_TOL * mag[written]).all()
        first = last = 0 if bt == 1 else 1
        wb, _, _ = ref.select(s, self.lens, cu, bt, topk, first, last)
        assert np.array_equal(blocks.cpu().numpy(), wb)
        for b, n in enumerate(self.lens):
            pos = [j for c in wb[b] if c >= 0 for j in range(c * bt, min(n, (c + 1) * bt))]
            ent = np.array([self.vals[self.tab[b, j // self.ps], j % self.ps] for j in pos]).reshape(-1, 576)
            o, l = ref.attend(ref.bf16_to_f64(bf16_bits(self.mq[b])), ent, 192 ** -0.5)
            assert_attn_close(out[b], o, f"request {b}")
            assert_lse_close(lse[b], l, f"request {b}")


class Declined:
    """A marshalling that serves nothing: every call takes its Python form."""
    insert = gather = scores = select = selected = staticmethod(lambda *a: None)


@pytest.mark.parametrize("topk,bt", [(64, 1), (4, 64)])
@pytest.mark.parametrize("given", [False, True])
def test_both_marshallings_give_the_same(m, monkeypatch, topk, bt, given):
    """The C marshalling of plain calls and the Python form, with new outputs and with buffers handed in (rows
    of wider tensors among them)."""
    def run():
        c = Chain(seed=11)
        B, Hi, H = c.B, c.Hi, c.H
        e = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device="cuda")
        bf = torch.bfloat16
        o = {}
        if given:
            o = dict(i=dict(q_out=e(B, Hi, 128, dtype=torch.int8), w_out=e(B, Hi, dtype=torch.float32)),
                     s=dict(scores=e(B, 1100, dtype=torch.float32)[:, 3:1080]), k=dict(blocks=e(B, topk + 5)[:, :topk]),
                     d=dict(out=e(B, H, 520, dtype=bf), lse=e(B, H, dtype=torch.float32), workspace=e(1 << 22, dtype=torch.uint8)),
                     g=dict(dst=e(300, 136, dtype=bf)[:, :128]))
            if bt == 1:
                o["k"]["slots"] = e(B, topk + 3)[:, :topk]
        qi, wi = m.index_q_cache_insert(c.q, c.k, c.w, c.cache, c.scales, c.slots, fmt="fp8", weight_scale=0.05, positions=c.pos,
                                        cos_sin_cache=c.cs, **o.get("i", {}))
        cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        sc = m.index_scores(qi, wi, c.cache, c.scales, c.table, c.seq, cu, fmt="fp8", block_tokens=bt, max_context=1024, **o.get("s", {}))
        table = dict(block_table=c.table, page_size=c.ps, num_blocks=c.nb) if bt == 1 else dict(first=1, last=1)
        blocks, slots = m.index_select(sc, c.seq, topk, cu, block_tokens=bt, **table, **o.get("k", {}))
        pages = blocks if bt > 1 else torch.zeros((B, 1), dtype=torch.int32, device="cuda")
        out, lse = m.selected_decode(c.mq, c.rec, c.table, c.seq, pages, cu, fmt="fp8_ds_mla", softmax_scale=0.07, return_lse=True,
                                     **o.get("d", {}))
        _, none = m.selected_decode(c.mq, c.rec, c.table, c.seq, pages, fmt="fp8_ds_mla", softmax_scale=0.07)
        lens = torch.clamp(c.seq, max=60)
        back = m.index_gather(c.cache, c.scales, c.table, torch.cat([cu[:1], torch.cumsum(lens, 0).int()]), cu[:-1] * 0, fmt="fp8",
                              num_tokens=300, **o.get("g", {}))
        assert none is None
        visible = torch.arange(sc.shape[1], device="cuda") < ((c.seq + bt - 1) // bt)[:, None]
        n = int(lens.sum())
        return [qi.view(torch.uint8), wi, torch.where(visible, sc, 0), blocks, blocks if slots is None else slots, out[..., :512], lse, back[:n]]

    m._plain()
    served = []
    real = m._marshal

    class Counted:
        def __getattr__(self, name):
            def call(*a):
                r = getattr(real, name)(*a)
                served.append(r is not None)
                return r
            return call

    monkeypatch.setattr(m, "_marshal", Counted())
    a = run()
    assert len(served) == 6 and all(served)
    monkeypatch.setattr(m, "_marshal", Declined())
    b = run()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_marshalling_declines_what_is_not_plain(m):
    """Calls that the C marshalling leaves to the Python form, which serves or refuses them."""
    p = m._plain()
    c = Chain(seed=3)
    ins = [c.q, c.k, c.w, c.cache, c.scales, c.slots, 1, 1.0, c.pos, c.cs, None, None]
    assert p.insert(*ins) is not None
    for i, v in [(0, c.q.cpu()), (0, c.q.float()), (0, c.q[:, :, :64]), (0, c.q.transpose(1, 2)), (1, c.k[:, None]), (1, c.k[:-1]),
                 (2, c.w.double()), (3, c.cache[..., :64]), (4, None), (4, c.scales[:, :-1]), (5, c.slots.int()), (6, 0), (7, 1),
                 (8, c.pos[:-1]), (9, c.cs[:, :32]), (10, torch.empty_like(c.q)), (11, c.w.t().contiguous().t()), (0, None), (0, 3)]:
        assert p.insert(*ins[:i], v, *ins[i + 1:]) is None, i
    x = torch.zeros((c.B, 64), device="cuda")
    sel = [x, c.seq, 4, None, 1, 0, 0, None, 0, 0, None, None]
    assert p.select(*sel) is not None
    for i, v in [(0, x.t()), (1, c.seq.long()), (1, c.seq[:-1]), (2, 0), (2, 2 ** 32 + 4), (2, 4.0), (4, 0), (5, 2 ** 31), (11, x.int())]:
        assert p.select(*sel[:i], v, *sel[i + 1:]) is None, i
    with pytest.raises(m.MLAError, match="first and last"):
        p.select(*sel[:5], 3, 3, *sel[7:])
    pages = torch.zeros((c.B, 2), dtype=torch.int32, device="cuda")
    dec = [c.mq, c.rec, c.table, c.seq, pages, None, 2, 0.1, 1.0, 1.0, None, False, None, None]
    assert p.selected(*dec) is not None
    for i, v in [(0, c.mq[..., :512]), (1, c.rec[:, None]), (2, c.table[:-1]), (3, c.seq[:0]), (4, pages[:-1]), (7, 1), (11, 1),
                 (10, torch.zeros((c.B, c.H, 256), dtype=torch.bfloat16, device="cuda")), (12, torch.zeros(8, device="cuda"))]:
        assert p.selected(*dec[:i], v, *dec[i + 1:]) is None, i
    with pytest.raises(m.MLAError, match="workspace too small"):
        p.selected(*dec[:12], torch.empty(0, dtype=torch.uint8, device="cuda"), None)
    assert p.insert() is None and p.gather(1) is None and p.scores() is None


@pytest.mark.parametrize("topk,bt", [(64, 1), (4, 64)])
def test_run_of_them_together(m, topk, bt):
    c = Chain(seed=topk)
    c.check(c.step(m, topk, bt), topk, bt)
    assert m.read_device_errors() == 0


@pytest.mark.parametrize("topk,bt", [(64, 1), (4, 64)])
def test_run_captured_and_replayed_with_new_inputs(m, topk, bt):
    a, b = Chain(seed=1), Chain(seed=2)
    a.step(m, topk, bt)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = a.step(m, topk, bt)
    g.replay()
    torch.cuda.synchronize()
    a.check(got, topk, bt)
    for name in ("q", "k", "w", "mq"):
        getattr(a, name).copy_(getattr(b, name))
    g.replay()
    torch.cuda.synchronize()
    a.check(got, topk, bt)


def test_two_runs_on_two_streams(m):
    cs = [Chain(seed=5), Chain(seed=6)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = []
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                got.append(c.step(m, 4, 64))
    torch.cuda.synchronize()
    for c, g in zip(cs, got):
        c.check(g, 4, 64)


# ------------------------------------------------------------------------------------------ refusals

def test_refusals(m):
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
    u8, bf, i32, i64 = torch.uint8, torch.bfloat16, torch.int32, torch.int64
    ok = dict(q=z(2, 4, 128, dt=bf), k=z(2, 128, dt=bf), w=z(2, 4), c=z(2, 16, 128, dt=u8), s=z(2, 16), slots=z(2, dt=i64))

    def insert(fmt="fp8", **kw):
        a = {**ok, **kw}
        return m.index_q_cache_insert(a["q"], a["k"], a["w"], a["c"], a["s"], a["slots"], fmt=fmt)
    insert()
    for bad in (dict(q=z(2, 4, 64, dt=bf)), dict(k=z(3, 128, dt=bf)), dict(w=z(2, 5)), dict(slots=z(3, dt=i64)), dict(c=z(2, 16, 64, dt=u8)),
                dict(s=z(2, 17)), dict(fmt="fp8_ds_mla"), dict(fmt="bf16"), dict(q=z(2, 4, 128))):
        with pytest.raises((ValueError, TypeError)):
            insert(**bad)
    with pytest.raises(m.MLAError, match="Hi must be"):
        insert(q=z(2, 65, 128, dt=bf), w=z(2, 65))

    def scores(**kw):
        a = dict(q=z(2, 4, 128, dt=u8), w=z(2, 4), c=ok["c"], s=ok["s"], t=z(2, 3, dt=i32), n=z(2, dt=i32), cu=None, bt=1, out=None, mc=48)
        a.update(kw)
        return m.index_scores(a["q"], a["w"], a["c"], a["s"], a["t"], a["n"], a["cu"], fmt="fp8", block_tokens=a["bt"],
                              max_context=a["mc"], scores=a["out"])
    scores()
    for bad in (dict(n=z(3, dt=i32)), dict(cu=z(2, dt=i32)), dict(t=z(1, 3, dt=i32)), dict(out=z(2, 47)), dict(w=z(2, 3)),
                dict(q=z(2, 4, 128, dt=bf))):
        with pytest.raises((ValueError, TypeError)):
            scores(**bad)
    for bad, msg in ((dict(bt=8), "block_tokens"), (dict(c=z(2, 48, 128, dt=u8), s=z(2, 48)), "block_size"),
                     (dict(q=z(2, 65, 128, dt=u8), w=z(2, 65)), "Hi must be")):
        with pytest.raises(m.MLAError, match=msg):
            scores(**bad)
    with pytest.raises(ValueError):
        m.index_select(z(2, 10), z(3, dt=i32), 4)
    with pytest.raises(ValueError):
        m.index_select(z(2, 10), z(2, dt=i32), 0)
    with pytest.raises(m.MLAError, match="first and last"):
        m.index_select(z(2, 10), z(2, dt=i32), 4, first=3, last=2)
    with pytest.raises(m.MLAError, match="page_size"):
        m.index_select(z(2, 10), z(2, dt=i32), 4, block_table=z(2, 1, dt=i32))
    with pytest.raises(m.MLAError, match="below 2"):
        m.index_select(z(2, 10), z(2, dt=i32), 4, block_table=z(2, 1, dt=i32), page_size=64, num_blocks=1 << 26)
    kv, q = z(4, 16, 576, dt=bf), z(2, 16, 576, dt=bf)
    sel = lambda **kw: m.selected_decode(kw.get("q", q), kv, z(2, 3, dt=i32), z(2, dt=i32), kw.get("blocks", z(2, 3, dt=i32)),
                                         fmt="bf16", softmax_scale=1.0, workspace=kw.get("ws"))
    sel()
    with pytest.raises(ValueError):
        sel(blocks=z(3, 3, dt=i32))
    with pytest.raises(m.MLAError, match="workspace"):
        sel(ws=z(256, dt=u8))
    with pytest.raises(m.MLAError, match="topk"):
        sel(blocks=z(2, 0, dt=i32))
    assert m.read_device_errors() == 1          # sel() listed a page of a request without keys


def test_problems_of_size_zero(m):
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device="cuda")
    u8, bf, i32, i64 = torch.uint8, torch.bfloat16, torch.int32, torch.int64
    q, w = m.index_q_cache_insert(z(0, 4, 128, dt=bf), z(0, 128, dt=bf), z(0, 4), z(2, 16, 128, dt=u8), z(2, 16), z(0, dt=i64), fmt="fp8")
    assert q.shape == (0, 4, 128)
    cu = t_i32([0, 0])
    assert m.index_scores(q, w, z(2, 16, 128, dt=u8), z(2, 16), z(1, 3, dt=i32), z(1, dt=i32), cu, fmt="fp8", max_context=8).shape == (0, 8)
    assert m.index_select(z(0, 8), z(1, dt=i32), 4, cu)[0].shape == (0, 4)
    out, _ = m.selected_decode(z(0, 16, 576, dt=bf), z(2, 16, 576, dt=bf), z(1, 3, dt=i32), z(1, dt=i32), z(0, 3, dt=i32), cu,
                               fmt="bf16", softmax_scale=1.0)
    assert out.shape == (0, 16, 512)
    blocks, slots = m.index_select(z(2, 8), t_i32([0, 0]), 4, block_table=z(2, 1, dt=i32), page_size=16, num_blocks=2)
    assert (blocks == -1).all() and (slots == -1).all()
    m.index_scores(z(2, 4, 128, dt=u8), z(2, 4), z(2, 16, 128, dt=u8), z(2, 16), z(2, 3, dt=i32), t_i32([0, 0]), fmt="fp8", max_context=8)
    torch.cuda.synchronize()
    assert m.read_device_errors() == 0


@pytest.mark.parametrize("n,k", [(200000, 8192), (9000, 8192), (300001, 2048), (65536, 1), (33000, 4000)])
@pytest.mark.parametrize("order", ["random", "ascending", "descending", "late"])
def test_select_long_rows_in_every_order(m, n, k, order):
    """Few rows: the row is shared by several CTAs.  Ascending scores cut the running list most often."""
    rng = np.random.default_rng(n)
    x = rng.standard_normal(n).astype(np.float32)
    if order != "random":
        x = np.sort(x) if order != "descending" else -np.sort(x)
    if order == "late":
        x[: n - n // 3] = x[0]
    check_select(m, np.stack([x, np.round(x * 4)]), [n, n - 1], [1, 1], 1, k, first=min(2, k), last=0)


@pytest.mark.parametrize("offset", [0, 1, 3])
def test_select_rows_off_the_16_byte_grid(m, offset):
    rng = np.random.default_rng(offset)
    x = rng.standard_normal((3, 9001 + 4)).astype(np.float32)
    t = f32(x)[:, offset:offset + 9001]
    got, _ = m.index_select(t, t_i32([9001, 500, 9000]), 100)
    want, _, _ = ref.select(x[:, offset:offset + 9001], [9001, 500, 9000], np.arange(4), 1, 100, 0, 0)
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("rows", [1, 160])      # rows shared by a cluster, and one CTA each
@pytest.mark.parametrize("n,k", [(9000, 600), (70001, 513), (140000, 2048)])
@pytest.mark.parametrize("kind", ["grid", "outlier", "infinite", "forced", "blocks", "waves", "periodic"])
def test_select_crowded_cuts(m, rows, n, k, kind):
    """Equal scores at the cut, a range that an outlier stretches, more infinities than places, forced blocks on
    both sides of the cut; rows whose neighbours resemble one another, or that repeat with the sample's stride."""
    rng = np.random.default_rng(n + k)
    x = rng.standard_normal((2, n)).astype(np.float32)
    if kind == "grid":
        x = (np.round(x * 256) / 256).astype(np.float32)
    elif kind == "outlier":
        x[0, n // 3] = 1e6
        x[1, n // 2] = np.inf
    elif kind == "infinite":
        x[0, rng.permutation(n)[:k + 40]] = np.inf
        x[1, rng.permutation(n)[:k // 2]] = np.inf
    elif kind == "blocks":
        x = np.repeat(x[:, :n // 16 + 1], 16, 1)[:, :n] + np.float32(0.02) * x
    elif kind == "waves":
        x = np.sin(np.arange(n) / np.array([[90.0], [700.0]])).astype(np.float32) + np.float32(0.1) * x
    elif kind == "periodic":
        x[:, :: max(1, n // 512)] += 9
        x[1] = -x[1]
    first, last = (5, 9) if kind == "forced" else (0, 0)
    if rows == 1:
        check_select(m, x[:1], [n], [1], 1, k, first, last, slots=True, ps=64, seed=n)
        check_select(m, x[1:], [n - 7], [1], 1, k, first, last, slots=True, ps=64, seed=n)
        return
    got, _ = m.index_select(f32(x).repeat(rows // 2, 1), t_i32([n, n - 7] * (rows // 2)), k, first=first, last=last)
    want, _, _ = ref.select(x, [n, n - 7], np.arange(3), 1, k, first, last)
    assert np.array_equal(got.cpu().numpy(), np.tile(want, (rows // 2, 1)))


def test_select_topk_limit(m):
    with pytest.raises(m.MLAError, match="topk must be"):
        m.index_select(torch.zeros((1, 10), device="cuda"), t_i32([10]), 8193)
