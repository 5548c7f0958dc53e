"""The 4-bit latent cache on the GPU against plain 64-bit references."""
import numpy as np
import pytest
import torch

import mxfp4_ref as ref

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
U8, BF, I32, I64 = torch.uint8, torch.bfloat16, torch.int32, torch.int64


@pytest.fixture(scope="module")
def m():
    import mla_latent_cache_attention_gb300 as mod
    mod.lib()
    return mod


def latents(rng, *shape, spread=0.5):
    chan = np.exp(spread * rng.standard_normal(512))
    return ref.bf16(rng.standard_normal((*shape, 512)) * chan)


def make_cache(rng, nb, bs, spread=0.5):
    lat, rope = latents(rng, nb, bs, spread=spread), ref.bf16(rng.standard_normal((nb, bs, 64)))
    return ref.records(lat.double().numpy(), rope)


def make_table(rng, lens, bs, nb, extra_cols=0):
    per = [-(-n // bs) for n in lens]
    ids = rng.permutation(nb)[:sum(per)]
    t = np.full((len(lens), max(1, max(per)) + extra_cols), -7, dtype=np.int32)
    at = 0
    for b, n in enumerate(per):
        t[b, :n] = ids[at:at + n]
        at += n
    return t


def check(out, lse, want, what=""):
    o, l, tol, ltol = want
    got = out.double().cpu().numpy()
    gl = lse.double().cpu().numpy()
    assert np.array_equal(np.isinf(gl), np.isinf(l)), what
    fin = np.isfinite(l)
    assert np.all(np.abs(gl[fin] - l[fin]) <= ltol[fin]), (what, np.max((np.abs(gl - l) / np.maximum(ltol, 1e-30))[fin]))
    assert np.all(np.abs(got - o) <= tol), (what, np.max(np.abs(got - o) / np.maximum(tol, 1e-300)))
    if o.size >= 4096 and np.any(o):        # and on the whole as good as the rounding of the output and of the weights: 2^-8
        assert np.linalg.norm(got - o) <= 2.0 ** -8 * np.linalg.norm(o), what


# ------------------------------------------------------------------------------------------ the record

CASES = {
    "ordinary": lambda r, n: latents(r, n),
    "wide": lambda r, n: ref.bf16(r.standard_normal((n, 512)) * np.exp2(r.integers(-20, 20, (n, 512)))),
    "tiny": lambda r, n: ref.bf16(r.standard_normal((n, 512)) * 1e-38),
    "huge": lambda r, n: ref.bf16(r.standard_normal((n, 512)).clip(-3, 3) * 1e38),
    "zero rows": lambda r, n: ref.bf16(r.standard_normal((n, 512)) * (np.arange(n)[:, None] % 2)),
    "zero groups": lambda r, n: ref.bf16(r.standard_normal((n, 512)) * (np.arange(512) // 32 % 3 == 0)),
    # whole steps, halves of them and the borders of the exponents
    "ties": lambda r, n: ref.bf16(r.choice([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 12, 48], (n, 512)) * r.choice([-1, 1], (n, 512))),
}


@pytest.mark.parametrize("kind", CASES)
@pytest.mark.parametrize("way", ["decode", "prefill"])
def test_records_are_the_definitions(m, kind, way):
    rng = np.random.default_rng(3)
    T, H, bs, nb = 37, 3, 16, 5
    lat, kpe = CASES[kind](rng, T), ref.bf16(rng.standard_normal((T, 64)))
    slots = torch.from_numpy(rng.permutation(nb * bs)[:T])
    slots[5] = -1
    cache = torch.full((nb, bs, 400), 171, dtype=U8, device="cuda")
    d = lambda t: t.cuda()
    if way == "decode":
        ql, qpe = ref.bf16(rng.standard_normal((T, H, 512))), ref.bf16(rng.standard_normal((T, H, 64)))
        out = m.q_concat_cache_insert(d(ql), d(qpe), d(lat), d(kpe), cache, d(slots), fmt="mxfp4")
        assert out.dtype == BF and torch.equal(out.cpu(), torch.cat([ql, qpe], -1))
    else:
        q, kn = ref.bf16(rng.standard_normal((T, H, 192))), ref.bf16(rng.standard_normal((T, H, 128)))
        q0 = d(q)
        out = m.key_concat_cache_insert(q0, d(kn), d(kpe), d(lat), cache, d(slots), fmt="mxfp4")
        assert torch.equal(q0.cpu(), q) and torch.equal(out.cpu(), torch.cat([kn, kpe[:, None].expand(T, H, 64)], -1))
    want = np.full((nb * bs, 400), 171, dtype=np.uint8)
    live = slots.numpy() >= 0
    want[slots.numpy()[live]] = ref.records(lat.double().numpy(), kpe)[live]
    got = cache.cpu().numpy().reshape(-1, 400)
    assert np.array_equal(got[:, 256:], want[:, 256:])
    assert np.array_equal(got, want)
    # read back: bf16 values (exact: one bit behind the point at a power of two) and the bytes
    table = torch.arange(nb, dtype=I32, device="cuda")[None]
    cu = torch.tensor([0, nb * bs], dtype=I32, device="cuda")
    raw = m.gather_context(cache, table, cu, fmt="mxfp4", num_tokens=nb * bs, raw=True)
    assert np.array_equal(raw.cpu().numpy(), got)
    vals = m.gather_context(cache, table, cu, fmt="mxfp4", num_tokens=nb * bs).double().cpu().numpy()
    vl, vr = ref.values(got)
    at = slots.numpy()[live]
    # (4 * 2^126 = 2^128, to which a value above 3.5 * 2^126 goes, is no bf16 number: read as an infinity)
    assert np.array_equal(vals[at, :512], ref.bf16(vl[at]).double().numpy()) and np.array_equal(vals[at, 512:], vr[at])
    # a value is off by at most half a step of its group (the steps between 4 and 6 are 2), and what is below 2^-14 of the
    # record's largest exponent by half of that step
    x = lat.double().numpy()[live].reshape(-1, 16, 32)
    step = 2.0 ** (want[at, 256:272].astype(np.float64) - 127)
    assert np.all(np.abs(vl[at].reshape(-1, 16, 32) - x) <= np.maximum(np.abs(x) / 4, step[..., None] / 4))
    assert m.read_device_errors() == 0


def test_infinities_and_nan(m):
    """A group with one is stored and read as NaN, the other groups and tokens as ever."""
    rng = np.random.default_rng(4)
    lat = latents(rng, 4)
    lat[1, 40], lat[2, 511], lat[3, 0], lat[3, 100] = float("nan"), float("inf"), float("-inf"), float("nan")
    kpe = ref.bf16(rng.standard_normal((4, 64)))
    z = torch.zeros((4, 1, 512), dtype=BF, device="cuda")
    cache = torch.zeros((1, 16, 400), dtype=U8, device="cuda")
    m.q_concat_cache_insert(z, z[..., :64].contiguous(), lat.cuda(), kpe.cuda(), cache, torch.arange(4, device="cuda"), fmt="mxfp4")
    assert np.array_equal(cache.cpu().numpy()[0, :4], ref.records(lat.double().numpy(), kpe))
    got = m.gather_context(cache, torch.zeros((1, 1), dtype=I32, device="cuda"), torch.tensor([0, 4], dtype=I32, device="cuda"), fmt="mxfp4", num_tokens=4)
    bad = torch.isnan(got[:, :512]).reshape(4, 16, 32)
    assert torch.equal(bad.all(-1), bad.any(-1))
    assert bad.all(-1).nonzero().tolist() == [[1, 1], [2, 15], [3, 0], [3, 3]]


@pytest.mark.parametrize("vec", [True, False])
@pytest.mark.parametrize("bs", [1, 7, 64])
def test_gather_layouts(m, vec, bs):
    """Chunks of contexts, padded entries, rows of no request left as they were, blocks out of range."""
    rng = np.random.default_rng(5)
    lens, starts = [0, 65, 1, 200], [0, 13, 3, 64]
    nb = sum(-(-(a + b) // bs) for a, b in zip(lens, starts)) + 2
    pitch = 416 if vec else 404
    full = torch.zeros((nb, bs, pitch), dtype=U8, device="cuda")
    full[..., :400] = torch.from_numpy(make_cache(rng, nb, bs)).cuda()
    cache = full[..., :400]
    table = make_table(rng, [a + b for a, b in zip(lens, starts)], bs, nb)
    cu = np.cumsum([0] + lens)
    n = int(cu[-1]) + 9
    t = lambda a, dt=I32: torch.tensor(np.asarray(a), dtype=dt, device="cuda")
    for raw in (False, True):
        dst = torch.full((n, 400 if raw else 576), 99, dtype=U8 if raw else BF, device="cuda")
        m.gather_context(cache, t(table), t(cu), t(starts), fmt="mxfp4", num_tokens=n, raw=raw, dst=dst)
        h = cache.cpu().numpy()
        rec = np.concatenate([ref.keys_of(h, table[b], s + L, bs)[s:] for b, (L, s) in enumerate(zip(lens, starts))])
        got = dst.cpu()
        assert bool((got[cu[-1]:] == 99).all())
        if raw:
            assert np.array_equal(got[:cu[-1]].numpy(), rec)
        else:
            assert np.array_equal(got[:cu[-1]].double().numpy(), np.concatenate(ref.values(rec), -1))
    assert m.read_device_errors() == 0
    table[1, -(-30 // bs)] = nb
    m.gather_context(cache, t(table), t(cu), t(starts), fmt="mxfp4", num_tokens=n)
    assert m.read_device_errors() == 2


def test_insert_rotates_like_the_other_caches(m):
    """RoPE of the query and the shared key, slots out of range: the same bits as with the bf16 cache."""
    rng = np.random.default_rng(6)
    T, H, nb, bs = 5, 2, 3, 8
    ql, qpe, lat, kpe = (ref.bf16(rng.standard_normal(s)).cuda() for s in ((T, H, 512), (T, H, 64), (T, 512), (T, 64)))
    pos, cs = torch.tensor([0, 5, 77, 131071, 9], device="cuda"), m.rope_table(131072, 64)
    slots = torch.tensor([3, nb * bs, 0, 23, -1], device="cuda")
    a, b = torch.zeros((nb, bs, 400), dtype=U8, device="cuda"), torch.zeros((nb, bs, 576), dtype=BF, device="cuda")
    qa = m.q_concat_cache_insert(ql, qpe, lat, kpe, a, slots, fmt="mxfp4", positions=pos, cos_sin_cache=cs)
    qb = m.q_concat_cache_insert(ql, qpe, lat, kpe, b, slots, fmt="bf16", positions=pos, cos_sin_cache=cs)
    assert torch.equal(qa, qb)
    assert torch.equal(a[..., 272:].contiguous().view(BF), b[..., 512:])
    assert m.read_device_errors() == 4


# ------------------------------------------------------------------------------------------ decode

def run_decode(m, rng, lens, *, q_len=1, H=16, bs=64, spread=0.5, scale=SCALE, max_context=None, cache=None, pad=0, strided=False, graph=False):
    nb = sum(-(-n // bs) for n in lens) + 3
    if cache is None:
        cache = make_cache(rng, nb, bs, spread)
    table = make_table(rng, lens, bs, nb, extra_cols=2)
    rows = len(lens) * q_len
    q = ref.bf16(rng.standard_normal((rows, H, 576)))
    want = ref.decode(q.double().numpy(), cache, table, lens, bs, q_len, scale)
    full = torch.zeros((*cache.shape[:2], 400 + pad), dtype=U8, device="cuda")
    full[..., :400] = torch.from_numpy(cache).cuda()
    kv = full[..., :400] if pad else full
    qd = q.cuda()
    out = lse = None
    if strided:
        big = torch.zeros((rows, H + 1, 584), dtype=BF, device="cuda")
        big[:, :H, :576] = qd
        qd = big[:, :H, :576]
        out = torch.full((rows, H + 2, 520), 7.0, dtype=BF, device="cuda")[:, :H]
    args = (qd, kv, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=I32, device="cuda"))
    kw = dict(fmt="mxfp4", q_len=q_len, max_context=max_context or max(1, max(lens)), softmax_scale=scale, return_lse=True)
    got, lse = m.paged_decode(*args, out=out, **kw)
    if strided:
        assert bool((got[..., 512:] == 7).all())
        got = got[..., :512]
    check(got, lse, want, (lens, q_len, H, bs))
    assert m.read_device_errors() == 0
    return args, kw, got, lse


@pytest.mark.parametrize("lens", [[1], [0, 5, 127], [128, 129, 0, 255, 256], [700, 1, 64, 385]])
@pytest.mark.parametrize("H", [1, 16, 17, 40])
def test_decode_lengths_and_heads(m, lens, H):
    run_decode(m, np.random.default_rng(len(lens) * 100 + H), lens, H=H)


@pytest.mark.parametrize("bs", [1, 3, 8, 16, 24, 48, 100, 128, 200, 256])
def test_decode_block_sizes(m, bs):
    run_decode(m, np.random.default_rng(bs), [300, 0, 17, 129], bs=bs)


@pytest.mark.parametrize("q_len,H", [(2, 8), (2, 16), (3, 11), (4, 16), (4, 96), (7, 5), (1, 96), (1, 128), (5, 128)])
def test_decode_speculative_rows(m, q_len, H):
    """Causal among the request's last rows; requests shorter than their rows have rows without any key."""
    run_decode(m, np.random.default_rng(q_len * 1000 + H), [q_len, 1, 0, 130, 261], q_len=q_len, H=H)


def test_decode_many_splits_and_items(m):
    """More work items than SMs, splits that most requests do not reach."""
    rng = np.random.default_rng(9)
    lens = [int(x) for x in rng.integers(0, 600, 70)] + [9000]
    run_decode(m, rng, lens, H=16, max_context=9000)


def test_decode_one_split(m):
    rng = np.random.default_rng(10)
    run_decode(m, rng, [1500, 40], H=32, max_context=300)       # longer than max_context: served all the same


def test_decode_long(m):
    """A long context: many moves of the reference, small weights."""
    run_decode(m, np.random.default_rng(11), [20011], H=16, scale=0.3)


@pytest.mark.parametrize("q_len,H,scale", [(1, 48, 0.3), (4, 16, SCALE), (1, 128, 0.1)])
def test_decode_long_of_many_columns(m, q_len, H, scale):
    run_decode(m, np.random.default_rng(H), [9011, 30, 2300], q_len=q_len, H=H, scale=scale)


@pytest.mark.parametrize("lens", [[111, 112, 113, 1], [224, 225, 0, 223, 336], [14, 15, 28, 98, 99]])
@pytest.mark.parametrize("bs", [3, 16, 64])
def test_decode_ends_of_short_tiles(m, lens, bs):
    """More than 32 columns take tiles of 112 keys, 14 a loader warp."""
    run_decode(m, np.random.default_rng(bs), lens, H=50, bs=bs)


@pytest.mark.parametrize("H", [16, 64])
def test_padded_batches(m, H):
    """Many requests without keys before, between and behind the others."""
    rng = np.random.default_rng(H)
    for where in ([0], [599], [0, 33, 64, 599], [31, 32, 300, 301, 450]):
        lens = [0] * 600
        for b in where:
            lens[b] = int(rng.integers(1, 900))
        run_decode(m, rng, lens, H=H)


@pytest.mark.parametrize("H", [16, 32, 40, 100])
def test_nan_keys_of_other_requests(m, H):
    """Several requests a CTA, every third with nothing but NaN keys: the others' results keep their bits."""
    rng = np.random.default_rng(H)
    bs, B = 64, 900
    lens = rng.integers(1, 300, B).astype(np.int32)
    nb = 24
    cache = make_cache(rng, 2 * nb, bs)
    table = rng.integers(0, nb, (B, 5)).astype(np.int32)
    table[::3] += nb                # of their own
    bad = cache.copy()
    bad[nb:, :, 256:] = 255
    q = ref.bf16(rng.standard_normal((B, H, 576))).cuda()
    run = lambda c: m.paged_decode(q, torch.from_numpy(c).cuda(), torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda(), fmt="mxfp4",
                                   max_context=300, softmax_scale=SCALE, return_lse=True)
    (out, lse), (o2, l2) = run(cache), run(bad)
    keep = torch.arange(B, device="cuda") % 3 != 0
    assert torch.equal(o2[keep], out[keep]) and torch.equal(l2[keep], lse[keep])
    assert bool(torch.isnan(o2[~keep]).all()) and not bool(torch.isnan(out).any())
    some = [1, 2, 4, 449, 898]
    want = ref.decode(q[some].double().cpu().numpy(), cache, table[some], [int(x) for x in lens[some]], bs, 1, SCALE)
    check(out[some], lse[some], want)


@pytest.mark.parametrize("scale", [0.0, -0.07, 1e-6, 4.0])
def test_decode_scales(m, scale):
    run_decode(m, np.random.default_rng(12), [333, 128], scale=scale)


@pytest.mark.parametrize("strided,pad", [(True, 0), (False, 16), (True, 112)])
def test_decode_layouts(m, strided, pad):
    run_decode(m, np.random.default_rng(13), [257, 100], H=20, q_len=2, strided=strided, pad=pad)


@pytest.mark.parametrize("kind", ["wide", "tiny", "huge", "zero rows", "zero groups"])
def test_decode_of_unusual_records(m, kind):
    """Exponents far apart within and between records: the key's power of two joins its weight."""
    rng = np.random.default_rng(14)
    nb, bs = 9, 64
    lat, rope = CASES[kind](rng, nb * bs).reshape(nb, bs, 512), ref.bf16(rng.standard_normal((nb, bs, 64)))
    cache = ref.records(lat.double().numpy(), rope)
    scale = {"huge": 1e-40, "wide": 1e-5}.get(kind, SCALE)
    lens, H = [300, 65], 16
    table = make_table(rng, lens, bs, nb)
    q = ref.bf16(rng.standard_normal((2, H, 576)))
    # 1e-40 is a subnormal of fp32; the kernel multiplies it by log2(e) and the query's 2^-e >= 2^-7 (no value of it passes
    # 7): off by 2^-150 / (1e-40 * 1.44 / 128) = 6.3e-4 of the scale at most, and 2^-150 / 1e-40 twice before
    want = ref.decode(q.double().numpy(), cache, table, lens, bs, 1, scale, eps=7e-4 if kind == "huge" else 0.0)
    assert q.abs().max() < 7
    out, lse = m.paged_decode(q.cuda(), torch.from_numpy(cache).cuda(), torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=I32, device="cuda"),
                              fmt="mxfp4", max_context=300, softmax_scale=scale, return_lse=True)
    o, l, tol, ltol = want
    if kind == "tiny":      # what is below 2^-74 reads as zero
        assert np.abs(o).max() < 2.0 ** -74
        o = np.zeros_like(o)
    check(out, lse, (o, l, tol, ltol), kind)


def test_garbage_where_no_key_is_seen(m):
    """NaN and infinities behind the last token, in unused blocks and in keys that only later rows see."""
    rng = np.random.default_rng(15)
    q_len, H, bs, lens = 2, 16, 64, [70, 130]
    nb = 6
    cache = make_cache(rng, nb, bs)
    table = make_table(rng, lens, bs, nb)
    q = ref.bf16(rng.standard_normal((4, H, 576)))
    want = ref.decode(q.double().numpy(), cache, table, lens, bs, q_len, SCALE)
    seen = np.zeros((nb, bs), bool)
    for b, L in enumerate(lens):
        pos = np.arange(L)
        seen[table[b][pos // bs], pos % bs] = True
    bad = cache.copy()
    bad[~seen] = 255                       # exponents 255 and NaN as rope values
    run = lambda c: m.paged_decode(q.cuda(), torch.from_numpy(c).cuda(), torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=I32, device="cuda"),
                                   fmt="mxfp4", q_len=q_len, max_context=130, softmax_scale=SCALE, return_lse=True)
    out, lse = run(bad)
    check(out, lse, want)
    # the last key of request 0: seen by its second row alone
    bad[table[0][69 // bs], 69 % bs, 256:] = 255
    o2, l2 = run(bad)
    assert torch.equal(o2[0], out[0]) and torch.equal(o2[2:], out[2:]) and torch.equal(l2[0], lse[0])
    assert bool(torch.isnan(o2[1]).all())


def test_bad_blocks_are_masked(m):
    """Keys of a block id out of range are left out, and the error word says so."""
    rng = np.random.default_rng(16)
    bs, L, H = 64, 200, 16
    cache = make_cache(rng, 5, bs)
    table = make_table(rng, [L], bs, 5)
    q = ref.bf16(rng.standard_normal((1, H, 576)))
    keep = [p for p in range(L) if p // bs != 1]
    lat, rope = ref.values(ref.keys_of(cache, table[0], L, bs)[keep])
    want = [x[None] for x in ref.attend(q[0].double().numpy(), lat, rope, SCALE)]
    for bad in (-1, 5, 2 ** 31 - 1, -2 ** 31):
        table[0, 1] = bad
        out, lse = m.paged_decode(q.cuda(), torch.from_numpy(cache).cuda(), torch.from_numpy(table).cuda(), torch.tensor([L], dtype=I32, device="cuda"),
                                  fmt="mxfp4", max_context=L, softmax_scale=SCALE, return_lse=True)
        check(out, lse, want)
        assert m.read_device_errors() == 2


def test_query_with_a_nan_or_infinity_spoils_its_own_row(m):
    rng = np.random.default_rng(17)
    args, kw, out, lse = run_decode(m, rng, [300, 40], H=16)
    q = args[0].clone()
    q[0, 3, 17], q[1, 5, 511] = float("nan"), float("inf")
    o2, l2 = m.paged_decode(q, *args[1:], **kw)
    assert bool(torch.isnan(o2[0, 3]).all()) and bool(torch.isnan(o2[1, 5]).all())
    same = torch.ones((2, 16), dtype=torch.bool, device="cuda")
    same[0, 3] = same[1, 5] = False
    assert torch.equal(o2[same], out[same]) and torch.equal(l2[same], lse[same])


def test_offsets_beyond_32_bits(m):
    """Blocks past 4 GB of the cache."""
    rng = np.random.default_rng(18)
    bs = 128
    nb = (1 << 33) // (bs * 400) + 8
    cache = torch.zeros((nb, bs, 400), dtype=U8, device="cuda")
    used = np.array([nb - 1, 3, nb - 2, nb // 2 + 1])
    part = make_cache(rng, 4, bs)
    cache[torch.from_numpy(used).cuda()] = torch.from_numpy(part).cuda()
    L, q = 4 * bs - 3, ref.bf16(rng.standard_normal((1, 16, 576)))
    want = ref.decode(q.double().numpy(), part, np.arange(4)[None], [L], bs, 1, SCALE)
    table = torch.tensor(used[None], dtype=I32, device="cuda")
    out, lse = m.paged_decode(q.cuda(), cache, table, torch.tensor([L], dtype=I32, device="cuda"), fmt="mxfp4", max_context=L, softmax_scale=SCALE, return_lse=True)
    check(out, lse, want)
    got = m.gather_context(cache, table, torch.tensor([0, L], dtype=I32, device="cuda"), fmt="mxfp4", num_tokens=L)
    assert np.array_equal(got.double().cpu().numpy(), np.concatenate(ref.values(part.reshape(-1, 400)[:L]), -1))
    slot = torch.tensor([int(nb - 3) * bs + 5], device="cuda")
    lat, z = latents(rng, 1), torch.zeros((1, 1, 512), dtype=BF, device="cuda")
    kpe = ref.bf16(rng.standard_normal((1, 64)))
    m.q_concat_cache_insert(z, z[..., :64].contiguous(), lat.cuda(), kpe.cuda(), cache, slot, fmt="mxfp4")
    assert np.array_equal(cache[nb - 3, 5].cpu().numpy(), ref.records(lat.double().numpy(), kpe)[0])
    assert m.read_device_errors() == 0


# ------------------------------------------------------------------------------------------ how it is called

def test_same_bits_alone_in_a_batch_and_again(m):
    rng = np.random.default_rng(19)
    args, kw, out, lse = run_decode(m, rng, [513, 77, 0, 900], H=48, q_len=2, max_context=900)
    for _ in range(3):
        o, l = m.paged_decode(*args, **kw)
        assert torch.equal(o, out) and torch.equal(l, lse)
    # the same split: the batch's max_context decides it with the number of rows, so one request of the batch repeated
    q, kv, table, seq = args
    o, l = m.paged_decode(q, kv, table, seq.flip(0).flip(0), **kw)
    assert torch.equal(o, out)


def test_captured_and_replayed(m):
    """A graph of insert, decode and read back, replayed on new inputs; two graphs with a workspace of their own."""
    rng = np.random.default_rng(20)
    bs, nb, B, H = 64, 20, 3, 16
    lens = [100, 500, 300]
    cache = torch.from_numpy(make_cache(rng, nb, bs)).cuda()
    table = torch.from_numpy(make_table(rng, lens, bs, nb)).cuda()
    seq = torch.tensor(lens, dtype=I32, device="cuda")
    slots = torch.tensor([int(table[b, (n - 1) // bs]) * bs + (n - 1) % bs for b, n in enumerate(lens)], device="cuda")
    ql, qpe, lat, kpe = (torch.zeros(s, dtype=BF, device="cuda") for s in ((B, H, 512), (B, H, 64), (B, 512), (B, 64)))

    def step(ws):
        q = m.q_concat_cache_insert(ql, qpe, lat, kpe, cache, slots, fmt="mxfp4")
        return m.paged_decode(q, cache, table, seq, fmt="mxfp4", max_context=9000, softmax_scale=SCALE, return_lse=True, workspace=ws)

    n = m.paged_decode_workspace_size(B, 1, H, 9000, fmt="mxfp4")
    graphs = []
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step(torch.empty(n, dtype=U8, device="cuda"))
    s.synchronize()
    for _ in range(2):
        ws = torch.empty(n, dtype=U8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            res = step(ws)
        graphs.append((g, res, ws))
    for i in range(4):
        for t in (ql, qpe, lat, kpe):
            t.copy_(ref.bf16(rng.standard_normal(t.shape)))
        torch.cuda.synchronize()
        g, res, _ = graphs[i % 2]
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in res]
        want = ref.decode(torch.cat([ql, qpe], -1).double().cpu().numpy(), cache.cpu().numpy(), table.cpu().numpy(), lens, bs, 1, SCALE)
        check(*got, want)
        again = step(torch.empty(n, dtype=U8, device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_two_streams_at_once(m):
    rng = np.random.default_rng(21)
    jobs = []
    for seed in (1, 2):
        args, kw, out, lse = run_decode(m, np.random.default_rng(seed), [2000 + seed, 700], H=32)
        jobs.append((args, kw, out, lse, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for args, kw, out, lse, st in jobs:
            with torch.cuda.stream(st):
                got.append((m.paged_decode(*args, **kw), out, lse))
    torch.cuda.synchronize()
    for (o, l), out, lse in got:
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_no_allocation_form_and_selected_pages(m):
    """The decode without a workspace gives the same bits; the decode over selected pages attends those."""
    import ctypes
    rng = np.random.default_rng(22)
    args, kw, out, lse = run_decode(m, rng, [900, 200], H=16, max_context=900)
    q, kv, table, seq = args
    o, l = torch.empty_like(out), torch.empty_like(lse)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    assert m.lib().mla_paged_decode_noalloc(p(q), q.stride(0), q.stride(1), p(kv), 3, kv.shape[0], kv.stride(0), kv.stride(1), 64, p(table), table.stride(0),
                                            p(seq), 2, 1, 16, 900, SCALE, 1.0, 1.0, p(o), o.stride(0), o.stride(1), p(l),
                                            ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    assert torch.equal(o, out) and torch.equal(l, lse)
    pages = [[0, 3, 14], [1, 3, -1]]
    blocks = torch.tensor(pages, dtype=I32, device="cuda")
    o, l = m.selected_decode(q, kv, table, seq, blocks, fmt="mxfp4", softmax_scale=SCALE, return_lse=True)
    want = []
    for b, L in enumerate([900, 200]):
        pos = [x for c in pages[b] if c >= 0 for x in range(c * 64, min(L, c * 64 + 64))]
        lat, rope = ref.values(ref.keys_of(kv.cpu().numpy(), table[b].cpu().numpy(), L, 64)[pos])
        want.append(ref.attend(q[b].double().cpu().numpy(), lat, rope, SCALE))
    check(o, l, [np.stack(z) for z in zip(*want)])


def test_both_marshallings_give_the_same(m, monkeypatch):
    rng = np.random.default_rng(23)
    args, kw, out, lse = run_decode(m, rng, [100, 300], H=16)
    q, kv, table, seq = args
    cu = torch.tensor([0, 100, 400], dtype=I32, device="cuda")

    def run():
        c = kv.clone()
        d = m.paged_decode(*args, **kw)
        g = m.gather_context(kv, table, cu, fmt="mxfp4", num_tokens=400)
        qc = m.q_concat_cache_insert(q[..., :512], q[..., 512:], q[:, 0, :512], q[:, 0, 512:], c, torch.tensor([1, 2], device="cuda"), fmt="mxfp4")
        kn = torch.ones((2, 16, 128), dtype=BF, device="cuda")
        q2 = torch.ones((2, 16, 192), dtype=BF, device="cuda")
        kc = m.key_concat_cache_insert(q2, kn, q[:, 0, 512:], q[:, 0, :512], c, torch.tensor([8, 9], device="cuda"), fmt="mxfp4")
        return [*d, g, qc, kc, c]

    served = []
    real = m._plain_step()

    class Counted:
        def __getattr__(self, name):
            def call(*a):
                r = getattr(real, name)(*a)
                served.append(r is not None)
                return r
            return call

    monkeypatch.setattr(m, "_step", Counted())
    a = run()
    assert len(served) == 4 and all(served)
    monkeypatch.setattr(m, "_step", m._DeclinedStep)
    b = run()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_wait_limit_is_reported(m):
    """The loaders write nothing (a test aid): every wait ends after 20 ms, the error word says so, and the next call is whole."""
    rng = np.random.default_rng(24)
    args, kw, out, lse = run_decode(m, rng, [300, 40], H=16)
    m.lib().mla_debug_stall_next_decode(20000)
    m.paged_decode(*args, **kw)
    assert m.read_device_errors() & 16
    o, l = m.paged_decode(*args, **kw)
    assert torch.equal(o, out) and torch.equal(l, lse) and m.read_device_errors() == 0


@pytest.mark.parametrize("H", [32, 48, 64, 128])
def test_wait_limit_of_more_columns(m, H):
    rng = np.random.default_rng(25)
    args, kw, out, lse = run_decode(m, rng, [300, 40, 700], H=H)
    m.lib().mla_debug_stall_next_decode(20000)
    m.paged_decode(*args, **kw)
    assert m.read_device_errors() & 16
    o, l = m.paged_decode(*args, **kw)
    assert torch.equal(o, out) and torch.equal(l, lse) and m.read_device_errors() == 0


@pytest.mark.parametrize("B,H", [(1, 16), (1, 48), (2, 128), (12, 16), (19, 16), (20, 16)])
def test_joins_of_many_and_few_parts(m, B, H):
    """Requests that many runs share, around the number from which on a join has fewer loads on their way."""
    rng = np.random.default_rng(B)
    run_decode(m, rng, [int(x) for x in rng.integers(2500, 4000, B)], H=H)


@pytest.mark.parametrize("seed", range(24))
def test_fuzz(m, seed):
    rng = np.random.default_rng(1000 + seed)
    q_len = int(rng.choice([1, 1, 1, 2, 3, 4]))
    lens = [int(x) for x in rng.integers(0, int(rng.choice([3, 130, 500, 1300])) + 1, int(rng.integers(1, 6)))]
    run_decode(m, rng, lens, q_len=q_len, H=int(rng.choice([1, 5, 16, 24, 33, 64, 128])), bs=int(rng.choice([5, 16, 32, 64, 128, 192])),
               spread=float(rng.choice([0.2, 1.0, 2.5])), scale=float(rng.choice([SCALE, 0.2])), max_context=max(lens) + int(rng.integers(1, 4000)))
