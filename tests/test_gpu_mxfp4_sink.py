"""The 4-bit cache's decode over rows with one dominating key and many small weights, against 64 bits on the GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
U8, BF, I32, F64 = torch.uint8, torch.bfloat16, torch.int32, torch.float64


@pytest.fixture(scope="module")
def m():
    import mla_latent_cache_attention_gb300 as mod
    mod.lib()
    return mod


def records(g, n):
    """Records whose channels have a mean of their own: magnitudes 0.5 to 4 of one sign a channel, groups of three exponents."""
    sign = torch.randint(0, 2, (512,), generator=g, device="cuda") * 8
    code = torch.randint(1, 7, (n, 512), generator=g, device="cuda") + sign
    rec = torch.empty((n, 400), dtype=U8, device="cuda")
    rec[:, :256] = (code[:, 0::2] + 16 * code[:, 1::2]).to(U8)
    rec[:, 256:272] = torch.randint(123, 126, (n, 16), generator=g, device="cuda").to(U8)
    rec[:, 272:] = (0.1 * torch.randn((n, 64), generator=g, device="cuda")).to(BF).view(U8)
    return rec


def values(rec):
    """Latents and rope values in 64 bits."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=F64, device="cuda")
    b = rec[:, :256].long()
    code = torch.stack([b & 15, b >> 4], -1).flatten(1)
    sc = torch.exp2(rec[:, 256:272].double() - 127).repeat_interleave(32, 1)
    return grid[code] * sc, rec[:, 272:].contiguous().view(BF).double()


def attend(q, lat, rope):
    """Row [H, 576] over keys: out, lse, and the bounds of their errors.

    A weight is off by at most 2^-10 of itself (2^-11 where its third term is rounded, 2^-11 where the whole is, to f16), or 2^-17
    on the scale on which the reference is 2^10: 2^-27 of the largest weight with its key's power of two, and 2^-10 of
    that over the 2^17 keys of the longest row, whatever the row's length.  In an output that is the bound times a key's
    largest code on that scale, 4 * 2^6 here, where the key of the largest weight has one of 2 * 2^6 at least (512
    codes of 0.5 to 4): twice the bound times its largest value.  Accumulators are cut off by 2^-23 a product: 2^-9.4 over three
    products a 32 of 2^17 keys; with the weights' 2^-10 below 2^-8 in all.  The output is rounded to bf16 (2^-8).  Logits:
    sums of 576 products in fp32, a query off by 2^-18 of its row's largest value where hi and lo terms share accumulators."""
    x = (q[:, :512] @ lat.T + q[:, 512:] @ rope.T) * SCALE
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[:, None])
    mag = q[:, :512].abs() @ lat.abs().T + q[:, 512:].abs() @ rope.abs().T
    dx = (SCALE * (576 * 2.0 ** -24 * mag + 2.0 ** -18 * q[:, :512].abs().amax(-1, keepdim=True) * lat.abs().sum(-1)) + 2.0 ** -20 * (1 + x.abs())).amax(-1, keepdim=True)
    out = p @ lat
    top = (p * lat.abs().amax(-1)).amax(-1, keepdim=True)
    return out, lse, 2.0 ** -8 * out.abs() + (2.0 ** -8 + dx) * (p @ lat.abs()) + 2 * 2.0 ** -10 * top, dx[:, 0] + 1e-6


def run(m, L, q_len, H, gaps, where, B, seed=0, bs=64):
    """B requests over the same L keys with the same queries; key where[i] stands gaps[i] nats above the mean of the others, whose
    logits are normal with a deviation of about 0.5."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    nb = -(-L // bs)
    rec = records(g, nb * bs)
    lat, rope = values(rec)
    q = torch.randn((q_len, H, 576), generator=g, device="cuda")
    q[..., :512] *= 1.8
    # the last 64 values of the queries are near 1, so that a key's constant rope values move its logits alike
    q[..., 512:] = 1 + 0.05 * q[..., 512:]
    q = q.to(BF)
    for gap, i in zip(gaps, where):
        rec[i] = rec[(i + L // 3 + 1) % L]
        rec[i, 272:] = torch.full((64,), gap / (64 * SCALE), device="cuda").to(BF).view(U8)
    lat, rope = values(rec)
    perm = torch.randperm(nb, generator=g, device="cuda")
    cache = torch.empty((nb, bs, 400), dtype=U8, device="cuda")
    cache[perm] = rec.view(nb, bs, 400)
    table = perm.to(I32)[None].expand(B, nb).contiguous()
    out, lse = m.paged_decode(q.repeat(B, 1, 1), cache, table, torch.full((B,), L, dtype=I32, device="cuda"), fmt="mxfp4", q_len=q_len, max_context=L,
                              softmax_scale=SCALE, return_lse=True)
    assert m.read_device_errors() == 0
    out, lse = out.view(B, q_len, H, 512), lse.view(B, q_len, H)
    for i in range(q_len):
        n = L - q_len + 1 + i
        o, l, tol, ltol = attend(q[i].double(), lat[:n], rope[:n])
        for b in {0, B // 2, B - 1}:
            err = (out[b, i].double() - o).abs()
            what = (b, i, (err.norm() / o.norm()).item(), (err / tol).max().item())
            assert bool(((lse[b, i].double() - l).abs() <= ltol).all()), what
            assert err.norm() <= 2.0 ** -8 * o.norm(), what
            assert bool((err <= tol).all()), what
    return out


def one_run_each():
    return torch.cuda.get_device_properties(0).multi_processor_count


COLUMNS = [(1, 16), (1, 32), (1, 48), (4, 16)]


@pytest.mark.parametrize("q_len,H", COLUMNS)
@pytest.mark.parametrize("L,gap", [(8192, 11), (32768, 11), (32768, 12), (131072, 11), (131072, 12), (131072, 15)])
def test_first_key_dominates_one_run_a_request(m, q_len, H, L, gap):
    """As many requests of equal length as SMs: every request is one run of tiles, whose reference is its first key."""
    out = run(m, L, q_len, H, [gap], [0], one_run_each())
    assert torch.equal(out, out[:1].expand_as(out))


@pytest.mark.parametrize("B", [1, 2, 7, 40])
@pytest.mark.parametrize("q_len,H", COLUMNS)
@pytest.mark.parametrize("L,gap", [(32768, 11), (131072, 12)])
def test_first_key_dominates_several_runs_a_request(m, q_len, H, L, gap, B):
    run(m, L, q_len, H, [gap], [0], B)


@pytest.mark.parametrize("q_len,H", COLUMNS)
@pytest.mark.parametrize("gap", [-5, 0, 3, 6, 9, 13, 17])
def test_any_distance(m, q_len, H, gap):
    run(m, 32768, q_len, H, [gap], [0], one_run_each(), seed=1)


@pytest.mark.parametrize("q_len,H", COLUMNS + [(1, 128), (2, 96)])
@pytest.mark.parametrize("gaps,where", [([12], [16000]), ([6, 9, 12], [0, 5000, 20000]), ([12, 9], [300, 30000]), ([11.5], [32767]), ([10, 10, 10], [0, 1, 127])])
def test_dominating_keys_elsewhere(m, q_len, H, gaps, where):
    """In the middle, at the end, several that rise or fall: what came before a larger one is small, too."""
    run(m, 32768, q_len, H, gaps, where, one_run_each(), seed=2)
