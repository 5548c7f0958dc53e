"""The plain fp8 cache's decode over rows with one dominating key and many small weights, against 64 bits on the GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
U8, I32 = torch.uint8, torch.int32


@pytest.fixture(scope="module")
def m():
    import mla_latent_cache_attention_gb300 as mod
    mod.lib()
    return mod


@pytest.mark.parametrize("q_len,H", [(1, 16), (1, 32), (4, 16), (1, 96)])
@pytest.mark.parametrize("L,gap", [(8192, 0), (8192, 11), (32768, 11), (32768, 12), (131072, 12)])
@pytest.mark.parametrize("B", [1, 152])
def test_first_key_dominates(m, q_len, H, L, gap, B):
    """B requests over the same keys: the first one gap nats above the others, whose logits are normal with a deviation of about half
    a nat.  A weight is an E4M3 term and an E5M2 one of the rest: to 2^-7 of itself down to 2^-10 of the reference, then to 2^-3
    (three bits) down to 2^-18.  The small ones' roundings go either way: their logits spread over three of the eighths
    of an octave on which E5M2 rounds, so that of their sum over thousands of keys less than 2^-10 is left; with the
    larger ones' 2^-7, which go either way too, and the output's bf16 the norm is within 2^-8."""
    g = torch.Generator(device="cuda").manual_seed(L + gap)
    bs, nb = 64, L // 64
    sign = torch.randint(0, 2, (512,), generator=g, device="cuda") * 2 - 1
    lat = (0.05 + 0.45 * torch.rand((L, 512), generator=g, device="cuda")) * sign
    kv = torch.cat([lat, 0.1 * torch.randn((L, 64), generator=g, device="cuda")], 1)
    q = torch.randn((q_len, H, 576), generator=g, device="cuda")
    q[..., :512] *= 2.3
    q[..., 512:] = 1
    kv[0, 512:] = gap / (64 * SCALE)
    kv, q = kv.to(torch.float8_e4m3fn), q.to(torch.float8_e4m3fn)
    perm = torch.randperm(nb, generator=g, device="cuda")
    cache = torch.empty((nb, bs, 576), dtype=U8, device="cuda")
    cache[perm] = kv.view(U8).view(nb, bs, 576)
    out, lse = m.paged_decode(q.view(U8).repeat(B, 1, 1), cache, perm.to(I32)[None].expand(B, nb).contiguous(), torch.full((B,), L, dtype=I32, device="cuda"),
                              fmt="fp8", q_len=q_len, max_context=L, softmax_scale=SCALE, return_lse=True)
    assert m.read_device_errors() == 0
    k = kv.double()
    for i in range(q_len):
        x = q[i].double() @ k[:L - q_len + 1 + i].T * SCALE
        want = torch.logsumexp(x, -1)
        o = torch.exp(x - want[:, None]) @ k[:L - q_len + 1 + i, :512]
        for b in {0, B - 1}:
            err = out[b * q_len + i].double() - o
            assert (lse[b * q_len + i].double() - want).abs().max() <= 1e-3
            assert err.norm() <= 2.0 ** -8 * o.norm(), (b, i, (err.norm() / o.norm()).item())
