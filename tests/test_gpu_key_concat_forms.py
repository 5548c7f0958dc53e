"""The key-concat epilogue in all its forms (wide and narrow CTAs, vector and scalar accesses) over the bf16, fp8_ds_mla and mxfp4
caches: keys and rotated queries bit for bit, records against their definition."""
import numpy as np
import pytest
import torch

import mxfp4_ref as ref

pytestmark = pytest.mark.gpu

BF, U8 = torch.bfloat16, torch.uint8
WIDTH = {"bf16": (576, BF), "fp8_ds_mla": (656, U8), "mxfp4": (400, U8)}


@pytest.fixture(scope="module")
def m():
    import mla_latent_cache_attention_gb300 as mod
    mod.lib()
    return mod


def unaligned(x):
    """The same values two bytes behind a 16-byte border."""
    flat = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")
    y = flat[1:].view(x.shape)
    y.copy_(x)
    return y


def run(m, fmt, T, H, dn, rope, crooked, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, kn, kpe, lat = (torch.randn(s, generator=g, device="cuda").to(BF) for s in ((T, H, dn + 64), (T, H, dn), (T, 64), (T, 512)))
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda") if rope else None
    tab = m.rope_table(5000, 64) if rope else None
    bs, nb = 16, -(-T // 16) + 2
    slots = torch.randperm(nb * bs, generator=g, device="cuda")[:T]
    slots[T // 2] = -1
    w, dt = WIDTH[fmt]
    cache = torch.full((nb, bs, w), 7, dtype=dt, device="cuda")
    q0 = unaligned(q) if "q" in crooked else q.clone()
    k = m.key_concat_cache_insert(q0, unaligned(kn) if "k" in crooked else kn, kpe, lat, cache, slots, fmt=fmt, positions=pos, cos_sin_cache=tab)
    assert m.read_device_errors() == 0
    # queries and keys: the same arithmetic as rope's
    turned = m.rope(kpe[:, None], pos, tab)[:, 0] if rope else kpe
    assert torch.equal(q0, m.rope(q, pos, tab) if rope else q)
    assert torch.equal(k[..., :dn], kn) and torch.equal(k[..., dn:], turned[:, None].expand(T, H, 64))
    live = (slots >= 0).cpu().numpy()
    got = cache.view(nb * bs, w)
    if fmt == "bf16":
        assert torch.equal(got[slots[slots >= 0]], torch.cat([lat, turned], 1)[slots >= 0])
    elif fmt == "mxfp4":
        want = ref.records(lat.double().cpu().numpy(), turned.cpu())[live]
        assert np.array_equal(got[slots[slots >= 0]].cpu().numpy(), want)
    else:
        assert torch.equal(got[slots[slots >= 0]][:, 528:].contiguous().view(BF), turned[slots >= 0])
    left = torch.ones(nb * bs, dtype=torch.bool, device="cuda")
    left[slots[slots >= 0]] = False
    assert bool((got[left] == 7).all())


@pytest.mark.parametrize("fmt", WIDTH)
@pytest.mark.parametrize("rope", [True, False])
@pytest.mark.parametrize("crooked", ["", "q", "k", "qk"])
@pytest.mark.parametrize("H", [1, 4, 5, 16, 17, 33])
def test_heads_and_alignment(m, fmt, rope, crooked, H):
    run(m, fmt, 37, H, 128, rope, crooked)


@pytest.mark.parametrize("fmt", WIDTH)
@pytest.mark.parametrize("dn", [8, 136, 264, 512])
@pytest.mark.parametrize("H", [3, 16, 20])
def test_widths(m, fmt, dn, H):
    run(m, fmt, 21, H, dn, True, "")


@pytest.mark.parametrize("fmt", WIDTH)
@pytest.mark.parametrize("T", [1, 1023, 1024, 1025])
@pytest.mark.parametrize("H", [2, 4, 5])
def test_prompts_of_few_heads(m, fmt, T, H):
    """Around the length from which few heads take the narrow CTAs."""
    run(m, fmt, T, H, 128, True, "")
