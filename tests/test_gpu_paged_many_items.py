"""Paged decode of batches that give every CTA several work items: the next items' first key tiles are in
shared memory while an item's softmax still moves its reference maximum."""
import numpy as np
import pytest
import torch

from tests import index_ref as ref
from tests.gpu_helpers import assert_attn_close, assert_lse_close, bf16_bits, t_i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["fp8", "bf16"])
@pytest.mark.parametrize("H", [16, 32, 80, 96, 128])
@pytest.mark.parametrize("selected", [False, True])
def test_many_items_a_cta(fmt, H, selected):
    import mla_latent_cache_attention_gb300 as m

    torch.manual_seed(H)
    B, W, ps, nb, scale = max(200, 6400 // H), 3, 64, 400, 0.05
    shape = [(B, H, 576), (nb, ps, 576)]
    if fmt == "fp8":
        q, kv = ((torch.randn(s, device="cuda") * 20).to(torch.float8_e4m3fn).view(torch.uint8) for s in shape)
        qv, vals = (ref.E4M3[x.cpu().numpy()] * scale for x in (q, kv))
    else:
        q, kv = (torch.randn(s, device="cuda").to(torch.bfloat16) for s in shape)
        qv, vals = (ref.bf16_to_f64(bf16_bits(x)) for x in (q, kv))
    rng = np.random.default_rng(H)
    lens = rng.integers(1, W * ps + 1, B).astype(np.int32)
    tab = rng.integers(0, nb, (B, W)).astype(np.int32)
    kw = dict(fmt=fmt, softmax_scale=192 ** -0.5, q_scale=scale, k_scale=scale, return_lse=True)
    if selected:
        pages = t_i32(np.where(np.arange(W) * ps < lens[:, None], np.arange(W), -1).astype(np.int32))
        run = lambda: m.selected_decode(q, kv, t_i32(tab), t_i32(lens), pages, **kw)
    else:
        run = lambda: m.paged_decode(q, kv, t_i32(tab), t_i32(lens), max_context=W * ps, **kw)
    want_o, want_l = np.zeros((B, H, 512)), np.zeros((B, H))
    for b in range(B):
        ent = vals[tab[b]].reshape(-1, 576)[:lens[b]]
        want_o[b], want_l[b] = ref.attend(qv[b], ent, 192 ** -0.5)
    for _ in range(3):
        out, lse = run()
        assert_attn_close(out, want_o, f"{fmt} H={H}")
        assert_lse_close(lse, want_l, f"{fmt} H={H}")
