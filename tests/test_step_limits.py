"""The largest sizes of rope and plan_step: refused on the host where a count would pass 32 bits in the kernel."""
import ctypes

import pytest

FAKE, FAR = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 50)
OK, INVALID, UNSUPPORTED = 0, -1, -2


@pytest.fixture(scope="module")
def L():
    from mla_latent_cache_attention_gb300 import build
    build.build()
    import mla_latent_cache_attention_gb300 as mod
    return mod.lib()


@pytest.mark.parametrize("H,D,want", [(1 << 21, 1024, UNSUPPORTED), (1 << 22, 512, UNSUPPORTED), ((1 << 31) - 1, 64, UNSUPPORTED)])
def test_rope_of_a_token_past_32_bits(L, H, D, want):
    s0 = H * D
    args = lambda h, q: L.mla_rope(0, q, s0, D, FAR, s0, D, h, D, 0, None, 0, 0, None, 0, 0, 0, 0, 0, FAKE, FAKE, 8, 64, 0, 0, 1, None)
    assert args(H, FAKE) == want
    # the largest that is served gets as far as the check of the pointers
    assert args(((1 << 31) - 1) // D, None) == INVALID


@pytest.mark.parametrize("kw", [dict(T=(1 << 31) - 1), dict(T=(1 << 31) - (1 << 13)), dict(B=(1 << 31) - 1), dict(B=(1 << 31) - (1 << 13))])
def test_plan_of_rows_or_requests_past_32_bits(L, kw):
    def plan(seq, B=2, T=4):
        return L.mla_plan_step(seq, FAKE, None, FAKE, 4, 4, FAKE, 16, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, B, T, 64, None)
    assert plan(FAKE, **kw) == UNSUPPORTED
    assert plan(None, **{k: (1 << 31) - (1 << 13) - 1 for k in kw}) == INVALID
