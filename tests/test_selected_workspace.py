"""One workspace for selected decodes of several row counts: the size of a call is not monotone in its rows."""
import random

import pytest


@pytest.fixture(scope="module")
def L():
    from mla_latent_cache_attention_gb300 import build
    build.build()
    import mla_latent_cache_attention_gb300 as mod
    return mod.lib()


def test_the_size_of_a_call_is_not_monotone(L):
    """32 rows are split over the SMs, 152 rows fill them."""
    n = lambda T: L.mla_selected_decode_workspace_size(0, T, 16, 64, 16, 152)
    assert n(32) > n(152)


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_the_bound_holds_every_smaller_call(L, fmt):
    rng = random.Random(fmt)
    shapes = [(152, 16, 64, 16, 152), (700, 64, 64, 1, 152), (90, 32, 64, 96, 152), (40, 1, 16, 128, 1), (33, 4096, 128, 128, 7)]
    shapes += [(rng.randint(1, 600), rng.randint(1, 200), rng.choice([16, 48, 64, 128]), rng.randint(1, 128), rng.choice([152, 132, 3]))
               for _ in range(12)]
    for T, topk, bs, H, sms in shapes:
        size = lambda t: L.mla_selected_decode_workspace_size(fmt, t, topk, bs, H, sms)
        bound = lambda t: L.mla_selected_decode_workspace_bound(fmt, t, topk, bs, H, sms)
        most = 0
        for t in range(1, T + 1):
            most = max(most, size(t))
            if t % 37 == 0 or t == T:
                assert bound(t) >= most, (t, topk, bs, H, sms)


def test_beyond_the_last_split_the_bound_grows_by_the_lists_alone(L):
    for fmt, H in ((0, 16), (1, 64), (2, 128)):
        n = lambda T: L.mla_selected_decode_workspace_bound(fmt, T, 16, 64, H, 152)
        lists = lambda T: -(-T * 16 * 4 // 256) * 256 + -(-T * 4 // 256) * 256
        assert n(100000) - n(20000) == lists(100000) - lists(20000)
        assert all(L.mla_selected_decode_workspace_size(fmt, t, 16, 64, H, 152) <= n(20000) for t in range(19000, 20001))


def test_no_size_without_a_shape(L):
    f = L.mla_selected_decode_workspace_bound
    assert f(0, 0, 4, 64, 16, 152) == 0 and f(0, 4, 0, 64, 16, 152) == 0 and f(0, 4, 1 << 24, 64, 16, 152) == 0
