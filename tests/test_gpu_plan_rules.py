"""Who is served by a planned step, from the words of mla.h; and the forms of the kernel that only large steps reach."""
import random

import pytest
import torch

from test_gpu_plan import State

pytestmark = pytest.mark.gpu

I32 = torch.int32


@pytest.fixture(scope="module")
def m():
    import mla_latent_cache_attention_gb300 as mod
    mod.lib()
    return mod


def rules(seq, new, cols, left, bs, T):
    """served, lengths and free blocks after a step without finished requests, one request after the other."""
    served, lens, rows, closed = [], [], 0, False
    up = lambda n: -(-n // bs)
    for L, n in zip(seq, new):
        rows += n
        need = up(L + n) - up(L)
        short = up(L + n) > cols                    # its table row
        if not short and need and (closed or need > left):
            closed, good = True, False
        else:
            good = not short and rows <= T
        if good:
            left -= need
        served.append(good)
        lens.append(L + n if good else L)
    return served, lens, left


def step(m, seq, new, cols, left, bs, T):
    B = len(seq)
    up = lambda n: -(-n // bs)
    dev = lambda x: torch.tensor(x, dtype=I32, device="cuda")
    table = torch.full((B, cols), -1, dtype=I32, device="cuda")
    at = 0
    for b, L in enumerate(seq):
        table[b, :up(L)] = torch.arange(at, at + up(L), dtype=I32, device="cuda")
        at += up(L)
    free = torch.arange(at, at + left + 3, dtype=I32, device="cuda")
    ok = torch.empty(B, dtype=torch.bool, device="cuda")
    slots, pos, cu, lens, nf = m.plan_step(dev(seq), dev(new), table, free, dev([left]), block_size=bs, num_tokens=T, served=ok)
    want = rules(seq, new, cols, left, bs, T)
    assert (ok.tolist(), lens.tolist(), nf.item()) == want
    assert m.read_device_errors() == (0 if all(want[0]) else 32)
    # every served request's blocks are its own
    own = [x for b, (good, L) in enumerate(zip(want[0], want[1])) for x in table[b, :up(L)].tolist()]
    assert len(set(own)) == len(own) and -1 not in own
    for b in range(B):
        rows = slice(cu[b].item(), cu[b + 1].item())
        assert (slots[rows] >= 0).all() if want[0][b] else (slots[rows] == -1).all()
    return want


def test_a_prompt_too_large_is_not_overtaken(m):
    """Five blocks are left, the first request needs ten: the second, which needs one, waits; the third needs none and goes on."""
    assert step(m, [0, 16, 5], [160, 1, 1], 20, 5, 16, 400)[0] == [False, False, True]


def test_a_table_row_too_short_holds_nobody_up(m):
    assert step(m, [0, 16, 5], [160, 1, 1], 9, 5, 16, 400)[0] == [False, True, True]


def test_what_is_left_is_enough_for_the_first(m):
    assert step(m, [16, 16, 16, 0, 15], [1, 33, 1, 1, 1], 20, 3, 16, 400)[0] == [True, False, False, False, True]


@pytest.mark.parametrize("seed", range(20))
def test_rules(m, seed):
    rng = random.Random(seed)
    B, bs = rng.choice([3, 20, 300, 1100]), rng.choice([1, 4, 16])
    seq = [rng.randrange(4 * bs) for _ in range(B)]
    new = [rng.choice([0, 1, 1, 1, rng.randrange(6 * bs)]) for _ in range(B)]
    need = sum(-(-(a + b) // bs) - -(-a // bs) for a, b in zip(seq, new))
    T = sum(new) + rng.choice([0, 5, 3000, -rng.randrange(1 + sum(new))])
    step(m, seq, new, rng.choice([9, 12]), rng.randrange(need + 3), bs, T)


@pytest.mark.parametrize("B,cols,cap", [(256, 64, None), (256, 64, 900), (1025, 20, None), (2500, 12, None), (2500, 12, 5000)])
def test_finished_requests_of_large_steps(m, B, cols, cap):
    """The copies that eight CTAs share, several chunks of requests, and a stack that runs over."""
    rng = random.Random(B + cols)
    bs = 16
    s = State([rng.choice([0, 1, 15, 16, rng.randrange(cols * bs // 2)]) for _ in range(B)], bs, cols, 2 * B, rng, cap=cap)
    for i in range(4):
        new = [rng.choice([0, 1, 1, rng.randrange(40)]) for _ in range(B)]
        s.step(m, new, sum(new) + rng.choice([0, 9, -3]), finished=[rng.random() < 0.4 for _ in range(B)], inplace=i % 2 == 0)


@pytest.mark.parametrize("T", [2047, 2048, 2049])
@pytest.mark.parametrize("finished", [False, True])
def test_rows_around_the_cluster_s_border(m, T, finished):
    rng = random.Random(T)
    B, bs = 40, 32
    s = State([rng.randrange(600) for _ in range(B)], bs, 200, 900, rng)
    new = [T // B + rng.randrange(-5, 6) for _ in range(B)]
    s.step(m, new, T, finished=[rng.random() < 0.3 for _ in range(B)] if finished else None)
