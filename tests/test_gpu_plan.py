"""Planned steps on the GPU against a plain reference, and a run of the step's operators together."""
import copy
import random

import numpy as np
import pytest
import torch

import mxfp4_ref
import plan_ref

pytestmark = pytest.mark.gpu

I32, I64 = torch.int32, torch.int64


@pytest.fixture(scope="module")
def m():
    import mla_latent_cache_attention_gb300 as mod
    mod.lib()
    return mod


class State:
    def __init__(self, seq, bs, cols, spare, rng, cap=None):
        per = [-(-max(n, 0) // bs) for n in seq]
        total = sum(per) + spare
        ids = list(range(total))
        rng.shuffle(ids)
        self.seq, self.bs = list(seq), bs
        self.table = [[-1 if c >= p else ids.pop() for c in range(cols)] for p in per]
        self.cap = total if cap is None else cap
        self.free = ids[:self.cap] + [-5] * (self.cap - len(ids[:self.cap]))
        self.num_free = min(len(ids), self.cap)
        self.dev = [torch.tensor(x, dtype=I32, device="cuda") for x in (self.seq, self.table, self.free, [self.num_free])]

    def step(self, m, new, T, finished=None, inplace=True, **kw):
        seq, table, free, nf = self.dev
        fin = None if finished is None else torch.tensor(finished, device="cuda")
        served = torch.empty(len(self.seq), dtype=torch.bool, device="cuda")
        out = m.plan_step(seq, torch.tensor(new, dtype=I32, device="cuda"), table, free, nf, block_size=self.bs, num_tokens=T, finished=fin,
                          served=served, **(dict(seq_lens_out=seq, num_free_out=nf) if inplace else {}), **kw)
        want = plan_ref.plan(self.seq, new, self.table, self.free, self.num_free, self.bs, T, finished)
        names = ("slots", "positions", "cu", "seq", "num_free", "served")
        got = [x.tolist() for x in out] + [served.tolist()]
        for name, g, w in zip(names, got, (*want[:4], [want[4]], want[5])):
            assert g == w, name
        assert table.tolist() == self.table and free.tolist() == self.free
        assert m.read_device_errors() == (0 if want[6] else 32)
        if not inplace:
            assert seq.tolist() == self.seq and nf.tolist() == [self.num_free]
            seq.copy_(out[3])
            nf.copy_(out[4])
        self.seq, self.num_free = want[3], want[4]
        return out


@pytest.mark.parametrize("B", [1, 2, 31, 33, 1024, 1025, 2500])
@pytest.mark.parametrize("bs", [1, 16, 64])
def test_decode_steps(m, B, bs):
    rng = random.Random(B * 100 + bs)
    seq = [rng.choice([0, 1, bs - 1, bs, rng.randrange(5 * bs)]) for _ in range(B)]
    s = State(seq, bs, 12 if bs > 1 else 40, 4 * B, rng)
    for i in range(3):
        s.step(m, [1] * B, B + 3 * i, inplace=i != 1)


@pytest.mark.parametrize("T", [0, 1, 4095, 4096, 4097, 20000])
def test_rows_of_one_cta_and_of_many(m, T):
    """Mixed chunks, requests without tokens, rows behind the last request."""
    rng = random.Random(T)
    B, bs = 40, 32
    s = State([rng.randrange(3000) for _ in range(B)], bs, 1000, 900, rng)
    new = [0] * B
    left = max(0, T - 5)
    for b in range(B):
        new[b] = min(left, rng.choice([0, 1, 1, rng.randrange(1500)]))
        left -= new[b]
    s.step(m, new, T)


@pytest.mark.parametrize("seed", range(30))
def test_fuzz_with_finished_requests(m, seed):
    """Long runs of steps: requests finish, their places are taken again, blocks run out, tables are too short."""
    rng = random.Random(seed)
    B, bs = rng.randrange(1, 70), rng.choice([1, 3, 16, 64])
    cols = rng.randrange(2, 30)
    s = State([rng.randrange(cols * bs) for _ in range(B)], bs, cols, rng.randrange(0, 60), rng)
    for _ in range(6):
        new = [rng.choice([0, 1, 1, -3, rng.randrange(4 * bs)]) for _ in range(B)]
        T = max(0, sum(max(n, 0) for n in new) + rng.choice([0, 0, 7, -2]))
        s.step(m, new, T, finished=rng.choice([None, [rng.random() < 0.3 for _ in range(B)]]), inplace=rng.random() < 0.5)


def test_the_stack_is_full(m):
    """Returned blocks that find no place are lost, and the error word says so."""
    rng = random.Random(5)
    s = State([64, 64, 64], 16, 8, 2, rng, cap=5)
    s.step(m, [0, 0, 0], 0, finished=[True, True, False])


def test_out_of_blocks_keeps_the_order(m):
    """The first requests get theirs; a later one that needs no block is served all the same."""
    rng = random.Random(6)
    s = State([16, 16, 5, 16], 16, 8, 1, rng)
    out = s.step(m, [1, 1, 1, 1], 4)
    assert [x >= 0 for x in out[0].tolist()] == [True, False, True, False]


def test_captured_steps_advance(m):
    """A graph of an in-place step, replayed: lengths, stack and table go on."""
    rng = random.Random(7)
    s = State([3, 17, 0], 16, 8, 9, rng)
    seq, table, free, nf = s.dev
    new = torch.ones(3, dtype=I32, device="cuda")
    outs = [torch.empty(5, dtype=I64, device="cuda"), torch.empty(5, dtype=I64, device="cuda"), torch.empty(4, dtype=I32, device="cuda"),
            torch.empty(3, dtype=torch.bool, device="cuda")]
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=st):
        m.plan_step(seq, new, table, free, nf, block_size=16, num_tokens=5, seq_lens_out=seq, num_free_out=nf, slot_mapping=outs[0],
                    positions=outs[1], cu_q_lens=outs[2], served=outs[3])
    for _ in range(20):
        g.replay()
        want = plan_ref.plan(s.seq, [1, 1, 1], s.table, s.free, s.num_free, 16, 5)
        s.seq, s.num_free = want[3], want[4]
        assert [outs[0].tolist(), outs[1].tolist(), outs[2].tolist(), seq.tolist(), nf.item()] == [*want[:4], want[4]]
        assert table.tolist() == s.table
    assert m.read_device_errors() == 0


def test_both_marshallings_give_the_same(m, monkeypatch):
    rng = random.Random(8)
    a, b = State([5, 70, 33], 16, 9, 12, rng), None
    b = copy.deepcopy(a)
    real, served = m._plain_step(), []

    class Counted:
        def plan(self, *x):
            r = real.plan(*x)
            served.append(r is not None)
            return r

    monkeypatch.setattr(m, "_step", Counted())
    x = a.step(m, [4, 40, 0], 50, finished=[False, False, True])
    assert served == [True]
    monkeypatch.setattr(m, "_step", m._DeclinedStep)
    y = b.step(m, [4, 40, 0], 50, finished=[False, False, True])
    assert all(torch.equal(i, j) for i, j in zip(x, y))


# ------------------------------------------------------------------------------------------ together

def test_a_server_s_steps(m):
    """Requests come, run and go: every step is planned on the GPU, its queries and keys rotated with the table, its
    latents written to the 4-bit cache, the context read back, and a decode step attends the cache.  Against a plain
    model of the same server in 64 bits."""
    rng, nrng = random.Random(9), np.random.default_rng(9)
    B, bs, cols, H, nb, scale = 4, 16, 12, 4, 40, 192 ** -0.5
    tab = m.rope_table(256, 64, scaling="yarn", factor=4.0, original=64)
    tab64 = tab.double().cpu().numpy()
    seq, nf = torch.zeros(B, dtype=I32, device="cuda"), torch.tensor([nb], dtype=I32, device="cuda")
    table, free = torch.zeros((B, cols), dtype=I32, device="cuda"), torch.randperm(nb, device="cuda").to(I32)
    cache = torch.zeros((nb, bs, 400), dtype=torch.uint8, device="cuda")
    kept = [np.zeros((0, 400), np.uint8) for _ in range(B)]             # the model's records of every request

    def turned(x, pos):
        c, s = tab64[pos][..., :32], tab64[pos][..., 32:]
        while c.ndim < x.ndim:
            c, s = c[:, None], s[:, None]
        y = np.empty_like(x)
        y[..., 0::2], y[..., 1::2] = x[..., 0::2] * c - x[..., 1::2] * s, x[..., 1::2] * c + x[..., 0::2] * s
        return y

    # prefill chunks, decode steps, two requests that end and a new one in the place of one of them
    plan = [([20, 1, 33, 0], None), ([1, 1, 1, 0], None), ([1, 40, 1, 17], None), ([1, 1, 1, 1], None), ([30, 1, 0, 1], [True, False, True, False]),
            ([1, 1, 0, 1], None)]
    for new, fin in plan:
        T = sum(new) + 3
        slots, pos, cu, seq, nf = m.plan_step(seq, torch.tensor(new, dtype=I32, device="cuda"), table, free, nf, block_size=bs, num_tokens=T,
                                              finished=None if fin is None else torch.tensor(fin, device="cuda"))
        lat = mxfp4_ref.bf16(nrng.standard_normal((T, 512)))
        ql, qpe, kpe = (mxfp4_ref.bf16(nrng.standard_normal(s)) for s in ((T, H, 512), (T, H, 64), (T, 64)))
        # the same rotation by the operator of its own and by the epilogue
        qr = m.rope(qpe.cuda(), pos, tab)
        q = m.q_concat_cache_insert(ql.cuda(), qpe.cuda(), lat.cuda(), kpe.cuda(), cache, slots, fmt="mxfp4", positions=pos, cos_sin_cache=tab)
        assert torch.equal(q[..., 512:], qr)
        back = m.gather_context(cache, table, torch.cat([torch.zeros(1, dtype=I32, device="cuda"), seq.cumsum(0).to(I32)]), fmt="mxfp4",
                                num_tokens=int(seq.sum()))
        # the model
        hp, hc = pos.cpu().numpy(), cu.tolist()
        assert (slots[sum(new):] == -1).all()
        krot = mxfp4_ref.bf16(turned(kpe.double().numpy(), hp))         # fp32 arithmetic: compared below with a rounding's room
        rec = mxfp4_ref.records(lat.double().numpy(), krot)
        for b in range(B):
            if fin and fin[b]:
                kept[b] = kept[b][:0]
            assert hp[hc[b]:hc[b + 1]].tolist() == list(range(len(kept[b]), len(kept[b]) + new[b]))
            kept[b] = np.concatenate([kept[b], rec[hc[b]:hc[b + 1]]])
        assert seq.tolist() == [len(k) for k in kept]
        want = np.concatenate([np.concatenate(mxfp4_ref.values(k), -1) for k in kept])
        got = back.double().cpu().numpy()
        assert np.array_equal(got[:, :512], want[:, :512])
        assert np.all(np.abs(got[:, 512:] - want[:, 512:]) <= 2.0 ** -7 * np.abs(want[:, 512:]) + 2.0 ** -20)
        # every request's last row attends its cache
        last = [hc[b + 1] - 1 for b in range(B)]
        if all(n > 0 for n in new):
            out, lse = m.paged_decode(q[last].contiguous(), cache, table, seq, fmt="mxfp4", max_context=cols * bs, softmax_scale=scale, return_lse=True)
            at = 0
            for b in range(B):
                n = len(kept[b])
                o, l, tol, ltol = mxfp4_ref.attend(q[last[b]].double().cpu().numpy(), got[at:at + n, :512], got[at:at + n, 512:], scale)
                assert np.all(np.abs(out[b].double().cpu().numpy() - o) <= tol) and np.all(np.abs(lse[b].double().cpu().numpy() - l) <= ltol)
                at += n
    assert m.read_device_errors() == 0


@pytest.mark.parametrize("B", [1, 5, 1024, 1025, 3000])
def test_without_the_served_flags(m, monkeypatch, B):
    """The same step whether anybody asks who was served or not, in both forms of the binding; a third of the requests do not fit."""
    g = torch.Generator(device="cuda").manual_seed(B)
    seq, new = (torch.randint(0, n, (B,), generator=g, device="cuda", dtype=torch.int32) for n in (90, 40))
    new[::3] = 1000
    done = torch.rand(B, generator=g, device="cuda") < 0.2

    def run(**kw):
        table = torch.arange(B * 12, dtype=torch.int32, device="cuda").view(B, 12)
        free = torch.arange(B * 12, B * 18, dtype=torch.int32, device="cuda")
        nf = torch.tensor([B * 5], dtype=torch.int32, device="cuda")
        out = m.plan_step(seq, new, table, free, nf, block_size=16, num_tokens=20 * B, finished=done, **kw)
        assert m.read_device_errors() == 32
        return [*out, table, free]

    want = run(served=torch.empty(B, dtype=torch.bool, device="cuda"))
    for _ in range(2):
        assert all(torch.equal(x, y) for x, y in zip(run(), want))
        monkeypatch.setattr(m, "_step", m._DeclinedStep)
