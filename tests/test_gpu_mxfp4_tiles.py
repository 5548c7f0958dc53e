"""The 4-bit cache's decode at the ends of its tiles (96 keys of 64 columns, else 128; 12 or 16 a loader warp), alone and in a batch."""
import numpy as np
import pytest
import torch

from test_gpu_mxfp4 import SCALE, check, make_cache, make_table, m, ref, run_decode      # noqa: F401  (m: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [16, 32, 40, 48, 64, 96])
@pytest.mark.parametrize("bs", [1, 12, 16, 64])
def test_ends_of_tiles(m, H, bs):
    rng = np.random.default_rng(H * 100 + bs)
    run_decode(m, rng, [95, 96, 97, 127, 128, 129, 0, 1, 12, 13, 16, 17], H=H, bs=bs)
    run_decode(m, rng, [191, 192, 193, 255, 256, 257, 287, 288, 289, 384], H=H, bs=bs)


@pytest.mark.parametrize("q_len,H", [(2, 24), (3, 16), (2, 48), (4, 16), (3, 32)])
def test_ends_of_tiles_of_speculative_rows(m, q_len, H):
    rng = np.random.default_rng(q_len * 100 + H)
    run_decode(m, rng, [q_len, 96, 97, 98, 128, 130, 194, 258], q_len=q_len, H=H)


@pytest.mark.parametrize("H,q_len", [(16, 1), (32, 1), (48, 1), (16, 4)])
def test_alone_and_in_a_batch(m, H, q_len):
    """A request's rows are cut into other runs in a batch than alone: both are within the bounds, and each call repeats its bits."""
    rng = np.random.default_rng(H + q_len)
    lens, bs, nb = [513, 77, 0, 900, 2000], 64, 70
    cache = make_cache(rng, nb, bs)
    table = make_table(rng, lens, bs, nb)
    q = ref.bf16(rng.standard_normal((len(lens) * q_len, H, 576)))
    want = ref.decode(q.double().numpy(), cache, table, lens, bs, q_len, SCALE)
    kv, tab, qd = torch.from_numpy(cache).cuda(), torch.from_numpy(table).cuda(), q.cuda()

    def run(which):
        rows = [b * q_len + i for b in which for i in range(q_len)]
        seq = torch.tensor([lens[b] for b in which], dtype=torch.int32, device="cuda")
        kw = dict(fmt="mxfp4", q_len=q_len, softmax_scale=SCALE, return_lse=True)
        out, lse = m.paged_decode(qd[rows], kv, tab[which].contiguous(), seq, max_context=2000, **kw)
        check(out, lse, [x[rows] for x in want], which)
        # the runs come from the lengths on the GPU: max_context changes nothing
        for ctx in (1, 300, 131072):
            o, l = m.paged_decode(qd[rows], kv, tab[which].contiguous(), seq, max_context=ctx, **kw)
            assert torch.equal(o, out) and torch.equal(l, lse)

    run([0, 1, 2, 3, 4])
    run([4, 3, 2, 1, 0])
    for b in range(len(lens)):
        run([b])
    assert m.read_device_errors() == 0
