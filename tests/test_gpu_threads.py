"""Calls from several host threads at once, each on a stream of its own: the same results as from one."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_selector_calls_of_four_threads():
    import mla_latent_cache_attention_gb300 as m
    m.lib()
    from tests.test_gpu_index import Chain
    chains = [Chain(seed=20 + i) for i in range(4)]
    want = [[t.clone() for t in c.step(m, 4, 64)] for c in chains]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in chains]
    start, failures = threading.Barrier(len(chains)), []

    def run(i):
        try:
            start.wait()
            with torch.cuda.stream(streams[i]):
                for _ in range(20):
                    got = chains[i].step(m, 4, 64)
                    streams[i].synchronize()
                    seen = torch.arange(want[i][0].shape[1], device="cuda") < ((chains[i].seq + 63) // 64)[:, None]
                    for a, b in zip(got, want[i]):
                        if a.shape == seen.shape and a.dtype == torch.float32:
                            a, b = torch.where(seen, a, 0), torch.where(seen, b, 0)
                        if not torch.equal(a, b):
                            failures.append(i)
        except Exception as e:      # a thread's exception would be lost
            failures.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(chains))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures
    assert m.read_device_errors() == 0
