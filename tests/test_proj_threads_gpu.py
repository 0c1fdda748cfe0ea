"""Projections from several host threads at once, each on its own stream, of different rows and with and without
adapters: their launches ask for different amounts of shared memory of the same kernels."""
import threading

import pytest
import torch

import gated_deltanet_verify_gb300 as gdn
from tests.test_lora_gpu import Case, shape_of

pytestmark = pytest.mark.gpu

ROUNDS = 1500


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(0)


def test_projections_from_several_threads():
    # (slots, tokens, rank or None); 1 x 16 asks for the most, 6 x 16 for the least
    jobs = [(1, 16, None), (6, 16, None), (2, 16, None), (1, 16, 16), (96, 1, 128), (6, 16, 8), (32, 1, 64)]
    cases, want, errors = [], [], []
    for i, (B, T, rank) in enumerate(jobs):
        c = Case(shape_of(n_slots=B, n_tokens=T), "in", 3, rank or 8, [k % 4 - 1 for k in range(B)], seed=i)
        c.out = torch.empty((c.M, c.N), dtype=torch.bfloat16, device="cuda")
        want.append(c.plain() if rank is None else c.run().clone())
        cases.append(c)
    torch.cuda.synchronize()
    start = threading.Barrier(len(jobs))

    def work(c, plain):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            start.wait()
            for k in range(ROUNDS):
                if plain:
                    gdn.gdn_project_in(c.dims, c.weights, c.x, c.out, None, 0, stream=stream)
                else:
                    gdn.gdn_project_in_lora(c.dims, c.weights, c.lora, c.ids, c.x, c.out, c.space, c.size, stream=stream)
                if k % 100 == 99:
                    stream.synchronize()
        except Exception as e:          # reported below
            errors.append((k, repr(e)))

    threads = [threading.Thread(target=work, args=(c, j[2] is None)) for c, j in zip(cases, jobs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for c, w in zip(cases, want):
        assert torch.equal(c.out, w), (c.M, c.rank)
