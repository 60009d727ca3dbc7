"""Results of the page and step calls, made inside and outside inference_mode by
one loop: each may be changed in place afterwards, and changes no other."""
import numpy as np
import pytest
import torch

from kv_cache_vector_gb300 import abi
from test_gpu_steps import books, gpu_table, kept_lists, pool, t32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_cache_vector_gb300 import build
    build.build()
    abi.lib()
    abi.tq_device_status(reset=True)


@pytest.mark.parametrize("first", [True, False])
def test_results_of_a_loop_in_two_modes(first):
    rng = np.random.default_rng(3)
    table, lens, refs, counts = books(rng, 11, 6, 90, 32)
    kept, n_keep = kept_lists(rng, counts, 4)
    layers = abi.PagedLayers(pool(rng, 1, len(refs), 1, 32, 32, 4, 2))
    tb, c, k, nk = gpu_table(table, lens, refs), t32(counts), t32(kept), t32(n_keep)
    T, made, values = int(counts.sum()) + 3, [], []
    side = torch.cuda.Stream()  # with nothing left over from other tests
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i in range(24):
            with torch.inference_mode((i % 2 == 0) == first):
                m = abi.tq_pages_slots(tb, c, T, 32)
                new = abi.tq_pages_keep(tb, c, k, nk, layers)
                _, info = abi.tq_pages_resize(tb, new, layers, out=gpu_table(table, lens, refs))
                made += [m.cu_q, m.positions, m.slots, new, info]
        values = [t.tolist() for t in made]
        for t in made:
            t.add_(1)
        for t, v in zip(made, values):
            assert t.tolist() == [x + 1 for x in v] and t._version <= 1
        weight = torch.ones(200, 4, device="cuda", requires_grad=True)
        a, b = abi.tq_pages_slots(tb, c, T, 32), abi.tq_pages_slots(tb, c, T, 32)
        loss = torch.nn.functional.embedding(a.positions, weight).sum()
        b.positions.add_(1)
        loss.backward()
        assert weight.grad.sum() == 4 * T
    assert abi.tq_device_status(reset=True) == 0


def test_batches_of_many_sizes_hold_no_memory():
    """Each call of tq_pages_keep has another number of rows than the one before."""
    most = 600
    layers = abi.PagedLayers(pool(np.random.default_rng(1), 1, 4, 1, 32, 32, 4, 2))
    table, zeros = abi.PageTable.empty(most, 1, 4), torch.zeros(most, dtype=torch.int32, device="cuda")
    lists = zeros[:, None]

    def all_sizes():
        for n in range(1, most + 1):
            part = abi.PageTable(table.block_table[:n], table.lens[:n], table.refs)
            new = abi.tq_pages_keep(part, zeros[:n], lists[:n], zeros[:n], layers)
            assert new.numel() == n

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        before = torch.cuda.memory_allocated()
        all_sizes()
        assert torch.cuda.memory_allocated() - before <= 2 ** 20
        new = [abi.tq_pages_keep(table, zeros, lists, zeros, layers) for _ in range(100)]
        assert len({t.data_ptr() for t in new}) == 100
    side.synchronize()
    assert abi.tq_device_status(reset=True) == 0
