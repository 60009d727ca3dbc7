"""Attention of few rows where cu_q steps back: the sequences whose entries are out
of range are left out, and all the others are there, also where rows that several
of them share make more items than the number of rows lets one expect.

Against the attention in 64 bits, with the tolerance of test_gpu_tree_sinks.py."""
import numpy as np
import pytest
import torch

from kv_cache_vector_gb300 import abi
from test_gpu_prefill_paged import Batch, check
from test_gpu_tree_sinks import pack, random_trees, sinks_seen, tree_seen, want

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kv_cache_vector_gb300 import build
    build.build()
    abi.lib()
    abi.tq_device_status(reset=True)


# (tokens of the sequence given `times` over, its context, times, tokens and context of the last one, Hq, Hkv).
# In front of each but the first a sequence out of range; sequences without tokens at the end.
CASES = [(64, 200, 5, 64, 190, 4, 4, 0), (32, 200, 10, 8, 100, 4, 4, 0), (12, 60, 3, 5, 129, 4, 1, 40),
         (60, 128, 2, 60, 127, 2, 2, 30)]


@pytest.mark.parametrize("d", [128, 64, 256, 32])
@pytest.mark.parametrize("first,ctx,times,last,end,Hq,Hkv,empty", CASES)
def test_all_other_sequences_are_there(first, ctx, times, last, end, Hq, Hkv, empty, d):
    bt = Batch(71, [(first, ctx), (last, end)], Hq, Hkv, d, 32, 4, 3)
    sees = random_trees(np.random.default_rng(2), bt.lens)[1]
    plan, q, _, cache, table, lens = bt.gpu()
    cu = [0, first] * times + [first + last] * (1 + empty)
    B = len(cu) - 1
    which = torch.tensor([0] * (2 * times - 1) + [1] * (1 + empty), device="cuda")
    args = (plan, q, torch.tensor(cu, dtype=torch.int32, device="cuda"), cache, table[which].contiguous(),
            lens[which].contiguous())
    assert q.shape[0] * (Hq // Hkv) <= 16 * B  # few rows
    mask = pack(sees, 4, first + last).cuda()
    for call, seen in ((lambda o: abi.tq_attn_sinks_paged(*args, 0.1, 100, 3, out=o), sinks_seen(bt, 100, 3)),
                       (lambda o: abi.tq_attn_tree_paged(*args, mask, 0.1, out=o), tree_seen(bt, sees))):
        ref = want(bt, 0.1, seen)
        out = torch.full(q.shape, 77.0, device="cuda")
        for _ in range(2):  # a second time over what the first left in the workspace's memory
            call(out)
            assert abi.tq_device_status(reset=True) == 71
            check(out, *ref, first + last, bf16=False)


def test_a_captured_call_follows_a_step_back():
    """The same launch, with a cu_q that ascends, one that steps back, and the first again."""
    bt = Batch(72, [(64, 200), (64, 190)], 4, 4, 128, 32, 4, 3)
    plan, q, _, cache, table, lens = bt.gpu()
    back, straight = [0, 64] * 5 + [128], [0] * 9 + [64, 128]
    which = torch.tensor([0] * 9 + [1], device="cuda")
    cu = torch.tensor(straight, dtype=torch.int32, device="cuda")
    out = torch.zeros(q.shape, device="cuda")
    ws = torch.empty(abi.tq_attn_sinks_paged_workspace_bytes(4, 4, 128), dtype=torch.uint8, device="cuda")
    args = (plan, q, cu, cache, table[which].contiguous(), lens[which].contiguous(), 0.1, 100, 3)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        abi.tq_attn_sinks_paged(*args, out=out, workspace=ws)
    ref = want(bt, 0.1, sinks_seen(bt, 100, 3))
    for entries, status in ((straight, 0), (back, 71), (straight, 0)):
        cu.copy_(torch.tensor(entries, dtype=torch.int32))
        out.fill_(77.0)
        g.replay()
        torch.cuda.synchronize()
        assert abi.tq_device_status(reset=True) == status
        check(out, *ref, 128, bf16=False)
