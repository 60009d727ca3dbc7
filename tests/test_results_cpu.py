"""The tensors that a call returns are its own, whatever other calls did before
it: writable in any mode, with version counters of their own.  On the CPU, by the
functions that make them."""
import pytest
import torch

from kv_cache_vector_gb300 import abi

CPU = torch.device("cpu")


@pytest.fixture(autouse=True)
def _no_capture(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False)


def _fields(step):
    return [t for t in (step.cu_q, step.positions, step.slots, step.mask) if t is not None]


MAKERS = {"fresh": lambda stream: [abi._fresh(CPU, stream, 7)],
          "step": lambda stream: _fields(abi._step(CPU, stream, 3, 5, 0)),
          "step with trees": lambda stream: _fields(abi._step(CPU, stream, 3, 5, 2))}


@pytest.mark.parametrize("make", MAKERS.values(), ids=MAKERS.keys())
@pytest.mark.parametrize("first", [True, False])
def test_results_are_writable_in_and_outside_inference_mode(make, first):
    """A loop that runs the model in inference_mode and the books outside, or the other way round."""
    made = []
    for k in range(40):
        with torch.inference_mode((k % 3 == 0) == first):
            made += make(-1 - first)
    for t in made:
        assert not t.is_inference()
        t.zero_()
        t.add_(1)
    with torch.inference_mode():
        for t in made:
            t.add_(1)
    assert all((t == 2).all() for t in made)


@pytest.mark.parametrize("make", MAKERS.values(), ids=MAKERS.keys())
def test_a_write_to_one_result_leaves_the_others_versions(make):
    """Autograd checks the versions of what it saved (the positions of an embedding)."""
    made = sum((make(-3) for _ in range(40)), [])
    assert len({t.data_ptr() for t in made}) == len(made)
    for t in made:
        t.zero_()
    for k, t in enumerate(made):
        assert t._version == 1 and not t._is_view()
        t.fill_(k)
    assert all((t == k).all() for k, t in enumerate(made))
    weight = torch.ones(4, 2, requires_grad=True)
    a, b = make(-4)[0], make(-4)[0]
    a.zero_(), b.zero_()
    loss = torch.nn.functional.embedding(a, weight).sum()
    b.add_(1)
    loss.backward()
    assert weight.grad[0, 0] == a.numel()
