"""Draft verification and step tables at their ends: steps without tokens."""

import numpy as np
import pytest
import torch

from quantized_memory_bound_amd import ocq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _batch(news):
    one = torch.ones(len(news), dtype=torch.int32, device=DEV)
    return ocq.TokenBatch(_ints([0] + list(np.cumsum(news))), one, one[:, None], max([1] + news), 1)


@pytest.mark.parametrize("probabilities", [False, True])
@pytest.mark.parametrize("temperature", [0.0, 0.7])
def test_drafts_of_a_step_without_tokens(probabilities, temperature):
    """Requests of which none brings a token accept no draft: given and allocated outputs, call after call."""
    none = torch.zeros((0, 50), device=DEV)
    empty = torch.zeros(0, device=DEV)
    for _ in range(3):
        junk = torch.full((3,), 77, dtype=torch.int32, device=DEV)
        given = junk.clone()
        del junk                                   # (what an allocation finds)
        for kw in (dict(), dict(accepted=given)):
            a, out = ocq.verify_drafts(none, _ints([]), _batch([0, 0, 0]), empty, torch.rand(3, device=DEV),
                                       temperature=temperature, probabilities=probabilities, **kw)
            assert a.tolist() == [0, 0, 0] and out.shape == (0,)
        assert given.tolist() == [0, 0, 0]


def test_drafts_of_a_step_without_tokens_on_another_stream_and_captured():
    none, empty, un = torch.zeros((0, 50), device=DEV), torch.zeros(0, device=DEV), torch.rand(2, device=DEV)
    batch, ids = _batch([0, 0]), _ints([])
    accepted = _ints([5, 6])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ocq.verify_drafts(none, ids, batch, empty, un, accepted=accepted, stream=side)
    side.synchronize()
    assert accepted.tolist() == [0, 0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ocq.verify_drafts(none, ids, batch, empty, un, accepted=accepted)
    for i in range(4):
        accepted.fill_(9 + i)
        graph.replay()
        torch.cuda.synchronize()
        assert accepted.tolist() == [0, 0], i


def test_drafts_of_rows_without_requests():
    empty = torch.zeros(0, device=DEV)
    for kw in (dict(), dict(out=_ints([3, 4, 5]))):
        a, out = ocq.verify_drafts(torch.zeros((3, 50), device=DEV), _ints([1, 2, 3]), _batch([]), torch.rand(3, device=DEV),
                                   empty, **kw)
        assert a.shape == (0,) and out.tolist() == [-1, -1, -1]
