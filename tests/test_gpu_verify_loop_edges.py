"""Whole verify steps at their ends: temperature 0."""

import pytest
import torch

from quantized_memory_bound_amd import ocq
from quantized_memory_bound_amd.verify_layer import VerifyLoop, random_layer

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SHAPE = dict(hidden=256, inter=512, heads=8, kv_heads=2, head_dim=64, page_size=16)
VOCAB = 500


def _loop(requests, drafts, per, pages=None, temperature=1.0, table=None, **kw):
    gen = torch.Generator(DEV).manual_seed(1)

    def bf(*shape, std=1.0):
        return (torch.randn(shape, device=DEV, generator=gen) * std).to(torch.bfloat16)
    pages = requests * per if pages is None else pages
    layer = random_layer(pages=pages, seed=3, device=DEV, **SHAPE, **kw)
    tables = ocq.PageTables.allocate(requests, per, pages, 16, device=DEV)
    return VerifyLoop(layer, bf(VOCAB, 256), bf(256, VOCAB, std=0.2), tables, drafts, per * 16, temperature), gen


def _prompts(requests, length, gen):
    return torch.randint(0, VOCAB, (requests, length), device=DEV, generator=gen)


def test_greedy_loops_accept_drafts():
    """The draft model's largest logit is often the target's: at temperature 0 such drafts stay, and the tokens are those
    of a loop without drafts.  (The layer changes the residual stream little here.)"""
    said, kept = [], 0
    for drafts in (0, 3):
        loop, gen = _loop(2, drafts, 12, temperature=0.0)
        loop.embed = loop.embed * 4
        prompts = _prompts(2, 20, gen)
        loop.prefill(prompts)
        tokens = [[], []]
        for _ in range(12):
            accepted, out = loop.step()
            kept += int(accepted.sum())
            for r in range(2):
                tokens[r] += [t for t in out[r].tolist() if t >= 0]
        said.append([t[:12] for t in tokens])
    assert said[0] == said[1] and kept > 0


@pytest.mark.parametrize("temperature", [-1.0, float("nan"), float("inf")])
def test_temperatures_that_are_none(temperature):
    with pytest.raises(ocq.OcqError) as e:
        _loop(1, 1, 4, temperature=temperature)
    assert e.value.status == ocq.ERR_INVALID_ARG
