"""Whole verify steps at their ends: temperature 0, prompts and steps that do not fit."""

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


@pytest.mark.parametrize("per,pages,length", [(4, 8, 66), (4, 7, 64), (2, 99, 100)])
def test_prompts_that_do_not_fit_are_refused(per, pages, length):
    """Too few entries in the table, too few pages in the ring."""
    loop, gen = _loop(2, 2, per, pages=pages)
    with pytest.raises(ocq.OcqError) as e:
        loop.prefill(_prompts(2, length, gen), chunk=17)
    assert e.value.status == ocq.ERR_BUFFER_TOO_SMALL


def test_steps_that_lack_pages_are_counted():
    loop, gen = _loop(1, 3, 2)
    loop.prefill(_prompts(1, 30, gen))
    for _ in range(4):
        loop.step()
    lacking = int(loop.missing)
    assert lacking > 0
    loop.step()
    assert int(loop.missing) > lacking
