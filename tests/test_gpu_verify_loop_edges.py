"""Whole verify steps at their ends: temperature 0, prompts and steps that do not fit, prompts after
steps, rows without a next token."""

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


def test_prompts_after_steps():
    """A prompt that begins with the loop's last tokens goes behind what was accepted: the cache is that of a loop which was
    given all of these tokens at once."""
    loop, gen = _loop(2, 4, 12)
    prompts = _prompts(2, 20, gen)
    loop.prefill(prompts)
    text = [p.tolist() for p in prompts]
    for _ in range(3):
        _, out = loop.step()
        for r in range(2):
            text[r] += [t for t in out[r].tolist() if t >= 0]
    more = _prompts(2, 9, gen)
    lens = [len(t) for t in text]
    loop.prefill(torch.cat([loop.last[:, None], more], 1))
    assert loop.tables.kv_lens.tolist() == [n + 8 for n in lens]
    assert loop.last.tolist() == more[:, -1].tolist()
    for r in range(2):
        other, _ = _loop(1, 4, 12)
        whole = torch.tensor([text[r]], device=DEV)
        other.prefill(torch.cat([whole, more[r:r + 1]], 1))
        for mine, its in ((loop.layer.cache.k, other.layer.cache.k), (loop.layer.cache.v, other.layer.cache.v)):
            j = torch.arange(lens[r] + 8, device=DEV)
            a = mine[loop.tables.page_table[r][j // 16].long(), :, j % 16].float()
            b = its[other.tables.page_table[0][j // 16].long(), :, j % 16].float()
            # (products of another number of rows may sum in another order: off by a rounding or two, other tokens by
            # values of order one)
            assert (a - b).abs().max() <= 2.0 ** -6 * b.abs().max()
    loop.step()
    # a prompt of one token changes nothing but the next step's token
    kv, last = loop.tables.kv_lens.tolist(), loop.accepted.tolist()
    loop.prefill(loop.last[:, None])
    loop.step()
    assert loop.tables.kv_lens.tolist() == [k - 5 + 1 + a + 5 for k, a in zip(kv, last)]


@pytest.mark.parametrize("why", ["a NaN", "-1"])
def test_requests_without_a_next_token_say_nothing_more(why):
    """Their rows are -1 from then on, no more of them stays in the cache, and the other requests go on as if nothing had
    happened; a new prompt takes them up again."""
    runs = []
    for bad in (False, True):
        loop, gen = _loop(3, 4, 12)
        prompts = _prompts(3, 20, gen).clamp(max=VOCAB - 2)
        if bad and why == "a NaN":
            loop.embed[VOCAB - 1] = float("nan")
            prompts[1, -1] = VOCAB - 1
        loop.prefill(prompts)
        steps = []
        for step in range(5):
            accepted, out = loop.step()
            if step == 0 and bad and why == "-1":
                loop.last[1] = -1
            steps.append((accepted.tolist(), out.tolist(), loop.tables.kv_lens.tolist()))
        runs.append(steps)
    for step, (a, b) in enumerate(zip(*runs)):
        for r in (0, 2):
            assert [x[r] for x in a] == [x[r] for x in b]
        if step > 0 or why == "a NaN":
            assert b[0][1] == 0 and b[1][1] == [-1] * 5
    first = runs[1][0]
    # (19 tokens of the prompt, its last one and what the first step accepted; 5 rows more during each step)
    assert [s[2][1] for s in runs[1]] == [24] + [20 + first[0][1] + 5] * 4
    loop.prefill(prompts.clamp(max=VOCAB - 2))
    assert (loop.last >= 0).all() and loop.tables.kv_lens.tolist()[1] == 20 + first[0][1] + 19
    if why == "-1":
        assert (loop.step()[1][:, 0] >= 0).all()
