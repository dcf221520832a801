"""Steps of speculative decoding with everything between them on the GPU: the same layer driven by lists on the host
gives the same bits, whatever was accepted; every accepted token and next token follows from the step's logits."""

import numpy as np
import pytest
import torch

from quantized_memory_bound_amd import ocq
from quantized_memory_bound_amd.verify_layer import VerifyLoop, batch_of, random_layer

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SHAPE = dict(hidden=256, inter=512, heads=8, kv_heads=2, head_dim=64, page_size=16)
VOCAB = 500


def _bf(gen, *shape, std=1.0):
    return (torch.randn(shape, device=DEV, generator=gen) * std).to(torch.bfloat16)


def _loop(requests, drafts, per, **kw):
    gen = torch.Generator(DEV).manual_seed(1)
    layer = random_layer(pages=requests * per, seed=3, device=DEV, **SHAPE, **kw)
    tables = ocq.PageTables.allocate(requests, per, requests * per, 16, device=DEV)
    return VerifyLoop(layer, _bf(gen, VOCAB, 256), _bf(gen, 256, VOCAB, std=0.2), tables, drafts, per * 16), gen


@pytest.mark.parametrize("kw", [dict(), dict(e4m3=True), dict(nvfp4=True)])
@pytest.mark.parametrize("requests,drafts", [(3, 4), (1, 0), (5, 12)])
def test_loop_against_lists_on_the_host(kw, requests, drafts):
    """The other side keeps its own cache and a page table that was never taken apart; rows are the same numbers, so
    that projections, cache and attention give the same bits, and so do the verifications that follow."""
    per, steps, n = 12, 6, 1 + drafts
    loop, gen = _loop(requests, drafts, per, **kw)
    prompts = torch.randint(0, VOCAB, (requests, 30), device=DEV, generator=gen)
    loop.prefill(prompts, chunk=17)
    other = random_layer(pages=requests * per, seed=3, device=DEV, **SHAPE, **kw)
    table = torch.arange(requests * per, dtype=torch.int32, device=DEV).flip(0).view(requests, per)
    lens = [0] * requests
    for at, end in ((0, 17), (17, 29)):
        m = end - at
        other(loop.embed[prompts[:, at:end].flatten()], None, batch_of([m] * requests, [end] * requests, table, DEV))
        lens = [end] * requests
    seen = []
    verify = ocq.verify_drafts

    def spy(target, ids, batch, ua, un, **k):
        seen.append((target, ids, ua, un, k))
        return verify(target, ids, batch, ua, un, **k)
    total = 0
    for step in range(steps):
        seen.clear()
        ocq.verify_drafts = spy
        try:
            accepted, out = loop.step()
        finally:
            ocq.verify_drafts = verify
        (logits, ids, ua, un, k), = seen
        assert loop.tables.kv_lens.tolist() == [l + n for l in lens] and int(loop.missing) == 0
        held = loop.tables.held.tolist()
        assert held == [-(-(l + n) // 16) for l in lens]
        pages = [p for r in range(requests) for p in loop.tables.page_table[r, : held[r]].tolist()]
        assert len(set(pages)) == len(pages) and min(pages) >= 0
        batch = batch_of([n] * requests, [l + n for l in lens], table, DEV)
        x, pending = other(loop.embed[ids], None, batch)
        assert torch.equal((x + pending) @ loop.head, logits)
        again = verify(logits, ids, batch, ua, un, **k)
        assert torch.equal(again[0], accepted) and torch.equal(again[1].view(requests, n), out)
        for r, a in enumerate(accepted.tolist()):
            assert out[r, :a].tolist() == ids.view(requests, n)[r, 1:1 + a].tolist() and int(loop.last[r]) == int(out[r, a])
            assert 0 <= int(out[r, a]) < VOCAB and (out[r, a + 1:] == -1).all()
            lens[r] += 1 + a
            total += a
    assert drafts == 0 or total > 0


def test_a_greedy_target_accepts_what_it_would_have_said():
    """Temperature 0: the tokens of a loop with drafts are those of one without."""
    said = []
    for drafts in (0, 3):
        loop, gen = _loop(2, drafts, 12)
        prompts = torch.randint(0, VOCAB, (2, 20), device=DEV, generator=gen)
        loop.prefill(prompts)
        tokens = [[], []]
        for _ in range(12):
            verify = ocq.verify_drafts
            ocq.verify_drafts = lambda *a, **k: verify(*a, **{**k, "temperature": 0.0})
            try:
                _, out = loop.step()
            finally:
                ocq.verify_drafts = verify
            for r in range(2):
                tokens[r] += [t for t in out[r].tolist() if t >= 0]
        said.append([t[:12] for t in tokens])
    # (the projections' library products may sum in another order for another number of rows: a tie could go
    # either way, which these inputs do not have)
    assert said[0] == said[1]
