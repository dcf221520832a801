"""Draft verification and step tables at their ends: steps without tokens, acceptances next to their border, tables without
requests or with far too few pages.

An acceptance compares u q(x) with p(x) = e_x / Z in 64 bits but for Z, whose exponentials are 32-bit: the kernel's bound of
its error is 2^-19 (subtraction, product with log2(e) / T and that factor's own rounding, 2^-24 each of an exponent whose
weighted mean over a lane's n <= 2^16 elements is below 8.1, Lambert's W of n / e; 2^-23 of the exponential, 3 2^-24 of a sum
of eight: 30 2^-24).  Decisions further than that from the border are certain: they are asked for at 1.05 2^-19.
"""

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


def _rows(kind, vocab, rows, gen):
    if kind == "tail":      # a maximum for each of 256 lanes, all else below half a last place of what is summed
        x = torch.full((rows, vocab), -18.75, device=DEV)
        x[:, :2048:8] = 0.0
        return x
    if kind == "rising":    # every lane's maximum moves with every vector
        return torch.linspace(-30.0, 0.0, vocab, device=DEV).expand(rows, -1) + torch.arange(rows, device=DEV)[:, None] * 0.37
    if kind == "flat":      # the weighted mean of the exponent is large: many unlikely ones beside one likely one
        x = torch.randn((rows, vocab), device=DEV, generator=gen) * 0.5
        x[:, vocab // 3] = 8.0
        return x
    return torch.randn((rows, vocab), device=DEV, generator=gen) * 3


@pytest.mark.parametrize("kind", ["tail", "rising", "flat", "random"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab,requests", [(131072, 400), (131072, 8), (50001, 400)])
def test_acceptances_next_to_their_border(kind, dtype, vocab, requests):
    """Two rows a request; u just below and just above the draft's probability, from one workgroup a row to many."""
    gen = torch.Generator(DEV).manual_seed(len(kind))
    some = min(8, requests)
    for temp in (1.0, 0.7):
        logits = _rows(kind, vocab, some, gen).to(dtype)
        p = torch.softmax(logits.double() * (1.0 / float(np.float32(temp))), -1)
        top = p.topk(40, -1).indices
        x = top[torch.arange(some, device=DEV), torch.randint(0, 40, (some,), device=DEV, generator=gen)]
        if kind == "tail":
            x = torch.arange(some, device=DEV) * 8
        px = p[torch.arange(some, device=DEV), x].cpu().numpy()
        assert (px < 0.999).all()
        of = torch.arange(requests, device=DEV) % some
        below = np.arange(requests) // some % 2 == 0
        u = px[of.cpu().numpy()] * np.where(below, 1 - 1.05 * 2.0 ** -19, 1 + 1.05 * 2.0 ** -19)
        ids = torch.zeros((requests, 2), dtype=torch.int32, device=DEV)
        ids[:, 1] = x[of].to(torch.int32)
        ua = torch.zeros((requests, 2), device=DEV)
        ua[:, 0] = torch.from_numpy(u.astype(np.float32)).to(DEV)
        target = logits[of].repeat_interleave(2, 0)
        a, out = ocq.verify_drafts(target, ids.flatten(), _batch([2] * requests), ua.flatten(),
                                   torch.rand(requests, device=DEV, generator=gen), temperature=temp)
        assert a.tolist() == below.astype(int).tolist()
        assert (out.view(-1, 2)[:, 0][torch.from_numpy(below).to(DEV)] == ids[:, 1][torch.from_numpy(below).to(DEV)]).all()


@pytest.mark.parametrize("start", [[0, 5, 3, 8], [0, 9, 2, 2], [-4, 90, 1, 7], [2 ** 31 - 1, -2 ** 31, 0, 8]])
@pytest.mark.parametrize("draft", [False, True])
def test_offsets_that_fall_write_nothing_elsewhere(start, draft):
    """q_start that no step gives: the outputs are any, the memory beside them stays, whatever the workspace holds; so it
    does where counters were left wrong by such a call."""
    gen = torch.Generator(DEV).manual_seed(3)
    target, ids = torch.randn((8, 3000), device=DEV, generator=gen), torch.randint(0, 3000, (8,), device=DEV, generator=gen)
    q = torch.softmax(torch.randn((8, 3000), device=DEV, generator=gen), -1) if draft else None
    one = torch.ones(3, dtype=torch.int32, device=DEV)
    batch = ocq.TokenBatch(_ints(start), one, one[:, None], 8, 1)
    for fill in (0x7F, 0x80, 0xFF, 0x01):
        accepted, out = _ints([99] * 5), _ints([99] * 10)
        workspace = torch.full((1 << 16,), fill, dtype=torch.uint8, device=DEV)
        ocq.verify_drafts(target, ids.to(torch.int32), batch, torch.rand(8, device=DEV, generator=gen),
                          torch.rand(3, device=DEV, generator=gen), draft_probs=q, accepted=accepted[1:-1], out=out[1:-1],
                          workspace=workspace)
        torch.cuda.synchronize()
        assert accepted[[0, -1]].tolist() == [99, 99] and out[[0, -1]].tolist() == [99, 99]
        assert (workspace[-(1 << 14):] == fill).all()


# ---------------------------------------------------------------- tables

@pytest.mark.parametrize("tokens", [0, 5, 40000])
@pytest.mark.parametrize("apart", [False, True])
def test_tables_without_requests(tokens, apart):
    """All rows are behind the last request; nothing lacks; the ring's counts go on."""
    def tables(counts):
        none = torch.zeros(0, dtype=torch.int32, device=DEV)
        return ocq.PageTables(_ints([7]), none, none, torch.tensor(counts, device=DEV), table, ring, 16)
    table, ring = torch.zeros((0, 4), dtype=torch.int32, device=DEV), _ints([0, 1, 2])
    before = tables([4, 6])
    after = tables([0, 0]) if apart else None
    outs = (torch.full((tokens,), 8, dtype=torch.int64, device=DEV), torch.full((tokens,), 8, dtype=torch.int32, device=DEV),
            torch.full((tokens,), 8, dtype=torch.int32, device=DEV), _ints([8]))
    got = ocq.step_tables(before, _ints([]), tokens, out=after, slots=outs[0], positions=outs[1], requests=outs[2],
                          missing=outs[3])
    assert all(a is b for a, b in zip(got, outs)) and all((t == -1).all() for t in got[:3]) and got[3].tolist() == [0]
    after = after or before
    assert after.q_start.tolist() == [0] and after.counts.tolist() == [4, 6] and ring.tolist() == [0, 1, 2]


def test_tables_without_requests_and_others_do_not_go_together():
    none, three = ocq.PageTables.allocate(0, 4, 12, 16, device=DEV), ocq.PageTables.allocate(3, 4, 12, 16, device=DEV)
    for before, after, news in ((none, three, _ints([])), (none, ocq.PageTables.allocate(0, 4, 12, 16, device=DEV), _ints([])),
                                (three, none, _ints([1, 1, 1]))):
        with pytest.raises(ocq.OcqError) as e:
            ocq.step_tables(before, news, 3, out=after)
        assert e.value.status == ocq.ERR_INVALID_ARG


@pytest.mark.parametrize("requests", [3, 1500])
def test_tables_that_lack_more_pages_than_a_number_holds(requests):
    """Lengths of nearly 2^31 in rows of four pages: what is missing stops at the largest int32."""
    t = ocq.PageTables.allocate(requests, 4, 12, 1, device=DEV)
    t.kv_lens.fill_(2 ** 31 - 1)
    missing = ocq.step_tables(t, torch.zeros(requests, dtype=torch.int32, device=DEV), 8)[3]
    assert missing.tolist() == [2 ** 31 - 1]
    assert t.kv_lens.tolist() == [2 ** 31 - 1] * requests and t.counts.tolist() == [12, 12]
    assert t.page_table[:3].tolist() == [[0, 1, 2, 3], [4, 5, 6, 7], [8, 9, 10, 11]]
    one = ocq.PageTables.allocate(1, 4, 12, 1, device=DEV)
    one.kv_lens.fill_(2 ** 31 - 1)
    assert ocq.step_tables(one, _ints([0]), 8)[3].tolist() == [2 ** 31 - 1 - 4]
