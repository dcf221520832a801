"""What stands between two verify steps, on the GPU: the drafts that stay and the token after them, and the next step's
tables, against plain implementations in 64 bits and in Python's whole numbers.

Everything returned is whole and has to be equal.  Random numbers are fixed by seeds; the 64-bit sums of both sides
differ by less than 2^-40 of the row's sum, and the acceptances' normalization by less than 2^-20, so that one of the
10^5 decisions made here could fall on the other side with a probability of about 10^5 2^-22 in all at the worst, where
the acceptances are within 2^-20 of a border; it has not to be allowed for, since the inputs are fixed.
"""

import numpy as np
import pytest
import torch

from quantized_memory_bound_amd import ocq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


# ---------------------------------------------------------------- drafts

def drafts_ref(target, ids, news, u_accept, u_next, draft, temps, probabilities):
    """Request by request, draft by draft, in 64 bits (numpy)."""
    accepted, out, at, drawn = [], [], 0, 0
    vocab = target.shape[1]
    for r, n in enumerate(news):
        if n == 0:
            accepted.append(0)
            continue
        p = target[at: at + n].astype(np.float64)
        bad = np.isnan(p).any(1)
        if not probabilities:
            if temps[r] == 0:
                bad |= ~(p > -np.inf).any(1)
                first = np.argmax(np.where(np.isnan(p), -np.inf, p), 1)
                p = np.zeros_like(p)
                p[np.arange(n), first] = 1.0
            else:
                with np.errstate(invalid="ignore"):
                    e = np.exp((p - p.max(1, keepdims=True)) * (1.0 / np.float64(temps[r])))
                    p = e / e.sum(1, keepdims=True)
                bad |= np.isnan(p).any(1)
        count, q = 0, None
        while count < n - 1:
            x = ids[at + count + 1]
            q = draft[drawn + count].astype(np.float64) if draft is not None else np.zeros(vocab)
            if draft is None and 0 <= x < vocab:
                q[x] = 1.0
            if not (0 <= x < vocab) or bad[count] or not float(u_accept[at + count]) * q[x] < p[count, x]:
                break
            count += 1
        w = p[count]
        if bad[count]:
            nxt = -1
        else:
            if count < n - 1:
                less = np.maximum(w - q, 0) if draft is not None else w * (1 - q)
                w = less if less.sum() > 0 else w
            c = np.cumsum(w)
            past = np.nonzero(c > float(u_next[r]) * c[-1])[0]
            nxt = -1 if not c[-1] > 0 else int(past[0]) if len(past) else int(np.nonzero(w > 0)[0][-1])
        accepted.append(count)
        out += [int(x) for x in ids[at + 1: at + 1 + count]] + [nxt] + [-1] * (n - 1 - count)
        at, drawn = at + n, drawn + n - 1
    return accepted, out


def make_drafts(news, vocab, seed, dtype=torch.bfloat16, q_dtype=torch.float32, temps=0.9, draft=True, probabilities=False,
                wide=0, shift=0, near=0.3, spread=2.0):
    """Inputs of a verify pass; rows `wide` elements further apart than vocab, `shift` elements past an aligned start."""
    g = torch.Generator(DEV).manual_seed(seed)
    tokens, rows = sum(news), sum(max(0, n - 1) for n in news)

    def place(x, dt):
        pool = torch.zeros(len(x) * (vocab + wide) + shift + 8, dtype=dt, device=DEV)
        t = pool[shift:].as_strided((len(x), vocab), (vocab + wide, 1), storage_offset=shift)
        t.copy_(x)
        return t
    logits = torch.randn((tokens, vocab), device=DEV, generator=g) * spread
    of = torch.cat([torch.arange(n - 1) + sum(news[:r]) for r, n in enumerate(news) if n > 1] or
                   [torch.zeros(0, dtype=torch.int64)]).to(DEV)
    q = torch.softmax(logits[of] + torch.randn((rows, vocab), device=DEV, generator=g) * near, -1)
    ids = torch.randint(0, vocab, (tokens,), device=DEV, generator=g)
    noise = -torch.log(torch.rand(q.shape, device=DEV, generator=g).clamp(min=1e-30))
    ids[of + 1] = (q / noise).argmax(-1) if draft else q.argmax(-1)
    start = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32, device=DEV)
    one = torch.ones(len(news), dtype=torch.int32, device=DEV)
    batch = ocq.TokenBatch(start, one, one[:, None], max(1, max(news)), 1)
    s = dict(target=place(torch.softmax(logits, -1) if probabilities else logits, dtype), ids=ids.to(torch.int32),
             news=news, batch=batch, u_accept=torch.rand(tokens, device=DEV, generator=g),
             u_next=torch.rand(len(news), device=DEV, generator=g), draft=place(q, q_dtype) if draft else None,
             temps=[temps] * len(news) if not isinstance(temps, (list, tuple)) else list(temps), probabilities=probabilities)
    return s


def check_drafts(s, **kw):
    temps = torch.tensor(s["temps"], dtype=torch.float32, device=DEV)
    accepted, out = ocq.verify_drafts(s["target"], s["ids"], s["batch"], s["u_accept"], s["u_next"], draft_probs=s["draft"],
                                      temperature=temps, probabilities=s["probabilities"], **kw)
    torch.cuda.synchronize()
    host = lambda t: None if t is None else t.float().cpu().numpy()  # noqa: E731
    want = drafts_ref(host(s["target"]), s["ids"].cpu().numpy(), s["news"], s["u_accept"].cpu().numpy(),
                      s["u_next"].cpu().numpy(), host(s["draft"]), temps.cpu().numpy(), s["probabilities"])
    assert accepted.tolist() == want[0]
    assert out[: len(want[1])].tolist() == want[1]
    assert (out[len(want[1]):] == -1).all() and not s["batch"].counters.any()
    return accepted, out


@pytest.mark.parametrize("vocab", [1, 7, 1000, 4096, 32000, 50001, 131072])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("dtype,q_dtype,probabilities", [
    (torch.bfloat16, torch.float32, False), (torch.float32, torch.bfloat16, False), (torch.float32, torch.float32, True),
    (torch.bfloat16, torch.bfloat16, True)])
def test_drafts(vocab, draft, dtype, q_dtype, probabilities):
    news = [5, 1, 13, 0, 2, 9] if vocab < 100000 else [5, 1, 4]
    temps = [0.7, 1.0, 0.0, 1.0, 1.5, 0.0][: len(news)]
    for seed in range(3):
        s = make_drafts(news, vocab, seed, dtype, q_dtype, temps, draft, probabilities)
        check_drafts(s)


@pytest.mark.parametrize("wide,shift", [(0, 1), (1, 0), (3, 5), (8, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_drafts_rows_at_any_alignment(wide, shift, dtype):
    for probabilities in (False, True):
        check_drafts(make_drafts([4, 3, 6], 5003, 5, dtype, dtype, probabilities=probabilities, wide=wide, shift=shift))


@pytest.mark.parametrize("news", [[1], [2], [64], [65], [130, 1, 64], [1] * 70, [0, 0, 3, 0], [3] * 300])
def test_drafts_batches(news):
    for draft in (True, False):
        check_drafts(make_drafts(news, 601, len(news), draft=draft, near=0.05))


def test_drafts_that_all_stay_and_that_none_does():
    """The target's own probabilities as the draft's: every draft stays but by rounding; far ones: none does."""
    s = make_drafts([6, 9], 3001, 1, torch.float32, near=0.0, temps=1.0)
    accepted, _ = check_drafts(s)
    assert accepted.tolist() == [5, 8]
    s["u_accept"][:] = 1 - 2.0 ** -24
    s["draft"][:] = 0
    s["draft"].scatter_(1, s["ids"][torch.tensor([1, 2, 3, 4, 5, 7, 8, 9, 10, 11, 12, 13, 14], device=DEV)].long()[:, None], 1.0)
    accepted, _ = check_drafts(s)
    assert accepted.tolist() == [0, 0]


@pytest.mark.parametrize("vocab", [50, 3001, 40000, 150000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_drafts_whose_probabilities_are_the_targets_but_for_roundings(vocab, dtype):
    """q is p rounded to bf16, random numbers next to 1 refuse where it was rounded up: the weights are what roundings
    left, far below p and q."""
    for seed in range(4):
        s = make_drafts([5, 3, 9], vocab, seed, dtype, torch.bfloat16, near=0.0, temps=[1.0, 0.8, 1.3])
        # of the logits as they are held
        p = torch.softmax(s["target"].double() / torch.tensor([1.0] * 5 + [0.8] * 3 + [1.3] * 9, device=DEV)[:, None], -1)
        of = torch.tensor([0, 1, 2, 3, 5, 6, 8, 9, 10, 11, 12, 13, 14, 15], device=DEV)
        s["draft"].copy_(p[of])
        s["u_accept"][:] = 1 - 2.0 ** -24
        check_drafts(s)


@pytest.mark.parametrize("u", [0.0, 2.0 ** -24, 0.5, 1 - 2.0 ** -24])
@pytest.mark.parametrize("vocab", [3, 2049, 20000])
def test_drafts_random_numbers_at_their_ends(u, vocab):
    for draft in (True, False):
        for probabilities in (False, True):
            s = make_drafts([3, 1, 4], vocab, 8, torch.float32, draft=draft, probabilities=probabilities)
            s["u_next"][:] = u
            check_drafts(s)
            s["u_accept"][:] = u
            check_drafts(s)


def test_drafts_places_of_the_next_token():
    """One token has all the weight, at the first and last places of lanes, workgroups and chunks, and two tokens with
    half of it each on either side of such a border; the others are ruled out."""
    vocab = 40000
    for at in (0, 7, 8, 511, 2047, 2048, 4095, 4096, 8191, 19999, 39999):
        s = make_drafts([1], vocab, 1, torch.float32)
        s["target"][:] = -float("inf")
        s["target"][0, at] = 3.0
        assert check_drafts(s)[1].tolist() == [at]
        if at + 1 < vocab:
            s["target"][0, at + 1] = 3.0
            for u, want in ((0.0, at), (0.5 - 2.0 ** -24, at), (0.5, at + 1), (0.75, at + 1)):
                s["u_next"][:] = u
                assert check_drafts(s)[1].tolist() == [want]


def test_drafts_weights_that_are_none():
    """q covers p: the next token is drawn from p.  Rows of -inf, of NaN, of +inf and of zeros: -1, and nothing before
    them is lost.  The largest of several equal logits is the first."""
    s = make_drafts([3, 3], 900, 2, torch.float32, probabilities=True)
    s["draft"][:] = 2.0
    s["u_accept"][:] = 0.999
    check_drafts(s)
    s = make_drafts([4, 4, 4, 4], 900, 3, torch.float32, near=0.0, temps=[1.0, 1.0, 0.0, 1.0])
    s["u_accept"][:] = 0.0
    s["target"][2] = -float("inf")
    s["target"][5, 77] = float("nan")
    s["target"][10] = float("-inf")
    s["target"][13, 5] = float("inf")
    accepted, out = check_drafts(s)
    assert [int(out[i]) for i in (2, 5, 13)] == [-1, -1, -1] and accepted[0] == 2
    s = make_drafts([2], 900, 3, torch.float32, probabilities=True, draft=False)
    s["target"][:] = 0
    assert check_drafts(s)[1].tolist() == [-1, -1]
    for dtype in (torch.bfloat16, torch.float32):
        s = make_drafts([1, 1], 70000, 4, dtype, temps=0.0)
        s["target"][:] = 1.0
        s["target"][0, [69999, 123, 40000]] = 5.0
        s["target"][1, 3] = float("nan")
        assert check_drafts(s)[1].tolist() == [123, -1]


def test_drafts_at_the_smallest_and_largest_temperatures():
    """Next to 0 the largest logits share all the weight, at 10^30 all tokens do (but those ruled out)."""
    s = make_drafts([1, 1, 1], 3000, 4, torch.float32, temps=[1e-40, 1e-30, 1e30])
    s["target"][:2, 17], s["target"][:2, 2900] = 50.0, 50.0
    s["target"][2, :1500] = -float("inf")
    for u, want in ((0.25, [17, 17, 1875]), (0.75, [2900, 2900, 2625])):
        s["u_next"][:] = u
        assert check_drafts(s)[1].tolist() == want


def test_drafts_ids_that_are_none():
    s = make_drafts([5, 5], 700, 6, torch.float32, near=0.0)
    s["ids"][2], s["ids"][6] = 700, -3
    accepted, _ = check_drafts(s)
    assert accepted.tolist() == [1, 0]


def test_drafts_many_requests():
    rng = np.random.default_rng(0)
    news = [int(x) for x in rng.integers(0, 4, 4096)]
    check_drafts(make_drafts(news, 333, 7, temps=[float(x) for x in rng.choice([0.0, 0.5, 1.0], 4096)]))


@pytest.mark.parametrize("requests", [64, 65, 130])
@pytest.mark.parametrize("draft", [True, False])
def test_drafts_of_batches_that_fill_the_chip(requests, draft):
    """Long rows of 64 requests and fewer are drawn from in 64 chunks, those of more in 32."""
    check_drafts(make_drafts([2] * requests, 70001, requests, torch.bfloat16, draft=draft, near=0.05))


def test_drafts_scalar_temperature_outputs_and_streams():
    s = make_drafts([5, 2, 7], 9001, 9)
    want = check_drafts(s)
    args = (s["target"], s["ids"], s["batch"], s["u_accept"], s["u_next"])
    # 0.9 is rounded to 32 bits on its way, as the tensor's is
    got = ocq.verify_drafts(*args, draft_probs=s["draft"], temperature=0.9)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    acc, out = torch.empty(3, dtype=torch.int32, device=DEV), torch.empty(14, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        acc.fill_(-5)
        side.wait_stream(torch.cuda.current_stream())
        ws = torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device=DEV)
        side.wait_stream(torch.cuda.current_stream())
        a, b = ocq.verify_drafts(*args, draft_probs=s["draft"], temperature=0.9, accepted=acc, out=out, workspace=ws,
                                 stream=side)
        side.synchronize()
        assert a is acc and b is out and torch.equal(a, want[0]) and torch.equal(b, want[1])


@pytest.mark.parametrize("news", [[5, 0, 3, 1, 0], [0, 2], [20]])
def test_drafts_greedy_for_all(news):
    """One temperature of 0 for all requests: as a tensor of zeros."""
    for dtype in (torch.bfloat16, torch.float32):
        s = make_drafts(news, 3001, 2, dtype, temps=0.0)
        want = check_drafts(s)
        got = ocq.verify_drafts(s["target"], s["ids"], s["batch"], s["u_accept"], s["u_next"], draft_probs=s["draft"],
                                temperature=0.0, accepted=torch.full((len(news),), 9, dtype=torch.int32, device=DEV))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_drafts_without_any():
    """Requests of one token each, with an empty matrix of draft probabilities and with none."""
    s = make_drafts([1, 1, 1], 5001, 3, torch.bfloat16, shift=1)
    assert s["draft"].shape[0] == 0
    want = check_drafts(s)
    s["draft"] = None
    got = check_drafts(s)
    assert torch.equal(want[1], got[1]) and got[0].tolist() == [0, 0, 0]


def test_drafts_rows_behind_the_last_request():
    """A padded batch: the rows that no request has are -1."""
    s = make_drafts([3, 4], 500, 10)
    start = s["batch"].q_start.clone()
    target = torch.cat([s["target"], s["target"]])
    ids, ua = torch.cat([s["ids"]] * 2), torch.cat([s["u_accept"]] * 2)
    one = torch.ones(2, dtype=torch.int32, device=DEV)
    batch = ocq.TokenBatch(start, one, one[:, None], 4, 1)
    draft = torch.cat([s["draft"], s["draft"], s["draft"]])
    want = check_drafts(s)
    a, out = ocq.verify_drafts(target, ids, batch, ua, s["u_next"], draft_probs=draft,
                               temperature=torch.tensor(s["temps"], device=DEV))
    assert torch.equal(a, want[0]) and torch.equal(out[:7], want[1]) and (out[7:] == -1).all()


def test_drafts_offsets_past_32_bits():
    """Logits of more than 2^32 bytes, the drawn rows at their end."""
    vocab, tokens = 1 << 20, 2200
    target = torch.zeros((tokens, vocab), dtype=torch.bfloat16, device=DEV)
    target[-1, 12345], target[-2, 54321] = 30.0, 30.0
    start = torch.tensor([0, tokens - 2, tokens], dtype=torch.int32, device=DEV)
    one = torch.ones(2, dtype=torch.int32, device=DEV)
    batch = ocq.TokenBatch(start, one, one[:, None], tokens, 1)
    ids = torch.zeros(tokens, dtype=torch.int32, device=DEV)
    ids[-1] = 54321
    zeros = torch.zeros(tokens, device=DEV)
    a, out = ocq.verify_drafts(target, ids, batch, zeros, torch.full((2,), 0.5, device=DEV))
    assert a.tolist() == [tokens - 3, 1] and out[-2:].tolist() == [54321, 12345]
    # the first request's next token: half of 2^20 equal weights lie before it
    assert int(out[tokens - 3]) == 1 << 19


# ---------------------------------------------------------------- tables

def tables_ref(t, news, tokens, accepted):
    """The step in whole numbers; t: lists q_start, kv, held, table, ring, counts and page."""
    page, table, ring = t["page"], [list(x) for x in t["table"]], list(t["ring"])
    taken, given = t["counts"]
    old, size, most = list(ring), len(ring), len(table[0])
    g0, o = given, dict(q_start=[0], kv=[], held=[], slots=[], positions=[], owners=[], missing=0)
    for r in range(len(news)):
        n = t["q_start"][r + 1] - t["q_start"][r]
        kept = 0 if news[r] < 0 else t["kv"][r] - n + (n if accepted is None else min(n, 1 + accepted[r]))
        new = max(0, news[r])
        kv = kept + new
        need = -(-kv // page)
        have = t["held"][r]
        for j in range(have, need):
            if j < most and taken < g0:
                table[r][j] = old[taken % size]
                taken, have = taken + 1, have + 1
            else:
                o["missing"] += 1
                if j < most:
                    table[r][j] = -1
        for j in range(need, t["held"][r]):
            ring[given % size] = table[r][j]
            given += 1
        o["held"].append(min(need, have))
        o["kv"].append(kv)
        o["q_start"].append(o["q_start"][-1] + new)
        for i in range(new):
            at = table[r][(kept + i) // page] if (kept + i) // page < most else -1
            o["slots"].append(at * page + (kept + i) % page if at >= 0 else -1)
            o["positions"].append(kept + i)
            o["owners"].append(r)
    for x in ("slots", "positions", "owners"):
        o[x] += [-1] * (tokens - len(o[x]))
    return dict(o, missing=[o["missing"]], counts=[taken, given], table=table, ring=ring, page=page)


def make_tables(requests, page, seed, longest=300, free=None, idle=0.2):
    """A server in the middle of its work: (lists as tables_ref takes them)."""
    rng = np.random.default_rng(seed)
    kv = [0 if rng.random() < idle else int(rng.integers(1, longest + 1)) for _ in range(requests)]
    held = [-(-x // page) for x in kv]
    olds = [0 if x == 0 else int(rng.integers(0, min(x, 14) + 1)) for x in kv]
    most = -(-longest // page) + 4
    free = sum(held) + 3 * requests if free is None else free
    pages = sum(held) + free
    order = [int(x) for x in rng.permutation(pages)]
    table, at = [], 0
    for h in held:
        table.append(order[at: at + h] + [-7] * (most - h))
        at += h
    taken = int(rng.integers(0, 1 << 40))
    ring = [-1] * pages
    for i, p in enumerate(order[at:]):
        ring[(taken + i) % pages] = p
    return dict(q_start=[0] + [int(x) for x in np.cumsum(olds)], kv=kv, held=held, table=table, ring=ring,
                counts=[taken, taken + free], page=page), olds, rng


def on_gpu(t):
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return ocq.PageTables(ints(t["q_start"]), ints(t["kv"]), ints(t["held"]),
                          torch.tensor(t["counts"], dtype=torch.int64, device=DEV), ints(t["table"]), ints(t["ring"]),
                          t["page"])


def check_tables(t, news, tokens, accepted, tables=None, **kw):
    tables = on_gpu(t) if tables is None else tables
    after = kw.get("out", tables)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    got = ocq.step_tables(tables, ints(news), tokens, accepted=None if accepted is None else ints(accepted), **kw)
    torch.cuda.synchronize()
    want = tables_ref(t, news, tokens, accepted)
    for x, name in zip(got, ("slots", "positions", "owners", "missing")):
        assert x.tolist() == want[name], name
    for x, name in ((after.q_start, "q_start"), (after.kv_lens, "kv"), (after.held, "held"), (after.counts, "counts"),
                    (after.page_table, "table"), (after.ring, "ring")):
        assert x.tolist() == want[name], name
    return want, tables


@pytest.mark.parametrize("requests", [1, 2, 63, 64, 65, 300, 1024, 1025, 2500])
@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("in_place", [True, False])
def test_tables(requests, page, in_place):
    """Decoding, verifying, ending and starting requests, call after call, in place or in turn."""
    t, olds, rng = make_tables(requests, page, requests + page, longest=40 if page == 1 else 300)
    tables, other = on_gpu(t), None
    if not in_place:
        other = ocq.PageTables(*(torch.full_like(x, 77) for x in (tables.q_start, tables.kv_lens, tables.held,
                                                                  tables.counts)), tables.page_table, tables.ring, page)
    for step in range(4):
        accepted = [int(rng.integers(0, max(1, n))) for n in olds]
        news = [int(rng.choice([-1, 0, 1, 5, 13])) for _ in range(requests)]
        if step == 1:
            news = [int(rng.integers(0, 30)) if kv == 0 else n for kv, n in zip(t["kv"], news)]
        total = sum(max(0, n) for n in news)
        t, tables = check_tables(t, news, total + step, accepted if step != 2 else None, tables,
                                 **({} if in_place else dict(out=other)))
        if not in_place:
            tables, other = other, tables
        olds = [b - a for a, b in zip(t["q_start"], t["q_start"][1:])]


@pytest.mark.parametrize("requests,prompt", [(1, 131072), (3, 20000), (40, 3000), (1500, 40)])
def test_tables_prompts(requests, prompt):
    """Empty requests that start on prompts: all pages are taken in one step, and given back in another."""
    page = 16
    most = -(-prompt // page)
    t = dict(q_start=[0] * (requests + 1), kv=[0] * requests, held=[0] * requests, table=[[-1] * most] * requests,
             ring=list(range(requests * most)), counts=[0, requests * most], page=page)
    news = [prompt - r % 17 for r in range(requests)]
    t, tables = check_tables(t, news, sum(news), None)
    t, tables = check_tables(t, [-1 if r % 2 == 0 else 1 for r in range(requests)], requests, None, tables)
    check_tables(t, [prompt if r % 2 == 0 else 0 for r in range(requests)], prompt * requests, None, tables)


@pytest.mark.parametrize("requests", [3, 700, 1300])
def test_tables_with_too_few_pages(requests):
    """The requests that come first get what there is; the others' entries are -1, and the next step tries again."""
    t, olds, rng = make_tables(requests, 16, requests, free=requests // 2)
    news = [33] * requests
    t, tables = check_tables(t, news, sum(news), None)
    assert t["missing"][0] > 0
    t, tables = check_tables(t, [-1] + [0] * (requests - 1), 4, None, tables)
    t, tables = check_tables(t, [0] * requests, 0, None, tables)


def test_tables_that_give_all_pages_back():
    """Many long requests end in a step of few tokens."""
    requests, most = 70, 8000
    t = dict(q_start=list(range(requests + 1)), kv=[16 * most - r for r in range(requests)], held=[most] * requests,
             table=[list(range(r * most, (r + 1) * most)) for r in range(requests)], ring=[-1] * (requests * most),
             counts=[5, 5], page=16)
    t, tables = check_tables(t, [-1] * requests, 3, [0] * requests)
    assert sorted(t["ring"]) == list(range(requests * most))
    check_tables(t, [16 * most if r == 3 else 0 for r in range(requests)], 16 * most, None, tables)


def test_tables_past_the_table():
    """Requests longer than their rows of the page table: the pages beyond it are missing, their tokens have no slot."""
    t, olds, rng = make_tables(5, 16, 1, longest=60)
    for news in ([200, 1, 0, 90, 1000], [1, 1, 1, 1, 1]):
        t, tables = check_tables(t, news, sum(news) + 3, None)
    assert t["missing"][0] > 0


def test_tables_of_any_contents_write_nothing_elsewhere():
    """Numbers that no step leaves (negative, huge, not sorted) give wrong tables, never a write outside them."""
    for requests in (40, 1500):
        t, olds, rng = make_tables(requests, 16, 3)
        tables = on_gpu(t)
        wide = torch.full((requests, tables.page_table.shape[1] + 2), 99, dtype=torch.int32, device=DEV)
        wide[:, 1:-1] = tables.page_table
        ring = torch.full((len(t["ring"]) + 2,), 99, dtype=torch.int32, device=DEV)
        gen = torch.Generator(DEV).manual_seed(requests)
        for trial in range(8):
            r = lambda n: torch.randint(-2 ** 31, 2 ** 31, (n,), device=DEV, generator=gen).to(torch.int32)  # noqa: E731
            odd = ocq.PageTables(r(requests + 1), r(requests), r(requests),
                                 torch.randint(-2 ** 62, 2 ** 62, (2,), device=DEV, generator=gen), wide[:, 1:-1],
                                 ring[1:-1], 16)
            out = torch.full((1002,), 99, dtype=torch.int64, device=DEV)
            news = r(requests) if trial % 2 else r(requests) % 50
            ocq.step_tables(odd, news, 1000, accepted=r(requests), slots=out[1:-1])
            torch.cuda.synchronize()
            assert (wide[:, [0, -1]] == 99).all() and (ring[[0, -1]] == 99).all() and (out[[0, -1]] == 99).all()


def test_tables_outputs_and_streams():
    t, olds, rng = make_tables(20, 16, 5)
    news = [3] * 20
    side = torch.cuda.Stream()
    a = on_gpu(t)
    side.wait_stream(torch.cuda.current_stream())
    ints = torch.tensor(news, dtype=torch.int32, device=DEV)
    side.wait_stream(torch.cuda.current_stream())
    got = ocq.step_tables(a, ints, 70, stream=side)
    side.synchronize()
    want = tables_ref(t, news, 70, None)
    assert got[0].tolist() == want["slots"] and a.kv_lens.tolist() == want["kv"]
    b = on_gpu(t)
    outs = [torch.empty(70, dtype=torch.int64, device=DEV)] + [torch.empty(n, dtype=torch.int32, device=DEV) for n in (70, 70, 1)]
    again = ocq.step_tables(b, ints, 70, slots=outs[0], positions=outs[1], requests=outs[2], missing=outs[3])
    assert all(x is y for x, y in zip(again, outs)) and torch.equal(again[0], got[0])


def test_tables_empty_ones():
    a = ocq.PageTables.allocate(3, 4, 12, 16, device=DEV)
    ocq.step_tables(a, torch.zeros(3, dtype=torch.int32, device=DEV), 0)
    assert a.kv_lens.tolist() == [0, 0, 0] and a.counts.tolist() == [0, 12] and a.q_start.tolist() == [0, 0, 0, 0]


# ---------------------------------------------------------------- graphs, refusals

def test_captured_steps_replay():
    """Tables, append, attention, drafts and tables again in one graph, replayed with other inputs: every replay as the
    eager calls on the same inputs."""
    requests, page, most, heads, dim, vocab = 3, 16, 40, 4, 64, 2000
    g = torch.Generator(DEV).manual_seed(2)
    sides = []
    for _ in range(2):
        tables = ocq.PageTables.allocate(requests, most, requests * most, page, device=DEV)
        batch = ocq.TokenBatch(tables.q_start, tables.kv_lens, tables.page_table, 5, most * page)
        cache = ocq.PagedKVCache.allocate(requests * most, page, 2, dim, nvfp4=True, device=DEV)
        sides.append((tables, batch, cache))
    rope = ocq.Rope.make(dim, device=DEV)
    news = torch.tensor([5, 3, 1], dtype=torch.int32, device=DEV)
    accepted = torch.full((requests,), 4, dtype=torch.int32, device=DEV)
    q = torch.zeros((9, heads + 4, dim), dtype=torch.bfloat16, device=DEV)
    target, ids = torch.zeros((9, vocab), device=DEV), torch.zeros(9, dtype=torch.int32, device=DEV)
    ua, un = torch.zeros(9, device=DEV), torch.zeros(requests, device=DEV)
    draft = torch.full((6, vocab), 1 / vocab, device=DEV)

    def step(tables, batch, cache):
        slots = ocq.step_tables(tables, news, 9, accepted=accepted)
        x = ocq.rope_append(q[:, :heads], q[:, heads:heads + 2], q[:, heads + 2:], rope, cache, batch)
        o, lse = ocq.paged_attention(x, cache, batch, want_lse=True)
        return slots + (o, lse) + ocq.verify_drafts(target, ids, batch, ua, un, draft_probs=draft, accepted=acc_of[id(tables)])
    acc_of = {id(s[0]): torch.zeros(requests, dtype=torch.int32, device=DEV) for s in sides}
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step(*sides[0])
    torch.cuda.current_stream().wait_stream(warm)
    step(*sides[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(*sides[0])
    for i in range(5):
        q.copy_(torch.randn(q.shape, device=DEV, generator=g))
        target.copy_(torch.randn(target.shape, device=DEV, generator=g) * 3)
        ids.copy_(torch.randint(0, vocab, ids.shape, device=DEV, generator=g))
        ua.copy_(torch.rand(ua.shape, device=DEV, generator=g) * 0.01)
        un.copy_(torch.rand(un.shape, device=DEV, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, step(*sides[1])):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
        accepted.copy_(got[-2])
        torch.cuda.synchronize()
    for x, y in zip(sides[0][0].__dict__.values(), sides[1][0].__dict__.values()):
        if isinstance(x, torch.Tensor):
            assert torch.equal(x, y)


def test_binding_refusals():
    s = make_drafts([3, 2], 100, 1)
    b, t = s["batch"], on_gpu(make_tables(4, 16, 1)[0])
    args = lambda **kw: {**dict(target=s["target"], tokens=s["ids"], batch=b, u_accept=s["u_accept"],  # noqa: E731
                                u_next=s["u_next"], draft_probs=s["draft"]), **kw}
    news = torch.zeros(4, dtype=torch.int32, device=DEV)
    other = ocq.PageTables.allocate(4, 8, 32, 16, device=DEV)
    for call in (lambda: ocq.verify_drafts(**args(target=s["target"].half())),
                 lambda: ocq.verify_drafts(**args(target=s["target"][:4])),
                 lambda: ocq.verify_drafts(**args(target=s["target"].t())),
                 lambda: ocq.verify_drafts(**args(tokens=s["ids"].long())),
                 lambda: ocq.verify_drafts(**args(u_accept=s["u_accept"].double())),
                 lambda: ocq.verify_drafts(**args(u_next=s["u_accept"])),
                 lambda: ocq.verify_drafts(**args(draft_probs=s["draft"][:2])),
                 lambda: ocq.verify_drafts(**args(draft_probs=s["draft"][:, :99])),
                 lambda: ocq.verify_drafts(**args(temperature=-1.0)),
                 lambda: ocq.verify_drafts(**args(temperature=float("nan"))),
                 lambda: ocq.verify_drafts(**args(temperature=torch.ones(3, device=DEV))),
                 lambda: ocq.verify_drafts(**args(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))),
                 lambda: ocq.verify_drafts(**args(out=torch.empty(4, dtype=torch.int32, device=DEV))),
                 lambda: ocq.step_tables(t, news.long(), 4), lambda: ocq.step_tables(t, news[:3], 4),
                 lambda: ocq.step_tables(t, news, -1), lambda: ocq.step_tables(t, news, 4, accepted=news[:2]),
                 lambda: ocq.step_tables(t, news, 4, out=other),
                 lambda: ocq.step_tables(t, news, 4, slots=torch.empty(4, dtype=torch.int32, device=DEV)),
                 lambda: ocq.PageTables(t.q_start, t.kv_lens, t.held, t.counts.int(), t.page_table, t.ring, 16),
                 lambda: ocq.PageTables(t.q_start[1:], t.kv_lens, t.held, t.counts, t.page_table, t.ring, 16),
                 lambda: ocq.PageTables(t.q_start, t.kv_lens, t.held, t.counts, t.page_table[:3], t.ring, 16),
                 lambda: ocq.step_tables(ocq.PageTables(t.q_start, t.kv_lens, t.held, t.counts, t.page_table, t.ring, 24),
                                         news, 4)):
        with pytest.raises(ocq.OcqError) as e:
            call()
        assert e.value.status in (ocq.ERR_INVALID_ARG, ocq.ERR_UNSUPPORTED, ocq.ERR_BUFFER_TOO_SMALL)
