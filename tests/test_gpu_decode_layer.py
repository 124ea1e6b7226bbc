"""PagedAttention, LogitRules behind ScoringHead, and the decode command: the operators together, as they are used."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.attention_cases import UNIT, Paged, attention_bounds, attention_oracle, f64  # noqa: E402


def note(msg):
    print(f"[case] {msg}", flush=True)


def make(heads=8, kv=2, dim=64, page=16, per_seq=12, seqs=3, tokens=200, seed=0, **kw):
    from binary_basis_lut_amd.paged import PagedAttention
    l = PagedAttention(heads, kv, dim, seqs * per_seq + 2, page, seqs, per_seq, tokens, **kw)
    g = torch.Generator().manual_seed(seed)
    l.page_table.copy_(torch.randperm(seqs * per_seq + 2, generator=g)[:seqs * per_seq].view(seqs, per_seq))
    return l, g


def check_step(l, out, news, lens):
    """out against the definition, of the queries and the cache as they stand."""
    c = Paged.__new__(Paged)
    c.dt, c.heads, c.kv, c.dim, c.page = "f16" if l.dtype == torch.float16 else "bf16", l.heads, l.kv_heads, l.dim, l.k_cache.shape[2]
    c.lengths, c.lens_host = [(n, t - n) for n, t in zip(news, lens)], lens
    c.rows = c.tokens = sum(news)
    c.starts_host = np.concatenate([[0], np.cumsum(news)])
    c.order, c.pages, c.per_seq, c.table_host = "heads", l.k_cache.shape[0], l.page_table.shape[1], l.page_table.cpu().numpy()
    c.q, c.k, c.v = l.q[:c.rows].cpu(), l.k_cache.cpu(), l.v_cache.cpu()
    want, _, mag, work, seen = attention_oracle(c, 1 / math.sqrt(c.dim), l.window)
    tol, _ = attention_bounds(c, want, mag, work, seen)
    assert (np.abs(f64(out).reshape(want.shape) - want) <= tol).all()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("window", [0, 20])
def test_prompts_then_single_tokens(dtype, window):
    """Two prompts and an empty place, then steps of one token each: rotation by the place in the cache throughout."""
    note(f"prompts then decode {dtype} window {window}")
    dt = getattr(torch, dtype)
    l, g = make(dtype=dt, window=window, rotary_dim=32, pairs=1)
    width = 12 * 64
    rows = [(torch.randn(60, width, generator=g) * 1.5).to(dt), (torch.randn(130, width, generator=g) * 1.5).to(dt)]
    lens = [40, 100, 0]
    l.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    qkv = torch.cat([rows[0][:40], rows[1][:100]]).cuda()
    starts = torch.tensor([0, 40, 140, 140], dtype=torch.int32, device="cuda")
    out = l.attend(qkv, starts)
    torch.cuda.synchronize()
    check_step(l, out, [40, 100, 0], lens)
    for step in range(15):
        lens = [n + 1 for n in lens[:2]]
        l.kv_lens[:2].add_(1)
        out = l.attend(torch.stack([rows[0][40 + step], rows[1][100 + step]]).cuda())
        torch.cuda.synchronize()
        check_step(l, out, [1, 1], lens)
    # the cache holds the rotated keys of all tokens, as if they had come at once
    again, _ = make(dtype=dt, window=window, rotary_dim=32, pairs=1)
    again.kv_lens.copy_(torch.tensor(lens + [0], dtype=torch.int32))
    again.attend(torch.cat([rows[0][:55], rows[1][:115]]).cuda(), torch.tensor([0, 55, 170, 170], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(again.k_cache, l.k_cache) and torch.equal(again.v_cache, l.v_cache)


def test_one_graph_serves_every_step_and_rows_behind_the_last_sequence_stay():
    note("one graph for all steps, padded rows")
    l, g = make(seqs=4)
    qkv = torch.randn(6, 12 * 64, generator=g).half().cuda()
    starts = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32, device="cuda")
    l.kv_lens.copy_(torch.tensor([3, 20, 47, 1], dtype=torch.int32))
    l.k_cache.copy_(torch.randn(l.k_cache.shape, generator=g))
    l.v_cache.copy_(torch.randn(l.v_cache.shape, generator=g))
    first = l.k_cache.clone(), l.v_cache.clone()
    l.out.fill_(9)

    def step():
        l.kv_lens.add_(1)
        return l.attend(qkv, starts)

    want = [step().clone() for _ in range(4)]
    torch.cuda.synchronize()
    assert all((w[4:] == 9).all() for w in want)
    l.kv_lens.copy_(torch.tensor([3, 20, 47, 1], dtype=torch.int32))
    l.k_cache.copy_(first[0])
    l.v_cache.copy_(first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for w in want:
        torch.randn(1 << 16, device="cuda").sum()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


def test_two_layers_on_two_streams():
    note("two layers on two streams at once")
    pairs = [make(heads=32, kv=8, dim=128, per_seq=260, seqs=2, tokens=8, seed=s) for s in (1, 2)]
    qkvs, want = [], []
    for l, g in pairs:
        l.kv_lens.copy_(torch.tensor([4000, 1500], dtype=torch.int32))
        l.k_cache.copy_(torch.randn(l.k_cache.shape, generator=g))
        l.v_cache.copy_(torch.randn(l.v_cache.shape, generator=g))
        qkvs.append(torch.randn(2, 48 * 128, generator=g).half().cuda())
        want.append(l.attend(qkvs[-1]).clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pairs]
    for _ in range(5):
        for (l, _), q, s in zip(pairs, qkvs, streams):
            with torch.cuda.stream(s):
                l.attend(q)
    torch.cuda.synchronize()
    for (l, _), w in zip(pairs, want):
        assert torch.equal(l.out[:2], w)


def test_rules_change_the_scores_of_a_head():
    from binary_basis_lut_amd.score_tokens import LogitRules, ScoringHead
    note("rules behind a head")
    rows, hidden, vocab = 5, 512, 3001
    g = torch.Generator().manual_seed(3)
    head = ScoringHead(torch.ones(hidden).half().cuda(), (torch.randn(vocab, hidden, generator=g) * 0.05).half().cuda(), 8)
    y, residual = (torch.randn(rows, hidden, generator=g).half().cuda() for _ in range(2))
    targets = torch.randint(0, vocab, (rows,), generator=g).cuda()
    plain = {n: v.clone() for n, v in head.score(y, residual, targets).items()}
    mask = torch.full((8, (vocab + 31) // 32), -1, dtype=torch.int32)
    best = plain["top_index"][:, 0].cpu()
    for r in range(rows):  # the best token of every row is forbidden, the second is penalised, the third favoured
        mask[r, best[r] // 32] ^= int(np.uint32(1 << int(best[r] % 32)).astype(np.int32))
    bias_index = torch.zeros(8, 1, dtype=torch.int32)
    bias_index[:rows, 0] = plain["top_index"][:, 2].int().cpu()
    rules = LogitRules(8, vocab, 4, repetition=torch.full((8,), 1.5, device="cuda"), frequency=torch.full((8,), 0.5, device="cuda"),
                       bias_index=bias_index.cuda(), bias_value=torch.full((8, 1), 20.0, device="cuda"), mask=mask.cuda())
    history = torch.zeros(8, 2, dtype=torch.int64, device="cuda")
    history[:rows] = plain["top_index"][:, 1:2]
    rules.append(history)  # twice the second best
    out = head.score(y, residual, targets, rules=rules)
    torch.cuda.synchronize()
    z = plain["logits"].double().cpu()
    row = torch.arange(rows)
    second, third = (plain["top_index"][:, i].cpu() for i in (1, 2))
    s = z[row, second]
    z[row, second] = torch.where(s > 0, s / 1.5, s * 1.5) - 1.0
    z[row, third] += 20
    z[row, best] = -math.inf
    got = out["logits"].cpu().double()
    assert torch.equal(torch.isinf(got), torch.isinf(z))
    assert (got - z)[~torch.isinf(z)].abs().max() <= 4 * 2.0 ** -24 * 30
    assert torch.equal(out["top_index"][:, 0].cpu(), third)
    lp = torch.log_softmax(got, 1)
    assert (out["top_logprob"].cpu().double() - lp.gather(1, out["top_index"].cpu())).abs().max() < 1e-4
    # the history holds what fits, and clear() forgets it
    rules.append(torch.full((8, 9), 7, dtype=torch.int64, device="cuda"))
    assert rules.total_len.tolist() == [4] * 8
    rules.clear()
    rules.mask.fill_(-1)
    rules.bias_value.zero_()
    assert torch.equal(head.score(y, residual, targets, rules=rules)["logits"], plain["logits"])


def test_the_command_runs():
    from binary_basis_lut_amd.decode_layer import run
    kw = dict(batch=3, steps=5, context=70, vocab=2000, heads=4, dim=64)
    r = run(**kw)
    assert r["kv_lens"] == [75] * 3
    assert all(0 <= t < 2000 and t % 32 for row in r["tokens"] for t in row)  # the mask forbids every 32nd token
    assert all(p <= 0 for row in r["logprobs"] for p in row) and np.shape(r["tokens"]) == (3, 5)
    again = run(**kw)
    assert again["tokens"] == r["tokens"] and again["logprobs"] == r["logprobs"]
