"""fluxbin_paged_attention and fluxbin_rope_append against their definitions in 64 bits (tests/attention_cases.py)."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.attention_cases import DT, TINY, U, UNIT, Paged, attention_bounds, attention_oracle, f64  # noqa: E402


@pytest.fixture(scope="module")
def fb():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    from binary_basis_lut_amd import fluxbin
    return fluxbin


def note(msg):
    print(f"[case] {msg}", flush=True)


def attend(fb, c, scale, window=0, lse=True, pad=0):
    """out and lse as the kernel leaves them, rows of out `pad` elements further apart; untouched places hold 7."""
    b = c.upload(fb)
    ld = c.heads * c.dim + pad
    q = torch.zeros(c.tokens, ld, dtype=DT[c.dt], device="cuda")
    q[:, :c.heads * c.dim] = c.dev["q"]
    out = torch.full((c.tokens, ld), 7.0, dtype=DT[c.dt], device="cuda")
    ls = torch.full((c.tokens, c.heads), 7.0, dtype=torch.float32, device="cuda") if lse else None
    need = fb.fluxbin_paged_attention_workspace_size(b)
    ws = torch.full((max(need, 16) // 4 + 4,), math.nan, dtype=torch.float32, device="cuda")
    torch.cuda.synchronize()
    fb.fluxbin_paged_attention(b, q, ld, scale, window, out, ld, ls, ws, need)
    torch.cuda.synchronize()
    assert (out[:, c.heads * c.dim:] == 7).all()
    assert (out[c.rows:] == 7).all() and (ls is None or (ls[c.rows:] == 7).all())  # rows behind the last sequence
    got = f64(out[:c.rows, :c.heads * c.dim]).reshape(c.rows, c.heads, c.dim)
    return got, None if ls is None else f64(ls[:c.rows])


def check(fb, c, window=0, pad=0):
    scale = 1 / math.sqrt(c.dim)
    got, ls = attend(fb, c, scale, window, pad=pad)
    out, lse, mag, work, seen = attention_oracle(c, scale, window)
    tol, tol_lse = attention_bounds(c, out, mag, work, seen)
    empty = seen == 0
    assert (got[empty] == 0).all() and np.isneginf(ls[empty]).all()
    off = np.abs(got - out)
    assert (off <= tol).all(), float((off / tol).max())
    live = ~empty
    assert (np.abs(ls - lse)[live] <= (tol_lse + 4 * U * np.abs(lse))[live]).all()


FEW = [(1, 0)], [(1, 15), (1, 16), (1, 31), (1, 32)], [(1, 1), (1, 700), (1, 63), (1, 128)]
CHUNK = [(1, 0), (40, 3)], [(64, 0)], [(130, 77), (3, 200), (65, 0)], [(33, 500)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [8, 40, 64, 72, 128, 136, 256])
@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 2), (6, 2)])
def test_decode(fb, dt, dim, heads, kv):
    for i, lengths in enumerate(FEW):
        note(f"decode {dt} dim {dim} heads {heads}/{kv} lengths {lengths}")
        check(fb, Paged(dt, heads, kv, dim, (16, 32, 64)[i], lengths, seed=dim + i), pad=(0, 1, 5)[i])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [8, 64, 72, 128, 256])
@pytest.mark.parametrize("heads,kv", [(2, 2), (6, 2)])
def test_chunks(fb, dt, dim, heads, kv):
    for i, lengths in enumerate(CHUNK):
        note(f"chunk {dt} dim {dim} heads {heads}/{kv} lengths {lengths}")
        check(fb, Paged(dt, heads, kv, dim, (16, 64, 32, 128)[i], lengths, seed=dim + i, order=("heads", "tokens")[i % 2], behind=i),
              pad=(0, 1, 8, 3)[i])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("lengths", [[(1, 5000)], [(3, 2000)], [(1, 300), (1, 4000), (1, 2)]])
def test_keys_split_over_workgroups(fb, dt, lengths):
    note(f"splits {dt} {lengths}")
    c = Paged(dt, 4, 1, 128, 16, lengths, seed=5, max_kv_len=8192)
    assert fb.fluxbin_paged_attention_workspace_size(c.upload(fb)) > 0
    check(fb, c)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv,lengths", [(64, 1, [(1, 300), (1, 7)]), (40, 1, [(1, 130)]), (33, 1, [(2, 90), (1, 0), (4, 9)]),
                                              (48, 2, [(3, 40)]), (16, 1, [(2, 100), (2, 0)])])
def test_many_query_heads_to_a_key_head(fb, dt, heads, kv, lengths):
    """More rows of single tokens than 32, exactly 32, and tiles that begin inside a group."""
    note(f"{heads} heads to {kv}, {dt} {lengths}")
    for dim in (64, 128):
        check(fb, Paged(dt, heads, kv, dim, 32, lengths, seed=heads, order="tokens"))


def test_lengths_that_the_host_does_not_know_of(fb):
    """max_kv_len only divides the work: sequences may be longer or shorter."""
    note("max_kv_len too small and too large")
    for max_kv in (1, 100, 1 << 20):
        for lengths in ([(1, 900), (1, 0)], [(1, 3000)], [(150, 2000)]):
            check(fb, Paged("f16", 4, 2, 64, 16, lengths, seed=max_kv, max_kv_len=max_kv, table_extra=100))


def mixed(seqs, seed, longest):
    """Sequences without a new token, with one, with a few, and one of them with `longest`."""
    rng = np.random.default_rng(seed)
    lengths = [(int(n), int(p)) for n, p in zip(rng.choice([0, 1, 1, 1, 2, 3], seqs), rng.integers(0, 70, seqs))]
    lengths[int(rng.integers(seqs))] = (longest, 50)
    return lengths


@pytest.mark.parametrize("seqs", [63, 64, 65, 200, 4200])
def test_many_sequences(fb, seqs):
    """One round of look-ups and several; single tokens beside a long chunk, in both forms; rows behind the last."""
    cases = [("single", 2, [(1, s % 40) for s in range(seqs)]), ("mixed", 2, mixed(seqs, seqs, 100))]
    if seqs <= 200:  # 8 rows to a token, and more than 32 to a sequence
        cases.append(("chunks", 8, mixed(seqs, seqs + 1, 4 * seqs)))
    for name, heads, lengths in cases:
        note(f"{seqs} sequences, {name}")
        c = Paged("f16", heads, 1, 64, 16, lengths, seed=seqs, behind=0 if name == "single" else 3)
        whole = {id(t): f64(t) for t in (c.k, c.v)}
        c.cached = lambda cache, s, c=c, whole=whole: np.array(
            [whole[id(cache)][c.table_host[s, j // 16], :, j % 16] for j in range(c.lens_host[s])]).reshape(-1, 1, 64)
        check(fb, c)


@pytest.mark.parametrize("seqs", [63, 64, 65, 200, 4200])
def test_rope_append_of_many_sequences(fb, seqs):
    """Keys and values as they are, without a rotation, each at its place; the queries too."""
    for lengths in ([(1, s % 40) for s in range(seqs)], mixed(seqs, seqs, 100)):
        note(f"rope_append, {seqs} sequences, {sum(n for n, _ in lengths)} rows")
        c = Paged("bf16", 2, 1, 64, 16, lengths, seed=seqs, behind=3 if max(lengths)[0] > 1 else 0)
        b = c.upload(fb)
        x = c.randn(c.tokens, 256)
        xd, q_out = x.cuda(), torch.full((c.tokens, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        fb.fluxbin_rope_append(b, xd, 256, xd[:, 128:], 256, xd[:, 192:], 256, None, None, 0.0, None, 0, 0, 1.0, None, q_out, 128)
        torch.cuda.synchronize()
        assert torch.equal(q_out[:c.rows].cpu(), x[:c.rows, :128]) and (q_out[c.rows:] == 7).all()
        want_k, want_v = c.k.clone(), c.v.clone()
        row = 0
        for s, (n, past) in enumerate(lengths):
            for t in range(past, past + n):
                page = c.table_host[s, t // 16]
                want_k[page, 0, t % 16], want_v[page, 0, t % 16] = x[row, 128:192], x[row, 192:]
                row += 1
        assert torch.equal(c.dev["k"].cpu(), want_k) and torch.equal(c.dev["v"].cpu(), want_v)


@pytest.mark.parametrize("window", [1, 2, 31, 100, 1000])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_windows(fb, window, dim):
    for lengths in ([(1, 0), (1, 99), (1, 100), (1, 777)], [(70, 130), (9, 0)], [(5, 1200)]):
        note(f"window {window} dim {dim} {lengths}")
        check(fb, Paged("f16", 4, 2, dim, 32, lengths, seed=window), window=window)


BALANCED = [(128, 4, 1, [(200, 3000)]), (64, 2, 2, [(300, 1700), (40, 5), (0, 0), (150, 900)]), (256, 2, 1, [(130, 1500)]),
            (72, 6, 2, [(90, 2500), (33, 0)]), (128, 2, 1, [(70, 0), (65, 4100)])]


def balanced(dt, dim, heads, kv, lengths, seed, page=16, **kw):
    """A table so long that the host takes the work for large: shares of key tiles are handed out."""
    rows = -(-sum(n for n, _ in lengths) * (heads // kv) // len(lengths))
    busy = len(lengths) * -(-rows // 128) * kv
    return Paged(dt, heads, kv, dim, page, lengths, seed=seed, decode=False, table_extra=(1 << 21) // busy // page + 1, max_kv_len=0, **kw)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("dim,heads,kv,lengths", BALANCED)
def test_shares_of_key_tiles(fb, dt, dim, heads, kv, lengths):
    note(f"shares {dt} dim {dim} heads {heads}/{kv} {lengths}")
    for window, order in ((0, "heads"), (1000, "tokens")):
        c = balanced(dt, dim, heads, kv, lengths, 7, order=order, behind=3)
        assert fb.fluxbin_paged_attention_workspace_size(c.upload(fb)) > 0  # without shares a chunk needs none
        check(fb, c, window=window)


def counting(c, seed):
    """q = 0 and values that name their key: every output is a number of keys over a number of keys."""
    c.q.zero_()
    g = torch.Generator().manual_seed(seed)
    for s in range(len(c.lengths)):
        for j in range(c.lens_host[s]):
            p = c.table_host[s, j // c.page] if j // c.page < c.per_seq else -1
            if 0 <= p < c.pages:
                view = c.v[p, :, j % c.page] if c.order == "heads" else c.v[p, j % c.page]
                view.zero_()
                view[:, int(torch.randint(0, c.dim, (1,), generator=g))] = 1


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("dim,heads,kv,lengths,window,max_kv", [
    (64, 4, 1, [(1, 17), (1, 160), (1, 333)], 0, None), (64, 2, 2, [(1, 500)], 77, 4096), (128, 8, 1, [(2, 90), (4, 0)], 0, None),
    (128, 2, 2, [(150, 40), (7, 300)], 0, None), (128, 2, 1, [(150, 40), (70, 300)], 50, 4096), (256, 2, 1, [(90, 33)], 0, None),
    (256, 2, 1, [(1, 400), (1, 3)], 100, None), (72, 3, 1, [(20, 100), (0, 50), (90, 0)], 0, None),
])
def test_every_key_counts_once(fb, dt, dim, heads, kv, lengths, window, max_kv):
    note(f"counting {dt} dim {dim} heads {heads}/{kv} {lengths} window {window}")
    for order in ("heads", "tokens"):
        c = Paged(dt, heads, kv, dim, 16, lengths, seed=3, order=order, max_kv_len=max_kv, decode=False)
        counting(c, 1)
        got, ls = attend(fb, c, 0.3, window)
        out, lse, _, _, seen = attention_oracle(c, 0.3, window)
        # sums of equal weights are exact; the quotient has two roundings, the output one
        assert (np.abs(got - out) <= (UNIT[dt] + 3 * U) * out).all()
        assert (np.abs(ls - lse) <= 4 * U * np.abs(lse) + 4 * U * np.log2(seen + 1.0)[:, None] + 8 * U).all()


@pytest.mark.parametrize("dim,heads,kv,lengths", BALANCED)
def test_every_key_counts_once_in_shares(fb, dim, heads, kv, lengths):
    note(f"counting in shares, dim {dim} {lengths}")
    for window in (0, 700):
        c = balanced("f16", dim, heads, kv, lengths, 2)
        counting(c, 5)
        got, ls = attend(fb, c, 0.3, window)
        out, lse, _, _, seen = attention_oracle(c, 0.3, window)
        assert (np.abs(got - out) <= (UNIT["f16"] + 3 * U) * out).all()
        live = seen > 0
        assert (np.abs(ls - lse) <= 4 * U * np.abs(lse) + 4 * U * np.log2(seen + 1.0)[:, None] + 8 * U)[live].all()


def test_shares_with_pages_that_are_not_there_and_values_that_are_not_numbers(fb):
    note("shares, missing pages and NaN")
    c = balanced("f16", 128, 4, 1, [(200, 3000), (50, 0)], 3)
    c.table_host[0, 3:70:2] = -1
    c.table_host[0, 190:] = c.pages
    check(fb, c)
    c = balanced("f16", 128, 4, 1, [(200, 3000)], 4)
    clean, _ = attend(fb, c, 0.1)
    out, _, mag, work, seen = attention_oracle(c, 0.1)
    tol, _ = attention_bounds(c, out, mag, work, seen)
    last = c.lens_host[0] - 1
    c.v[c.table_host[0, last // 16], :, last % 16] = math.nan
    got, _ = attend(fb, c, 0.1)
    assert np.isnan(got[-1]).all() and (np.abs(got - clean) <= 2 * tol)[:-1].all()
    c.table_host[:] = -1
    check(fb, c)
    c.lens_host = [7]  # shorter than the new tokens
    check(fb, c)


@pytest.mark.parametrize("dim,heads,kv,lengths", [(128, 4, 2, [(1, 200), (1, 90)]), (64, 2, 2, [(100, 60), (40, 0)]),
                                                  (256, 2, 1, [(80, 60)])])
def test_pages_that_are_not_there(fb, dim, heads, kv, lengths):
    """Numbers outside the cache, in the middle and at the ends, and an index beyond the table."""
    note(f"missing pages dim {dim} {lengths}")
    c = Paged("f16", heads, kv, dim, 16, lengths, seed=8, decode=False)
    c.table_host[0, 0] = -1
    c.table_host[0, 3] = c.pages
    c.table_host[-1, 1] = 2 ** 31 - 1
    c.table_host[0, 5] = -2 ** 31
    check(fb, c)
    check(fb, c, window=40)
    c.lens_host = [n + 64 for n in c.lens_host]  # now the new tokens lie beyond the table
    check(fb, c)
    c.table_host[:] = -1
    check(fb, c)
    c.lens_host = [1 for _ in c.lens_host]  # shorter than the new tokens: their first ones have no index
    c.table_host[:, 0] = 0
    check(fb, c)
    c.lens_host = [0 for _ in c.lens_host]
    check(fb, c)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("dim,heads,kv,lengths,window", [
    (128, 8, 2, [(1, 100), (1, 37)], 0), (128, 8, 2, [(1, 100), (1, 37)], 20), (64, 4, 1, [(4, 70), (8, 3)], 0),
    (128, 2, 2, [(150, 20), (60, 100)], 0), (128, 2, 2, [(150, 20)], 33), (256, 2, 1, [(70, 50)], 30), (256, 4, 1, [(1, 50)], 0),
])
def test_what_a_row_does_not_see_does_not_matter(fb, dt, dim, heads, kv, lengths, window):
    """Pages of nobody, places behind the lengths, and later tokens' keys and values hold NaN and infinities."""
    note(f"NaN in unseen places {dt} dim {dim} {lengths} window {window}")
    bad = torch.tensor([math.nan, math.inf, -math.inf])
    c = Paged(dt, heads, kv, dim, 32, lengths, seed=4, decode=False)
    scale = 1 / math.sqrt(dim)
    clean, ls_clean = attend(fb, c, scale, window)
    out, _, mag, work, seen = attention_oracle(c, scale, window)
    tol, tol_lse = attention_bounds(c, out, mag, work, seen)
    mine = np.zeros((c.pages, c.page), dtype=bool)
    for s in range(len(lengths)):
        for j in range(c.lens_host[s]):
            if not window or j > c.lens_host[s] - lengths[s][0] - window:
                mine[c.table_host[s, j // 32], j % 32] = True
    for cache in (c.k, c.v):
        nobody = torch.from_numpy(~mine)[:, None, :, None].expand(cache.shape)
        cache[nobody] = bad[torch.randint(0, 3, (int(nobody.sum()),))].to(DT[dt])
    got, ls = attend(fb, c, scale, window)
    assert np.array_equal(got, clean) and np.array_equal(ls, ls_clean)
    # the last new token's key and value of sequence 0: its own row is NaN, the rows before are as they were
    last = c.lens_host[0] - 1
    for which in range(3):
        c.v[c.table_host[0, last // 32], :, last % 32, dim // 2] = bad[which].to(DT[dt])
        got, ls = attend(fb, c, scale, window)
        row = c.lengths[0][0] - 1
        others = np.arange(c.rows) != row
        want = clean.copy()
        want[row, :, dim // 2] = bad[which].item()
        # computed key by key, products and sums in another order: both are within their bounds of the definition, so within
        # twice those of each other
        assert ((np.abs(got - want) <= 2 * tol) | (np.isnan(got) & np.isnan(want)) | (got == want)).all()
        assert np.isfinite(got[others]).all() and (np.abs(ls - ls_clean) <= 2 * (tol_lse + 4 * U * np.abs(ls_clean))).all()
    c.k[c.table_host[0, last // 32], :, last % 32, 3] = math.nan
    got, ls = attend(fb, c, scale, window)
    assert np.isnan(got[row]).all() and np.isnan(ls[row]).all() and np.isfinite(got[others]).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("dim,heads,kv,lengths", [(128, 4, 2, [(1, 300), (1, 20)]), (64, 4, 2, [(130, 100)]), (256, 2, 1, [(70, 200)])])
def test_values_without_bounds_that_rows_do_see(fb, dt, dim, heads, kv, lengths):
    """An infinity among the values of an old key: its dimension is infinite, the others are as they were."""
    note(f"infinite values that are seen {dt} dim {dim} {lengths}")
    c = Paged(dt, heads, kv, dim, 16, lengths, seed=12, decode=False)
    clean, _ = attend(fb, c, 0.1)
    out, _, mag, work, seen = attention_oracle(c, 0.1)
    tol, _ = attention_bounds(c, out, mag, work, seen)
    p = c.table_host[0, 0]
    c.v[p, 0, 5, 3], c.v[p, 0, 6, 4], c.v[p, 0, 7, 5], c.v[p, 0, 8, 5] = math.inf, -math.inf, math.inf, -math.inf
    got, _ = attend(fb, c, 0.1)
    rows, mine = np.arange(lengths[0][0]), np.arange(heads // kv)
    want = clean.copy()
    for d, v in ((3, math.inf), (4, -math.inf), (5, math.nan)):
        want[np.ix_(rows, mine, [d])] = v
    same = (np.abs(got - want) <= 2 * tol) | (got == want) | (np.isnan(got) & np.isnan(want))
    assert same.all(), np.argwhere(~same)[:5]


@pytest.mark.parametrize("lengths", [[(1, 300)], [(130, 100)]])
def test_large_scores(fb, lengths):
    """Scores far apart and large: the weights of all but the largest vanish, and the maximum moves often."""
    note(f"large scores {lengths}")
    for dt in ("f16", "bf16"):
        c = Paged(dt, 4, 2, 128, 16, lengths, seed=6)
        c.q *= 30
        for s in range(len(lengths)):  # ascending keys: every tile raises the maximum
            for j in range(c.lens_host[s]):
                c.k[c.table_host[s, j // 16], :, j % 16] *= 0.02 * (j + 1)
        check(fb, c)


@pytest.mark.parametrize("lengths,max_kv", [([(1, 1000)], None), ([(1, 50), (1, 2000)], 4096), ([(300, 100)], None),
                                            ([(300, 2000), (20, 0)], 0)])
def test_repeats_streams_and_graphs(fb, lengths, max_kv):
    note(f"repeats and graphs {lengths}")
    c = balanced("bf16", 128, 8, 2, lengths, 9) if max_kv == 0 else Paged("bf16", 8, 2, 128, 16, lengths, seed=9, max_kv_len=max_kv)
    b = c.upload(fb)
    out = torch.empty_like(c.dev["q"])
    need = fb.fluxbin_paged_attention_workspace_size(b)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    q, scale, ld = c.dev["q"], 0.1, c.heads * c.dim

    def call():
        fb.fluxbin_paged_attention(b, q, ld, scale, 0, out, ld, None, ws, need)

    call()
    torch.cuda.synchronize()
    want = out.clone()
    side = torch.cuda.Stream()
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        out.fill_(i)
        ws.fill_(255)
        q2 = q.clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        assert torch.equal(q, q2)
    # the same graph serves the next step: the lengths are read when it runs
    c.lens_host = [n - 7 for n in c.lens_host]
    c.lengths = [(n, p - 7) for n, p in c.lengths]
    c.dev["lens"].sub_(7)
    graph.replay()
    torch.cuda.synchronize()
    o, _, mag, work, seen = attention_oracle(c, scale)
    tol, _ = attention_bounds(c, o, mag, work, seen)
    assert (np.abs(f64(out).reshape(o.shape) - o) <= tol).all()


def test_offsets_beyond_32_bits(fb):
    """Pages whose first element lies beyond 2^32 bytes and 2^31 elements."""
    note("a cache beyond 2^31 elements")
    c = Paged("f16", 2, 1, 64, 16, [(1, 40), (1, 3)], seed=2)
    b = c.upload(fb)
    want, _ = attend(fb, c, 0.125)
    far = (1 << 31) // c.pages // 8 * 8 + 4096
    big = torch.zeros(far * (c.pages - 1) + 16 * 64, dtype=torch.float16, device="cuda")
    big_v = torch.zeros_like(big)
    for p in range(c.pages):
        big[far * p:far * p + 1024] = c.dev["k"][p].reshape(-1)
        big_v[far * p:far * p + 1024] = c.dev["v"][p].reshape(-1)
    b = c.upload(fb)
    b.k_cache, b.v_cache, b.page_stride = big.data_ptr(), big_v.data_ptr(), far
    out = torch.empty_like(c.dev["q"])
    need = fb.fluxbin_paged_attention_workspace_size(b)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    fb.fluxbin_paged_attention(b, c.dev["q"], 128, 0.125, 0, out, 128, None, ws, need)
    torch.cuda.synchronize()
    assert np.array_equal(f64(out).reshape(want.shape), want)


# ------------------------------------------------------------------ rope_append

def rope_oracle(x, w, pos, freq, rot, pairs, eps, scale):
    """x [tokens][heads][dim] in 64 bits -> the definition, and the magnitude that its roundings go by."""
    u = x if w is None else x * w / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    y, mag = u.copy(), np.abs(u)
    a = pos.astype(np.float64)[:, None, None] * freq
    c, s = np.cos(a) * scale, np.sin(a) * scale
    first, second = (np.s_[..., :rot // 2], np.s_[..., rot // 2:rot]) if pairs == "half" else (np.s_[..., 0:rot:2], np.s_[..., 1:rot:2])
    p, q = u[first], u[second]
    y[first], y[second] = p * c - q * s, q * c + p * s
    mag[first] = mag[second] = (np.abs(p) + np.abs(q)) * max(1.0, abs(scale))
    return y, mag


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("dim,rot,heads,kv", [(128, 128, 4, 2), (64, 32, 3, 1), (8, 8, 2, 2), (40, 24, 5, 1), (72, 72, 2, 1),
                                              (256, 64, 4, 2), (136, 136, 1, 1), (80, 0, 2, 2)])
@pytest.mark.parametrize("pairs", ["half", "near"])
@pytest.mark.parametrize("norm", [False, True])
def test_rope_append(fb, dt, dim, rot, heads, kv, pairs, norm):
    for i, lengths in enumerate(([(1, 0)], [(1, 33), (1, 500), (1, 15)], [(5, 11), (0, 9), (130, 40), (1, 0)], [(700, 3)])):
        note(f"rope_append {dt} dim {dim} rot {rot} heads {heads}/{kv} {pairs} norm {norm} {lengths}")
        c = Paged(dt, heads, kv, dim, (16, 32, 64, 128)[i], lengths, seed=i + dim, order=("heads", "tokens")[i % 2], behind=2 * (i // 2))
        b = c.upload(fb)
        width = (heads + 2 * kv) * dim
        ld = width + (0, 1, 3, 8)[i]
        x = c.randn(c.tokens, ld, scale=2.0)
        w = [(1 + 0.2 * c.randn(dim).float()).to(DT[dt]) for _ in range(2)] if norm else [None, None]
        far = i >= 2
        pos = torch.randint(0, 1 << 20, (c.tokens,), generator=c.g).to(torch.int32) if far else None
        freq = 10000.0 ** (-np.arange(0, max(rot, 2), 2) / max(rot, 2))
        scale = 1.0 if i % 2 else 0.75
        xd, wd = x.cuda(), [None if t is None else t.cuda() for t in w]
        pd, fd = None if pos is None else pos.cuda(), torch.from_numpy(freq).cuda()
        q_out = torch.full((c.tokens, heads * dim + i), 7.0, dtype=DT[dt], device="cuda")
        fb.fluxbin_rope_append(b, xd, ld, xd[:, heads * dim:], ld, xd[:, (heads + kv) * dim:], ld, wd[0], wd[1], 1e-5, fd, rot,
                               {"half": fb.ROPE_HALF, "near": fb.ROPE_NEAR}[pairs], scale, pd, q_out, heads * dim + i)
        torch.cuda.synchronize()
        x64 = f64(x)[:c.rows, :width].reshape(c.rows, heads + 2 * kv, dim)
        at = np.concatenate([np.arange(p, p + n) for n, p in lengths])
        where = at if pos is None else pos.numpy()[:c.rows]
        # the norm: half the relative error of a sum of dim squares and of its quotient, the root, two products; the
        # rotation: sincospi (4 units), its argument (pi / 2 units), the scale, two products and a sum
        units = (dim / 2 + 6 if norm else 0) + 12
        wq, mq = rope_oracle(x64[:, :heads], None if w[0] is None else f64(w[0]), where, freq, rot, pairs, 1e-5, scale)
        wk, mk = rope_oracle(x64[:, heads:heads + kv], None if w[1] is None else f64(w[1]), where, freq, rot, pairs, 1e-5, scale)
        got = f64(q_out)
        assert (got[:, heads * dim:] == 7).all() and (got[c.rows:] == 7).all()
        got = got[:c.rows, :heads * dim].reshape(c.rows, heads, dim)
        assert (np.abs(got - wq) <= UNIT[dt] * np.abs(wq) + units * U * mq * (1 + UNIT[dt]) + TINY[dt]).all()
        kd, vd = c.dev["k"].cpu(), c.dev["v"].cpu()
        want_k, want_v = c.k.clone(), c.v.clone()  # what no token came to is as it was
        seq = np.concatenate([np.full(n, s) for s, (n, _) in enumerate(lengths)]).astype(int)
        for row in range(c.rows):
            p, o = c.table_host[seq[row], at[row] // c.page], at[row] % c.page
            gk = kd[p, :, o] if c.order == "heads" else kd[p, o]
            assert (np.abs(f64(gk) - wk[row]) <= UNIT[dt] * np.abs(wk[row]) + units * U * mk[row] * (1 + UNIT[dt]) + TINY[dt]).all()
            (want_k[p, :, o] if c.order == "heads" else want_k[p, o]).copy_(gk)
            (want_v[p, :, o] if c.order == "heads" else want_v[p, o]).copy_(x[row, (heads + kv) * dim:width].view(kv, dim))
        assert torch.equal(kd, want_k) and torch.equal(vd, want_v)


def test_rope_append_where_pages_are_not_there(fb):
    note("rope_append, missing pages")
    c = Paged("f16", 2, 1, 64, 16, [(40, 0), (1, 90)], seed=1, decode=False)
    c.table_host[0, 1], c.table_host[1, 5] = c.pages, -1
    b = c.upload(fb)
    x = c.randn(c.tokens, 256).cuda()
    q_out = torch.zeros(c.tokens, 128, dtype=torch.float16, device="cuda")
    fb.fluxbin_rope_append(b, x, 256, x[:, 128:], 256, x[:, 192:], 256, None, None, 0.0, None, 0, 0, 1.0, None, q_out, 128)
    torch.cuda.synchronize()
    assert torch.equal(q_out, x[:, :128])  # the queries are written all the same
    k = c.k.clone()
    xk = x[:, 128:192].cpu()
    k[c.table_host[0, 0], 0, :], k[c.table_host[0, 2], 0, :8] = xk[:16], xk[32:40]
    assert torch.equal(c.dev["k"].cpu(), k)
    # lengths shorter than the new tokens, and beyond the table: nothing is stored
    for lens in ([0, 0], [1 << 30, 1 << 30]):
        c.dev["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        before = c.dev["k"].clone()
        fb.fluxbin_rope_append(b, x, 256, x[:, 128:], 256, x[:, 192:], 256, None, None, 0.0, None, 0, 0, 1.0, None, q_out, 128)
        torch.cuda.synchronize()
        assert torch.equal(c.dev["k"], before)


def test_rope_append_in_place_without_queries_and_special_rows(fb):
    note("rope_append in place, without queries, rows of infinities and zeros")
    c = Paged("bf16", 4, 2, 128, 32, [(3, 5), (6, 0)], seed=2)
    b = c.upload(fb)
    x = c.randn(c.tokens, 1024)
    x[0, :128], x[1, :128], x[2, 512:640] = 0, 1e30, math.inf
    x[3, 5] = math.nan
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    freq = torch.full((64,), 0.1, dtype=torch.float64, device="cuda")
    out = []
    for way in range(3):
        xd = x.cuda()
        c.dev["k"].zero_()
        c.dev["v"].zero_()
        q = xd if way != 2 else None
        dst = torch.zeros_like(xd) if way == 0 else q
        fb.fluxbin_rope_append(b, q, 1024, xd[:, 512:], 1024, xd[:, 768:], 1024, w, w, 0.0, freq, 128, fb.ROPE_HALF, 1.0, None, dst,
                               1024)
        torch.cuda.synchronize()
        out.append((None if way == 2 else dst[:, :512].clone(), c.dev["k"].clone(), c.dev["v"].clone()))
    same = lambda s, t: torch.equal(s.view(torch.int16), t.view(torch.int16))  # noqa: E731
    assert same(out[0][0], out[1][0]) and all(same(out[0][1], o[1]) and same(out[0][2], o[2]) for o in out[1:])
    q = out[0][0].float()
    assert torch.isnan(q[0, :128]).all()  # eps 0 and a row of zeros: 0 times infinity
    assert torch.isnan(q[1, :128]).all() and torch.isnan(q[3, :128]).all() and torch.isfinite(q[3, 128:]).all()


def test_rope_append_replays(fb):
    note("rope_append in a graph")
    c = Paged("f16", 8, 2, 128, 16, [(1, 20), (1, 47)], seed=3)
    b = c.upload(fb)
    x = c.randn(2, 12 * 128).cuda()
    freq = torch.full((64,), 0.3, dtype=torch.float64, device="cuda")
    q = torch.empty(2, 1024, dtype=torch.float16, device="cuda")

    def call():
        fb.fluxbin_rope_append(b, x, 1536, x[:, 1024:], 1536, x[:, 1280:], 1536, None, None, 0.0, freq, 128, 0, 1.0, None, q, 1024)

    graph = torch.cuda.CUDAGraph()
    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for step in range(3):
        c.dev["lens"].sub_(1)
        got = []
        for run in (call, graph.replay):
            q.fill_(step)
            c.dev["k"].copy_(c.k)
            c.dev["v"].copy_(c.v)
            run()
            torch.cuda.synchronize()
            got.append([t.clone() for t in (q, c.dev["k"], c.dev["v"])])
        assert all(torch.equal(e, r) for e, r in zip(*got)), step
        assert not torch.equal(got[0][1].cpu(), c.k)
