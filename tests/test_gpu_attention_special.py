"""fluxbin_paged_attention where scores or values are not numbers, infinite or at the ends of fp32: every division of the keys
gives what the definition gives (tests/attention_cases.py)."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.attention_cases import U, Paged, attention_bounds, attention_oracle, f64  # noqa: E402
from tests.test_gpu_attention_ops import attend, balanced, fb, note  # noqa: E402,F401

# how the keys are divided: rows of single tokens in one workgroup or over several, rows of a chunk in one or in shares
FORMS = ["whole", "splits", "chunk", "shares"]


def make(form, dt, dim=128, heads=4, seed=0, past=None):
    if form in ("whole", "splits"):
        return Paged(dt, heads, 1, dim, 16, [(1, past or 5000), (3, past or 2000)], seed=seed, decode=False,
                     max_kv_len={"whole": 1, "splits": 8192}[form])
    lengths = [(130, past or 1500)]
    return Paged(dt, heads, 1, dim, 16, lengths, seed=seed, decode=False, max_kv_len=1) if form == "chunk" else \
        balanced(dt, dim, heads, 1, lengths, seed)


def workspace_of(fb, c):
    return fb.fluxbin_paged_attention_workspace_size(c.upload(fb))


def keys(c, s, js):
    """Key and value rows [dim] of the places js of sequence s, as (page, place in it)."""
    return [(c.table_host[s, j // c.page], j % c.page) for j in js]


def same_as(got, ls, out, lse, tol, tol_lse):
    """Equal infinities, NaN for NaN, and finite numbers within the tolerance."""
    for g, w, t in ((got, out, tol), (ls, lse, tol_lse + 4 * U * np.abs(lse))):
        fine = np.isfinite(w)
        assert np.array_equal(np.isnan(g), np.isnan(w)), np.argwhere(np.isnan(g) != np.isnan(w))[:5]
        assert np.array_equal(g[np.isinf(w)], w[np.isinf(w)])
        assert (np.abs(g[fine] - w[fine]) <= t[fine]).all()


@pytest.mark.parametrize("what", ["query", "all of a split", "one key", "one key of small scores", "infinity", "minus infinity"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("form", FORMS)
def test_scores_that_are_not_numbers(fb, form, dt, what):
    note(f"{what}, {form} {dt}")
    c = make(form, dt)
    assert (workspace_of(fb, c) > 0) == (form in ("splits", "shares"))
    scale = 0.05
    seqs = range(len(c.lengths))
    if what in ("infinity", "minus infinity", "one key of small scores"):
        c.q.abs_()
    if what == "one key of small scores":  # 1/2 or less each times -64: far below the others, and a weight of 0 beside theirs
        scale = 1.0
        c.k.mul_(0.01)
        c.q.clamp_(min=0.25, max=0.5)
        for s in seqs:
            for p, i in keys(c, s, range(512, 1024)):
                c.k[p, :, i] = -16
    _, _, mag, work, seen = attention_oracle(c, scale)
    if what == "query":
        c.q[0, c.dim + 5] = math.nan
    elif what == "all of a split":
        for p, i in keys(c, 0, range(512, 1024)):
            c.k[p, :, i] = math.nan
    else:
        p, i = keys(c, 0, [700])[0]
        c.k[p, 0, i, 9] = {"i": math.inf, "m": -math.inf}.get(what[0], math.nan)
    out, lse, *_ = attention_oracle(c, scale)
    assert np.isnan(out).any() == (what != "minus infinity")
    tol, tol_lse = attention_bounds(c, np.nan_to_num(out), mag, work, seen)
    got, ls = attend(fb, c, scale)
    # without the key of weight p the others weigh 1 / (1 - p) times as much, p being less than 1/2
    same_as(got, ls, out, lse, 2 * tol, 2 * tol_lse)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("form", FORMS)
def test_scores_at_the_ends_of_fp32(fb, form, dt, sign):
    """z = scale q . k of 2.7e38, z log2(e) beyond fp32: the keys of the largest one share the weight."""
    note(f"scores of {sign} 2.7e38, {form} {dt}")
    c = make(form, dt, past=1100)
    workspace_of(fb, c)
    c.q.zero_()
    c.q[:, ::c.dim] = 16384
    for s in range(len(c.lengths)):
        for j, (p, i) in enumerate(keys(c, s, range(c.lens_host[s]))):
            c.k[p, 0, i, 0] = sign * (16384, 16512)[(j % 3 == 0) == (sign > 0)]
    out, lse, mag, work, seen = attention_oracle(c, float(np.float32(1e30)))
    assert (np.abs(lse) > 2.6e38).all() and (np.abs(lse) < 3e38).all()
    # the weights are 1 or 0: a product's rounding moves no score past another, so only sums and roundings count in out
    tol, _ = attention_bounds(c, out, mag, 0 * work, seen)
    _, tol_lse = attention_bounds(c, out, mag, work, seen)
    same_as(*attend(fb, c, 1e30), out, lse, tol, tol_lse)


@pytest.mark.parametrize("dim", [64, 72, 128, 256])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("form", FORMS)
def test_infinite_values_under_vanishing_weights(fb, form, dt, dim):
    """A weight is positive however small: an infinity shows, whether it comes before the maximum or after it."""
    note(f"infinities under weights of e^-300, {form} {dt} dim {dim}")
    c = make(form, dt, dim)
    workspace_of(fb, c)
    c.q.fill_(1)
    c.k.mul_(0.01)
    n = c.lens_host[0] - c.lengths[0][0]
    for p, i in keys(c, 0, list(range(64)) + list(range(n - 20, n - 8))):
        c.k[p, :, i] = -300 / dim
    _, _, mag, work, seen = attention_oracle(c, 1.0)
    for j, d, v in ((5, 3, math.inf), (n - 10, 4, -math.inf), (7, 5, math.inf), (n - 12, 5, -math.inf), (9, 6, math.nan), (n - 13, 7, math.nan)):
        p, i = keys(c, 0, [j])[0]
        c.v[p, 0, i, d] = v
    out, lse, *_ = attention_oracle(c, 1.0)
    row = out[:c.lengths[0][0]]
    assert (row[..., 3] == math.inf).all() and (row[..., 4] == -math.inf).all() and np.isnan(row[..., 5:8]).all()
    tol, tol_lse = attention_bounds(c, np.nan_to_num(out, posinf=0, neginf=0), mag, work, seen)
    same_as(*attend(fb, c, 1.0), out, lse, tol, tol_lse)


@pytest.mark.parametrize("form", FORMS)
def test_rows_before_the_first_sequence(fb, form):
    """They are left as they were, as those behind the last one are."""
    note(f"rows before the first sequence, {form}")
    few = form in ("whole", "splits")
    before, lengths = (9, [(1, 5000), (6, 2000)]) if few else (140, [(130, 1500)])
    c = Paged("f16", 4, 1, 128, 16, lengths, seed=1, decode=False, max_kv_len={"whole": 1, "splits": 8192, "chunk": 1, "shares": 0}[form],
              behind=before, table_extra=1 << 16 if form == "shares" else 0)
    b = c.upload(fb)
    c.dev["starts"].add_(before)
    q = torch.zeros_like(c.dev["q"])
    q[before:] = c.dev["q"][:c.rows]
    out, ls = torch.full_like(q, 7.0), torch.full((c.tokens, 4), 7.0, device="cuda")
    need = fb.fluxbin_paged_attention_workspace_size(b)
    assert (need > 0) == (form in ("splits", "shares"))
    ws = torch.full((max(need, 16) // 4 + 4,), math.nan, dtype=torch.float32, device="cuda")
    fb.fluxbin_paged_attention(b, q, 512, 0.1, 0, out, 512, ls, ws, need)
    torch.cuda.synchronize()
    assert (out[:before] == 7).all() and (ls[:before] == 7).all()
    want, lse, mag, work, seen = attention_oracle(c, 0.1)
    tol, tol_lse = attention_bounds(c, want, mag, work, seen)
    same_as(f64(out[before:]).reshape(want.shape), f64(ls[before:]), want, lse, tol, tol_lse)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("form", FORMS)
def test_outputs_over_the_queries(fb, form, dt):
    """The same bits as apart, also where rows are computed key by key and read their query again."""
    note(f"out is q, {form} {dt}")
    for bad in (False, True):
        c = make(form, dt, seed=2)
        if bad:
            p, i = keys(c, 0, [100])[0]
            c.v[p, 0, i, 9] = math.inf
        b = c.upload(fb)
        need = fb.fluxbin_paged_attention_workspace_size(b)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        ld = c.heads * c.dim + 8
        q = torch.full((c.tokens, ld), 7.0, dtype=c.dev["q"].dtype, device="cuda")
        q[:, :-8] = c.dev["q"]
        apart = torch.full_like(q, 7.0)
        for out in (apart, q):
            fb.fluxbin_paged_attention(b, q, ld, 0.1, 0, out, ld, None, ws, need)
        torch.cuda.synchronize()
        assert torch.isinf(apart).any() == bad
        assert torch.equal(q, apart)


@pytest.mark.parametrize("dim", [64, 72, 256])
@pytest.mark.parametrize("form", FORMS)
def test_a_query_that_is_not_a_number(fb, form, dim):
    note(f"NaN query, {form} dim {dim}")
    c = make(form, "bf16", dim, seed=4)
    assert (workspace_of(fb, c) > 0) == (form in ("splits", "shares"))
    _, _, mag, work, seen = attention_oracle(c, 0.05)
    c.q[-1, dim - 1] = math.nan
    out, lse, *_ = attention_oracle(c, 0.05)
    assert np.isnan(lse).sum() == 1 and np.isnan(out[-1, 0]).all()
    tol, tol_lse = attention_bounds(c, np.nan_to_num(out), mag, work, seen)
    same_as(*attend(fb, c, 0.05), out, lse, tol, tol_lse)
