"""Host-side checks of the attention operators: refusals, plans, grids, the classes' checks (no GPU needed)."""
import ctypes
import math

import pytest

from tests import attention_launches as L
from tests import launches as L8

A = 1 << 20


@pytest.fixture(scope="module")
def fb():
    from binary_basis_lut_amd import build as B
    if B.is_stale():
        B.build()
    from binary_basis_lut_amd import fluxbin
    return fluxbin


def refused(fb, name, args, status):
    st = fb.raw_status(name, *args)
    assert st == status, (st, fb.fluxbin_last_error())
    assert fb.fluxbin_last_error()


BATCHES = [
    (dict(abi_version=7), 1), (dict(dtype=4), 2), (dict(dtype=0), 2), (dict(heads=7), 1), (dict(heads=0), 1), (dict(kv_heads=0), 1),
    (dict(heads=1026, kv_heads=2), 2), (dict(dim=0), 2), (dict(dim=4), 2), (dict(dim=100), 2), (dict(dim=264, token_stride=264), 2),
    (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=131072), 2), (dict(page_size=0), 2), (dict(page_size=-16), 2),
    (dict(tokens=-1), 1), (dict(seqs=-1), 1), (dict(tokens=5), 1), (dict(tokens=(1 << 24) + 1, seqs=(1 << 24) + 1), 2),
    (dict(tokens=1 << 24, seqs=1 << 24, heads=128), 2), (dict(max_kv_len=-1), 1), (dict(table_pages=-1), 1), (dict(table_ld=63), 1),
    (dict(table_pages=1 << 27, table_ld=1 << 27), 2), (dict(cache_pages=-1), 1), (dict(cache_pages=1 << 31), 2),
    (dict(page_stride=4100), 1), (dict(head_stride=-8), 1), (dict(token_stride=120), 1), (dict(token_stride=132), 1),
    (dict(token_stride=(1 << 24) + 8), 2), (dict(kv_lens=None), 1), (dict(page_table=None), 1), (dict(k_cache=None), 1),
    (dict(v_cache=None), 1), (dict(k_cache=A + 8), 1), (dict(v_cache=A + 2), 1), (dict(kv_lens=A + 2), 1), (dict(page_table=A + 1), 1),
    (dict(seq_starts=A + 2), 1),
]


@pytest.mark.parametrize("kw,status", BATCHES)
def test_batches_that_are_refused(fb, kw, status):
    b = fb.PagedBatch(**L.batch(**kw))
    refused(fb, "fluxbin_paged_attention", [ctypes.byref(b), A, 1 << 20, 0.1, 0, A, 1 << 20, None, A, 72 << 20, None], status)
    refused(fb, "fluxbin_rope_append", [ctypes.byref(b), A, 1 << 20, A, 1 << 20, A, 1 << 20, None, None, 0.0, A, 0, 0, 1.0, None, A, 1 << 20,
                                        None], status)
    refused(fb, "fluxbin_paged_attention_workspace_size", [ctypes.byref(b), ctypes.byref(ctypes.c_size_t())], status)


def attention_args(fb, **kw):
    d = dict(batch=fb.PagedBatch(**L.batch()), q=A, ldq=1024, scale=0.1, window=0, out=A, ldo=1024, lse=A, workspace=A, workspace_bytes=72 << 20,
             stream=None)
    assert set(kw) <= set(d)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(batch=None), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(ldq=1023), 1), (dict(ldo=1023), 1), (dict(q=A + 1), 1),
    (dict(out=A + 1), 1), (dict(lse=A + 2), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=math.nan), 1),
    (dict(scale=math.inf), 1), (dict(window=-1), 1),
])
def test_paged_attention_refuses(fb, kw, status):
    refused(fb, "fluxbin_paged_attention", attention_args(fb, **kw), status)


def test_paged_attention_refuses_a_workspace_that_does_not_do(fb):
    b = fb.PagedBatch(**L.batch(table_pages=4096, table_ld=4096))
    need = fb.fluxbin_paged_attention_workspace_size(b)
    assert need > 0
    for kw, status in ((dict(workspace=None), 3), (dict(workspace_bytes=need - 1), 3), (dict(workspace=A + 4), 1)):
        refused(fb, "fluxbin_paged_attention", attention_args(fb, batch=b, **kw), status)
    with pytest.raises(fb.FluxbinError):
        fb.fluxbin_paged_attention_workspace_size(None)
    assert fb.raw_status("fluxbin_paged_attention_workspace_size", ctypes.byref(b), None) == 1


def append_args(fb, **kw):
    d = dict(batch=fb.PagedBatch(**L.batch()), q=A, ldq=1024, k=A, ldk=256, v=A, ldv=256, q_norm=A, k_norm=A, eps=1e-5, freq=A,
             rotary_dim=128, pairs=0, rope_scale=1.0, positions=A, q_out=A, ldqo=1024, stream=None)
    assert set(kw) <= set(d)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(batch=None), 1), (dict(q=None), 1), (dict(q_out=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(freq=None), 1),
    (dict(ldq=1023), 1), (dict(ldk=255), 1), (dict(ldv=255), 1), (dict(ldqo=1000), 1), (dict(rotary_dim=-8), 1), (dict(rotary_dim=12), 1),
    (dict(rotary_dim=136), 1), (dict(pairs=2), 1), (dict(pairs=-1), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1),
    (dict(rope_scale=math.inf), 1), (dict(rope_scale=math.nan), 1), (dict(q=A + 1), 1), (dict(k=A + 1), 1), (dict(v=A + 1), 1),
    (dict(q_out=A + 1), 1), (dict(q_norm=A + 1), 1), (dict(k_norm=A + 1), 1), (dict(positions=A + 2), 1), (dict(freq=A + 4), 1),
])
def test_rope_append_refuses(fb, kw, status):
    refused(fb, "fluxbin_rope_append", append_args(fb, **kw), status)


def test_appending_in_place_with_another_stride_is_refused(fb):
    for q, ldq, ldqo in ((A, 1024, 1032), (A, 2048, 1024)):
        refused(fb, "fluxbin_rope_append", append_args(fb, q=q, ldq=ldq, q_out=q, ldqo=ldqo), 1)


def adjust_args(**kw):
    d = dict(logits=A, ld=1000, dtype=1, rows=4, vocab=1000, history=A, ldh=50, history_cols=50, prompt_len=A, total_len=A, repetition=A,
             frequency=A, presence=A, bias_index=A, bias_value=A, ldb=8, biases=8, mask=A, ldm=32, out=2 * A, ldo=1000, stream=None)
    assert set(kw) <= set(d)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), 2), (dict(dtype=2), 2), (dict(rows=-1), 1), (dict(vocab=0), 1), (dict(rows=(1 << 22) + 1), 2),
    (dict(vocab=(1 << 28) + 1, ld=1 << 30, ldo=1 << 30), 2), (dict(rows=1 << 22, vocab=10000, ld=10000, ldo=10000, ldm=400), 2),
    (dict(history_cols=-1), 1), (dict(history_cols=1 << 30, ldh=1 << 30), 2), (dict(biases=-1), 1), (dict(biases=4097, ldb=5000), 2),
    (dict(logits=None), 1), (dict(out=None), 1), (dict(ld=999), 1), (dict(ldo=999), 1), (dict(out=A, ldo=1001), 1), (dict(history=None), 1),
    (dict(ldh=49), 1), (dict(bias_index=None), 1), (dict(bias_value=None), 1), (dict(ldb=7), 1), (dict(ldm=31), 1), (dict(logits=A + 1), 1),
    (dict(out=A + 1), 1), (dict(dtype=4, logits=A + 2), 1), (dict(history=A + 2), 1), (dict(prompt_len=A + 1), 1), (dict(total_len=A + 2), 1),
    (dict(repetition=A + 2), 1), (dict(frequency=A + 1), 1), (dict(presence=A + 3), 1), (dict(bias_index=A + 2), 1),
    (dict(bias_value=A + 2), 1), (dict(mask=A + 2), 1),
])
def test_adjust_logits_refuses(fb, kw, status):
    refused(fb, "fluxbin_adjust_logits", adjust_args(**kw), status)


def test_nothing_to_do_is_no_error(fb):
    for kw in (dict(tokens=0, seqs=0), dict(tokens=0, seqs=0, seq_starts=A), dict(tokens=0, seq_starts=A), dict(seqs=0, seq_starts=A)):
        b = fb.PagedBatch(**L.batch(kv_lens=None, **kw))
        assert fb.raw_status("fluxbin_paged_attention", *attention_args(fb, batch=b, q=None, out=None, workspace=None)) == fb.OK
        assert fb.raw_status("fluxbin_rope_append", *append_args(fb, batch=b, k=None, v=None)) == fb.OK
        assert fb.fluxbin_paged_attention_workspace_size(b) == 0
    assert fb.raw_status("fluxbin_adjust_logits", *adjust_args(rows=0, logits=None)) == fb.OK


def shapes():
    for tokens, seqs in ((1, 1), (2, 1), (7, 7), (64, 64), (300, 300), (4096, 4096), (40, 5), (517, 1), (4096, 1), (9000, 12), (70000, 400),
                         (3, 900), (1 << 20, 3), (5000000, 5000000), (8200000, 8200000), (9000000, 9000000), (1 << 24, 1 << 24)):
        for heads, kv in ((1, 1), (8, 1), (64, 8), (32, 32), (48, 48), (512, 4)):
            if tokens * heads <= 1 << 30:
                for dim in (8, 64, 128, 136, 256):
                    for pages in (0, 1, 8, 300, 8192, 60000):
                        yield dict(tokens=tokens, seqs=seqs, seq_starts=None if tokens == seqs else L.A, heads=heads, kv_heads=kv, dim=dim,
                                   table_pages=pages, table_ld=pages, page_stride=kv * 16 * dim, head_stride=16 * dim, token_stride=dim)


def test_workspaces_stay_below_what_the_header_says(fb):
    for kw in shapes():
        assert fb.fluxbin_paged_attention_workspace_size(fb.PagedBatch(**L.batch(**kw))) <= 72 << 20, kw


recorded = pytest.mark.skipif(not L8.available(), reason="gcc and c++filt not available")


def fits(launch):
    (x, y, z), (bx, by, bz) = launch["grid"], launch["block"]
    return 0 < x and x * bx < 1 << 32 and y == z == by == bz == 1 and bx <= 1024


@recorded
def test_grids_fit_or_are_refused(fb):
    calls = [f(L.batch(dtype=3, **kw)) for kw in shapes() if kw["table_pages"] in (1, 8192) for f in (L.attend, L.append)]
    calls += [L.adjust(r, v, biases=n) for r, v in ((1, 1), (1, 1 << 28), (1 << 22, 100), (70000, 262144), (1 << 17, 131072)) for n in (0, 5)]
    refusals = 0
    for call, r in zip(calls, L.record(calls)[1]):
        assert r["status"] in (0, 2), (call, r)
        refusals += r["status"] == 2
        assert bool(r["launches"]) == (r["status"] == 0) and all(fits(x) for x in r["launches"]), (call, r)
    assert 0 < refusals < len(calls) // 2


# every kernel of the operators and a call that takes it
def one_of_each():
    for dt in ("f16", "bf16"):
        t = dt.upper()
        for dim, d in ((8, 64), (64, 64), (72, 128), (128, 128), (136, 256), (256, 256)):
            b = lambda **kw: L.batch(**{**dict(dtype=L.TYPES[dt], dim=dim, token_stride=dim, head_stride=16 * dim, page_stride=32 * dim), **kw})  # noqa: E731
            few, chunk = f"attention_few_kernel<{t}, {d}>", f"attention_chunk_kernel<{t}, {d}, 1>"
            yield L.attend(b(table_pages=16)), [few]
            yield L.attend(b(tokens=1, seqs=1, table_pages=512, table_ld=512)), [few, f"attention_join_kernel<{t}>"]
            yield L.attend(b(tokens=100, seqs=2, seq_starts=L.A, table_pages=16)), [chunk]
            yield L.attend(b(tokens=100, seqs=2, seq_starts=L.A, table_pages=8192, table_ld=8192)), \
                ["attention_count_kernel<128>", f"attention_balanced_kernel<{t}, {d}, 1>", f"attention_gather_kernel<{t}, 128>"]
        for dim, rot, params in ((64, 64, "8, 4"), (128, 64, "8, 8"), (256, 256, "8, 16"), (24, 24, "4, 4"), (64, 24, "4, 8"), (104, 104, "4, 16"),
                                 (256, 40, "4, 32")):
            b = L.batch(dtype=L.TYPES[dt], dim=dim, token_stride=dim)
            for norm in (False, True):
                yield L.append(b, norm=norm, rot=rot), [f"rope_append_kernel<{t}, {params}, {'true' if norm else 'false'}>"]
    for dt in ("f16", "bf16", "f32"):
        for biases in (0, 3):
            s = "true" if biases else "false"
            for vocab, params in ((5, "true, 256, 4096"), (8, "false, 256, 4096"), (4096, "false, 256, 4096"),
                                  (4097, "false, 1024, 8192" if biases else "false, 1024, 16384")):
                yield L.adjust(3, vocab, dt, biases), [f"adjust_logits_kernel<{dt.upper()}, {s}, {params}>"]


@recorded
def test_every_kernel_is_reached_by_a_rule(fb):
    calls, want = zip(*one_of_each())
    kernels, results = L.record(list(calls))
    for call, names, r in zip(calls, want, results):
        assert r["status"] == 0 and [x["kernel"] for x in r["launches"]] == names, (call, r)
    mine = {k for k in kernels if k.startswith(("attention_", "rope_append_", "adjust_logits_"))}
    assert mine == {n for names in want for n in names}


@recorded
def test_a_window_never_takes_more_workspace_than_none(fb):
    """The size is asked for without the window: whatever a window makes of the plan has to fit it."""
    base = [dict(tokens=t, seqs=s, seq_starts=L.A, heads=h, kv_heads=k, table_pages=p, table_ld=p)
            for t, s in ((1, 1), (5, 1), (517, 1), (64, 64), (300, 3), (3000, 12)) for h, k in ((8, 8), (64, 8), (8, 1)) for p in (8, 500, 8192)]
    calls = []
    for kw in base:
        for window in (0, 1, 100, 5000, 100000, 2 ** 31 - 1):
            calls.append(L.attend(L.batch(**kw), window=window))
    sizes = {}
    for call, r in zip(calls, L.record(calls)[1]):
        call["args"][8] = sizes.setdefault(str(call["batch"]), r["workspace"])
    for call, r in zip(calls, L.record(calls)[1]):
        assert r["status"] == 0, (call, r)


# ------------------------------------------------------------------ the classes, on fake tensors

torch = pytest.importorskip("torch")


@pytest.fixture
def calls(monkeypatch, fb):
    from torch._subclasses.fake_tensor import FakeTensorMode

    class Stream:
        cuda_stream = 0

        def synchronize(self):
            pass

    seen = []
    for name in ("fluxbin_quantize_rows", "fluxbin_add_rmsnorm", "fluxbin_gemm_w8a8", "fluxbin_token_logprobs", "fluxbin_rope_append",
                 "fluxbin_paged_attention", "fluxbin_adjust_logits"):
        monkeypatch.setattr(fb, name, lambda *a, _n=name: seen.append((_n, *a)))
    monkeypatch.setattr(fb, "fluxbin_paged_attention_workspace_size", lambda b: 0)
    monkeypatch.setattr(fb, "PagedBatch", lambda: type("Batch", (), {})())
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda t: 0, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    with FakeTensorMode():
        yield seen


def cuda(*shape, dtype=torch.float16, device="cuda"):
    return torch.empty(shape, dtype=dtype, device=device)


def layer(**kw):
    from binary_basis_lut_amd.paged import PagedAttention
    return PagedAttention(**{**dict(heads=8, kv_heads=2, dim=64, pages=10, page_size=16, max_seqs=4, max_pages=5, max_tokens=20), **kw})


WIDTH = 12 * 64


@pytest.mark.parametrize("kw", [dict(dtype=torch.float32), dict(freq=31), dict(q_norm=(64, torch.float32)),
                                dict(k_norm=(32, torch.float16))], ids=str)
def test_layers_that_are_refused(calls, kw):
    if "freq" in kw:
        kw = dict(freq=cuda(31, dtype=torch.float64, device="cpu"))
    elif "dtype" not in kw:
        kw = {n: cuda(v[0], dtype=v[1]) for n, v in kw.items()}
    with pytest.raises(ValueError):
        layer(**kw)
    assert not calls


@pytest.mark.parametrize("make", [
    lambda: dict(qkv=cuda(21, WIDTH)), lambda: dict(qkv=cuda(3, WIDTH - 1)), lambda: dict(qkv=cuda(3, WIDTH, dtype=torch.bfloat16)),
    lambda: dict(qkv=cuda(3, WIDTH, device="cpu")), lambda: dict(qkv=cuda(3, 2 * WIDTH)[:, ::2]), lambda: dict(qkv=cuda(WIDTH, 3).t()),
    lambda: dict(qkv=cuda(3, WIDTH), seqs=2), lambda: dict(qkv=cuda(5, WIDTH)),
    lambda: dict(qkv=cuda(3, WIDTH), seq_starts=cuda(3, dtype=torch.int64)), lambda: dict(qkv=cuda(3, WIDTH), seq_starts=cuda(7, dtype=torch.int32)),
    lambda: dict(qkv=cuda(3, WIDTH), seq_starts=cuda(6, dtype=torch.int32)[::2]),
    lambda: dict(qkv=cuda(3, WIDTH), seq_starts=cuda(3, dtype=torch.int32), seqs=3),
    lambda: dict(qkv=cuda(3, WIDTH), positions=cuda(3, dtype=torch.int64)), lambda: dict(qkv=cuda(3, WIDTH), positions=cuda(2, dtype=torch.int32)),
    lambda: dict(qkv=cuda(3, WIDTH), positions=cuda(6, dtype=torch.int32)[::2]),
], ids=range(15))
def test_calls_that_would_be_misread_are_refused(calls, make):
    l = layer()
    with pytest.raises(ValueError):
        l.attend(**make())
    assert not calls


def test_what_attend_hands_on(calls):
    l = layer()
    qkv = cuda(3, WIDTH + 5)[:, :WIDTH]
    assert l.attend(qkv).shape == (3, 512)
    append, attention = calls
    assert append[0] == "fluxbin_rope_append" and append[2] is qkv and append[3] == WIDTH + 5
    assert append[4].storage_offset() == 512 and append[6].storage_offset() == 640
    assert attention[0] == "fluxbin_paged_attention" and attention[4] == 1 / 8 and attention[8] is None
    calls.clear()
    l.attend(cuda(1, 9 * WIDTH)[:, :WIDTH].as_strided((1, WIDTH), (1, 1)))  # one row, whatever its stride
    assert calls[0][3] == WIDTH
    calls.clear()
    l.attend(cuda(20, WIDTH), seq_starts=cuda(3, dtype=torch.int32))
    assert calls[0][1].seqs == 2 and calls[0][1].tokens == 20


def test_another_current_device_is_refused(calls, monkeypatch):
    l = layer()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        l.attend(cuda(3, WIDTH))
    assert not calls


def test_frequencies():
    from binary_basis_lut_amd.paged import rope_frequencies
    f = rope_frequencies(64)
    assert f.dtype == torch.float64 and f.shape == (32,) and f[0] == 1 and abs(float(f[16]) - 0.01) < 1e-15
    assert torch.equal(rope_frequencies(64, linear=4.0), f / 4)
    g = rope_frequencies(64, by_parts=(8.0, 1.0, 4.0, 8192))
    turns = 8192 * f / (2 * math.pi)
    assert torch.equal(g[turns >= 4], f[turns >= 4]) and torch.allclose(g[turns <= 1], f[turns <= 1] / 8, rtol=1e-15)
    assert (g <= f).all() and (g >= f / 8).all() and (g[1:] < g[:-1]).all()
    with pytest.raises(ValueError):
        rope_frequencies(64, by_parts=(8.0, 4.0, 4.0, 8192))


def rules(**kw):
    from binary_basis_lut_amd.score_tokens import LogitRules
    return LogitRules(**{**dict(max_rows=4, vocab=1000, max_history=30), **kw})


@pytest.mark.parametrize("make", [
    lambda: dict(repetition=cuda(4)), lambda: dict(frequency=cuda(3, dtype=torch.float32)), lambda: dict(presence=cuda(4, dtype=torch.float64)),
    lambda: dict(prompt_len=cuda(4, dtype=torch.int64)), lambda: dict(bias_index=cuda(4, 3, dtype=torch.int32)),
    lambda: dict(bias_index=cuda(4, 3, dtype=torch.int32), bias_value=cuda(4, 2, dtype=torch.float32)),
    lambda: dict(mask=cuda(4, 31, dtype=torch.int32)), lambda: dict(mask=cuda(4, 32, dtype=torch.bool)),
    lambda: dict(mask=cuda(4, 64, dtype=torch.int32)[:, ::2]), lambda: dict(repetition=cuda(4, dtype=torch.float32, device="cpu")),
], ids=range(10))
def test_rules_that_would_be_misread_are_refused(calls, make):
    with pytest.raises(ValueError):
        rules(**make())


def test_rules_stand_between_the_head_and_the_scores(calls):
    from binary_basis_lut_amd.score_tokens import ScoringHead
    head = ScoringHead(cuda(512), cuda(1000, 512), 8)
    r = rules(bias_index=cuda(4, 3, dtype=torch.int32), bias_value=cuda(4, 3, dtype=torch.float32))
    calls.clear()
    head.score(cuda(3, 512), cuda(3, 512), cuda(3, dtype=torch.int64), rules=r)
    assert [c[0] for c in calls] == ["fluxbin_add_rmsnorm", "fluxbin_gemm_w8a8", "fluxbin_adjust_logits", "fluxbin_token_logprobs"]
    adjust = calls[2]
    assert adjust[1] is head.logits and adjust[-2] is head.logits and adjust[4] == 3 and adjust[16] == adjust[17] == 3
    calls.clear()
    for bad in (rules(vocab=999), rules(max_rows=2)):
        with pytest.raises(ValueError, match="rules"):
            head.score(cuda(3, 512), cuda(3, 512), cuda(3, dtype=torch.int64), rules=bad)
    assert not calls


def test_a_history_that_is_full_keeps_the_latest_token():
    r = rules(max_rows=2, max_history=5, device="cpu:0")
    new = lambda *t: torch.tensor([t, [x + 100 for x in t]])
    r.append(new(1, 2, 3))
    r.append(new(4))
    assert r.history.tolist() == [[1, 2, 3, 4, -1], [101, 102, 103, 104, -1]] and r.total_len.tolist() == [4, 4]
    r.append(new(5, 6, 7))
    assert r.history.tolist() == [[1, 2, 3, 4, 7], [101, 102, 103, 104, 107]] and r.total_len.tolist() == [5, 5]
    r.append(new(8))
    r.append(torch.zeros(2, 0, dtype=torch.int64))
    assert r.history.tolist() == [[1, 2, 3, 4, 8], [101, 102, 103, 104, 108]] and r.total_len.tolist() == [5, 5]
    for bad in (torch.zeros(1, 1, dtype=torch.int64), torch.zeros(2, 1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="tokens"):
            r.append(bad)


def test_no_history_takes_no_tokens():
    r = rules(max_rows=2, max_history=0, device="cpu:0")
    r.append(torch.ones(2, 3, dtype=torch.int64))
    assert r.history.shape == (2, 0) and r.total_len.tolist() == [0, 0]
