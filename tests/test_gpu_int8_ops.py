"""The 8-bit operators against plain implementations in 64 bits (numpy on the host).

Tolerances are first-order bounds of the stated arithmetic, u = 2^-24 being fp32's rounding unit and
2^-11, 2^-8, 2^-24 the output type's.  Integers and indices are compared for equality.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -126}  # half a subnormal step (fp32: flush)


@pytest.fixture(scope="module")
def fb():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    from binary_basis_lut_amd import fluxbin
    return fluxbin


def code(fb, dt):
    return {"f16": fb.DT_F16, "bf16": fb.DT_BF16, "f32": fb.DT_F32}[dt]


def note(msg):
    print(f"[case] {msg}", flush=True)


def randn(rows, cols, dt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * scale
    x[:, torch.rand(cols, generator=g) < 0.02] *= 20
    return x.to(DT[dt])


def strided(x, ld, offset=0):
    """x on the GPU with row stride ld, its first element `offset` elements into the allocation."""
    rows, cols = x.shape
    buf = torch.zeros(rows * ld + offset + 16, dtype=x.dtype, device="cuda")
    view = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(x)
    return view


def f64(t):
    return t.detach().cpu().double().numpy()


def quant_oracle(t32):
    """q and a of the written rule, from fp32 rows, in numpy's IEEE arithmetic."""
    a = np.maximum(np.abs(t32).max(axis=1), np.float32(2.0 ** -100)).astype(np.float32)
    with np.errstate(all="ignore"):
        q = np.rint(t32 * (np.float32(127.0) / a)[:, None])
    good = np.isfinite(t32).all(axis=1)
    q = np.where(good[:, None], q, 0).astype(np.int64)
    return q, np.where(good, a, np.nan)


# ------------------------------------------------------------------ quantize_rows

COLS = [1, 2, 7, 8, 9, 63, 511, 512, 513, 2047, 2049, 4096, 4099, 8192, 8193, 16385, 32768, 32771]


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("cols", COLS)
def test_quantize_rows(fb, dt, cols):
    rows = 5
    note(f"quantize_rows {dt} {rows} x {cols}")
    x = randn(rows, cols, dt, 11 + cols)
    xd = strided(x, cols + 3, offset=1)  # odd stride and start: element alignment only
    q = torch.full((rows, cols + 5), 77, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, dtype=torch.float32, device="cuda")
    fb.fluxbin_quantize_rows(xd, cols + 3, code(fb, dt), rows, cols, q, cols + 5, s)
    torch.cuda.synchronize()
    want, a = quant_oracle(x.float().numpy())
    got = q.cpu().numpy().astype(np.int64)
    assert np.array_equal(got[:, :cols], want)
    assert (got[:, cols:] == 77).all()  # nothing written past the row
    assert np.array_equal(s.cpu().numpy(), a / np.float32(127.0))
    # and against the definition in 64 bits: half a step and the roundings of 127 / a and of the product
    x64 = f64(x)
    assert (np.abs(got[:, :cols] - 127.0 * x64 / a[:, None].astype(np.float64)) <= 0.5 + 127 * 3 * U).all()


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("cols", [40, 700, 5000, 33000])
def test_quantize_rows_special_rows(fb, dt, cols):
    note(f"quantize_rows special rows {dt} x {cols}")
    x = randn(8, cols, dt, 5)
    x[0] = 0
    x[1, 3] = math.inf
    x[2, cols - 1] = -math.inf
    x[3, cols // 2] = math.nan
    x[4] = 0
    x[4, 1] = torch.finfo(DT[dt]).tiny if dt != "f16" else 2.0 ** -24
    x[5] = torch.finfo(DT[dt]).max
    x[5, 1] = -torch.finfo(DT[dt]).max
    xd = x.cuda()
    q = torch.empty((8, cols), dtype=torch.int8, device="cuda")
    s = torch.empty(8, dtype=torch.float32, device="cuda")
    fb.fluxbin_quantize_rows(xd, cols, code(fb, dt), 8, cols, q, cols, s)
    torch.cuda.synchronize()
    want, a = quant_oracle(x.float().numpy())
    assert np.array_equal(q.cpu().numpy().astype(np.int64), want)
    got = s.cpu().numpy()
    assert np.isnan(got[1:4]).all() and np.isfinite(np.delete(got, [1, 2, 3])).all()
    assert np.array_equal(got, (a / np.float32(127.0)).astype(np.float32), equal_nan=True)


# ------------------------------------------------------------------ add_rmsnorm

def norm_oracle(x, res, w, dt, eps):
    h = x if res is None else (x.float() + res.float()).to(DT[dt])
    h64, w64 = f64(h), f64(w)
    rms = np.sqrt((h64 ** 2).mean(axis=1) + eps)
    q, a = quant_oracle(h.float().numpy() * w.float().numpy())
    return h, h64 * w64 / rms[:, None], q, a.astype(np.float64) / 127 / rms


def ss_roundings(cols):
    """Roundings on the longest path of a sum of squares: a thread's elements, the wave, the workgroup."""
    return max(32, -(-cols // 1024)) + 6 + 16


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("mode", ["all", "q", "y"])
def test_add_rmsnorm(fb, dt, cols, mode):
    rows = 6
    note(f"add_rmsnorm {dt} {rows} x {cols} {mode}")
    x, res = randn(rows, cols, dt, 3 + cols), randn(rows, cols, dt, 4 + cols, 3.0)
    w = (1 + 0.1 * randn(1, cols, "f32", 9)[0]).to(DT[dt])
    if mode == "y":
        res = None  # no residual
    xd, wd = strided(x, cols + 1, 1), strided(w[None], cols, 1)
    rd = None if res is None else strided(res, cols + 2)
    ro = torch.empty((rows, cols + 3), dtype=DT[dt], device="cuda") if mode == "all" else None
    y = torch.empty((rows, cols), dtype=DT[dt], device="cuda") if mode != "q" else None
    q = torch.empty((rows, cols + 7), dtype=torch.int8, device="cuda") if mode != "y" else None
    s = torch.empty(rows, dtype=torch.float32, device="cuda") if mode != "y" else None
    fb.fluxbin_add_rmsnorm(xd, cols + 1, rd, cols + 2, wd, code(fb, dt), rows, cols, 1e-5, ro, cols + 3, y, cols, q,
                           cols + 7, s)
    torch.cuda.synchronize()
    h, y64, q_want, s64 = norm_oracle(x, res, w, dt, 1e-5)
    # inv: half the relative error of the mean (its sum, the product with 1 / cols, eps), the root, the quotient
    rel = ((ss_roundings(cols) + 4) / 2 + 3) * U
    if ro is not None:
        assert torch.equal(ro[:, :cols].cpu(), h)
    if y is not None:
        assert (np.abs(f64(y) - y64) <= (rel + 2 * U + UNIT[dt]) * np.abs(y64) + TINY[dt]).all()
    if q is not None:
        assert np.array_equal(q[:, :cols].cpu().numpy().astype(np.int64), q_want)
        assert (np.abs(f64(s) - s64) <= (rel + 3 * U) * s64).all()


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("cols,out", [(96, "x"), (5120, "residual"), (8200, "x"), (40000, "x"), (40000, "residual")])
def test_add_rmsnorm_in_place(fb, dt, cols, out):
    note(f"add_rmsnorm in place {dt} x {cols} into {out}")
    rows = 3
    x, res, w = randn(rows, cols, dt, 1), randn(rows, cols, dt, 2), torch.ones(cols, dtype=DT[dt])
    xd, rd, wd = x.cuda(), res.cuda(), w.cuda()
    ro = xd if out == "x" else rd
    q = torch.empty((rows, cols), dtype=torch.int8, device="cuda")
    s = torch.empty(rows, dtype=torch.float32, device="cuda")
    fb.fluxbin_add_rmsnorm(xd, cols, rd, cols, wd, code(fb, dt), rows, cols, 1e-6, ro, cols, None, cols, q, cols, s)
    torch.cuda.synchronize()
    h, _, q_want, s64 = norm_oracle(x, res, w, dt, 1e-6)
    assert torch.equal(ro.cpu(), h)
    assert np.array_equal(q.cpu().numpy().astype(np.int64), q_want)
    assert (np.abs(f64(s) - s64) <= ((ss_roundings(cols) + 4) / 2 + 6) * U * s64).all()


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("cols", [200, 4096, 36000])
def test_add_rmsnorm_special_rows(fb, dt, cols):
    note(f"add_rmsnorm special rows {dt} x {cols}")
    x = randn(6, cols, dt, 21)
    x[0] = 0
    x[1, 5] = math.inf
    x[2, cols - 1] = math.nan
    x[3, :] = 1e30 if dt != "f16" else 6e4  # beyond fp16 the sum of squares leaves fp32
    res = torch.zeros_like(x)
    res[4, 0], x[4, 0] = math.inf, -math.inf
    w = torch.ones(cols, dtype=DT[dt])
    y = torch.empty((6, cols), dtype=DT[dt], device="cuda")
    q = torch.empty((6, cols), dtype=torch.int8, device="cuda")
    s = torch.empty(6, dtype=torch.float32, device="cuda")
    fb.fluxbin_add_rmsnorm(x.cuda(), cols, res.cuda(), cols, w.cuda(), code(fb, dt), 6, cols, 1e-5, None, cols, y, cols, q,
                           cols, s)
    torch.cuda.synchronize()
    y, q, s = f64(y), q.cpu().numpy(), f64(s)
    assert (y[0] == 0).all() and (q[0] == 0).all() and np.isfinite(s[0])
    for r in (1, 2, 4):
        assert np.isnan(y[r]).all() and np.isnan(s[r]) and (q[r] == 0).all()
    if dt == "f16":
        assert np.abs(y[3] - 1).max() < 2e-3 and (q[3] == 127).all()
    else:
        assert np.isnan(y[3]).all() and np.isnan(s[3])  # never a wrong finite number
    assert np.isfinite(y[5]).all() and np.isfinite(s[5])


# ------------------------------------------------------------------ gemm_w8a8

def gemm_case(fb, m, n, k, dt, bias=False, extreme=False, pad=0, seed=0, ldy_pad=0):
    g = torch.Generator().manual_seed(seed + 7 * m + 3 * n + k)
    ld = (k + 15) // 16 * 16 + pad
    if extreme:
        a, w = torch.full((m, ld), -128, dtype=torch.int8), torch.full((n, ld), -128, dtype=torch.int8)
    else:
        a = torch.randint(-128, 128, (m, ld), generator=g, dtype=torch.int8)  # the padding holds values too
        w = torch.randint(-128, 128, (n, ld), generator=g, dtype=torch.int8)
    sa = torch.rand(m, generator=g) * 0.02 + 0.001
    sw = torch.rand(n, generator=g) * 0.002 + 0.0001
    b = torch.randn(n, generator=g) if bias else None
    y = torch.full((m, n + ldy_pad), 3.0, dtype=DT[dt], device="cuda")
    fb.fluxbin_gemm_w8a8(a.cuda(), ld, sa.cuda(), w.cuda(), ld, sw.cuda(), None if b is None else b.cuda(), m, n, k, y,
                         n + ldy_pad, code(fb, dt))
    torch.cuda.synchronize()
    acc = a[:, :k].double() @ w[:, :k].double().t()  # exact: below 2^53
    v = (acc * sa.double()[:, None] * sw.double()).numpy()
    want = v if b is None else v + b.double().numpy()
    mag = np.abs(v) + (0 if b is None else np.abs(b.double().numpy()))
    got = f64(y)
    limit = np.where(np.abs(want) > 65504, np.inf, 0) if dt == "f16" else 0
    tol = UNIT[dt] * np.abs(want) + 5 * U * mag + TINY[dt] + limit
    bad = np.abs(got[:, :n] - want) > tol
    assert not bad.any(), (m, n, k, dt, np.argwhere(bad)[:5], got[:, :n][bad][:5], want[bad][:5])
    assert (got[:, n:] == 3).all()  # nothing written past a row


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 33, 64, 65, 100, 129, 255, 257, 300])
@pytest.mark.parametrize("n,k", [(1, 1), (3, 17), (16, 64), (127, 255), (130, 129), (257, 1000), (512, 2048)])
def test_gemm_w8a8_sizes(fb, m, n, k):
    note(f"gemm_w8a8 {m} x {n} x {k}")
    gemm_case(fb, m, n, k, "f32", bias=m % 2 == 0, pad=16 * (m % 3), ldy_pad=n % 3)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (8, 4097, 1111), (48, 1024, 11008), (200, 700, 4100), (513, 1000, 640),
                                   (1025, 2049, 300), (2048, 2048, 1024)])
def test_gemm_w8a8_types(fb, dt, m, n, k):
    note(f"gemm_w8a8 {dt} {m} x {n} x {k}")
    gemm_case(fb, m, n, k, dt, bias=True)


# (tokens, channels) that take different tiles, some by k
@pytest.mark.parametrize("m,n", [(61, 8190), (61, 16390), (333, 4093), (1030, 2050), (3500, 4499)])
@pytest.mark.parametrize("k", [1, 16, 127, 128, 129, 256, 300, 513, 650])
def test_gemm_w8a8_tiles(fb, m, n, k):
    """Fewer stages than a tile holds, as many, and more, each with and without a tail of k."""
    note(f"gemm_w8a8 tile {m} x {n} x {k}")
    gemm_case(fb, m, n, k, "bf16" if k % 2 else "f16", bias=k > 200, ldy_pad=k % 2)


@pytest.mark.parametrize("m,n,k", [(m, n, k) for m, n in ((20, 16384), (7, 30001), (300, 3000)) for k in (1, 127, 256, 257, 511, 700, 1300)]
                         + [(61, 8190, 1300), (333, 4093, 1100), (3500, 4499, 1000), (3500, 4499, 1024), (3500, 4499, 1153)])
def test_gemm_w8a8_more_tiles(fb, m, n, k):
    """64 x 32 and 64 x 64 at all numbers of stages; the largest tile, which takes long k, with and without a tail."""
    note(f"gemm_w8a8 tile {m} x {n} x {k}")
    gemm_case(fb, m, n, k, "f32" if k % 2 else "bf16", bias=True, pad=16, ldy_pad=k % 3)


def test_gemm_w8a8_wide_strides(fb):
    """Row strides of more than 8 MiB, whose 256 rows pass 32-bit offsets."""
    note("gemm_w8a8 strides of 2^23 + 16")
    m, n, k, ld = 20, 40, 100, (1 << 23) + 16
    g = torch.Generator().manual_seed(1)
    a = torch.randint(-128, 128, (m, k), generator=g, dtype=torch.int8)
    w = torch.randint(-128, 128, (n, k), generator=g, dtype=torch.int8)
    ad, wd = strided(a, ld), strided(w, ld)
    y = torch.empty((m, n), device="cuda")
    one = torch.ones(max(m, n), device="cuda")
    fb.fluxbin_gemm_w8a8(ad, ld, one, wd, ld, one, None, m, n, k, y, n, fb.DT_F32)
    torch.cuda.synchronize()
    assert torch.equal(y.cpu().double(), a.double() @ w.double().t())  # below 2^24: exact in fp32


def test_gemm_w8a8_most_channels(fb):
    """2^27 channels: tiles of 16 channels by 512 threads would make a grid of 2^32 threads."""
    m, n, k = 1, 1 << 27, 304
    note(f"gemm_w8a8 {m} x {n} x {k}")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 42 GB of GPU memory")
    w = torch.zeros((n, k), dtype=torch.int8, device="cuda")
    at = torch.tensor([0, 1 << 26, n - 17, n - 1], device="cuda")
    w[at, 300] = torch.tensor([1, -2, 3, 127], dtype=torch.int8, device="cuda")
    a = torch.full((m, k), 2, dtype=torch.int8, device="cuda")
    one = torch.ones(n, device="cuda")
    y = torch.full((m, n), 9.0, device="cuda")
    fb.fluxbin_gemm_w8a8(a, k, one, w, k, one, None, m, n, k, y, n, fb.DT_F32)
    torch.cuda.synchronize()
    assert y[0, at].tolist() == [2.0, -4.0, 6.0, 254.0]
    y[0, at] = 0
    assert not y.any()


def test_outputs_beyond_32_bit_offsets(fb):
    note("gemm_w8a8, quantize_rows and token_logprobs over more than 2^31 elements")
    m, n, k = 40000, 60000, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    a = torch.randint(-128, 128, (m, k), generator=g, dtype=torch.int8, device="cuda")
    w = torch.randint(-128, 128, (n, k), generator=g, dtype=torch.int8, device="cuda")
    sa, sw = torch.rand(m, generator=g, device="cuda") * 1e-3, torch.rand(n, generator=g, device="cuda") * 1e-2
    y = torch.empty((m, n), dtype=torch.float16, device="cuda")
    fb.fluxbin_gemm_w8a8(a, k, sa, w, k, sw, None, m, n, k, y, n, fb.DT_F16)
    rows = torch.tensor([0, 1, 20000, 35791, 35792, 35793, m - 2, m - 1])
    want = (a[rows].cpu().double() @ w.cpu().double().t()) * sa[rows].cpu().double()[:, None] * sw.cpu().double()
    got = y[rows].cpu().double()
    assert ((got - want).abs() <= (UNIT["f16"] + 5 * U) * want.abs() + TINY["f16"]).all()
    q = torch.empty((m, n), dtype=torch.int8, device="cuda")
    s = torch.empty(m, device="cuda")
    fb.fluxbin_quantize_rows(y, n, fb.DT_F16, m, n, q, n, s)
    q_want, _ = quant_oracle(y[rows].cpu().float().numpy())
    assert np.array_equal(q[rows].cpu().numpy().astype(np.int64), q_want)
    del q
    top, idx = torch.empty((m, 3), device="cuda"), torch.empty((m, 3), dtype=torch.int64, device="cuda")
    lp, ent = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    targets = torch.full((m,), n - 1, device="cuda")
    assert fb.fluxbin_token_logprobs_workspace_size(m, n, 3) == 0
    fb.fluxbin_token_logprobs(y, n, fb.DT_F16, m, n, 1.0, targets, lp, ent, 3, top, idx, None, 0)
    check_scores(y[rows].cpu(), {"logprob": f64(lp[rows]), "entropy": f64(ent[rows]), "top": f64(top[rows]),
                                 "index": idx[rows].cpu().numpy()}, 1.0, 3, targets[rows].cpu())


@pytest.mark.parametrize("m", [1, 20, 70, 300])
def test_gemm_w8a8_largest_sums(fb, m):
    """-128 * -128 over the longest k: every sum is 131071 * 2^14, just below 2^31."""
    note(f"gemm_w8a8 extreme m = {m}")
    gemm_case(fb, m, 33, 131071, "f32", extreme=True)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_gemm_w8a8_poisoned_token_shows(fb, m):
    k, n = 512, 300
    a = torch.ones((m, k), dtype=torch.int8, device="cuda")
    w = torch.ones((n, k), dtype=torch.int8, device="cuda")
    sa = torch.ones(m, device="cuda")
    sa[m // 2] = math.nan
    y = torch.empty((m, n), dtype=torch.float32, device="cuda")
    fb.fluxbin_gemm_w8a8(a, k, sa, w, k, torch.ones(n, device="cuda"), None, m, n, k, y, n, fb.DT_F32)
    torch.cuda.synchronize()
    y = y.cpu().numpy()
    assert np.isnan(y[m // 2]).all() and (np.delete(y, m // 2, axis=0) == k).all()


# ------------------------------------------------------------------ token_logprobs

def score(fb, x, dt, top_k, scale=1.0, targets=None, ld=None, offset=0, entropy=True):
    rows, vocab = x.shape
    ld = ld or vocab
    xd = strided(x, ld, offset)
    out = {"logprob": torch.full((rows,), 9.0, device="cuda") if targets is not None else None,
           "entropy": torch.full((rows,), 9.0, device="cuda") if entropy else None,
           "top": torch.full((rows, top_k), 9.0, device="cuda") if top_k else None,
           "index": torch.full((rows, top_k), -9, dtype=torch.int64, device="cuda") if top_k else None}
    need = fb.fluxbin_token_logprobs_workspace_size(rows, vocab, top_k)
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device="cuda")  # its contents do not matter
    td = None if targets is None else targets.cuda()
    fb.fluxbin_token_logprobs(xd, ld, code(fb, dt), rows, vocab, scale, td, out["logprob"], out["entropy"], top_k,
                              out["top"], out["index"], ws if need else None, need)
    torch.cuda.synchronize()
    return {n: None if v is None else v.cpu().numpy() for n, v in out.items()}


def score_oracle(x, scale, top_k):
    x64 = f64(x)
    z = x64 * np.float64(np.float32(scale))
    zmax = z.max(axis=1, keepdims=True)
    with np.errstate(all="ignore"):
        d = np.where(np.isinf(zmax) & (zmax < 0), -np.inf, z - zmax)
        e = np.exp(d)
        total = e.sum(axis=1, keepdims=True)
        lp = np.where(total > 0, d - np.log(total), -np.inf)
        p = np.where(total > 0, e / total, 0)
        entropy = -np.where(p > 0, p * np.where(p > 0, lp, 0), 0).sum(axis=1)
    order = np.argsort(-x64, axis=1, kind="stable")[:, :top_k]
    return lp, entropy, order


def check_scores(x, got, scale, top_k, targets):
    lp, entropy, order = score_oracle(x, scale, top_k)
    vocab = x.shape[1]

    # A log probability is c (x - max) with a relative error of a few u, minus log2 of a sum whose terms are off by
    # that times their own exponent; weighted with p these exponents average at most ln(vocab) + 1.
    def tol(v):
        return 8 * U * (np.abs(np.where(np.isfinite(v), v, 0)) + 2 * math.log(vocab) + 8)

    def close(a, b):
        same = np.isfinite(b)
        assert np.array_equal(a[~same], b[~same]), (a[~same], b[~same])
        assert (np.abs(a[same] - b[same]) <= tol(b[same])).all(), np.abs(a[same] - b[same]).max()

    if targets is not None:
        t = targets.numpy()
        want = np.where(t < 0, 0.0, lp[np.arange(len(t)), np.maximum(t, 0)])
        close(got["logprob"].astype(np.float64), want)
    if got["entropy"] is not None:
        assert (np.abs(got["entropy"] - entropy) <= tol(entropy) * 2).all()
    if top_k:
        assert np.array_equal(got["index"], order)
        close(got["top"].astype(np.float64), np.take_along_axis(lp, order, axis=1))


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab", [1, 2, 5, 64, 255, 257, 2048, 2049, 8191, 8192, 8193, 20001, 32000, 100003])
@pytest.mark.parametrize("rows", [1, 3])
def test_token_logprobs(fb, dt, vocab, rows):
    top_k = min(vocab, [0, 1, 5, 20, 64][(vocab + rows) % 5])
    note(f"token_logprobs {dt} {rows} x {vocab} top {top_k}")
    g = torch.Generator().manual_seed(vocab)
    x = (torch.randn(rows, vocab, generator=g) * 4).to(DT[dt])
    targets = torch.randint(0, vocab, (rows,), generator=g)
    targets[rows // 2] = -1 if vocab % 2 else targets[rows // 2]
    got = score(fb, x, dt, top_k, 0.75, targets, ld=vocab + 5, offset=3)
    check_scores(x, got, 0.75, top_k, targets)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,top_k", [(1100, 3000, 20), (700, 9001, 64), (2000, 33, 5), (40, 50001, 1)])
def test_token_logprobs_many_rows(fb, dt, rows, vocab, top_k):
    note(f"token_logprobs {dt} {rows} x {vocab} top {top_k}")
    g = torch.Generator().manual_seed(rows)
    x = (torch.randn(rows, vocab, generator=g) * 3).to(DT[dt])
    targets = torch.randint(-2, vocab, (rows,), generator=g)
    check_scores(x, score(fb, x, dt, top_k, 1.0, targets), 1.0, top_k, targets)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,vocab,top_k", [(9, 2050, 64), (2, 32760, 20), (40, 32768, 5), (2, 32769, 64), (256, 2100, 5), (257, 2100, 5),
                                              (7, 512, 32), (7, 512, 33), (7, 513, 32), (3000, 257, 20), (3000, 60, 32)])
def test_token_logprobs_around_the_plans_borders(fb, dt, rows, vocab, top_k):
    note(f"token_logprobs {dt} {rows} x {vocab} top {top_k}")
    g = torch.Generator().manual_seed(vocab)
    x = (torch.randn(rows, vocab, generator=g) * 3).to(DT[dt])
    targets = torch.randint(-2, vocab, (rows,), generator=g)
    check_scores(x, score(fb, x, dt, top_k, 1.0, targets, ld=vocab + 3, offset=1), 1.0, top_k, targets)


@pytest.mark.parametrize("rows", [1, 2, 5, 1500])
@pytest.mark.parametrize("top_k", [1, 5, 30, 64])
@pytest.mark.parametrize("pattern", ["equal", "two values", "ascending", "descending", "few left", "none left", "zeros of both signs",
                                     "lowest value", "lowest throughout", "peaked", "huge"])
def test_token_logprobs_hard_rows(fb, rows, top_k, pattern):
    vocab = {1: 17000, 2: 40000, 5: 500}.get(rows, 9000)
    note(f"token_logprobs {pattern} {rows} x {vocab} top {top_k}")
    g = torch.Generator().manual_seed(5)
    x = torch.randn(rows, vocab, generator=g)
    if pattern == "equal":
        x[:] = 1.5
    elif pattern == "two values":
        x = (x > 0.3).float()
    elif pattern == "ascending":
        x = torch.arange(vocab).float().repeat(rows, 1) * 2.0 ** -7
    elif pattern == "descending":
        x = -torch.arange(vocab).float().repeat(rows, 1) * 2.0 ** -7
    elif pattern == "few left":
        keep = torch.zeros(vocab, dtype=torch.bool)
        keep[[7, vocab // 2, vocab - 1]] = True
        x[:, ~keep] = -math.inf
    elif pattern == "none left":
        x[:] = -math.inf
    elif pattern == "zeros of both signs":
        x = torch.where(x > 0, 0.0, -0.0)
    elif pattern == "lowest value":
        x[:, ::2] = torch.finfo(torch.float32).min
    elif pattern == "lowest throughout":
        x[:] = torch.finfo(torch.float32).min
    elif pattern == "peaked":
        x[:, min(4321, vocab // 2)] = 200.0
    elif pattern == "huge":
        x = x * 3000
    targets = torch.full((rows,), 8 if pattern == "lowest value" else 7, dtype=torch.int64)
    check_scores(x, score(fb, x, "f32", top_k, 1.0, targets), 1.0, top_k, targets)


@pytest.mark.parametrize("rows,vocab", [(3, 700), (3, 40000), (2000, 700)])
def test_token_logprobs_poisoned_rows(fb, rows, vocab):
    note(f"token_logprobs poisoned {rows} x {vocab}")
    x = torch.randn(rows, vocab, generator=torch.Generator().manual_seed(3))
    x[0, vocab // 2] = math.nan
    x[1, vocab - 1] = math.inf
    targets = torch.zeros(rows, dtype=torch.int64)
    targets[2] = vocab  # out of range
    got = score(fb, x, "f32", 5, 1.0, targets)
    assert np.isnan(got["logprob"][:3]).all() and np.isnan(got["entropy"][:2]).all() and np.isfinite(got["entropy"][2])
    assert np.isnan(got["top"][:2]).all() and np.isfinite(got["top"][2]).all()
    assert got["index"][1, 0] == vocab - 1  # +inf is the best alternative, a NaN is none
    row = np.where(np.isnan(x[0].numpy()), -np.inf, x[0].numpy())
    assert np.array_equal(got["index"][0], np.argsort(-row, kind="stable")[:5])
    assert np.isfinite(got["logprob"][3:]).all()
    x[0] = math.nan
    got = score(fb, x, "f32", 5, 1.0, targets)
    assert (got["index"][0] == -1).all() and np.isnan(got["top"][0]).all()


def test_token_logprobs_outputs_are_optional(fb):
    x = torch.randn(4, 5000, generator=torch.Generator().manual_seed(1))
    targets = torch.arange(4)
    full = score(fb, x, "f32", 5, 1.0, targets)
    only = score(fb, x, "f32", 0, 1.0, targets, entropy=False)
    assert np.array_equal(only["logprob"], full["logprob"])
    only = score(fb, x, "f32", 5, 1.0, None, entropy=False)
    assert np.array_equal(only["top"], full["top"]) and np.array_equal(only["index"], full["index"])


# ------------------------------------------------------------------ streams, graphs, repeats

def chain(fb, t, stream=None):
    """norm -> head product -> scores on preallocated tensors."""
    rows, cols, vocab = t["rows"], t["cols"], t["vocab"]
    fb.fluxbin_add_rmsnorm(t["x"], cols, t["res"], cols, t["nw"], fb.DT_F16, rows, cols, 1e-5, None, cols, None, cols, t["q"],
                           cols, t["qs"], stream)
    fb.fluxbin_quantize_rows(t["w16"], cols, fb.DT_F16, vocab, cols, t["w"], cols, t["ws"], stream)
    fb.fluxbin_gemm_w8a8(t["q"], cols, t["qs"], t["w"], cols, t["ws"], None, rows, vocab, cols, t["logits"], vocab, fb.DT_F32,
                         stream)
    fb.fluxbin_token_logprobs(t["logits"], vocab, fb.DT_F32, rows, vocab, 1.0, t["targets"], t["lp"], t["ent"], 4, t["top"],
                              t["idx"], t["work"], t["work"].numel(), stream)


def chain_tensors(rows, cols, vocab):
    d = "cuda"
    return {"rows": rows, "cols": cols, "vocab": vocab, "x": randn(rows, cols, "f16", 1).to(d), "res": randn(rows, cols, "f16", 2).to(d),
            "nw": torch.ones(cols, dtype=torch.float16, device=d), "q": torch.empty((rows, cols), dtype=torch.int8, device=d),
            "qs": torch.empty(rows, device=d), "w16": randn(vocab, cols, "f16", 3, 0.02).to(d),
            "w": torch.empty((vocab, cols), dtype=torch.int8, device=d), "ws": torch.empty(vocab, device=d),
            "logits": torch.empty((rows, vocab), device=d), "targets": torch.arange(rows, device=d),
            "lp": torch.empty(rows, device=d), "ent": torch.empty(rows, device=d), "top": torch.empty((rows, 4), device=d),
            "idx": torch.empty((rows, 4), dtype=torch.int64, device=d), "work": torch.empty(4 << 20, dtype=torch.uint8, device=d)}


OUT = ("q", "qs", "logits", "lp", "ent", "top", "idx")


@pytest.mark.parametrize("rows", [1, 16, 150, 600])
def test_chain_repeats_bitwise_on_a_side_stream_and_in_a_graph(fb, rows):
    note(f"chain, {rows} rows")
    t = chain_tensors(rows, 1024, 5000)
    chain(fb, t)
    torch.cuda.synchronize()
    want = {n: t[n].clone() for n in OUT}

    def clear():
        for n in OUT:
            t[n].zero_()

    side = torch.cuda.Stream()
    clear()
    side.wait_stream(torch.cuda.current_stream())
    chain(fb, t, side)
    torch.cuda.synchronize()
    for n in OUT:
        assert torch.equal(t[n], want[n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(fb, t)
    for _ in range(3):
        clear()
        t["work"].fill_(170)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in OUT:
            assert torch.equal(t[n], want[n]), n
    # the head's logits against 64 bits, from the integers and scales of the steps before
    acc = t["q"].cpu().double() @ t["w"].cpu().double().t()
    logits = (acc * t["qs"].cpu().double()[:, None] * t["ws"].cpu().double()).numpy()
    assert (np.abs(f64(t["logits"]) - logits) <= 5 * U * np.abs(logits) + 2.0 ** -126).all()
    check_scores(t["logits"].cpu(), {"logprob": f64(t["lp"]), "entropy": f64(t["ent"]), "top": f64(t["top"]),
                                     "index": t["idx"].cpu().numpy()}, 1.0, 4, torch.arange(rows))
