"""Paths of the 8-bit operators that sizes, strides and types choose, against 64 bits on the host."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests import int8_cases as C  # noqa: E402
from tests.test_gpu_int8_ops import DT, check_scores, code, f64, fb, note, score  # noqa: E402,F401

WIDE = (1 << 23) + 16  # a row stride whose 256 rows pass 32-bit offsets


# ------------------------------------------------------------------ the product over wide strides

@pytest.mark.parametrize("m,n", [(2, (1 << 26) + 20), ((1 << 19) + 20, 3), (1, 5000), (5000, 1)])
def test_product_over_wide_strides_in_several_launches(fb, m, n):
    """More channels or tokens than one launch of the kernel without tiles takes; a single row's stride is no matter."""
    k = 16
    note(f"gemm_w8a8 {m} x {n} x {k}, strides of {WIDE}")
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB of GPU memory")
    g = torch.Generator(device="cuda").manual_seed(m)

    def operand(rows):
        if rows > 40:
            return torch.randint(-128, 128, (rows, k), generator=g, dtype=torch.int8, device="cuda"), k
        buf = torch.zeros((rows - 1) * WIDE + k, dtype=torch.int8, device="cuda")
        view = buf.as_strided((rows, k), (WIDE, 1))
        view.copy_(torch.randint(-128, 128, (rows, k), generator=g, dtype=torch.int8, device="cuda"))
        return view, WIDE

    (a, lda), (w, ldw) = operand(m), operand(n)
    sa = 2.0 ** torch.randint(-3, 4, (m,), generator=g, device="cuda").float()  # powers of two: the outputs are exact
    sw = 2.0 ** torch.randint(-3, 4, (n,), generator=g, device="cuda").float()
    bias = torch.arange(n, device="cuda").remainder(7).float() / 64
    y = torch.full((m, n), math.nan, device="cuda")
    fb.fluxbin_gemm_w8a8(a, lda, sa, w, ldw, sw, bias, m, n, k, y, n, fb.DT_F32)
    torch.cuda.synchronize()
    # |sum| <= 16 * 2^14 = 2^18 in steps of 2^-6 and the bias in steps of 2^-6, times up to 2^6: 24 bits but for the largest
    # outputs, where one rounding of the addition remains
    step = max(1, (1 << 24) // m)
    for at in range(0, n, step):
        part = slice(at, min(n, at + step))
        want = (a.double() @ w[part].double().t().contiguous()) * sa.double()[:, None] * sw[part].double() + bias[part].double()
        assert torch.equal(y[:, part], want.float())


# ------------------------------------------------------------------ every instance of the product

def product(fb, m, n, k, dt, bias=True, pad=0, ldy_pad=0, loud=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * m + 3 * n + k)
    ld = (k + 15) // 16 * 16 + pad
    a = torch.randint(-128, 128, (m, ld), generator=g, dtype=torch.int8, device="cuda")  # the padding holds values too
    w = torch.randint(-128, 128, (n, ld), generator=g, dtype=torch.int8, device="cuda")
    sa = (torch.rand(m, generator=g, device="cuda") * 0.02 + 0.001) * loud
    sw = torch.rand(n, generator=g, device="cuda") * 0.002 + 0.0001
    b = torch.randn(n, generator=g, device="cuda") if bias else None
    y = torch.full((m, n + ldy_pad), 3.0, dtype=DT[dt], device="cuda")
    fb.fluxbin_gemm_w8a8(a, ld, sa, w, ld, sw, b, m, n, k, y, n + ldy_pad, code(fb, dt))
    torch.cuda.synchronize()
    v = torch.mm(a[:, :k].double(), w[:, :k].double().t().contiguous())  # exact: below 2^53
    v = (v * sa.double()[:, None] * sw.double()).cpu().numpy()
    b64 = np.zeros(n) if b is None else f64(b)
    got, want = f64(y), v + b64
    bad = C.product_errors(got[:, :n], want, np.abs(v) + np.abs(b64), dt)
    assert not bad.any(), (m, n, k, dt, np.argwhere(bad)[:5], got[:, :n][bad][:5], want[bad][:5])
    assert (got[:, n:] == 3).all()  # nothing written past a row
    return want


@pytest.mark.parametrize("dt", C.TYPES)
@pytest.mark.parametrize("tile", C.TILES)
def test_every_instance_at_its_numbers_of_stages(fb, tile, dt):
    m, n = C.TILES[tile][1]
    for k in C.tile_ks(tile):
        note(f"gemm_w8a8 {tile} {dt} {m} x {n} x {k}")
        product(fb, m, n, k, dt, bias=k % 2 == 0, pad=16 * (k % 3), ldy_pad=k % 4)


@pytest.mark.parametrize("dt", C.TYPES)
@pytest.mark.parametrize("n,k", [(1, 1), (3, 17), (16, 64), (127, 255), (130, 129), (257, 1000), (600, 16), (600, 64), (600, 200), (600, 513), (512, 2048)])
def test_product_sizes(fb, n, k, dt):
    for m in (1, 2, 15, 16, 17, 33, 64, 65, 100, 129, 255, 257, 300):
        note(f"gemm_w8a8 {dt} {m} x {n} x {k}")
        product(fb, m, n, k, dt, bias=m % 2 == 0, pad=16 * (m % 3), ldy_pad=n % 3)


@pytest.mark.parametrize("dt", C.TYPES)
def test_the_largest_tile_over_a_long_k(fb, dt):
    note(f"gemm_w8a8 {dt} 1024 x 8192 x 8192")
    product(fb, 1024, 8192, 8192, dt)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_outputs_beyond_fp16_are_infinite(fb, m):
    note(f"gemm_w8a8 f16 overflow, {m} tokens")
    # a sum's deviation is 2^5 * 74^2 = 1.7e5, the scales are about 0.011 * 4e4 and 0.0011: outputs of about 8e4
    size = np.abs(product(fb, m, 500, 1024, "f16", loud=4e4))
    over, under = float((size > 65520).mean()), float((size < 65504).mean())
    assert over > 0.05 and under > 0.05


# ------------------------------------------------------------------ every plan of the scores

def hard_rows(rows, vocab, dt):
    """Rows that defeat the bound of the best, or have little or nothing left, one pattern after the other."""
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = torch.randn(rows, vocab, generator=g, device="cuda") * 3
    at = torch.arange(vocab, device="cuda")
    low = torch.finfo(DT[dt]).min

    def few(*left):
        keep = torch.zeros(vocab, dtype=torch.bool, device="cuda")
        keep[list(left)] = True
        return lambda r: torch.where(keep, r, -math.inf)

    patterns = [
        lambda r: r,
        lambda r: torch.full_like(r, 1.5),
        lambda r: (r > 0.3).float(),
        lambda r: at.float() * 2.0 ** -7,
        lambda r: -at.float() * 2.0 ** -7,
        lambda r: r + torch.div(at, 1000, rounding_mode="floor"),  # later columns larger, in steps
        few(7, vocab // 2, vocab - 1),
        few(vocab - 1),
        few(*range(0, vocab, max(1, vocab // 70))),
        few(*range(vocab - 66, vocab)),
        lambda r: torch.where(at < vocab - 300, -math.inf, r),
        lambda r: torch.full_like(r, -math.inf),
        lambda r: torch.where(r > 0, 0.0, -0.0),
        lambda r: torch.where(at % 2 == 0, low, r),
        lambda r: torch.full_like(r, low),
        lambda r: torch.where(at == vocab // 2, 200.0, r),
        lambda r: r * 1000,
        lambda r: torch.where(at % 5 == 0, -math.inf, r),
    ]
    for i in range(rows):
        if i < 2 * len(patterns) or i >= rows - len(patterns):
            x[i] = patterns[i % len(patterns)](x[i])
    return x.to(DT[dt]), len(patterns)


@pytest.mark.parametrize("dt", C.TYPES)
@pytest.mark.parametrize("plan", C.PLANS)
def test_every_plan_of_the_scores(fb, plan, dt):
    rows, vocab = C.PLANS[plan][:2]
    x, patterns = hard_rows(max(rows, 18), vocab, dt)
    assert patterns == 18
    groups = [x[i:i + rows] for i in range(0, x.shape[0], rows)]  # of few rows a call several calls
    for top_k in C.plan_top_ks(plan):
        for x in groups:
            note(f"token_logprobs {plan} {dt} {tuple(x.shape)} top {top_k}")
            n = x.shape[0]
            targets = torch.randint(-2, vocab, (n,), generator=torch.Generator().manual_seed(n + top_k))
            got = score(fb, x, dt, top_k, 0.75, targets, ld=vocab + 3, offset=1)
            see = torch.cat([torch.arange(min(n, patterns)), torch.arange(max(min(n, patterns), n - 2), n)])
            part = {name: None if v is None else v[see.numpy()] for name, v in got.items()}
            check_scores(x[see.cuda()].cpu(), part, 0.75, top_k, targets[see])


@pytest.mark.parametrize("dt", C.TYPES)
@pytest.mark.parametrize("plan", C.PLANS)
def test_poisoned_rows_in_every_plan(fb, plan, dt):
    rows, vocab = C.PLANS[plan][:2]
    note(f"token_logprobs poisoned, {plan} {dt}")
    x = torch.randn(rows, vocab, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(DT[dt])
    x[0, vocab // 2] = math.nan
    x[1, vocab - 1] = math.inf
    x[2] = math.nan
    targets = torch.zeros(rows, dtype=torch.int64)
    got = score(fb, x, dt, 5, 1.0, targets)
    assert np.isnan(got["logprob"][:3]).all() and np.isnan(got["entropy"][:3]).all() and np.isnan(got["top"][:3]).all()
    row = f64(x[0])
    assert np.array_equal(got["index"][0], np.argsort(-np.where(np.isnan(row), -np.inf, row), kind="stable")[:5])
    assert got["index"][1, 0] == vocab - 1 and (got["index"][2] == -1).all()
    assert np.isfinite(got["logprob"][3:]).all() and np.isfinite(got["entropy"][3:]).all() and np.isfinite(got["top"][3:]).all()
