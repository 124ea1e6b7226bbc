"""Paths of the 8-bit operators that sizes, strides and types choose, against 64 bits on the host."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.test_gpu_int8_ops import fb, note  # noqa: E402,F401

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
