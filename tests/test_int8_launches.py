"""The launches of the 8-bit operators, watched on the host (tests/launches.py)."""
import pytest

from tests import launches as L

pytestmark = pytest.mark.skipif(not L.available(), reason="gcc and c++filt not available")

BYTES = {"F16": 2, "BF16": 2, "F32": 4}


@pytest.fixture(scope="module", autouse=True)
def built():
    from binary_basis_lut_amd import build as B
    if B.is_stale():
        B.build()


def recorded(calls):
    results = L.record(calls)[1]
    for call, r in zip(calls, results):
        assert r["status"] == 0, (call, r["error"])
    return [r["launches"] for r in results]


def cdiv(a, b):
    return -(-a // b)


def check_grid(launch):
    """What HIP devices take: fewer than 2^32 threads along x, at most 65535 workgroups along y and z."""
    (x, y, z), (bx, by, bz) = launch["grid"], launch["block"]
    assert x > 0 and x * bx < 1 << 32, launch
    assert 0 < y <= 65535 and z == 1 and by == bz == 1 and bx <= 1024, launch


def check_gemm(call, launches):
    """Every launch's grid fits, and together they compute every output once, from its own operands."""
    a, lda, _, w, ldw, _, bias, m, n, k, y, ldy, _ = call[1]
    area = set()
    for launch in launches:
        check_grid(launch)
        g, kernel = launch["args"], launch["kernel"]
        elem = BYTES[kernel.split("<")[1].split(",")[0]]
        assert (g["lda"], g["ldw"], g["ldy"], g["k"]) == (lda, ldw, ldy, k)
        m0, n0 = (g["a_scale"] - L.A) // 4, (g["w_scale"] - L.A) // 4
        assert g["a"] == a + m0 * lda and g["w"] == w + n0 * ldw and g["y"] == y + (m0 * ldy + n0) * elem
        assert g["bias"] == (bias + 4 * n0 if bias else None)
        if "rows" in kernel:
            assert launch["grid"] == [cdiv(g["n"], 16), cdiv(g["m"], 16), 1]
        else:
            bn, bm = (int(v) for v in kernel.split(", ")[1:3])
            assert launch["grid"] == [cdiv(g["n"], bn) * cdiv(g["m"], bm), 1, 1]
        area.add((m0, n0, g["m"], g["n"]))
    assert len(area) == len(launches) and sum(r[2] * r[3] for r in area) == m * n
    for m0, n0, dm, dn in area:
        assert dm > 0 and dn > 0 and m0 + dm <= m and n0 + dn <= n
    rows = {r[0]: r[2] for r in area}
    cols = {r[1]: r[3] for r in area}
    assert len(area) == len(rows) * len(cols) and sum(rows.values()) == m and sum(cols.values()) == n  # a lattice


WIDE = (1 << 23) + 16  # a stride whose 256 rows pass 32-bit offsets


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("m,n,k,kw", [
    (1, 1 << 27, 304, dict(lda=2 * WIDE)), (2, 1 << 27, 16, dict(lda=WIDE)), (2, (1 << 27) - 5, 16, dict(lda=WIDE, bias=False)),
    ((1 << 21) + 5, 16, 16, dict(ldw=WIDE)), (1 << 27, 1, 16, dict(ldw=WIDE)), ((1 << 27) - 3, 2, 16, dict(ldw=WIDE)),
    (20, 40, 100, dict(lda=WIDE, ldw=WIDE)),
])
def test_products_over_wide_strides_fit_their_grids(m, n, k, kw, dt):
    call = L.gemm(m, n, k, dt, **kw)
    check_gemm(call, recorded([call])[0])


def test_products_of_all_sizes_fit_their_grids():
    calls = [L.gemm(m, n, k) for m in (1, 2, 16, 17, 333, 8192, 1 << 20, 1 << 27) for n in (1, 31, 4096, 57344, 1 << 20, 1 << 27)
             for k in (1, 128, 4096, 131071) if m * n <= 1 << 37]
    for call, launches in zip(calls, recorded(calls)):
        check_gemm(call, launches)
        assert len(launches) == 1
