"""The launches of the 8-bit operators, watched on the host (tests/launches.py)."""
import numpy as np
import pytest

from tests import int8_cases as C
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


def instances(kernels, prefix):
    return {k for k in kernels if k.startswith(prefix)}


@pytest.fixture(scope="module")
def kernels():
    return L.record([])[0]


def test_the_table_of_tiles_reaches_every_instance_of_the_product(kernels):
    calls, want = [], []
    for tile, (params, (m, n), _, _) in C.TILES.items():
        for dt in C.TYPES:
            for k in C.tile_ks(tile):
                calls.append(L.gemm(m, n, k, dt))
                want.append(f"gemm_w8a8_{'rows' if tile == '16x16' else 'tile'}_kernel<{dt.upper()}, {params}>")
    got = recorded(calls)
    for call, launches, name in zip(calls, got, want):
        assert [x["kernel"] for x in launches] == [name], call
        check_gemm(call, launches)
    assert set(want) == instances(kernels, "gemm_w8a8_")


def test_the_table_of_plans_reaches_every_instance_of_the_scores(kernels):
    seen = set()
    for plan, (rows, vocab, params, splits, slices) in C.PLANS.items():
        calls = [L.score(rows, vocab, k, dt) for dt in C.TYPES for k in C.plan_top_ks(plan)]
        for call, launches in zip(calls, recorded(calls)):
            dt = {v: k for k, v in L.TYPES.items()}[call[1][2]].upper()
            names = [f"logprob_rows_kernel<{dt}, {params}>"] + [f"logprob_join_kernel<{dt}>"] * (splits > 1)
            assert [x["kernel"] for x in launches] == names, (plan, call)
            a, threads = launches[0]["args"], int(params.split(", ")[1])
            assert a["splits"] == splits and launches[0]["grid"] == [rows * splits, 1, 1], (plan, a)
            assert cdiv(min(a["split_len"], vocab), threads * 8 * (1 if "true" in params else 4)) == slices, (plan, a)
            assert splits * a["split_len"] >= vocab > (splits - 1) * a["split_len"]
            for x in launches:
                check_grid(x)
            seen.update(names)
    assert seen == instances(kernels, "logprob_")


@pytest.mark.parametrize("dt", C.TYPES)
def test_the_products_comparison_sees_what_is_wrong(dt):
    want = np.array([1.0, -2.0, 0.0, 70000.0, -70000.0, 1000.0])
    mag = np.abs(want)
    right = want.copy()
    if dt == "f16":
        right[3:5] = np.inf, -np.inf
    assert not C.product_errors(right, want, mag, dt).any()
    for i in range(len(want)):
        for wrong in (np.nan, -right[i] if right[i] else 1e-3, 3.0, np.inf if right[i] != np.inf else 65504.0):
            got = right.copy()
            got[i] = wrong
            assert C.product_errors(got, want, mag, dt).tolist() == [j == i for j in range(len(want))], (i, wrong)
    # the border of fp16's largest number and infinity
    border = np.array([65519.0, 65521.0])
    if dt == "f16":
        assert not C.product_errors(np.array([65504.0, np.inf]), border, border, dt).any()
        assert C.product_errors(np.array([np.inf, 65504.0]), border, np.zeros(2), dt).all()
