"""The comparison that the GPU tests of adjusted logits use has to reject what is wrong (no GPU needed)."""
import numpy as np
import pytest

from tests.adjust_compare import EDGE, MOST, compare
from tests.attention_cases import DT, UNIT

torch = pytest.importorskip("torch")


def rounded(x, dt):
    return torch.tensor(x, dtype=torch.float64).to(torch.float32).to(DT[dt]).double().numpy()


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_what_is_wrong_is_rejected(dt):
    rng = np.random.default_rng(1)
    z = rng.standard_normal((3, 200)) * 4
    masked = rng.random(z.shape) < 0.5
    want, mag = np.where(masked, -np.inf, z), np.abs(z)
    want[0, :4] = np.nan, np.inf, 2 * MOST[dt], -2 * MOST[dt]
    with np.errstate(over="ignore"):
        good = rounded(want, dt)
    compare(dt, good, want, mag, 6)
    row, col = np.argwhere(masked[1:])[0]
    free = np.argwhere(~masked[1:])[0]
    wrong = [((row + 1, col), v) for v in (z[row + 1, col], np.inf, np.nan, -MOST[dt], 0.0)]  # a mask that was not applied, and worse
    wrong += [((0, 0), 0.0), ((0, 1), -np.inf), ((0, 1), MOST[dt]), ((0, 2), -np.inf), ((0, 2), MOST[dt]), ((0, 3), np.inf), ((0, 3), np.nan)]
    at = (free[0] + 1, free[1])
    wrong += [(at, v) for v in (np.nan, np.inf, -np.inf, z[at] * (1 + 3 * UNIT[dt] + 2.0 ** -20), -z[at])]
    for where, v in wrong:
        bad = good.copy()
        bad[where] = v
        with pytest.raises(AssertionError):
            compare(dt, bad, want, mag, 6)
    with pytest.raises(AssertionError):
        compare(dt, rounded(z, dt), want, mag, 6)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_values_at_the_end_of_the_type(dt):
    edge = EDGE[dt]
    with np.errstate(over="ignore"):
        below = rounded(np.array([edge * (1 - 1e-5)]), dt)[0]
    for want, got, ok in ((edge * (1 + 1e-5), np.inf, True), (edge * (1 + 1e-5), MOST[dt], False), (edge * (1 - 1e-5), np.inf, False),
                          (edge * (1 - 1e-5), below, True), (-edge * 1.1, -np.inf, True), (-edge * 1.1, np.inf, False)):
        call = lambda: compare(dt, np.array([got]), np.array([want]), np.array([abs(want)]), 6)  # noqa: E731, B023
        if ok:
            call()
        else:
            with pytest.raises(AssertionError):
                call()
