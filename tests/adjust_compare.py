"""Adjusted logits against their definition, where both may be infinite or NaN (numpy)."""
import numpy as np

from tests.attention_cases import TINY, U, UNIT

MOST = {"f16": 65504.0, "bf16": float.fromhex("0x1.fep127"), "f32": float.fromhex("0x1.fffffep127")}
EDGE = {"f16": 65520.0, "bf16": MOST["bf16"] + 2.0 ** 119, "f32": MOST["f32"] + 2.0 ** 103}  # half a step beyond: infinity from there on


def compare(dt, got, want, mag, units):
    """Raises unless every element is as it has to be.

    want: the value in 64 bits, mag: the magnitude that `units` fp32 roundings go by.  A forbidden token is -inf
    and nothing else, NaN is NaN.  A finite value is within its roundings; one that may round past the type's
    largest number may be the infinity of its sign, and has to be where no rounding could bring it back.
    """
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fine = np.isfinite(want)
    with np.errstate(all="ignore"):
        tol = np.where(fine, UNIT[dt] * np.abs(want) + units * U * mag * (1 + UNIT[dt]) + TINY[dt], 0.0)
        over = fine & (np.abs(want) + units * U * mag >= EDGE[dt])
        must = fine & (np.abs(want) - units * U * mag >= EDGE[dt])
        near = fine & ~must & (np.abs(got - want) <= tol)
        infinite = over & np.isinf(got) & (np.sign(got) == np.sign(want))
    ok = near | infinite | (~fine & ((got == want) | (np.isnan(got) & np.isnan(want))))
    assert ok.all(), (dt, np.argwhere(~ok)[:5], got[~ok][:5], want[~ok][:5])
