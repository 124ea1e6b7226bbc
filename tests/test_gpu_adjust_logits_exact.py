"""fluxbin_adjust_logits where the definition gives infinities and NaN: each has to be the same one."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.adjust_compare import MOST, compare  # noqa: E402
from tests.attention_cases import DT, f64  # noqa: E402
from tests.test_gpu_adjust_logits import Case, fb, note  # noqa: E402,F401


def check(c, got):
    want, mag = c.want()
    compare(c.dt, got, want, mag, 6 + (c.biases if c.bi is not None else 0))
    return want


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab", [1, 5, 7, 8, 9, 31, 33, 1000, 4095, 4096, 4097, 4099, 8192, 8195, 12293, 16385, 32000])
def test_forbidden_tokens(fb, dt, vocab):  # noqa: F811
    """Everything at once, a mask alone, and a mask that forbids all of a row or nothing of it."""
    note(f"adjust_logits, forbidden tokens, {dt} {vocab}")
    for i, (hist, biases) in enumerate([(1, 1), (300, 20), (2000, 0), (0, 5), (0, 0)]):
        c = Case(dt, 4, vocab, max(hist, 1), biases, seed=100 + vocab + i)
        c.mask[1], c.mask[2] = 0, 0xffffffff
        if hist == 0:
            c.history = None
        if biases == 0:
            c.bi = None
        want = check(c, c.run(fb, in_place=i % 2 == 1, stride=(0, 1, 3, 8, 0)[i]))
        assert np.isneginf(want[1]).all() and np.isfinite(want[2]).all()


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("mask", [False, True])
def test_infinite_logits_and_ends_of_the_type(fb, dt, mask):  # noqa: F811
    """-inf, inf, NaN, zeros and the type's largest numbers, which penalties and biases may push beyond it."""
    note(f"adjust_logits, special logits, {dt}, mask {mask}")
    c = Case(dt, 5, 4500, 100, 8, seed=11)
    big = torch.finfo(DT[dt]).max
    for start, step, v in ((0, 7, -math.inf), (3, 11, math.inf), (5, 13, math.nan), (6, 17, -big), (8, 19, big), (9, 23, 0.0), (10, 29, big / 2)):
        c.x[:, start::step] = v
    # every kind of logit comes up in the history, and under a bias that may carry it beyond the type
    c.history[:, :60] = np.concatenate([np.arange(s, s + 6 * 7 * 11, 7 * 11) for s in (0, 3, 5, 6, 8, 9, 10, 17, 25, 39)])[None]
    c.total[:], c.prompt[:] = (100, 60, 30, 100, 0), (0, 30, 30, 100, 0)
    c.bi[:, :] = (6, 8, 0, 3, 5, 9, 8 + 19, 6 + 17)
    c.bv[:, :] = (-MOST[dt] / 3, MOST[dt] / 3, 1.0, -1.0, 2.0, MOST[dt], -1.0, 1.0)
    if not mask:
        c.mask = None
    want = check(c, c.run(fb))
    x = f64(c.x)
    assert np.isnan(want).any() and (want == np.inf).any() and (want == -np.inf).any() and (np.abs(want[np.isfinite(want)]) > MOST[dt]).any()
    assert np.isfinite(x[:, 6]).all()


def test_infinite_biases(fb):  # noqa: F811
    """A bias of -inf forbids as a mask does; one of +inf leaves no other choice."""
    note("adjust_logits, infinite biases")
    for dt in ("f16", "bf16", "f32"):
        c = Case(dt, 3, 700, 50, 6, seed=12)
        c.bi[:, :] = (1, 2, 650, 650, 699, 8)
        c.bv[:, :] = (-np.inf, np.inf, -np.inf, 5.0, np.inf, np.nan)
        want = check(c, c.run(fb))
        free = np.unpackbits(c.mask.view(np.uint8), axis=1, bitorder="little")[:, :700] == 1
        assert np.isneginf(want[:, 1]).all() and (want[:, 2][free[:, 2]] == np.inf).all()
