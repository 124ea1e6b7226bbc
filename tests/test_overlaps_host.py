"""Outputs that overlap inputs: refused unless they are the same rows (no GPU needed)."""
import random

import pytest

from tests import attention_launches as L
from tests import launches as L8

pytestmark = pytest.mark.skipif(not L8.available(), reason="gcc and c++filt not available")

DIMS = dict(heads=2, kv_heads=1, dim=8, token_stride=8, head_stride=128, page_stride=128)  # rows of 16 elements


def attention(tokens, x, ldx, y, ldy):
    c = L.attend(L.batch(tokens=tokens, seqs=tokens, table_pages=4, **DIMS))
    c["args"][0], c["args"][1], c["args"][4], c["args"][5] = L.A + 2 * x, ldx, L.A + 2 * y, ldy
    return c


def append(tokens, x, ldx, y, ldy):
    c = L.append(L.batch(tokens=tokens, seqs=tokens, **DIMS))
    c["args"][0], c["args"][1], c["args"][-2], c["args"][-1] = L.A + 2 * x, ldx, L.A + 2 * y, ldy
    return c


def adjust(tokens, x, ldx, y, ldy):
    c = L.adjust(tokens, 16)
    c["args"][0], c["args"][1], c["args"][-2], c["args"][-1] = L.A + 2 * x, ldx, L.A + 2 * y, ldy
    return c


def meet(tokens, x, ldx, y, ldy):
    places = [{p + i * ld + e for i in range(tokens) for e in range(16)} for p, ld in ((x, ldx), (y, ldy))]
    return bool(places[0] & places[1])


def layouts():
    yield from [(4, 0, 16, 64, 16), (4, 0, 16, 63, 16), (4, 0, 32, 16, 32), (4, 0, 32, 15, 32), (4, 16, 32, 0, 32), (4, 17, 32, 0, 32),
                (4, 0, 16, 0, 16), (4, 0, 32, 0, 32), (4, 0, 32, 0, 16), (1, 0, 16, 15, 16), (1, 0, 16, 16, 99), (2, 0, 64, 16, 20),
                (4, 0, 32, 48, 32), (4, 0, 32, 128, 32), (4, 0, 32, 96, 40), (3, 0, 16, 100, 1 << 40), (3, 50, 1 << 62, 0, 16)]
    rng = random.Random(5)
    for _ in range(400):
        yield rng.randint(1, 6), rng.randint(0, 200), rng.randint(16, 70), rng.randint(0, 200), rng.randint(16, 70)
    for _ in range(200):
        ld = rng.randint(16, 70)
        yield rng.randint(1, 6), rng.randint(0, 200), ld, rng.randint(0, 200), ld


@pytest.mark.parametrize("op", [attention, append, adjust], ids=lambda f: f.__name__)
def test_overlapping_rows_are_refused_and_no_others(op):
    cases = list(layouts())
    answers = [0, 0]
    for case, r in zip(cases, L.record([op(*c) for c in cases])[1]):
        bad = meet(*case) and case[1:3] != case[3:5]
        assert (r["status"] == 1) == bad and bool(r["launches"]) == (not bad), (case, r)
        answers[bad] += 1
    assert min(answers) > 100
