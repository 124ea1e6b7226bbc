"""fluxbin_adjust_logits against its definition in 64 bits (numpy on the host)."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.attention_cases import DT, TINY, U, UNIT, f64  # noqa: E402


@pytest.fixture(scope="module")
def fb():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible GPU")
    from binary_basis_lut_amd import fluxbin
    return fluxbin


def note(msg):
    print(f"[case] {msg}", flush=True)


def code(fb, dt):
    return {"f16": fb.DT_F16, "bf16": fb.DT_BF16, "f32": fb.DT_F32}[dt]


class Case:
    """Rows with histories, penalties, biases and a mask; any of them may be None afterwards."""

    def __init__(self, dt, rows, vocab, hist, biases, seed=0):
        r = self.r = np.random.default_rng(seed)
        self.dt, self.rows, self.vocab, self.hist, self.biases = dt, rows, vocab, hist, biases
        g = torch.Generator().manual_seed(seed)
        self.x = (torch.randn(rows, vocab, generator=g) * 4).to(DT[dt])
        # from all of the vocabulary, again and again from a few places, and some outside it
        self.history = r.integers(0, vocab, (rows, hist)).astype(np.int32)
        again = r.random((rows, hist)) < 0.5
        self.history[again] = r.integers(0, min(vocab, 5), again.sum())
        outside = r.random((rows, hist)) < 0.1
        self.history[outside] = r.choice([-1, vocab, 2 ** 31 - 1, -2 ** 31], outside.sum())
        self.prompt = r.integers(0, hist + 1, rows).astype(np.int32)
        self.total = r.integers(0, hist + 1, rows).astype(np.int32)
        self.rep = (0.5 + r.random(rows) * 1.5).astype(np.float32)
        self.freq, self.pres = (r.standard_normal(rows).astype(np.float32) for _ in range(2))
        self.bi = r.integers(0, vocab, (rows, biases)).astype(np.int32)
        if biases > 3:
            self.bi[:, 3] = self.bi[:, 1]
            self.bi[:, -1] = self.bi[:, 0]
            self.bi[:, 2] = r.choice([-1, vocab, -2 ** 31])
        self.bv = r.standard_normal((rows, biases)).astype(np.float32) * 3
        self.mask = r.integers(0, 1 << 32, (rows, -(-vocab // 32)), dtype=np.uint64).astype(np.uint32)

    def run(self, fb, in_place=False, stride=0, stream=None):
        up = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a).view(  # noqa: E731
            np.int32 if a.dtype == np.uint32 else a.dtype)).cuda()
        ld = self.vocab + stride
        x = torch.full((self.rows, ld), 5.0, dtype=DT[self.dt], device="cuda")
        x[:, :self.vocab] = self.x.cuda()
        out = x if in_place else torch.full((self.rows, ld), 5.0, dtype=DT[self.dt], device="cuda")
        t = [up(a) for a in (self.history, self.prompt, self.total, self.rep, self.freq, self.pres, self.bi, self.bv, self.mask)]
        h, nb = 0 if self.history is None else self.hist, 0 if self.bi is None else self.biases
        torch.cuda.synchronize()
        fb.fluxbin_adjust_logits(x, ld, code(fb, self.dt), self.rows, self.vocab, t[0], h, h, t[1], t[2], t[3], t[4], t[5], t[6], t[7],
                                 nb, nb, t[8], -(-self.vocab // 32), out, ld, stream)
        torch.cuda.synchronize()
        assert (out[:, self.vocab:] == 5).all()
        if not in_place:
            assert torch.equal(x[:, :self.vocab].cpu().view(torch.uint8), self.x.view(torch.uint8))
        return f64(out[:, :self.vocab])

    def want(self):
        z = f64(self.x)
        mag = np.abs(z)
        masked = np.zeros(z.shape, dtype=bool)
        with np.errstate(all="ignore"):
            for i in range(self.rows):
                given, made = np.zeros(self.vocab, dtype=bool), np.zeros(self.vocab)
                if self.history is not None:
                    n = self.hist if self.total is None else self.total[i]
                    p = 0 if self.prompt is None else self.prompt[i]
                    for k, tok in enumerate(self.history[i, :n]):
                        if 0 <= tok < self.vocab:
                            if k < p:
                                given[tok] = True
                            else:
                                made[tok] += 1
                seen = given | (made > 0)
                rho = 1.0 if self.rep is None else float(self.rep[i])
                z[i] = np.where(seen, np.where(z[i] > 0, z[i] / rho, z[i] * rho), z[i])
                mag[i] = np.where(seen, np.maximum(mag[i], np.abs(z[i])), mag[i])
                for f, c in ((self.freq, made), (self.pres, made > 0)):
                    if f is not None:
                        z[i] -= np.where(made > 0, float(f[i]) * c, 0.0)
                        mag[i] += abs(float(f[i])) * c
                if self.bi is not None:
                    for tok, v in zip(self.bi[i], self.bv[i]):
                        if 0 <= tok < self.vocab:
                            z[i, tok] += float(v)
                            mag[i, tok] += abs(float(v))
                if self.mask is not None:
                    bits = np.unpackbits(self.mask[i].view(np.uint8), bitorder="little")[:self.vocab]
                    masked[i] = bits == 0
        return np.where(masked, -np.inf, z), mag


def check(c, got):
    want, mag = c.want()
    # roundings: the quotient or product, two penalties of two each, the sum of the biases of one token and its addition
    units = 6 + (c.biases if c.bi is not None else 0)
    with np.errstate(all="ignore"):
        ok = np.abs(got - want) <= UNIT[c.dt] * np.abs(want) + units * U * mag * (1 + UNIT[c.dt]) + TINY[c.dt]
    ok |= got == want
    ok |= np.isnan(got) & np.isnan(want)
    assert ok.all(), np.argwhere(~ok)[:5]


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab", [1, 5, 7, 8, 9, 31, 33, 1000, 4095, 4096, 4097, 4099, 8192, 12293, 32000])
def test_everything(fb, dt, vocab):
    note(f"adjust_logits {dt} {vocab}")
    for i, (hist, biases) in enumerate([(1, 1), (300, 20), (2000, 0), (0, 5)]):
        c = Case(dt, 4, vocab, max(hist, 1), biases, seed=vocab + i)
        if hist == 0:
            c.history = None
        if biases == 0:
            c.bi = None
        check(c, c.run(fb, in_place=i % 2 == 1, stride=(0, 1, 3, 8)[i]))


@pytest.mark.parametrize("left", ["history", "prompt", "total", "rep", "freq", "pres", "bi", "mask", "all"])
def test_what_may_be_left_out(fb, left):
    note(f"adjust_logits without {left}")
    for dt in ("f16", "f32"):
        c = Case(dt, 3, 5003, 400, 12, seed=7)
        for n in ("history", "prompt", "total", "rep", "freq", "pres", "bi", "mask"):
            if left in (n, "all"):
                setattr(c, n, None)
        check(c, c.run(fb))


def test_without_anything_the_logits_are_copied(fb):
    c = Case("bf16", 3, 5003, 4, 4, seed=1)
    c.x.view(torch.int16).copy_(torch.randint(-2 ** 15, 2 ** 15, c.x.shape, generator=torch.Generator().manual_seed(0)).to(torch.int16))
    for n in ("history", "prompt", "total", "rep", "freq", "pres", "bi", "mask"):
        setattr(c, n, None)
    got, x = c.run(fb), f64(c.x)
    assert np.array_equal(got, x, equal_nan=True)


def test_special_logits_and_lengths(fb):
    note("adjust_logits, infinities, NaN, lengths out of range")
    for dt in ("f16", "bf16", "f32"):
        c = Case(dt, 5, 4500, 100, 8, seed=3)
        c.x[:, ::7] = -math.inf
        c.x[:, 3::11] = math.inf
        c.x[:, 5::13] = math.nan
        c.x[:, 6::17] = torch.finfo(DT[dt]).min
        c.x[:, 8::19] = 0.0
        c.total[:3], c.prompt[2:4] = (100, 0, 50), (0, 100)
        got = c.run(fb)
        check_overflow = f64(c.x)
        want, _ = c.want()
        if dt == "f16":  # beyond fp16's largest number: the infinity of the sign
            over = np.abs(want) > 65519
            assert (np.isinf(got[over & ~np.isnan(want)])).all()
            got = np.where(over, want, got)
        if dt != "f16":
            big = np.abs(check_overflow) > 1e38
            got = np.where(big, want, got)  # times a penalty: past the type's range, or not
        check(c, got)
        c.total[:] = (1 << 30, -5, 101, 100, 0)
        c.prompt[:] = (-3, 5, 1 << 30, 7, -1)
        got = c.run(fb)
        c.total, c.prompt = c.total.clip(0, 100), c.prompt.clip(0, 100)
        again = c.run(fb)
        assert np.array_equal(got, again, equal_nan=True)


def test_many_rows_and_biases(fb):
    note("adjust_logits, 700 rows; 4096 biases with repeats")
    check(*(lambda c: (c, c.run(fb)))(Case("f16", 700, 333, 40, 3, seed=2)))
    c = Case("f32", 2, 6000, 10, 4096, seed=4)
    check(c, c.run(fb))


def test_repeats_and_graphs(fb):
    note("adjust_logits in a graph")
    c = Case("f32", 6, 20000, 900, 30, seed=5)
    want = c.run(fb)
    for _ in range(3):
        assert np.array_equal(c.run(fb), want)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a).view(np.int32 if a.dtype == np.uint32 else a.dtype)).cuda()  # noqa: E731
    t = [up(a) for a in (c.history, c.prompt, c.total, c.rep, c.freq, c.pres, c.bi, c.bv, c.mask)]
    x, out = c.x.cuda(), torch.empty_like(c.x, device="cuda")
    args = (x, 20000, fb.DT_F32, 6, 20000, t[0], 900, 900, *t[1:6], t[6], t[7], 30, 30, t[8], 625, out, 20000)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.fluxbin_adjust_logits(*args)
    for i in range(3):
        out.fill_(i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(f64(out), want)
