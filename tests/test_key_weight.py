"""The weight of a single key (csrc/key_weight.hpp) on the host, over the ends of fp32."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "binary_basis_lut_amd", "csrc")
SOURCE = """
#include "key_weight.hpp"
extern "C" void weights(int n, const bool *there, const float *s, const float *m, const float *c, float *w) {
  for (int i = 0; i < n; ++i) w[i] = fluxbin::key_weight(there[i], s[i], m[i], c[i]);
}
"""


@pytest.fixture(scope="module")
def weights(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    d = tmp_path_factory.mktemp("weights")
    (d / "w.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-ffp-contract=off", "-shared", "-fPIC", "-I", CSRC, "-o", str(d / "w.so"),
                    str(d / "w.cpp")], check=True)
    lib = ctypes.CDLL(str(d / "w.so"))

    def run(there, s, m, c):
        a = [np.ascontiguousarray(x, dtype=t) for x, t in zip(np.broadcast_arrays(there, s, m, c), (np.bool_, *3 * [np.float32]))]
        w = np.empty(a[0].shape, dtype=np.float32)
        lib.weights(w.size, *(x.ctypes.data_as(ctypes.c_void_p) for x in (*a, w)))
        return w

    return run


M = np.array([0, 1, 1e-40, 3e8, 2.7e8, 1e20, 3.4e38], dtype=np.float32)
C = np.array([1e-45, 1e-30, 1.44, 1.44e30], dtype=np.float32)  # scale is at most 1e30


def test_a_key_that_is_not_there_weighs_nothing(weights):
    """Its score is -inf.  Only a weight other than 0 makes the kernel look for a key's values."""
    m, c = (x.ravel() for x in np.meshgrid(np.concatenate([M, -M, [np.inf]]), C))
    assert (weights(False, -np.inf, m, c) == 0).all()


def test_weights_over_all_of_fp32(weights):
    """2^(c (s - m) + 7): the difference rounds once, its product and the sum once more."""
    m, d, c = (x.ravel() for x in np.meshgrid(np.concatenate([M, -M]), [0, 1e-38, 1e-30, 1e-20, 0.5, 1, 3, 40, 1e10, 1e38, 3.4e38], C))
    with np.errstate(all="ignore"):
        s = (m - d.astype(np.float32)).astype(np.float32)
    s = np.maximum(s, -np.finfo(np.float32).max)
    got = weights(True, s, m, c).astype(np.float64)
    e = np.maximum(c.astype(np.float64) * (s.astype(np.float64) - m.astype(np.float64)) + 7, -2000)  # 2^-2000 is 0
    want = np.exp2(e)
    tol = want * (np.exp2(3 * 2.0 ** -24 * (np.abs(e) + 14)) - 1 + 2.0 ** -22) + 2.0 ** -149
    off = ~(np.abs(got - want) <= tol)
    assert not off.any(), np.stack([m, s, c, got, want], 1)[off][:5]
    assert (weights(True, np.float32(-np.inf), m, c) == 0).all()
