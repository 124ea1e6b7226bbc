"""Host-side checks of the 8-bit operators: every refusal happens before any launch (no GPU needed)."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # an aligned stand-in address: a refused call never looks at it


@pytest.fixture(scope="module")
def fb():
    from binary_basis_lut_amd import build as B
    if B.is_stale():
        B.build()
    from binary_basis_lut_amd import fluxbin
    return fluxbin


def refused(fb, name, args, status):
    st = fb.raw_status(name, *args.values())
    assert st == status, (st, fb.fluxbin_last_error())
    assert fb.fluxbin_last_error()


def quant_args(**kw):
    d = dict(x=A, ldx=64, dtype=1, rows=4, cols=64, q=A, ldq=64, scale=A, stream=None)
    assert set(kw) <= set(d)
    d.update(kw)
    return d


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), 2), (dict(dtype=2), 2), (dict(dtype=5), 2), (dict(rows=-1), 1), (dict(cols=0), 1),
    (dict(cols=(1 << 30) + 1), 2), (dict(x=None), 1), (dict(q=None), 1), (dict(scale=None), 1), (dict(ldx=63), 1),
    (dict(ldq=63), 1), (dict(x=A + 1), 1), (dict(dtype=4, x=A + 2), 1), (dict(scale=A + 2), 1),
])
def test_quantize_rows_refuses(fb, kw, status):
    refused(fb, "fluxbin_quantize_rows", quant_args(**kw), status)


def norm_args(**kw):
    d = dict(x=A, ldx=64, residual=A, ldr=64, weight=A, dtype=1, rows=4, cols=64, eps=1e-5, residual_out=A, ldro=64, y=A,
             ldy=64, q=A, ldq=64, scale=A, stream=None)
    assert set(kw) <= set(d)
    d.update(kw)
    return d


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 2), (dict(rows=-1), 1), (dict(cols=0), 1), (dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(y=None, q=None), 1), (dict(residual=None), 1), (dict(x=None), 1),
    (dict(weight=None), 1), (dict(scale=None), 1), (dict(ldx=63), 1), (dict(ldr=63), 1), (dict(ldro=63), 1),
    (dict(ldy=63), 1), (dict(ldq=63), 1), (dict(x=A + 1), 1), (dict(weight=A + 1), 1), (dict(residual=A + 1), 1),
    (dict(residual_out=A + 1), 1), (dict(y=A + 1), 1), (dict(scale=A + 1), 1),
])
def test_add_rmsnorm_refuses(fb, kw, status):
    refused(fb, "fluxbin_add_rmsnorm", norm_args(**kw), status)


def gemm_args(**kw):
    d = dict(a=A, lda=64, a_scale=A, w=A, ldw=64, w_scale=A, bias=None, m=4, n=8, k=64, y=A, ldy=8, dtype=1, stream=None)
    assert set(kw) <= set(d)
    d.update(kw)
    return d


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), 2), (dict(m=-1), 1), (dict(n=-1), 1), (dict(k=0), 1), (dict(k=131072, lda=131072, ldw=131072), 2),
    (dict(m=(1 << 27) + 1), 2), (dict(n=(1 << 27) + 1), 2), (dict(a=None), 1), (dict(w=None), 1), (dict(a_scale=None), 1),
    (dict(w_scale=None), 1), (dict(y=None), 1), (dict(a=A + 8), 1), (dict(w=A + 8), 1), (dict(lda=72), 1), (dict(ldw=72), 1),
    (dict(lda=48), 1), (dict(k=65, lda=80), 1), (dict(ldy=7), 1), (dict(y=A + 1), 1), (dict(dtype=4, y=A + 2), 1),
    (dict(bias=A + 2), 1), (dict(a_scale=A + 1), 1), (dict(w_scale=A + 1), 1),
])
def test_gemm_w8a8_refuses(fb, kw, status):
    refused(fb, "fluxbin_gemm_w8a8", gemm_args(**kw), status)


def score_args(**kw):
    d = dict(logits=A, ld=32000, dtype=1, rows=4, vocab=32000, logit_scale=1.0, targets=A, logprob=A, entropy=A, top_k=5,
             top_logprob=A, top_index=A, workspace=A, workspace_bytes=1 << 22, stream=None)
    assert set(kw) <= set(d)
    d.update(kw)
    d["workspace_bytes"] = ctypes.c_size_t(d["workspace_bytes"])
    return d


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 2), (dict(rows=-1), 1), (dict(rows=(1 << 22) + 1), 2), (dict(vocab=0), 1), (dict(vocab=(1 << 28) + 1), 2),
    (dict(top_k=-1), 1), (dict(top_k=65), 2), (dict(vocab=4, top_k=5), 1), (dict(logit_scale=0.0), 1),
    (dict(logit_scale=-1.0), 1), (dict(logit_scale=float("nan")), 1), (dict(logit_scale=float("inf")), 1),
    (dict(targets=None), 1), (dict(logprob=None), 1), (dict(targets=None, logprob=None, entropy=None, top_k=0), 1),
    (dict(logits=None), 1), (dict(top_index=None), 1), (dict(top_logprob=None), 1), (dict(ld=31999), 1),
    (dict(logits=A + 1), 1), (dict(targets=A + 4), 1), (dict(logprob=A + 2), 1), (dict(entropy=A + 2), 1),
    (dict(top_index=A + 4), 1), (dict(top_logprob=A + 2), 1), (dict(vocab=300000, ld=300000, workspace=None), 3),
    (dict(vocab=300000, ld=300000, workspace_bytes=8), 3), (dict(vocab=300000, ld=300000, workspace=A + 8), 1),
])
def test_token_logprobs_refuses(fb, kw, status):
    refused(fb, "fluxbin_token_logprobs", score_args(**kw), status)


def test_zero_sizes_are_no_ops(fb):
    assert fb.raw_status("fluxbin_quantize_rows", *quant_args(rows=0, x=None, q=None, scale=None).values()) == fb.OK
    assert fb.raw_status("fluxbin_add_rmsnorm", *norm_args(rows=0).values()) == fb.OK
    assert fb.raw_status("fluxbin_gemm_w8a8", *gemm_args(m=0, a=None, y=None).values()) == fb.OK
    assert fb.raw_status("fluxbin_gemm_w8a8", *gemm_args(n=0, w=None, y=None).values()) == fb.OK
    assert fb.raw_status("fluxbin_token_logprobs", *score_args(rows=0, logits=None).values()) == fb.OK


def test_logprob_workspace_stays_small(fb):
    size = fb.fluxbin_token_logprobs_workspace_size
    for rows in (0, 1, 2, 3, 7, 64, 333, 512, 1024, 4096, 1 << 22):
        for vocab in (1, 255, 2048, 2049, 32000, 131072, 262144, 1 << 28):
            for top_k in (0, 1, 20, 64):
                if top_k <= vocab:
                    assert size(rows, vocab, top_k) <= 4 << 20
    assert size(4096, 32000, 5) == 0  # enough rows: one workgroup each
    with pytest.raises(fb.FluxbinError):
        size(1, 4, 5)
    assert fb.raw_status("fluxbin_token_logprobs_workspace_size", 1, 100, 5, None) == fb.ERR_INVALID_ARGUMENT


C_PROGRAM = r"""
#include <stdio.h>
#include "fluxbin.h"
int main(void) {
  size_t ws = 1;
  if (fluxbin_token_logprobs_workspace_size(4096, 32000, 5, &ws) != FLUXBIN_OK || ws != 0) return 1;
  if (fluxbin_quantize_rows(NULL, 8, FLUXBIN_DT_BF16, 0, 8, NULL, 8, NULL, NULL) != FLUXBIN_OK) return 2;
  if (fluxbin_add_rmsnorm(NULL, 8, NULL, 8, NULL, FLUXBIN_DT_F32, 1, 8, 0.0f, NULL, 8, NULL, 8, NULL, 8, NULL, NULL) !=
      FLUXBIN_ERR_INVALID_ARGUMENT) return 3;
  if (fluxbin_gemm_w8a8(NULL, 16, NULL, NULL, 16, NULL, NULL, 1, 1, 16, NULL, 1, FLUXBIN_DT_F16, NULL) !=
      FLUXBIN_ERR_INVALID_ARGUMENT) return 4;
  if (fluxbin_token_logprobs(NULL, 8, FLUXBIN_DT_F16, 1, 8, 1.0f, NULL, NULL, NULL, 0, NULL, NULL, NULL, 0, NULL) !=
      FLUXBIN_ERR_INVALID_ARGUMENT) return 5;
  printf("%s\n", fluxbin_last_error());
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_plain_c_program_reaches_the_operators(fb, tmp_path):
    src, exe = tmp_path / "ops.c", tmp_path / "ops"
    src.write_text(C_PROGRAM)
    lib = str(fb.LIB_PATH.parent)
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    "-o", str(exe), str(src), "-L", lib, "-lfluxbin", f"-Wl,-rpath,{lib}"], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.returncode
    assert "nothing to write" in res.stdout
