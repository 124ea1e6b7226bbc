"""Which kernels the library launches, and how, for given calls: the host side alone, without a GPU.

`record(calls)` runs them in a process of its own, where tests/launch_recorder.c stands in for the HIP
launch interface.  A call is (entry point, its arguments up to the stream); pointers are plain numbers,
which nothing follows.
"""
import ctypes
import json
import os
import re
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
A = 1 << 40  # a stand-in address, aligned for everything


class GemmArgs(ctypes.Structure):
    """csrc/gemm_w8a8_kernel.hpp"""
    _fields_ = [(n, ctypes.c_void_p) for n in ("a", "w", "a_scale", "w_scale", "bias", "y")] + \
               [(n, ctypes.c_int64) for n in ("lda", "ldw", "ldy")] + [(n, ctypes.c_int32) for n in ("m", "n", "k")]


class LogprobArgs(ctypes.Structure):
    """csrc/logprob_kernels.hpp"""
    _fields_ = [(n, ctypes.c_void_p) for n in ("logits", "targets", "logprob", "entropy", "top_logprob", "top_index", "workspace")] + \
               [(n, ctypes.c_int64) for n in ("rows", "ld")] + \
               [(n, ctypes.c_int32) for n in ("vocab", "top_k", "splits", "split_len")] + [("scale", ctypes.c_float)]


ARGS = {"fluxbin_gemm_w8a8": GemmArgs, "fluxbin_token_logprobs": LogprobArgs}
TYPES = {"f16": 1, "bf16": 3, "f32": 4}


def available():
    return shutil.which("gcc") is not None and shutil.which("c++filt") is not None


def gemm(m, n, k, dt="f16", lda=None, ldw=None, bias=True):
    ld = (k + 15) // 16 * 16
    return ["fluxbin_gemm_w8a8", [A, lda or ld, A, A, ldw or ld, A, A if bias else None, m, n, k, A, n, TYPES[dt]]]


def score(rows, vocab, top_k, dt="f16"):
    return ["fluxbin_token_logprobs", [A, vocab, TYPES[dt], rows, vocab, 1.0, A, A, A, top_k, A, A, A, 4 << 20]]


def _demangled(names):
    out = subprocess.run(["c++filt"], input="\n".join(names), capture_output=True, text=True, check=True).stdout.split("\n")
    return {n: re.sub(r"fluxbin::|^void |\(.*$", "", o) for n, o in zip(names, out)}


def record(calls):
    """(all kernels of the library, for every call its status and its launches as dicts)."""
    with tempfile.TemporaryDirectory() as tmp:
        so = os.path.join(tmp, "recorder.so")
        subprocess.run(["gcc", "-std=c11", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-o", so,
                        os.path.join(HERE, "launch_recorder.c")], check=True)
        res = subprocess.run([sys.executable, os.path.abspath(__file__), so], input=json.dumps(calls), capture_output=True,
                             text=True, cwd=ROOT, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    kernels, results = json.loads(res.stdout)
    names = _demangled(sorted(set(kernels)))
    for r in results:
        for launch in r["launches"]:
            launch["kernel"] = names.get(launch["kernel"], launch["kernel"])
    return sorted(names.values()), results


def _main():
    class Launch(ctypes.Structure):
        _fields_ = [("kernel", ctypes.c_char_p), ("grid", ctypes.c_uint32 * 3), ("block", ctypes.c_uint32 * 3),
                    ("args", ctypes.c_uint8 * 256)]

    rec = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)  # before the library, whose calls then end here
    rec.recorder_launch.restype = ctypes.POINTER(Launch)
    rec.recorder_kernel.restype = ctypes.c_char_p
    rec.recorder_start.argtypes = [ctypes.c_size_t]
    sys.path.insert(0, ROOT)
    from binary_basis_lut_amd import fluxbin as F
    out = []
    for name, args in json.load(sys.stdin):
        kind = ARGS[name]
        rec.recorder_start(ctypes.sizeof(kind))
        st = F.raw_status(name, *args, None)
        launches = []
        for i in range(rec.recorder_count()):
            l = rec.recorder_launch(i).contents
            a = kind.from_buffer_copy(bytes(l.args))
            launches.append({"kernel": l.kernel.decode(), "grid": list(l.grid), "block": list(l.block),
                             "args": {n: getattr(a, n) for n, _ in kind._fields_}})
        out.append({"status": st, "error": F.fluxbin_last_error(), "launches": launches})
    print(json.dumps([[rec.recorder_kernel(i).decode() for i in range(rec.recorder_kernels())], out]))


if __name__ == "__main__":
    _main()
