"""Which kernels the attention operators launch, and how, for given calls: the host side alone, without a GPU.

As tests/launches.py does for the 8-bit operators: tests/launch_recorder.c takes the place of the HIP launch
interface in a process of its own.  A call is a dict; pointers are plain numbers, which nothing follows.
"""
import ctypes
import json
import os
import re
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
A = 1 << 40
TYPES = {"f16": 1, "bf16": 3, "f32": 4}
BATCH = dict(abi_version=8, dtype=1, heads=8, kv_heads=2, dim=128, page_size=16, tokens=4, seqs=4, max_kv_len=0, seq_starts=None,
             kv_lens=A, page_table=A, table_ld=64, table_pages=64, k_cache=A, v_cache=A, cache_pages=1000, page_stride=4096,
             head_stride=2048, token_stride=128)


def batch(**kw):
    assert set(kw) <= set(BATCH)
    return {**BATCH, **kw}


def attend(b, scale=0.1, window=0, lse=True):
    ld = b["heads"] * b["dim"]
    return {"name": "fluxbin_paged_attention", "batch": b, "args": [A, ld, scale, window, A, ld, A if lse else None, A, 72 << 20]}


def append(b, norm=False, rot=None, pairs=0, q=True):
    q_ld, k_ld = b["heads"] * b["dim"], b["kv_heads"] * b["dim"]
    n = A if norm else None
    return {"name": "fluxbin_rope_append", "batch": b,
            "args": [A if q else None, q_ld, A, k_ld, A, k_ld, n, n, 1e-5, A, b["dim"] if rot is None else rot, pairs, 1.0, None,
                     A if q else None, q_ld]}


def adjust(rows, vocab, dt="f16", biases=0, history=100):
    return {"name": "fluxbin_adjust_logits", "batch": None,
            "args": [A, vocab, TYPES[dt], rows, vocab, A if history else None, history, history, None, None, None, None, None,
                     A if biases else None, A if biases else None, biases, biases, A, (vocab + 31) // 32, A, vocab]}


def record(calls):
    """(all kernels of the library, for every call its status, workspace size and launches as dicts)."""
    with tempfile.TemporaryDirectory() as tmp:
        so = os.path.join(tmp, "recorder.so")
        subprocess.run(["gcc", "-std=c11", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-o", so,
                        os.path.join(HERE, "launch_recorder.c")], check=True)
        res = subprocess.run([sys.executable, os.path.abspath(__file__), so], input=json.dumps(calls), capture_output=True,
                             text=True, cwd=ROOT, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    kernels, results = json.loads(res.stdout)
    names = sorted(set(kernels))
    out = subprocess.run(["c++filt"], input="\n".join(names), capture_output=True, text=True, check=True).stdout.split("\n")
    plain = {n: re.sub(r"fluxbin::|^void |\(.*$", "", o) for n, o in zip(names, out)}
    for r in results:
        for launch in r["launches"]:
            launch["kernel"] = plain.get(launch["kernel"], launch["kernel"])
    return sorted(plain.values()), results


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
    for c in json.load(sys.stdin):
        args, need = list(c["args"]), None
        if c["batch"] is not None:
            b = F.PagedBatch(**c["batch"])
            args.insert(0, ctypes.byref(b))
            if c["name"] == "fluxbin_paged_attention":
                size = ctypes.c_size_t(0)
                need = size.value if F.raw_status("fluxbin_paged_attention_workspace_size", ctypes.byref(b), ctypes.byref(size)) else size.value
        rec.recorder_start(0)
        st = F.raw_status(c["name"], *args, None)
        launches = []
        for i in range(rec.recorder_count()):
            l = rec.recorder_launch(i).contents
            launches.append({"kernel": l.kernel.decode(), "grid": list(l.grid), "block": list(l.block)})
        out.append({"status": st, "error": F.fluxbin_last_error(), "workspace": need, "launches": launches})
    print(json.dumps([[rec.recorder_kernel(i).decode() for i in range(rec.recorder_kernels())], out]))


if __name__ == "__main__":
    _main()
