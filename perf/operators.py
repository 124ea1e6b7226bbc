"""The 8-bit operators around the binary-basis layers, as cases to be timed and compared.

Four operators of one path: a token's activations are added to the residual stream, normalised and
quantised to int8 (`norm`), or quantised alone (`quant`), multiplied with an int8 weight matrix that
has a scale per output channel (`gemm`: a projection at prefill, or the output head), and the head's
logits are turned into log probabilities of given tokens with the entropy and the best alternatives
(`score`).

`run` computes a case either in a plain form (torch's elementary operations, 32-bit arithmetic, one
rounding at the end) or, where `own` is true, through `binary_basis_lut_amd.fluxbin`.

int8 results are returned as they are held, with their scales beside them: the quantisation rule
(see `_quantize`) leaves no freedom in the integers, so they are compared as whole numbers.
"""
import math

import torch

own = False  # set from outside: whether run() calls the library's kernels or computes the plain form

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
AMAX_FLOOR = 2.0 ** -100  # a row's largest magnitude counts as at least this, so that 127 / amax stays finite
EPS = 1e-5
WORKSPACE = 4 << 20  # bytes a program keeps for `score` at any size: the library asks for no more than this


def listed():
    return [
        # One token's attention output or MLP activation before an int8 projection: pure latency.
        {"name": "quant one token", "op": "quant", "dtype": "f16", "rows": 1, "cols": 11008},
        # Offline: a whole 70B down-projection matrix to int8, one scale per output channel.
        {"name": "quant weights 8192x28672", "op": "quant", "dtype": "f16", "rows": 8192, "cols": 28672},
        # One decode step's norm between two layers: latency.
        {"name": "norm one token", "op": "norm", "dtype": "f16", "rows": 1, "cols": 4096},
        # A ragged batch of prompts, bf16, with the normalised row kept beside its int8 form.
        {"name": "norm 333x5120 bf16", "op": "norm", "dtype": "bf16", "rows": 333, "cols": 5120, "keep": True},
        # A long prefill at the 70B hidden size.
        {"name": "norm 8192x8192", "op": "norm", "dtype": "f16", "rows": 8192, "cols": 8192},
        # One token through a 4096 x 4096 projection (decode): the weights are read once.
        {"name": "gemm 1x4096x4096", "op": "gemm", "dtype": "f16", "m": 1, "n": 4096, "k": 4096},
        # A decode batch through the output head, logits in 32 bits.
        {"name": "gemm 16x32000x4096 f32", "op": "gemm", "dtype": "f32", "m": 16, "n": 32000, "k": 4096},
        # A ragged prefill batch through the 7B down projection, with a bias.
        {"name": "gemm 333x4096x11008 bf16", "op": "gemm", "dtype": "bf16", "m": 333, "n": 4096, "k": 11008, "bias": True},
        # A long prefill through one 70B MLP matrix.
        {"name": "gemm 8192x28672x8192", "op": "gemm", "dtype": "f16", "m": 8192, "n": 28672, "k": 8192},
        # One generated token's log probability and five alternatives: latency.
        {"name": "score 1x32000", "op": "score", "dtype": "f16", "rows": 1, "vocab": 32000, "top": 5},
        # A decode batch over a large vocabulary, part of it masked out, twenty alternatives.
        {"name": "score 64x131072 bf16", "op": "score", "dtype": "bf16", "rows": 64, "vocab": 131072, "top": 20, "masked": True},
        # Perplexity of a 4096-token text: every position scored, padding positions without a target.
        {"name": "score 4096x32000 f32", "op": "score", "dtype": "f32", "rows": 4096, "vocab": 32000, "top": 1},
    ]


def _log_int(rng, lo, hi):
    """A whole number whose logarithm is spread evenly; half of them multiples of 64 where there is room."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v > 256 and rng.random() < 0.5:
        v = max(lo, v // 64 * 64)
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["quant", "norm", "norm", "gemm", "gemm", "gemm", "score", "score"])
    dtype = rng.choice(["f16", "f16", "bf16", "f32"])
    if op in ("quant", "norm"):
        cols = _log_int(rng, 64, 28672)
        most = (8192 * 28672 if op == "quant" else 8192 * 8192) * 2 // SIZE[dtype]
        case = {"op": op, "dtype": dtype, "rows": _log_int(rng, 1, max(1, min(65536, most // cols))), "cols": cols}
        if op == "norm":
            case["keep"] = rng.random() < 0.3
        return case
    if op == "gemm":
        n, k = _log_int(rng, 128, 57344), _log_int(rng, 64, 28672)
        most = min(8192, 8192 * 28672 * 8192 // (n * k) if dtype == "f16" else 4096 * 28672 * 8192 // (n * k))
        return {"op": op, "dtype": dtype, "m": _log_int(rng, 1, max(1, most)), "n": n, "k": k, "bias": rng.random() < 0.5}
    vocab = _log_int(rng, 256, 262144)
    most = 4096 * 32000 * 4 // (vocab * max(4, SIZE[dtype]))
    return {"op": op, "dtype": dtype, "rows": _log_int(rng, 1, max(1, min(16384, most))), "vocab": vocab,
            "top": rng.choice([0, 1, 5, 20, 64]), "masked": rng.random() < 0.3}


def _up16(v):
    return (v + 15) // 16 * 16


def _activations(g, rows, cols, dtype):
    """Normal values with 1 % of the channels twenty times as large, the profile of transformer activations."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    loud = torch.rand(cols, device="cuda", generator=g) < 0.01
    return (x * torch.where(loud, 20.0, 1.0)).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}
    empty = lambda *shape, **kw: torch.empty(*shape, device="cuda", **kw)  # noqa: E731
    if op in ("quant", "norm"):
        rows, cols = case["rows"], case["cols"]
        s["x"] = _activations(g, rows, cols, dt)
        s["q"] = empty(rows, _up16(cols), dtype=torch.int8)
        s["scale"] = empty(rows, dtype=torch.float32)
        if op == "norm":
            s["residual"] = (_activations(g, rows, cols, torch.float32) * 3).to(dt)
            s["weight"] = (1 + 0.1 * torch.randn(cols, device="cuda", generator=g)).to(dt)
            s["residual_out"] = empty(rows, cols, dtype=dt)
            s["y"] = empty(rows, cols, dtype=dt) if case.get("keep") else None
    elif op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        for name, r in (("a", m), ("w", n)):
            v = torch.randn(r, _up16(k), device="cuda", generator=g).mul_(32).round_().clamp_(-127, 127)
            s[name] = v.to(torch.int8)  # the columns past k, which pad a row to 16 bytes, hold no zeros on purpose
        s["a_scale"] = 0.01 + 0.02 * torch.rand(m, device="cuda", generator=g)
        s["w_scale"] = 0.001 * (0.5 + torch.rand(n, device="cuda", generator=g))
        s["bias"] = torch.randn(n, device="cuda", generator=g) if case.get("bias") else None
        s["y"] = empty(m, n, dtype=dt)
    else:
        rows, vocab, top = case["rows"], case["vocab"], case["top"]
        s["logits"] = torch.randn(rows, vocab, device="cuda", generator=g).mul_(3).to(dt)
        if case.get("masked"):
            s["logits"][:, torch.rand(vocab, device="cuda", generator=g) < 0.25] = -math.inf
        s["targets"] = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
        s["targets"][torch.rand(rows, device="cuda", generator=g) < 0.05] = -100
        s["logit_scale"] = 1.0 if seed % 2 else 1.25
        s["logprob"], s["entropy"] = empty(rows, dtype=torch.float32), empty(rows, dtype=torch.float32)
        s["top_logprob"] = empty(rows, top, dtype=torch.float32)
        s["top_index"] = empty(rows, top, dtype=torch.int64)
        s["workspace"] = empty(WORKSPACE, dtype=torch.uint8)
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from binary_basis_lut_amd import fluxbin as F
    case = s["case"]
    op, dt = case["op"], {"f16": F.DT_F16, "bf16": F.DT_BF16, "f32": F.DT_F32}[case["dtype"]]
    if op == "quant":
        rows, cols, ldq = case["rows"], case["cols"], s["q"].shape[1]
        F.fluxbin_quantize_rows(s["x"], cols, dt, rows, cols, s["q"], ldq, s["scale"])
        return {"q": s["q"][:, :cols], "scale": s["scale"]}
    if op == "norm":
        rows, cols, ldq = case["rows"], case["cols"], s["q"].shape[1]
        F.fluxbin_add_rmsnorm(s["x"], cols, s["residual"], cols, s["weight"], dt, rows, cols, EPS, s["residual_out"], cols,
                              s["y"], cols, s["q"], ldq, s["scale"])
        out = {"q": s["q"][:, :cols], "scale": s["scale"], "residual": s["residual_out"]}
        if s["y"] is not None:
            out["y"] = s["y"]
        return out
    if op == "gemm":
        m, n, k, ld = case["m"], case["n"], case["k"], s["a"].shape[1]
        F.fluxbin_gemm_w8a8(s["a"], ld, s["a_scale"], s["w"], ld, s["w_scale"], s["bias"], m, n, k, s["y"], n, dt)
        return s["y"]
    rows, vocab, top = case["rows"], case["vocab"], case["top"]
    F.fluxbin_token_logprobs(s["logits"], vocab, dt, rows, vocab, s["logit_scale"], s["targets"], s["logprob"], s["entropy"],
                             top, s["top_logprob"], s["top_index"], s["workspace"], s["workspace"].numel())
    return _scores(s["logprob"], s["entropy"], s["top_logprob"], s["top_index"])


def _scores(logprob, entropy, top_logprob, top_index):
    out = {"logprob": logprob, "entropy": entropy}
    if top_index.shape[1]:
        out["top_logprob"], out["top_index"] = top_logprob, top_index
    return out


def _quantize(t):
    """Symmetric int8 of each row of t (32 bits): q = rint(t * (127 / amax)), and amax / 127."""
    amax = t.abs().amax(dim=1, keepdim=True).clamp_min(AMAX_FLOOR)
    full = torch.full_like(amax, 127.0)
    q = torch.round(t * torch.div(full, amax)).to(torch.int8)
    return q, torch.div(amax, full)[:, 0]


def _run_plain(s):
    case = s["case"]
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "quant":
        q, scale = _quantize(s["x"].float())
        return {"q": q, "scale": scale}
    if op == "norm":
        # The norm is taken of the sum as the residual stream holds it. The root mean square is a
        # factor of the whole row, so it cancels in the integers and enters the scale alone.
        held = (s["x"].float() + s["residual"].float()).to(dt)
        h, w = held.float(), s["weight"].float()
        inv = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS)
        q, scale = _quantize(h * w)
        out = {"q": q, "scale": scale * inv[:, 0], "residual": held}
        if case.get("keep"):
            out["y"] = (h * inv * w).to(dt)
        return out
    if op == "gemm":
        k = case["k"]
        y = (s["a"][:, :k].float() @ s["w"][:, :k].float().t()) * s["a_scale"][:, None] * s["w_scale"]
        return (y if s["bias"] is None else y + s["bias"]).to(dt)
    x = s["logits"].float() * s["logit_scale"]
    d = x - x.amax(dim=1, keepdim=True)
    e = torch.exp(d)
    total = e.sum(dim=1, keepdim=True)
    lp = d - torch.log(total)
    target = s["targets"]
    logprob = torch.where(target < 0, 0.0, lp.gather(1, target.clamp_min(0)[:, None])[:, 0])
    p = e / total
    entropy = -torch.where(p > 0, p * lp, 0.0).sum(dim=1)
    # Distinct keys of which the larger is the larger logit or, of equal ones, the lower index.
    bits = (s["logits"].float() + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64)
    keys = (order << 32) - torch.arange(case["vocab"], device=x.device)
    top = torch.topk(keys, min(case["top"], case["vocab"]), dim=1).indices
    return _scores(logprob, entropy, lp.gather(1, top), top)


def work(case):
    op, b = case["op"], SIZE[case["dtype"]]
    if op == "quant":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (b + 1) + 4 * case["rows"], "flops": 3 * n}
    if op == "norm":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (3 * b + 1 + (b if case.get("keep") else 0)) + 4 * case["rows"] + b * case["cols"],
                "flops": 8 * n}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + m * n * b + 4 * (m + n) + (4 * n if case.get("bias") else 0), "flops": 2 * m * n * k}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * b + case["rows"] * (16 + 12 * case["top"]), "flops": 6 * n}


def exact(case, seed):
    """The definition in 64 bits. The int8 integers and the token indices have no value here."""
    s, op = prepare(case, seed), case["op"]
    if op == "quant":
        largest = torch.maximum(s["x"].double().amax(1), -s["x"].double().amin(1))
        return {"q": None, "scale": torch.clamp(largest, min=AMAX_FLOOR) / 127}
    if op == "norm":
        dt = DTYPES[case["dtype"]]
        held = (s["x"].double() + s["residual"].double()).to(dt).double()
        rms = (held.pow(2).sum(1) / case["cols"] + EPS).sqrt()
        y = held * s["weight"].double() / rms[:, None]
        out = {"q": None, "scale": (held * s["weight"].double()).abs().amax(1).clamp(min=AMAX_FLOOR) / rms / 127, "residual": held}
        if case.get("keep"):
            out["y"] = y
        return out
    if op == "gemm":
        k = case["k"]
        a = s["a"][:, :k].double() * s["a_scale"].double()[:, None]
        w = s["w"][:, :k].double() * s["w_scale"].double()[:, None]
        y = torch.mm(a, w.t())
        return y if s["bias"] is None else y + s["bias"].double()
    x = s["logits"].double() * s["logit_scale"]
    lp = torch.log_softmax(x, dim=1)
    del x
    rows = torch.arange(case["rows"], device=lp.device)
    logprob = lp[rows, s["targets"].clamp(min=0)].masked_fill(s["targets"] < 0, 0.0)
    entropy = -(lp.exp() * lp.clamp(min=-1e4)).sum(1)
    out = {"logprob": logprob, "entropy": entropy}
    if case["top"]:
        out["top_logprob"] = torch.topk(lp, min(case["top"], case["vocab"]), dim=1).values
        out["top_index"] = None
    return out
