"""The operators between a decoder layer's products, and between the head and its scores, as cases.

`append`: the rows of a QKV product become queries, and keys and values of a paged cache (a norm of every
head where the model has one, the position rotation, the store to the cache's pages). `attend`: the new
tokens' attention over that cache, a chunk of tokens or one for each sequence. `adjust`: repetition,
frequency and presence penalties, biases and a grammar's mask on the logits before they are scored.

`run` computes a case either in a plain form (torch's elementary operations, 32-bit arithmetic, one
rounding at the end; 64 bits for the angles) or, where `own` is true, through
`binary_basis_lut_amd.fluxbin`.
"""
import math
import random

import torch

own = False  # set from outside: whether run() calls the library's kernels or computes the plain form

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-5
THETA = 10000.0
SPARE = 3  # pages of the cache that no sequence has


def listed():
    return [
        # One token of a 7B layer (32 heads, no sharing) between its QKV product and its attention: pure latency.
        {"name": "append one token", "op": "append", "dtype": "f16", "heads": 32, "kv": 32, "dim": 128, "seqs": 1, "new": 1,
         "past": 1000, "page": 16, "rot": 128, "pairs": "half"},
        # A decode batch, half of each head rotated by neighbours, positions of a long document given apart from the cache.
        {"name": "append 64 tokens, part", "op": "append", "dtype": "bf16", "heads": 48, "kv": 8, "dim": 128, "seqs": 64, "new": 1,
         "past": 300, "page": 32, "rot": 64, "pairs": "near", "far": 200000},
        # A long prefill at the 70B layer's heads (64, 8 shared), queries and keys normed: the bytes.
        {"name": "append 8192 tokens, normed", "op": "append", "dtype": "bf16", "heads": 64, "kv": 8, "dim": 128, "seqs": 2,
         "new": 4096, "past": 77, "page": 64, "rot": 128, "pairs": "half", "norm": True},
        # One sequence's next token at the 7B heads: a few thousand keys, little to share the work among.
        {"name": "attend one token over 4000", "op": "attend", "dtype": "f16", "heads": 32, "kv": 32, "dim": 128, "seqs": 1,
         "new": 1, "past": 4000, "page": 16},
        # A decode batch at the 70B heads, sequences of all lengths: the cache's bytes.
        {"name": "attend 64 tokens over 8192", "op": "attend", "dtype": "bf16", "heads": 64, "kv": 8, "dim": 128, "seqs": 64,
         "new": 1, "past": 8192, "ragged": True, "page": 64},
        # A whole prompt at the 7B heads: the matrix instructions.
        {"name": "attend 4096 new", "op": "attend", "dtype": "f16", "heads": 32, "kv": 32, "dim": 128, "seqs": 1, "new": 4096,
         "past": 0, "page": 64},
        # The last chunk of a long prompt, its log-sum-exp kept to be joined with other parts.
        {"name": "attend 517 new over 31000", "op": "attend", "dtype": "bf16", "heads": 64, "kv": 8, "dim": 128, "seqs": 1,
         "new": 517, "past": 31000, "page": 16, "lse": True},
        # Prompts of all lengths together, small heads, a sliding window.
        {"name": "attend 12 ragged, window 500", "op": "attend", "dtype": "f16", "heads": 16, "kv": 4, "dim": 64, "seqs": 12,
         "new": 1500, "past": 700, "ragged": True, "page": 32, "window": 500, "lse": True},
        # One generated token's logits with its penalties: latency.
        {"name": "adjust 1x32000", "op": "adjust", "dtype": "f16", "rows": 1, "vocab": 32000, "history": 600, "biases": 8},
        # A decode batch over a large vocabulary, every row under a grammar.
        {"name": "adjust 64x131072 bf16", "op": "adjust", "dtype": "bf16", "rows": 64, "vocab": 131072, "history": 4000,
         "biases": 50, "mask": True},
        # All positions of drafted tokens, logits in 32 bits as the int8 head gives them: the bytes.
        {"name": "adjust 2048x32000 f32", "op": "adjust", "dtype": "f32", "rows": 2048, "vocab": 32000, "history": 300,
         "biases": 0, "mask": True},
    ]


def _log_int(rng, lo, hi):
    """A whole number whose logarithm is spread evenly; half of them multiples of 64 where there is room."""
    hi = max(lo, int(hi))
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v > 256 and rng.random() < 0.5:
        v = max(lo, v // 64 * 64)
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "attend", "adjust", "adjust"])
    if op == "adjust":
        vocab = _log_int(rng, 256, 262144)
        return {"op": op, "dtype": rng.choice(["f16", "bf16", "f32"]), "rows": _log_int(rng, 1, min(4096, 2048 * 32000 // vocab)),
                "vocab": vocab, "history": _log_int(rng, 1, 4000), "biases": rng.choice([0, 0, 1, 17, 64]) if vocab > 1000 else 0,
                "mask": rng.random() < 0.5}
    dim, kv, group = rng.choice([64, 80, 96, 128, 128, 128, 256]), rng.choice([1, 2, 4, 8, 8, 32]), rng.choice([1, 1, 4, 6, 8, 16])
    group = min(group, 64 // kv)
    case = {"op": op, "dtype": rng.choice(["f16", "bf16"]), "heads": kv * group, "kv": kv, "dim": dim,
            "page": rng.choice([16, 32, 64, 128]), "ragged": rng.random() < 0.6}
    if op == "append":
        tokens = _log_int(rng, 1, min(16384, 8192 * 80 * 128 // ((group + 2) * kv * dim)))
        seqs = _log_int(rng, 1, min(256, tokens))
        case.update(seqs=seqs, new=max(1, tokens // seqs) if rng.random() < 0.7 else 1, past=rng.randrange(300),
                    rot=rng.choice([dim, dim, dim // 2, 32]), pairs=rng.choice(["half", "near"]), norm=rng.random() < 0.4)
        if rng.random() < 0.3:
            case["far"] = rng.choice([5000, 200000, 1000000])
        return case
    if rng.random() < 0.5:  # a decode step
        seqs = _log_int(rng, 1, 256)
        case.update(seqs=seqs, new=1, past=_log_int(rng, 1, min(32768, 64 * 8192 * 8 * 128 // (seqs * kv * dim))))
    else:
        new = _log_int(rng, 2, 4096)
        most = min(4096 * 2048 * 32 * 128 // (new * kv * group * dim), 64 * 517 * 31517 // (new * kv * group))  # pairs, scores
        past = rng.choice([0, _log_int(rng, 1, 32768)])
        past = max(0, min(past, most - new))
        new = min(new, most)
        seqs = min(32, most // (new + past), 64 * 8192 * 8 * 128 // ((new + past) * kv * dim))
        case.update(seqs=_log_int(rng, 1, max(1, seqs)), new=new, past=past)
    if rng.random() < 0.3:
        case["window"] = _log_int(rng, 1, 4096)
    case["lse"] = rng.random() < 0.3
    return case


def _lengths(case):
    """(new tokens, cached tokens before them) of every sequence: as the case has them, or spread up to them."""
    seqs, new, past = case["seqs"], case["new"], case["past"]
    if not case.get("ragged"):
        return [(new, past)] * seqs
    rng = random.Random(1000003 * seqs + 1009 * new + past)
    return [(new, past)] + [(rng.randint(1, new), rng.randint(0, past)) for _ in range(seqs - 1)]


def _up(v, m):
    return (v + m - 1) // m * m


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}
    randn = lambda *shape: torch.randn(*shape, device="cuda", generator=g)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    if op == "adjust":
        rows, vocab, hist, nb = case["rows"], case["vocab"], case["history"], case["biases"]
        s["logits"] = randn(rows, vocab).mul_(3).to(dt)
        # A few tokens come again and again; the last of each row's places are not filled.
        few = torch.rand(rows, hist, device="cuda", generator=g).pow_(3).mul_(vocab).to(torch.int32).clamp_(max=vocab - 1)
        total = torch.randint(max(1, hist // 2), hist + 1, (rows,), device="cuda", generator=g).to(torch.int32)
        s["history"] = torch.where(torch.arange(hist, device="cuda") < total[:, None], few, -1).contiguous()
        s["total"], s["prompt"] = total, total // 3
        s["repetition"] = 1 + 0.3 * torch.rand(rows, device="cuda", generator=g)
        s["frequency"] = torch.rand(rows, device="cuda", generator=g) * 0.5
        s["presence"] = torch.rand(rows, device="cuda", generator=g) - 0.3
        s["bias_index"] = s["bias_value"] = None
        if nb:
            first = torch.randint(0, vocab, (rows, 1), device="cuda", generator=g)
            s["bias_index"] = ((first + torch.arange(nb, device="cuda") * (vocab // nb)) % vocab).to(torch.int32)
            s["bias_value"] = randn(rows, nb) * 5
        s["mask"] = None
        if case.get("mask"):
            s["mask"] = torch.randint(-2 ** 31, 2 ** 31, (rows, (vocab + 31) // 32), device="cuda", generator=g).to(torch.int32)
        s["out"] = torch.empty_like(s["logits"])
        return s
    heads, kv, dim, page, seqs = case["heads"], case["kv"], case["dim"], case["page"], case["seqs"]
    lengths = _lengths(case)
    news, lens = [n for n, _ in lengths], [n + p for n, p in lengths]
    tokens, per_seq = sum(news), max(-(-n // page) for n in lens)
    s["starts"] = None if case["new"] == 1 else ints([sum(news[:i]) for i in range(seqs + 1)])
    s["lens"], s["most"] = ints(lens), max(lens)
    used = [-(-n // page) for n in lens]
    pages = sum(used) + SPARE
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    have = torch.arange(per_seq, device="cuda") < ints(used)[:, None]
    at = (have.cumsum(1) + ints([sum(used[:i]) for i in range(seqs)])[:, None] - 1).clamp_min(0)
    s["table"] = torch.where(have, order[at], -1).contiguous()
    s["k_cache"], s["v_cache"] = randn(pages, kv, page, dim).to(dt), randn(pages, kv, page, dim).to(dt)
    s["tokens"] = tokens
    if op == "append":
        s["qkv"] = randn(tokens, (heads + 2 * kv) * dim).to(dt)
        s["q_norm"] = s["k_norm"] = None
        if case.get("norm"):
            s["q_norm"], s["k_norm"] = ((1 + 0.1 * randn(dim)).to(dt) for _ in range(2))
        s["freq"] = THETA ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        s["positions"] = None
        if case.get("far"):
            s["positions"] = torch.randint(0, case["far"], (tokens,), device="cuda", generator=g).to(torch.int32)
        s["q_out"] = torch.empty(tokens, heads * dim, dtype=dt, device="cuda")
    else:
        s["q"] = (randn(tokens, heads * dim) * 1.5).to(dt)
        s["out"] = torch.empty(tokens, heads * dim, dtype=dt, device="cuda")
        s["lse"] = torch.empty(tokens, heads, dtype=torch.float32, device="cuda") if case.get("lse") else None
    if own:
        from binary_basis_lut_amd import fluxbin as F
        s["batch"] = b = F.PagedBatch()
        b.abi_version, b.dtype = F.ABI_VERSION, {"f16": F.DT_F16, "bf16": F.DT_BF16}[case["dtype"]]
        b.heads, b.kv_heads, b.dim, b.page_size = heads, kv, dim, page
        b.tokens, b.seqs, b.max_kv_len = tokens, seqs, s["most"]
        b.seq_starts = None if s["starts"] is None else s["starts"].data_ptr()
        b.kv_lens, b.page_table, b.table_ld, b.table_pages = s["lens"].data_ptr(), s["table"].data_ptr(), per_seq, per_seq
        b.k_cache, b.v_cache, b.cache_pages = s["k_cache"].data_ptr(), s["v_cache"].data_ptr(), pages
        b.page_stride, b.head_stride, b.token_stride = kv * page * dim, page * dim, dim
        if op == "attend":
            need = F.fluxbin_paged_attention_workspace_size(b)
            s["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from binary_basis_lut_amd import fluxbin as F
    case = s["case"]
    if case["op"] == "adjust":
        rows, vocab, hist, nb = case["rows"], case["vocab"], case["history"], case["biases"]
        dt = {"f16": F.DT_F16, "bf16": F.DT_BF16, "f32": F.DT_F32}[case["dtype"]]
        F.fluxbin_adjust_logits(s["logits"], vocab, dt, rows, vocab, s["history"], hist, hist, s["prompt"], s["total"],
                                s["repetition"], s["frequency"], s["presence"], s["bias_index"], s["bias_value"], nb, nb,
                                s["mask"], (vocab + 31) // 32, s["out"], vocab)
        return s["out"]
    b, heads, kv, dim = s["batch"], case["heads"], case["kv"], case["dim"]
    if case["op"] == "append":
        ld = (heads + 2 * kv) * dim
        x = s["qkv"]
        F.fluxbin_rope_append(b, x, ld, x[:, heads * dim:], ld, x[:, (heads + kv) * dim:], ld, s["q_norm"], s["k_norm"], EPS,
                              s["freq"], case["rot"], F.ROPE_HALF if case["pairs"] == "half" else F.ROPE_NEAR, 1.0,
                              s["positions"], s["q_out"], heads * dim)
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    F.fluxbin_paged_attention(b, s["q"], heads * dim, 1 / math.sqrt(dim), case.get("window", 0), s["out"], heads * dim, s["lse"],
                              s["workspace"], s["workspace"].numel())
    return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}


def _rows_of(s):
    """For every token its sequence, its number among that sequence's new tokens, and its index in the cache."""
    case, dev = s["case"], s["lens"].device
    starts = s["starts"] if s["starts"] is not None else torch.arange(case["seqs"] + 1, device=dev, dtype=torch.int32)
    row = torch.arange(s["tokens"], device=dev, dtype=torch.int32)
    seq = torch.searchsorted(starts, row, right=True) - 1
    nth = row - starts[seq]
    return seq, nth, s["lens"][seq] - (starts[seq + 1] - starts[seq]) + nth


def _run_plain(s):
    return {"append": _append, "attend": _attend, "adjust": _adjust}[s["case"]["op"]](s)


def _normed(x, w):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _rotated(x, c, sn, rot, pairs):
    """x [tokens][heads][dim], c and sn [tokens][1][rot / 2]"""
    y = x.clone()
    if pairs == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * sn, b * c + a * sn
    else:
        a, b = x[..., :rot:2], x[..., 1:rot:2]
        y[..., :rot:2], y[..., 1:rot:2] = a * c - b * sn, b * c + a * sn
    return y


def _append(s):
    case = s["case"]
    heads, kv, dim, page = case["heads"], case["kv"], case["dim"], case["page"]
    x = s["qkv"].view(s["tokens"], heads + 2 * kv, dim)
    q, k, v = x[:, :heads].float(), x[:, heads:heads + kv].float(), x[:, heads + kv:]
    seq, _, at = _rows_of(s)
    pos = at if s["positions"] is None else s["positions"]
    angle = pos.double()[:, None, None] * s["freq"]
    c, sn = torch.cos(angle).float(), torch.sin(angle).float()
    q = _rotated(_normed(q, s["q_norm"]), c, sn, case["rot"], case["pairs"])
    k = _rotated(_normed(k, s["k_norm"]), c, sn, case["rot"], case["pairs"])
    s["q_out"].copy_(q.reshape(s["tokens"], heads * dim))
    to = s["table"][seq, at // page].long()
    s["k_cache"][to, :, (at % page).long()] = k.to(s["k_cache"].dtype)
    s["v_cache"][to, :, (at % page).long()] = v
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attend(s):
    case = s["case"]
    heads, kv, dim, page, seqs = case["heads"], case["kv"], case["dim"], case["page"], case["seqs"]
    group, most, n = heads // kv, s["most"], case["new"]
    seq, nth, at = _rows_of(s)
    j = torch.arange(most, device=at.device)
    pages = s["table"][:, j // page].clamp_min(0).long()
    k = s["k_cache"][pages, :, j % page].float().permute(0, 2, 3, 1).contiguous()  # [seqs][kv][dim][most]
    v = s["v_cache"][pages, :, j % page].float().permute(0, 2, 1, 3).contiguous()
    q = torch.zeros(seqs, n, heads, dim, device=at.device)
    q[seq, nth] = s["q"].view(s["tokens"], heads, dim).float()
    q = q.view(seqs, n, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kv, group * n, dim)
    z = torch.matmul(q, k).view(seqs, kv, group, n, most).mul_(1 / math.sqrt(dim))
    p = torch.full((seqs, n), -1, device=at.device)  # rows that a shorter sequence has not: nothing to see
    p[seq, nth] = at.to(p.dtype)
    hidden = j > p[..., None]
    if case.get("window"):
        hidden |= j <= p[..., None] - case["window"]
    z.masked_fill_(hidden[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp_(z.sub_(top))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(seqs, kv, group * n, most), v).view(seqs, kv, group, n, dim) / total
    s["out"].copy_(o.permute(0, 3, 1, 2, 4)[seq, nth].reshape(s["tokens"], heads * dim))
    if s["lse"] is None:
        return {"out": s["out"]}
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2)[seq, nth]
    s["lse"].copy_(lse.reshape(s["tokens"], heads))
    return {"out": s["out"], "lse": s["lse"]}


def _adjust(s):
    case = s["case"]
    rows, vocab = case["rows"], case["vocab"]
    z = s["logits"].float()
    place = torch.arange(case["history"], device=z.device)
    token = torch.where(place < s["total"][:, None], s["history"], -1)
    token = torch.where(token < 0, vocab, token).long()
    counts = lambda which: torch.zeros(rows, vocab + 1, dtype=torch.int32, device=z.device).scatter_add_(  # noqa: E731
        1, token, which.to(torch.int32))[:, :vocab]
    made = counts(place >= s["prompt"][:, None])
    seen = counts(torch.ones_like(token)) > 0
    rho = s["repetition"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / rho, z * rho), z)
    z = z - s["frequency"][:, None] * made - s["presence"][:, None] * (made > 0)
    if s["bias_index"] is not None:
        z.scatter_add_(1, s["bias_index"].long(), s["bias_value"])
    if s["mask"] is not None:
        j = torch.arange(vocab, device=z.device)
        z.masked_fill_((s["mask"][:, j // 32] >> (j % 32).to(torch.int32)) & 1 == 0, -math.inf)
    return s["out"].copy_(z)


def _pairs(case):
    """Visible (query, key) pairs of one head, and the keys that some query of their sequence sees."""
    pairs = keys = 0
    w = case.get("window") or 1 << 40
    for n, past in _lengths(case):
        pairs += sum(min(past + i + 1, w) for i in range(n))
        keys += min(n + past, w + n - 1)
    return pairs, keys


def work(case):
    b = SIZE[case["dtype"]]
    if case["op"] == "adjust":
        n = case["rows"] * case["vocab"]
        return {"bytes": 2 * n * b + case["rows"] * (4 * case["history"] + 8 * case["biases"] + 20) + (n // 8 if case.get("mask") else 0),
                "flops": 4 * n}
    tokens, heads, kv, dim = sum(n for n, _ in _lengths(case)), case["heads"], case["kv"], case["dim"]
    if case["op"] == "append":
        n = tokens * (heads + 2 * kv) * dim
        return {"bytes": 2 * n * b, "flops": 6 * n}
    pairs, keys = _pairs(case)
    return {"bytes": 2 * tokens * heads * dim * b + 2 * keys * kv * dim * b + (4 * tokens * heads if case.get("lse") else 0),
            "flops": 4 * pairs * heads * dim}


def exact(case, seed):
    """The definitions in 64 bits, sequence by sequence."""
    s, op = prepare(case, seed), case["op"]
    if op == "adjust":
        return _exact_adjust(case, s)
    heads, kv, dim, page = case["heads"], case["kv"], case["dim"], case["page"]
    first, out = 0, []
    if op == "append":
        rot, q_all = case["rot"], []
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for i, (n, past) in enumerate(_lengths(case)):
            x = s["qkv"][first:first + n].double().view(n, heads + 2 * kv, dim)
            at = past + torch.arange(n, device=x.device)
            pos = at.double() if s["positions"] is None else s["positions"][first:first + n].double()
            turn = torch.polar(torch.ones(n, 1, rot // 2, device=x.device, dtype=torch.float64), (pos[:, None] * s["freq"])[:, None])
            both = []
            for y, w in ((x[:, :heads], s["q_norm"]), (x[:, heads:heads + kv], s["k_norm"])):
                if w is not None:
                    y = y / (y.pow(2).sum(-1, keepdim=True) / dim + EPS).sqrt() * w.double()
                part = y[..., :rot]
                part = part.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if case["pairs"] == "half" else part.unflatten(-1, (rot // 2, 2))
                part = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
                part = (part.transpose(-1, -2) if case["pairs"] == "half" else part).flatten(-2)
                both.append(torch.cat([part, y[..., rot:]], -1))
            q_all.append(both[0].reshape(n, heads * dim))
            slot = s["table"][i].long()[at // page]
            kc[slot, :, at % page], vc[slot, :, at % page] = both[1], x[:, heads + kv:]
            first += n
        return {"q": torch.cat(q_all), "k_cache": kc, "v_cache": vc}
    lse = []
    w = case.get("window") or 1 << 40
    for i, (n, past) in enumerate(_lengths(case)):
        t = past + n
        pages = s["table"][i, :-(-t // page)].long()
        k, v = (s[c][pages].transpose(0, 1).reshape(kv, -1, dim)[:, :t].double() for c in ("k_cache", "v_cache"))
        q = s["q"][first:first + n].double().view(n, kv, heads // kv, dim)
        key, query = torch.arange(t, device=q.device), past + torch.arange(n, device=q.device)[:, None]
        seen = (key <= query) & (key > query - w)
        o, l = [], []
        for h in range(kv):
            z = q[:, h].reshape(-1, dim) @ k[h].t().contiguous() / math.sqrt(dim)
            z = z.view(n, heads // kv, t).masked_fill_(~seen[:, None], -math.inf)
            l.append(torch.logsumexp(z, -1))
            o.append(torch.exp(z - l[-1][..., None]).view(-1, t).mm(v[h]).view(n, -1))
        out.append(torch.cat(o, 1))
        lse.append(torch.cat(l, 1))
        first += n
    return {"out": torch.cat(out), "lse": torch.cat(lse)} if case.get("lse") else {"out": torch.cat(out)}


def _exact_adjust(case, s):
    vocab = case["vocab"]
    z = s["logits"].double()
    token = s["history"].long()  # a row's unfilled places hold -1: a column of their own behind the vocabulary
    token[token < 0] = vocab
    generated = torch.arange(case["history"], device=z.device)[None] >= s["prompt"][:, None]
    n_all, n_gen = (torch.zeros(case["rows"], vocab + 1, dtype=torch.float64, device=z.device) for _ in range(2))
    n_all.scatter_add_(1, token, torch.ones(token.shape, dtype=torch.float64, device=z.device))
    n_gen.scatter_add_(1, token, generated.double())
    n_all, n_gen = n_all[:, :vocab], n_gen[:, :vocab]
    rho = s["repetition"].double()[:, None].expand_as(z)
    z = torch.where(n_all > 0, z * torch.where(z > 0, 1 / rho, rho), z)
    z = z - s["frequency"].double()[:, None] * n_gen - s["presence"].double()[:, None] * n_gen.clamp(max=1)
    if case["biases"]:
        z = z.scatter_add(1, s["bias_index"].long(), s["bias_value"].double())
    if case.get("mask"):
        words = s["mask"].long()[..., None] >> torch.arange(32, device=z.device) & 1
        z = torch.where(words.flatten(1)[:, :vocab] > 0, z, -math.inf)
    return z
