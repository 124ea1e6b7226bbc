"""Paged batches for the attention operators' tests, and their definitions in 64 bits on the host (numpy)."""
import numpy as np
import torch

U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -126}  # half a subnormal step (fp32: flush)


def f64(t):
    return t.detach().cpu().double().numpy()


class Paged:
    """Sequences of (new, past) tokens over a cache whose pages are handed out in a random order.

    order: "heads" (a page holds its tokens head by head) or "tokens".  behind: rows of q behind the last
    sequence.  spare: pages that are nobody's.  Everything lives on the GPU unless device says otherwise.
    """

    def __init__(self, dt, heads, kv, dim, page, lengths, seed=0, order="heads", behind=0, spare=2, decode=None, table_extra=0,
                 max_kv_len=None, device="cuda"):
        self.dt, self.heads, self.kv, self.dim, self.page, self.lengths = dt, heads, kv, dim, page, lengths
        self.g = torch.Generator().manual_seed(seed)
        self.decode = all(n == 1 for n, _ in lengths) and behind == 0 if decode is None else decode
        news, lens = [n for n, _ in lengths], [n + p for n, p in lengths]
        self.starts_host = np.concatenate([[0], np.cumsum(news)]).astype(np.int64)
        self.rows, self.tokens, self.lens_host = int(sum(news)), int(sum(news)) + behind, lens
        used = [-(-n // page) for n in lens]
        self.per_seq = max([1] + used) + table_extra
        self.pages = sum(used) + spare
        ids = torch.randperm(self.pages, generator=self.g)[:sum(used)].tolist()
        table = np.full((len(lengths), self.per_seq), -1, dtype=np.int32)
        for s, u in enumerate(used):
            table[s, :u] = [ids.pop() for _ in range(u)]
        self.table_host = table
        shape = (self.pages, kv, page, dim) if order == "heads" else (self.pages, page, kv, dim)
        self.order, self.shape, self.device, self.max_kv_len = order, shape, device, max_kv_len
        self.k, self.v = self.randn(*shape), self.randn(*shape)
        self.q = self.randn(self.tokens, heads * dim)

    def randn(self, *shape, scale=1.0):
        return (torch.randn(*shape, generator=self.g) * scale).to(DT[self.dt])

    def cached(self, cache, s, length=None):
        """[length][kv][dim] of sequence s (float64), NaN where there is no page."""
        n = self.lens_host[s] if length is None else length
        c = cache if self.order == "heads" else cache.transpose(1, 2)
        c = f64(c)
        out = np.full((n, self.kv, self.dim), np.nan)
        for j in range(n):
            if j // self.page < self.per_seq:
                p = self.table_host[s, j // self.page]
                if 0 <= p < self.pages:
                    out[j] = c[p, :, j % self.page]
        return out

    def there(self, s, j):
        i = j // self.page
        return (i < self.per_seq) & (0 <= self.table_host[s, np.minimum(i, self.per_seq - 1)]) & \
               (self.table_host[s, np.minimum(i, self.per_seq - 1)] < self.pages)

    def upload(self, F):
        """The description, with its tensors kept in self.dev."""
        d = self.dev = {n: t.to(self.device).contiguous() for n, t in (("k", self.k), ("v", self.v), ("q", self.q))}
        d["table"] = torch.from_numpy(self.table_host).to(self.device)
        d["starts"] = None if self.decode else torch.from_numpy(self.starts_host.astype(np.int32)).to(self.device)
        d["lens"] = torch.tensor(self.lens_host, dtype=torch.int32, device=self.device)
        b = F.PagedBatch()
        b.abi_version, b.dtype = F.ABI_VERSION, {"f16": F.DT_F16, "bf16": F.DT_BF16}[self.dt]
        b.heads, b.kv_heads, b.dim, b.page_size = self.heads, self.kv, self.dim, self.page
        b.tokens, b.seqs = self.tokens, len(self.lengths)
        b.max_kv_len = max([0] + self.lens_host) if self.max_kv_len is None else self.max_kv_len
        b.seq_starts = None if self.decode else d["starts"].data_ptr()
        b.kv_lens, b.page_table, b.table_ld, b.table_pages = d["lens"].data_ptr(), d["table"].data_ptr(), self.per_seq, self.per_seq
        b.k_cache, b.v_cache, b.cache_pages = d["k"].data_ptr(), d["v"].data_ptr(), self.pages
        b.page_stride = self.kv * self.page * self.dim
        b.head_stride, b.token_stride = (self.page * self.dim, self.dim) if self.order == "heads" else (self.dim, self.kv * self.dim)
        return b


def attention_oracle(c, scale, window=0):
    """out, lse, and the bound's parts: sum p |v|, sum |q k| of the largest, keys seen, for every row of a sequence."""
    out = np.zeros((c.rows, c.heads, c.dim))
    lse = np.full((c.rows, c.heads), -np.inf)
    mag = np.zeros((c.rows, c.heads, c.dim))
    work = np.zeros((c.rows, c.heads))
    seen = np.zeros(c.rows, dtype=np.int64)
    q = f64(c.q).reshape(c.tokens, c.heads, c.dim)
    group = c.heads // c.kv
    for s, (n, past) in enumerate(c.lengths):
        length = c.lens_host[s]
        if n == 0:
            continue
        k, v = c.cached(c.k, s), c.cached(c.v, s)
        j = np.arange(length)
        ok = c.there(s, j) if length else np.zeros(0, dtype=bool)
        for i in range(n):
            t, row = length - n + i, c.starts_host[s] + i
            vis = ok & (j <= t) & ((j > t - window) if window else True)
            seen[row] = vis.sum()
            if not vis.any():
                continue
            for h in range(c.heads):
                kk, vv = k[vis, h // group], v[vis, h // group]
                with np.errstate(all="ignore"):
                    z = scale * (kk @ q[row, h])
                    top = z.max()
                    e = np.exp(z - top)
                    p = e / e.sum()
                    out[row, h], lse[row, h] = p @ vv, top + np.log(e.sum())
                    mag[row, h] = p @ np.abs(vv)
                    work[row, h] = scale * (np.abs(kk) @ np.abs(q[row, h])).max()
    return out, lse, mag, work, seen


def attention_bounds(c, out, mag, work, seen):
    """How far out and lse may be off.

    A product q . k: at most dim + 2 fp32 roundings of sum |q k| (its sum in any order), and the exponent another
    three of that; 2^x and the shift's rounding four units, and 2^-22 for v_exp's own error; so a weight's relative
    error is e.  Sums over the keys: a rounding for every key and for every rescaling (of 32 keys).  The weights of the second
    product are rounded to the type (twice nothing smaller than 2^-25 of a weight of 2^7 in fp16: 2^-31 each).
    """
    n = seen[:, None]
    e = ((c.dim + 5) * U * work + 2.0 ** -22 + 4 * U + 20 * U)
    sums = (n * 1.04 + 16) * U
    tol = mag * (UNIT[c.dt] + 2 * e + 2 * sums)[..., None] + UNIT[c.dt] * np.abs(out) + TINY[c.dt]
    if c.dt == "f16":
        tol = tol + 2.0 ** -31 * (n * 4)[..., None] * np.abs(out).max(initial=1.0)
    return tol, e + sums + 8 * U
