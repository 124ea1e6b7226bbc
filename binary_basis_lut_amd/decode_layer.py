"""Decode steps through one attention layer of binary bases, from a token to the next.

  python3 -m binary_basis_lut_amd.decode_layer --batch 4 --steps 16 --context 1000

runs, on synthetic weights of the LLaMA-2-7B shapes and a random cache, what stands around a layer's
attention for a batch of sequences, as one HIP graph per step:

  h        = norm(x), x the embeddings of the last tokens            fluxbin_add_rmsnorm
  q, k, v  = LUT GEMV of the QKV projection (12288 x 4096, g = 4)    fluxbin_gemv
  queries rotated, keys rotated and appended with the values         fluxbin_rope_append
  o        = attention over the paged cache                          fluxbin_paged_attention
  y        = LUT GEMV of the output projection (4096 x 4096)         fluxbin_gemv
  logits   = int8 head of norm(y + x)                                fluxbin_add_rmsnorm, fluxbin_gemm_w8a8
  penalties for the tokens so far, biases and a mask                 fluxbin_adjust_logits
  the best alternatives, of which the first is the next token        fluxbin_token_logprobs

Prints the tokens, their log probabilities and the time of a step.
"""
from __future__ import annotations

import argparse


def run(batch: int, steps: int, context: int, vocab: int = 32000, heads: int = 32, dim: int = 128, page_size: int = 16,
        repetition: float = 1.2, seed: int = 11) -> dict:
    import numpy as np
    import torch

    from . import fluxbin as F
    from . import inputs as I
    from .paged import PagedAttention
    from .score_tokens import LogitRules, ScoringHead

    hidden = heads * dim
    layer = lambda n, k, which: F.DeviceLayer(  # noqa: E731
        I.make_layer(n, k, 2, 1, 4, s=max(32, k // 64 * 2), outlier_frac=0.01, seed=(6, which, seed)), max_batch=batch)
    qkv_proj, out_proj = layer(3 * hidden, hidden, 0), layer(hidden, hidden, 1)
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    per_seq = -(-(context + steps) // page_size)
    attention = PagedAttention(heads, heads, dim, batch * per_seq, page_size, batch, per_seq, batch)
    attention.page_table.copy_(torch.randperm(batch * per_seq, generator=g, device="cuda").view(batch, per_seq))
    attention.k_cache.copy_(randn(*attention.k_cache.shape))
    attention.v_cache.copy_(randn(*attention.v_cache.shape))
    attention.kv_lens.fill_(context)
    head = ScoringHead((1 + 0.1 * randn(hidden)).half(), (randn(vocab, hidden) * 0.02).half(), batch)
    norm = (1 + 0.1 * randn(hidden)).half()
    embedding = randn(vocab, hidden).half()
    rules = LogitRules(batch, vocab, steps + 1, repetition=torch.full((batch,), repetition, device="cuda"),
                       mask=torch.full((batch, (vocab + 31) // 32), -2, dtype=torch.int32, device="cuda"))  # never token 0, 32, ..
    tokens = torch.randint(1, vocab, (batch, 1), generator=g, device="cuda")
    targets = torch.full((batch,), -1, dtype=torch.int64, device="cuda")
    half = lambda *shape: torch.empty(shape, dtype=torch.float16, device="cuda")  # noqa: E731
    h, qkv, y = half(batch, hidden), half(batch, 3 * hidden), half(batch, hidden)

    def step():
        x = embedding[tokens[:, 0]]
        rules.append(tokens)
        attention.kv_lens.add_(1)
        F.fluxbin_add_rmsnorm(x, hidden, None, 0, norm, F.DT_F16, batch, hidden, 1e-5, None, 0, h, hidden, None, 0, None)
        qkv_proj.gemv(h, qkv, batch)
        out_proj.gemv(attention.attend(qkv), y, batch)
        out = head.score(y, x, targets, rules=rules)
        tokens.copy_(out["top_index"][:, :1])
        return out

    start = tokens.clone()
    step()  # the graph records launches only: first uses stand before it
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    tokens.copy_(start)
    attention.kv_lens.fill_(context)
    rules.clear()
    made, logprobs, ms = [], [], []
    before, after = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(steps):
        before.record()
        graph.replay()
        after.record()
        torch.cuda.synchronize()
        ms.append(before.elapsed_time(after))
        made.append(tokens[:, 0].tolist())
        logprobs.append(out["top_logprob"][:, 0].tolist())
    result = {"tokens": np.array(made).T.tolist(), "logprobs": np.array(logprobs).T.tolist(), "us_per_step": 1e3 * sorted(ms)[len(ms) // 2],
              "kv_lens": attention.kv_lens.tolist()}
    qkv_proj.close()
    out_proj.close()
    return result


def main() -> int:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--context", type=int, default=1000)
    a = ap.parse_args()
    r = run(a.batch, a.steps, a.context)
    print(f"{a.steps} steps of {a.batch} sequences over {a.context} tokens: {r['us_per_step']:.1f} us a step")
    for b, (t, p) in enumerate(zip(r["tokens"], r["logprobs"])):
        print(f"sequence {b}: " + ", ".join(f"{i} ({v:.2f})" for i, v in zip(t[:8], p)) + (" ..." if len(t) > 8 else ""))
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
