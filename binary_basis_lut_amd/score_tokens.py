"""The end of a decode step on binary-basis layers: the last layer's output to token scores.

  python3 -m binary_basis_lut_amd.score_tokens --batch 4 --steps 8

runs, on synthetic weights of the LLaMA-2-7B shapes, what a model does after
its last MLP for a batch of sequences, as one HIP graph per step:

  y      = LUT GEMV of the down projection (4096 x 11008, two global bases and
           one salient basis, g = 4)                       fluxbin_gemv
  q, s   = int8(norm(y + residual))                        fluxbin_add_rmsnorm
  logits = q . head, int8 weights with a scale per token   fluxbin_gemm_w8a8
  log p of each sequence's next token, the entropy and     fluxbin_token_logprobs
  the best alternatives

The head's weights are quantised once, by fluxbin_quantize_rows.  Prints the
mean log probability, the perplexity of the given tokens, the best
alternatives of the last step and the time of a step.
"""
from __future__ import annotations

import argparse


def _check(name, t, dtype, device, shape) -> None:
    """Raises ValueError unless `t` is what the kernels, which see its address only, will take it for."""
    if t.dtype != dtype or t.device != device or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, not {dtype} {tuple(shape)} on {device}")
    if t.dim() == 2 and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the elements of a row lie {t.stride(1)} apart, not side by side")


def _check_current(device) -> None:
    import torch

    if torch.cuda.current_device() != device.index:  # where the launches go
        raise ValueError(f"the head is on {device}, the current device is cuda:{torch.cuda.current_device()}")


def _row_stride(t) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]  # a single row's stride can be any number


class ScoringHead:
    """Final norm, int8 output head and scoring for up to `max_rows` rows at a time.

    norm_weight: fp16 [hidden]; head: fp16 [vocab][hidden] (quantised here, per
    output channel; the tensor is not kept; the constructor waits for it, so
    that score() may run on any stream).  score() enqueues three calls on
    the current stream, and a copy of the targets where they are not adjacent,
    and returns views of buffers that the next call overwrites; it allocates
    nothing, so it can be captured in a graph.  Calls of one head share these
    buffers: the caller orders calls on different streams, and of the inputs
    only `residual` may be one of the views (the last call's, all its rows).
    """

    def __init__(self, norm_weight, head, max_rows: int, top_k: int = 5, eps: float = 1e-5):
        import torch
        from . import fluxbin as F

        self.F, self.top_k, self.eps = F, top_k, eps
        if head.dim() != 2 or not head.is_cuda:
            raise ValueError(f"head: {tuple(head.shape)} on {head.device}, not [vocab][hidden] on a GPU")
        self.vocab, self.hidden = head.shape
        dev = self.device = head.device
        _check("head", head, torch.float16, dev, head.shape)
        _check("norm_weight", norm_weight, torch.float16, dev, (self.hidden,))
        _check_current(dev)
        self.norm_weight = norm_weight.contiguous()
        self.ld = (self.hidden + 15) // 16 * 16  # the int8 product wants rows of whole 16-byte pieces
        empty = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=dev)
        self.head_q, self.head_scale = empty(self.vocab, self.ld, dtype=torch.int8), empty(self.vocab)
        F.fluxbin_quantize_rows(head, _row_stride(head), F.DT_F16, self.vocab, self.hidden, self.head_q, self.ld, self.head_scale)
        self.residual = empty(max_rows, self.hidden, dtype=torch.float16)
        self.q, self.scale = empty(max_rows, self.ld, dtype=torch.int8), empty(max_rows)
        self.logits = empty(max_rows, self.vocab)
        self.targets = empty(max_rows, dtype=torch.int64)
        self.logprob, self.entropy = empty(max_rows), empty(max_rows)
        self.top_logprob, self.top_index = empty(max_rows, top_k), empty(max_rows, top_k, dtype=torch.int64)
        need = max(F.fluxbin_token_logprobs_workspace_size(r, self.vocab, top_k) for r in range(1, max_rows + 1))
        self.workspace = empty(max(need, 16), dtype=torch.uint8)
        torch.cuda.current_stream().synchronize()  # the quantised head is there for a score() on any stream

    def score(self, y, residual, targets, logit_scale: float = 1.0) -> dict:
        """y, residual: fp16 [rows][hidden], any row stride; targets: int64 [rows], any stride, negative where there is none."""
        import torch

        F, rows = self.F, y.shape[0]
        if rows > self.logits.shape[0]:
            raise ValueError(f"y {tuple(y.shape)}: at most {self.logits.shape[0]} rows of {self.hidden}")
        _check("y", y, torch.float16, self.device, (rows, self.hidden))
        _check("residual", residual, torch.float16, self.device, (rows, self.hidden))
        _check("targets", targets, torch.int64, self.device, (rows,))
        _check_current(self.device)
        if not targets.is_contiguous():  # one step's column of a [rows][steps] matrix
            targets = self.targets[:rows].copy_(targets)
        F.fluxbin_add_rmsnorm(y, _row_stride(y), residual, _row_stride(residual), self.norm_weight, F.DT_F16, rows, self.hidden,
                              self.eps, self.residual, self.hidden, None, 0, self.q, self.ld, self.scale)
        F.fluxbin_gemm_w8a8(self.q, self.ld, self.scale, self.head_q, self.ld, self.head_scale, None, rows, self.vocab,
                            self.hidden, self.logits, self.vocab, F.DT_F32)
        F.fluxbin_token_logprobs(self.logits, self.vocab, F.DT_F32, rows, self.vocab, logit_scale, targets, self.logprob,
                                 self.entropy, self.top_k, self.top_logprob, self.top_index, self.workspace,
                                 self.workspace.numel())
        return {"residual": self.residual[:rows], "logits": self.logits[:rows], "logprob": self.logprob[:rows],
                "entropy": self.entropy[:rows], "top_logprob": self.top_logprob[:rows], "top_index": self.top_index[:rows]}


def run(batch: int, steps: int, vocab: int, top_k: int) -> dict:
    import math

    import numpy as np
    import torch

    from . import fluxbin as F
    from . import inputs as I

    hidden, inner = 4096, 11008
    layer = I.make_layer(hidden, inner, 2, 1, 4, s=224, outlier_frac=0.01, seed=(2, 0, 7))
    down = F.DeviceLayer(layer, max_batch=batch)
    g = torch.Generator(device="cuda").manual_seed(7)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    head = ScoringHead((1 + 0.1 * randn(hidden)).half(), (randn(vocab, hidden) * 0.02).half(), batch, top_k)
    x = torch.empty((batch, inner), dtype=torch.int16, device="cuda")
    y = torch.empty((batch, hidden), dtype=torch.float16, device="cuda")
    residual = torch.empty_like(y)
    targets = torch.empty(batch, dtype=torch.int64, device="cuda")

    def step():
        down.gemv(x, y)
        return head.score(y, residual, targets)

    def feed(i):
        x.copy_(torch.from_numpy(I.make_x(layer, batch, seed=(2, i, 7)).view(np.int16)))
        residual.copy_(randn(batch, hidden) * 10)
        targets.copy_(torch.randint(0, vocab, (batch,), generator=g, device="cuda"))

    feed(0)
    step()  # the graph records launches only: first uses stand before it
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    total, ms = 0.0, []
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(steps):
        feed(i)
        start.record()
        graph.replay()
        stop.record()
        torch.cuda.synchronize()
        ms.append(start.elapsed_time(stop))
        total += float(out["logprob"].sum())
    mean = total / (steps * batch)
    best = [list(zip(t, p)) for t, p in zip(out["top_index"].tolist(), out["top_logprob"].tolist())]
    result = {"mean_logprob": mean, "perplexity": math.exp(-mean), "best": best, "entropy": out["entropy"].tolist(),
              "us_per_step": 1e3 * sorted(ms)[len(ms) // 2], "uniform_logprob": -math.log(vocab)}
    down.close()
    return result


def main() -> int:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--top", type=int, default=5)
    a = ap.parse_args()
    r = run(a.batch, a.steps, a.vocab, a.top)
    print(f"{a.steps} steps of {a.batch} sequences: mean log probability {r['mean_logprob']:.4f} (uniform "
          f"{r['uniform_logprob']:.4f}), perplexity {r['perplexity']:.0f}, {r['us_per_step']:.1f} us a step")
    for b, (best, h) in enumerate(zip(r["best"], r["entropy"])):
        print(f"sequence {b}: entropy {h:.3f}, best " + ", ".join(f"{t} ({p:.3f})" for t, p in best))
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
