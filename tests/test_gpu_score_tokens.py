"""ScoringHead (norm, int8 head, scores) behind a LUT layer, against 64 bits and captured in a graph."""
import numpy as np
import pytest

from binary_basis_lut_amd import inputs as I

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def make(batch, hidden, vocab, top_k=5):
    from binary_basis_lut_amd.score_tokens import ScoringHead
    g = torch.Generator().manual_seed(batch + vocab)
    norm = (1 + 0.1 * torch.randn(hidden, generator=g)).half()
    head = (torch.randn(vocab, hidden, generator=g) * 0.05).half()
    y, residual = torch.randn(batch, hidden, generator=g).half(), (3 * torch.randn(batch, hidden, generator=g)).half()
    targets = torch.randint(0, vocab, (batch,), generator=g)
    targets[batch // 2] = -100
    return ScoringHead(norm.cuda(), head.cuda(), batch, top_k), norm, head, y, residual, targets


@pytest.mark.parametrize("batch,hidden,vocab", [(1, 512, 3000), (7, 1000, 2049), (90, 768, 5000)])
def test_scores_follow_from_the_quantised_head(batch, hidden, vocab):
    print(f"[case] score_tokens {batch} x {hidden} -> {vocab}", flush=True)
    head, norm, w, y, residual, targets = make(batch, hidden, vocab)
    out = head.score(y.cuda(), residual.cuda(), targets.cuda())
    torch.cuda.synchronize()
    h = (y.float() + residual.float()).half()
    assert torch.equal(out["residual"].cpu(), h)
    h64, n64 = h.double(), norm.double()
    normed = h64 * n64 / (h64.pow(2).mean(1, keepdim=True) + 1e-5).sqrt()
    # both quantisations are off by half a step per element: |error| <= sum |a| dw + |w| da + da dw
    da = normed.abs().amax(1, keepdim=True) / 254 * 1.001
    dw = w.double().abs().amax(1, keepdim=True) / 254 * 1.001
    exact = normed @ w.double().t()
    bound = normed.abs().sum(1, keepdim=True) * dw.t() + da * w.double().abs().sum(1) + hidden * da * dw.t()
    logits = out["logits"].cpu().double()
    assert ((logits - exact).abs() <= bound + 1e-5 * (1 + exact.abs())).all()
    # and the scores are those of the logits
    lp = torch.log_softmax(logits, 1)
    want = torch.where(targets < 0, 0.0, lp[torch.arange(batch), targets.clamp_min(0)])
    tol = 8 * 2.0 ** -24 * (lp.abs().amax() + 2 * np.log(vocab) + 8)
    assert ((out["logprob"].cpu().double() - want).abs() <= tol).all()
    assert ((out["entropy"].cpu().double() + (lp.exp() * lp).sum(1)).abs() <= 2 * tol).all()
    order = np.argsort(-logits.numpy(), axis=1, kind="stable")[:, :5]
    assert np.array_equal(out["top_index"].cpu().numpy(), order)


def test_refuses_what_does_not_fit():
    head, norm, w, y, residual, targets = make(3, 512, 1000)
    with pytest.raises(ValueError):
        head.score(torch.zeros((4, 512), dtype=torch.float16, device="cuda"), residual.cuda(), targets.cuda())
    with pytest.raises(ValueError):
        head.score(y.cuda()[:, :256], residual.cuda()[:, :256], targets.cuda())
    from binary_basis_lut_amd.score_tokens import ScoringHead
    with pytest.raises(ValueError):
        ScoringHead(norm.cuda().float(), w.cuda(), 3)


def test_a_decode_step_replays_bitwise_behind_a_lut_layer():
    from binary_basis_lut_amd import fluxbin as F
    print("[case] LUT layer 512 x 1024 -> norm -> head -> scores, graph", flush=True)
    batch, hidden, vocab = 3, 512, 4000
    layer = I.make_layer(hidden, 1024, 2, 1, 4, s=64, outlier_frac=0.01, seed=(5, 0, 1))
    down = F.DeviceLayer(layer, max_batch=batch)
    head, _, _, _, residual, targets = make(batch, hidden, vocab)
    x = torch.from_numpy(I.make_x(layer, batch, seed=(5, 0, 1)).view(np.int16)).cuda()
    y = torch.empty((batch, hidden), dtype=torch.float16, device="cuda")
    rd, td = residual.cuda(), targets.cuda()

    def step():
        down.gemv(x, y)
        return head.score(y, rd, td)

    want = {n: v.clone() for n, v in step().items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        for v in out.values():
            v.zero_()
        y.fill_(i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, v in out.items():
            assert torch.equal(v, want[n]), n
    down.close()


def test_the_command_runs():
    from binary_basis_lut_amd.score_tokens import run
    r = run(batch=2, steps=2, vocab=1000, top_k=3)
    assert np.isfinite(r["mean_logprob"]) and r["perplexity"] > 1 and len(r["best"]) == 2 and len(r["best"][0]) == 3
    assert all(0 < h <= np.log(1000) + 1e-4 for h in r["entropy"])
