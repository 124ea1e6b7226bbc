"""ScoringHead on inputs that do not lie in memory as its buffers do."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HIDDEN, VOCAB = 512, 3000


def make(rows):
    from binary_basis_lut_amd.score_tokens import ScoringHead
    g = torch.Generator().manual_seed(rows)
    norm = (1 + 0.1 * torch.randn(HIDDEN, generator=g)).half().cuda()
    head = (torch.randn(VOCAB, HIDDEN, generator=g) * 0.05).half().cuda()
    y, residual = torch.randn(rows, HIDDEN, generator=g).half().cuda(), torch.randn(rows, HIDDEN, generator=g).half().cuda()
    return ScoringHead(norm, head, rows), y, residual, g


def kept(out):
    torch.cuda.synchronize()
    return {n: v.clone() for n, v in out.items()}


def same(a, b):
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("rows", [1, 4, 33])
def test_a_step_of_a_token_matrix_scores_its_own_tokens(rows):
    print(f"[case] score, {rows} strided targets", flush=True)
    head, y, residual, g = make(rows)
    tokens = torch.randint(0, VOCAB, (rows, 7), generator=g).cuda()
    for t in range(7):
        want = kept(head.score(y, residual, tokens[:, t].contiguous()))
        same(kept(head.score(y, residual, tokens[:, t])), want)
    # first-order bound of the kernel's fp32: see check_scores of the operators' tests
    lp = torch.log_softmax(want["logits"].double(), 1).gather(1, tokens[:, 6:])[:, 0]
    tol = 8 * 2.0 ** -24 * (lp.abs() + 2 * math.log(VOCAB) + 8)
    assert ((want["logprob"].double() - lp).abs() <= tol).all()


def test_strided_targets_are_read_anew_by_every_replay():
    rows = 5
    print("[case] score, strided targets in a graph", flush=True)
    head, y, residual, g = make(rows)
    tokens = torch.randint(0, VOCAB, (rows, 4), generator=g).cuda()
    head.score(y, residual, tokens[:, 1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = head.score(y, residual, tokens[:, 1])
    for _ in range(3):
        tokens.copy_(torch.randint(0, VOCAB, (rows, 4), generator=g))
        graph.replay()
        got = kept(out)
        same(kept(head.score(y, residual, tokens[:, 1].contiguous())), got)


def test_rows_that_lie_apart_score_as_adjacent_ones():
    rows = 6
    print("[case] score, y and residual with row strides", flush=True)
    head, y, residual, g = make(rows)
    targets = torch.randint(0, VOCAB, (rows,), generator=g).cuda()
    want = kept(head.score(y, residual, targets))
    wide, twice = torch.zeros(rows, HIDDEN + 9, dtype=y.dtype, device="cuda"), torch.zeros(2 * rows, HIDDEN, dtype=y.dtype, device="cuda")
    wide[:, 3:3 + HIDDEN], twice[::2] = y, residual
    same(kept(head.score(wide[:, 3:3 + HIDDEN], twice[::2], targets)), want)


def test_a_head_made_on_one_stream_scores_on_another():
    rows = 4
    print("[case] score on another stream than the constructor's", flush=True)
    head, y, residual, g = make(rows)
    targets = torch.randint(0, VOCAB, (rows,), generator=g).cuda()
    want = kept(head.score(y, residual, targets))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = make(rows)[0]
    same(kept(other.score(y, residual, targets)), want)


def test_the_last_residual_is_taken_in_place():
    rows = 5
    print("[case] score with the residual view of the call before", flush=True)
    head, y, residual, g = make(rows)
    targets = torch.randint(0, VOCAB, (rows,), generator=g).cuda()
    between = kept(head.score(y, residual, targets))["residual"]
    want = kept(head.score(y, between, targets))
    out = head.score(y, residual, targets)
    same(kept(head.score(y, out["residual"], targets)), want)
