"""What ScoringHead refuses and what it hands to the kernels, without a GPU.

The tensors are fake ones that say they are on cuda:0 and hold nothing, and the launching entry points
are replaced by recorders, so a call that is let through is seen by its arguments.
"""
import pytest

torch = pytest.importorskip("torch")

HIDDEN, VOCAB, ROWS = 512, 1000, 3


@pytest.fixture
def calls(monkeypatch):
    from torch._subclasses.fake_tensor import FakeTensorMode

    from binary_basis_lut_amd import build as B
    if B.is_stale():
        B.build()
    from binary_basis_lut_amd import fluxbin

    class Stream:
        cuda_stream = 0

        def synchronize(self):
            seen.append(("synchronize",))

    seen = []
    for name in ("fluxbin_quantize_rows", "fluxbin_add_rmsnorm", "fluxbin_gemm_w8a8", "fluxbin_token_logprobs"):
        monkeypatch.setattr(fluxbin, name, lambda *a, _n=name: seen.append((_n, *a)))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    with FakeTensorMode():
        yield seen


def fp16(*shape, device="cuda"):
    return torch.empty(shape, dtype=torch.float16, device=device)


def int64(*shape, device="cuda"):
    return torch.empty(shape, dtype=torch.int64, device=device)


def make(rows=8):
    from binary_basis_lut_amd.score_tokens import ScoringHead
    return ScoringHead(fp16(HIDDEN), fp16(VOCAB, HIDDEN), rows)


def scored(calls, head, y, residual, targets):
    calls.clear()
    head.score(y, residual, targets)
    return {c[0]: c[1:] for c in calls}


def refused(calls, head, y, residual, targets, name):
    calls.clear()
    with pytest.raises(ValueError, match=name):
        head.score(y, residual, targets)
    assert not calls  # before any launch


@pytest.mark.parametrize("targets", [
    lambda: int64(ROWS).to(torch.int32), lambda: int64(ROWS - 1), lambda: int64(ROWS + 1), lambda: int64(0),
    lambda: int64(ROWS, 1), lambda: int64(ROWS, device="cpu"), lambda: fp16(ROWS),
], ids=["int32", "too few", "too many", "none", "2-D", "host memory", "fp16"])
def test_targets_that_would_be_misread_are_refused(calls, targets):
    refused(calls, make(), fp16(ROWS, HIDDEN), fp16(ROWS, HIDDEN), targets(), "targets")


@pytest.mark.parametrize("rows", [1, 2, ROWS, 8])
def test_targets_of_one_step_of_a_token_matrix_arrive_one_behind_the_other(calls, rows):
    tokens = int64(rows, 17)
    given = scored(calls, make(), fp16(rows, HIDDEN), fp16(rows, HIDDEN), tokens[:, 5])["fluxbin_token_logprobs"][6]
    assert given.dtype == torch.int64 and given.shape == (rows,) and given.is_contiguous()


def test_adjacent_targets_are_passed_as_they_are(calls):
    targets = int64(9)[4:4 + ROWS]
    assert scored(calls, make(), fp16(ROWS, HIDDEN), fp16(ROWS, HIDDEN), targets)["fluxbin_token_logprobs"][6] is targets


@pytest.mark.parametrize("bad", [
    lambda: fp16(ROWS, HIDDEN).to(torch.bfloat16), lambda: fp16(ROWS, HIDDEN).float(), lambda: fp16(ROWS, 2 * HIDDEN)[:, ::2],
    lambda: fp16(HIDDEN, ROWS).t(), lambda: fp16(ROWS, HIDDEN, device="cpu"),
], ids=["bf16", "fp32", "every other column", "transposed", "host memory"])
@pytest.mark.parametrize("which", ["y", "residual"])
def test_activations_that_would_be_misread_are_refused(calls, which, bad):
    t = {"y": fp16(ROWS, HIDDEN), "residual": fp16(ROWS, HIDDEN), which: bad()}
    refused(calls, make(), t["y"], t["residual"], int64(ROWS), which)


@pytest.mark.parametrize("shape", [(HIDDEN,), (ROWS, HIDDEN, 1), (0, HIDDEN + 1)])
def test_activations_of_another_shape_are_refused(calls, shape):
    refused(calls, make(), fp16(*shape), fp16(*shape), int64(ROWS), "y")


def test_activations_whose_rows_lie_apart_go_with_their_stride(calls):
    norm = scored(calls, make(), fp16(ROWS, 2 * HIDDEN)[:, :HIDDEN], fp16(2 * ROWS, HIDDEN)[::2], int64(ROWS))["fluxbin_add_rmsnorm"]
    assert norm[1] == 2 * HIDDEN and norm[3] == 2 * HIDDEN


def test_a_single_row_is_scored_whatever_its_row_stride_says(calls):
    row = fp16(HIDDEN, 1).t()  # adjacent elements; a stride between rows that are not there
    assert row.is_contiguous() and row.stride(0) < HIDDEN
    norm = scored(calls, make(), row, row, int64(1))["fluxbin_add_rmsnorm"]
    assert norm[1] >= HIDDEN and norm[3] >= HIDDEN  # below that fluxbin_add_rmsnorm refuses the call


@pytest.mark.parametrize("norm,head,name", [
    (lambda: fp16(HIDDEN - 1), lambda: fp16(VOCAB, HIDDEN), "norm_weight"), (lambda: fp16(HIDDEN + 1), lambda: fp16(VOCAB, HIDDEN), "norm_weight"),
    (lambda: fp16(1, HIDDEN), lambda: fp16(VOCAB, HIDDEN), "norm_weight"),
    (lambda: fp16(HIDDEN, device="cpu"), lambda: fp16(VOCAB, HIDDEN), "norm_weight"),
    (lambda: fp16(HIDDEN).to(torch.bfloat16), lambda: fp16(VOCAB, HIDDEN), "norm_weight"),
    (lambda: fp16(HIDDEN), lambda: fp16(HIDDEN, VOCAB).t(), "head"), (lambda: fp16(HIDDEN), lambda: fp16(VOCAB, 2 * HIDDEN)[:, ::2], "head"),
    (lambda: fp16(HIDDEN), lambda: fp16(VOCAB, HIDDEN).float(), "head"), (lambda: fp16(HIDDEN), lambda: fp16(VOCAB * HIDDEN), "head"),
    (lambda: fp16(HIDDEN, device="cpu"), lambda: fp16(VOCAB, HIDDEN, device="cpu"), "head"),
], ids=["short norm", "long norm", "2-D norm", "norm in host memory", "bf16 norm", "transposed head", "every other column", "fp32 head",
        "flat head", "host memory"])
def test_weights_that_would_be_misread_are_refused(calls, norm, head, name):
    from binary_basis_lut_amd.score_tokens import ScoringHead
    with pytest.raises(ValueError, match=name):
        ScoringHead(norm(), head(), 4)
    assert not calls


def test_weights_with_strides_are_taken(calls):
    from binary_basis_lut_amd.score_tokens import ScoringHead
    h = ScoringHead(fp16(2 * HIDDEN)[::2], fp16(VOCAB, HIDDEN + 8)[:, :HIDDEN], 4)
    assert h.norm_weight.is_contiguous() and calls[0][:3] == ("fluxbin_quantize_rows", calls[0][1], HIDDEN + 8)


def test_the_quantised_head_is_finished_before_a_score_on_any_stream(calls):
    make()
    names = [c[0] for c in calls]
    assert names == ["fluxbin_quantize_rows", "synchronize"]


def test_a_score_waits_for_nothing(calls):
    head = make()
    scored(calls, head, fp16(ROWS, HIDDEN), fp16(ROWS, HIDDEN), int64(ROWS, 2)[:, 0])
    assert ("synchronize",) not in calls


def test_another_current_device_is_refused(calls, monkeypatch):
    """The launches go to the current device, which need not reach another one's memory."""
    from binary_basis_lut_amd.score_tokens import ScoringHead
    head = make()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    refused(calls, head, fp16(ROWS, HIDDEN), fp16(ROWS, HIDDEN), int64(ROWS), "cuda:1")
    with pytest.raises(ValueError, match="cuda:1"):
        ScoringHead(fp16(HIDDEN, device="cuda:0"), fp16(VOCAB, HIDDEN, device="cuda:0"), 4)
    assert not calls
