"""The embedding and the linear cross entropy at their limits: waits that run out, sums of many terms of one sign,
sure targets, and forms that the other tests leave out.

Bounds.  u = 2^-24 and ut are half a step of fp32 and of the operands' type."""
import pytest
import torch

from test_embedding import _check_grad, _grad, _tokens
from test_linear_cross_entropy import _forward, _grads
from train_reference import TYPES


@pytest.fixture(scope="module")
def b(cuda_ready):
    from gemm_conv_epilogues_gb300 import binding
    yield binding
    assert binding.tf_read_device_error() == (0, 0)


# ---------------------------------------------------------------- embedding

@pytest.mark.gpu
@pytest.mark.parametrize("hidden", [256, 512, 1024, 4096])
def test_ring_waits_that_run_out(b, hidden):
    """A limit of nothing: copies that are not there at the first looks are given up, and the error word says so; copies
    under way have landed before the kernel ends (no drain runs out), and later calls are not touched by it.
    One, two and four pieces to a CTA, and rows of several slices."""
    rows, vocab = 60000, 5000
    tokens = _tokens("zipf", rows, vocab)
    dy = torch.randn(rows, hidden, device="cuda").bfloat16()
    want = torch.empty(vocab, hidden, device="cuda")
    ws = _grad(b, dy, tokens, want, 1.0, 0, "bf16")
    assert b.tf_read_device_error() == (0, 0)
    old = b.tf_get_wait_limit_ns()
    try:
        b.tf_set_wait_limit_ns(0)
        for _ in range(5):
            dtable = torch.full((vocab, hidden), float("nan"), device="cuda")
            _grad(b, dy, tokens, dtable, 1.0, 0, "bf16", ws=ws)
            status, word = b.tf_read_device_error()
            if status == b.TF_OK:
                assert torch.equal(dtable, want)
            else:
                assert status == b.TF_ERR_TIMEOUT and word == b.TF_DEVERR_PRODUCER_WAIT
    finally:
        b.tf_set_wait_limit_ns(old)
    dtable = torch.full((vocab, hidden), float("nan"), device="cuda")
    _grad(b, dy, tokens, dtable, 1.0, 0, "bf16", ws=ws)
    assert b.tf_read_device_error() == (0, 0) and torch.equal(dtable, want)


# ---------------------------------------------------------------- linear cross entropy

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,vocab,hidden", [(60, 900, 256), (300, 900, 1100), (130, 70, 257), (4200, 40001, 512)])
def test_sure_targets_have_no_gradient(b, rows, vocab, hidden, dtype):
    """Targets whose logits, of some hundred, leave every other word's exponential below the smallest number: the
    loss is exactly 0, and so is every gradient, in one piece of the vocabulary and in several."""
    g = torch.Generator("cuda").manual_seed(rows)
    w = torch.randn(vocab, hidden, generator=g, device="cuda").to(TYPES[dtype])
    targets = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    size = 400.0 / hidden
    x = (size * (w[targets].float() + 0.1 * torch.randn(rows, hidden, generator=g, device="cuda"))).to(TYPES[dtype])
    l = x.double() @ w.double().t()
    hit = l.gather(1, targets[:, None])
    assert (l.scatter(1, targets[:, None], float("-inf")) < hit - 100).all()   # e^-88 is the smallest
    loss, lse = _forward(b, x, w, targets, dtype)
    assert (loss == 0).all() and ((lse.double() - hit[:, 0]).abs() <= 1e-2).all()
    dloss = torch.full((rows,), 1.0 / rows, device="cuda")
    dx, dw = _grads(b, x, w, targets, lse, dloss, None, dtype)
    assert (dx == 0).all() and (dw == 0).all()
