"""The embedding and the linear cross entropy at their limits: waits that run out, sums of many terms of one sign,
sure targets, and forms that the other tests leave out.

Bounds.  u = 2^-24 and ut are half a step of fp32 and of the operands' type."""
import pytest
import torch

from test_embedding import _check_grad, _grad, _tokens


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
