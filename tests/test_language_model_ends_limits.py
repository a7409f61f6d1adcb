"""The embedding and the linear cross entropy at their limits: waits that run out, sums of many terms of one sign,
sure targets, and forms that the other tests leave out.

Bounds.  u = 2^-24 and ut are half a step of fp32 and of the operands' type."""
import pytest
import torch

from test_embedding import _check_grad, _grad, _tokens
from test_linear_cross_entropy import _check_grads, _forward, _grads, _inputs, _weights
from train_reference import TYPES, U, half_step


@pytest.fixture(scope="module")
def b(cuda_ready):
    from gemm_conv_epilogues_gb300 import binding
    yield binding
    assert binding.tf_read_device_error() == (0, 0)


# ---------------------------------------------------------------- refusals (no GPU)

def test_scale_whose_exponents_overflow(native_lib):
    """The exponents take scale*log2(e): where that is infinite, a largest logit's 0*infinity would make every loss NaN."""
    from gemm_conv_epilogues_gb300 import binding as b
    p = 1 << 20
    n0 = b.tf_launch_count()

    def calls(scale):   # no rows: where the scale is accepted there is nothing to do
        return [b.tf_linear_cross_entropy_forward(None, 64, p, None, 1, None, None, 0, 100, 64, scale, -100, 1, None, 0, 0,
                                                  check=False),
                b.tf_linear_cross_entropy_backward(None, 64, p, None, 1, None, None, None, p, 64, None, 0, 100, 64, scale, -100, 0,
                                                   1, 1, None, 0, 0, check=False)]

    assert calls(3.0e38) == [b.TF_ERR_INVALID_ARG] * 2
    assert calls(2.35e38) == [b.TF_OK] * 2   # 2.35e38*log2(e) is 3.39e38, and the largest number 3.40e38
    assert b.tf_launch_count() == n0


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


def _one_rounding(value, dtype, unit):
    """A gradient of a logit as its type holds it in these units; that 1e-5 of its value does not change the rounding."""
    held = torch.tensor([value * unit * s for s in (1.0, 1 - 1e-5, 1 + 1e-5)], dtype=torch.float64).to(TYPES[dtype])
    assert held[0] == held[1] == held[2]
    return held[0].double().item() / unit


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [5000, 70001, (1 << 20) + 777])
def test_weight_gradient_of_many_rows_of_one_sign(b, rows, dtype):
    """Equal logits, so that every row's gradients of them are the same numbers, whose rounding is known; x positive.
    A part of a sum has 4096 terms, 256 accumulations, each truncated by at most 2u; the parts' sum rounds by u each."""
    vocab, hidden = 200, 24
    g = torch.Generator("cuda").manual_seed(rows)
    x = (1 + torch.rand(rows, hidden, generator=g, device="cuda")).to(TYPES[dtype])
    w = torch.zeros(vocab, hidden, dtype=TYPES[dtype], device="cuda")
    targets = torch.full((rows,), 3, device="cuda")
    loss, lse = _forward(b, x, w, targets, dtype)
    unit = 1.0 if dtype == "bf16" else 2.0 ** 14
    d = torch.full((vocab, 1), _one_rounding(1 / vocab, dtype, unit), dtype=torch.float64, device="cuda")
    d[3] = _one_rounding(1 / vocab - 1, dtype, unit)
    want = d * x.double().sum(0)
    _, dw = _grads(b, x, w, targets, lse, None, None, dtype, want=("dw",), dw_dtype="fp32")
    parts = (rows + 4095) // 4096
    assert ((dw.double() - want).abs() <= (2 * 256 + parts + 4) * U * want.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [4, 200])
def test_input_gradient_of_many_words_of_one_sign(b, rows, dtype):
    """Equal logits of four million words; positive weights, and dlse alone.  A part of a sum has 16384 terms, 1024
    accumulations, each truncated by at most 2u; up to 64 parts, splits and pieces are added to one result."""
    vocab, hidden = (1 << 22) - 333, 64
    g = torch.Generator("cuda").manual_seed(rows)
    w = torch.rand(vocab, hidden, generator=g, device="cuda").add_(1).to(TYPES[dtype])
    x = torch.zeros(rows, hidden, dtype=TYPES[dtype], device="cuda")
    targets = torch.arange(rows, device="cuda")
    loss, lse = _forward(b, x, w, targets, dtype)
    total = torch.zeros(hidden, dtype=torch.float64, device="cuda")
    for part in w.split(1 << 19):
        total += part.double().sum(0)
    d = _one_rounding(1 / vocab, dtype, 1.0 if dtype == "bf16" else 2.0 ** 14)
    zero, one = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dx, _ = _grads(b, x, w, targets, lse, zero, one, dtype, want=("dx",))
    off = half_step(dtype) + (2 * 1024 + 64) * U
    assert ((dx.double() - d * total).abs() <= off * d * total).all()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(4097, 1500, 328), (9001, 9001, 72), (100, 140001, 200), (140, 70001, 1002), (9000, 300, 65)], ids=str)
def test_gradients_in_several_parts(b, shape):
    """More than 4096 rows, words of a split, or both; tiles of every width, some of them empty."""
    x, w, targets = _inputs(*shape, "bf16", "some", pad=8, seed=18)
    loss, lse = _forward(b, x, w, targets, "bf16")
    dloss, dlse = _weights(targets)
    before = torch.randn(shape[1], shape[2], device="cuda")
    dw = before.clone()
    dx, _ = _grads(b, x, w, targets, lse, dloss, dlse, "bf16", dw=dw, dw_dtype="fp32", accumulate=1)
    _check_grads(x, w, targets, lse, dloss, dlse, "bf16", 1.0, dx, dw, "fp32", before)
    _, dw = _grads(b, x, w, targets, lse, dloss, dlse, "bf16")
    _check_grads(x, w, targets, lse, dloss, dlse, "bf16", 1.0, None, dw)
