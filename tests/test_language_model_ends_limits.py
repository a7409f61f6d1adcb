"""The embedding and the linear cross entropy at their limits: waits that run out, sums of many terms of one sign,
sure targets, and forms that the other tests leave out.

Bounds.  u = 2^-24 and ut are half a step of fp32 and of the operands' type."""
import pytest
import torch

from test_embedding import _check_grad, _grad, _tokens
from test_linear_cross_entropy import IGNORE, _check_grads, _forward, _grads, _inputs, _weights
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
    """A limit of nothing: a copy that has not come when a wait's looks are over (each waits some microseconds itself, so
    that all may come) is given up, and the error word says so; copies under way have landed before the kernel ends (no drain
    runs out), and later calls are not touched by it.  One, two and four pieces to a CTA, and rows of several slices."""
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


def _other_words(tokens, padding, vocab):
    """The tokens whose rows have a gradient; -1 in the others' places."""
    return torch.where((tokens == padding) | (tokens < 0) | (tokens >= vocab), -1, tokens)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [1, 0])
@pytest.mark.parametrize("vocab", [150001, 262144, 262145, 600001])
@pytest.mark.parametrize("rows", [900, 40000, 140000])
def test_orders_of_either_token_type(b, vocab, rows, wide):
    """One pass and two, tokens that a warp keeps marks of and those that it reads again, a padding that is a word, and
    tokens outside the vocabulary, far outside too."""
    g = torch.Generator("cuda").manual_seed(rows)
    padding = vocab // 3
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    tokens[::5] = tokens[0]          # a frequent word
    tokens[1::5] = tokens[1] % 262144 + 262144 * (vocab // 262144 - 1 if vocab > 262144 else 0)
    tokens[2::9] = padding
    dy = torch.randn(rows, 8, generator=g, device="cuda").half()
    for outside in (False, True):
        if outside:
            tokens[3::11] = vocab
            tokens[4::11] = (1 << 40) + 5 if wide else (1 << 31) - 1
            tokens[5::11] = -7
        keep = _other_words(tokens, padding, vocab)
        dy[keep < 0] = float("nan")
        before = torch.randn(vocab, 8, generator=g, device="cuda")
        for accumulate in (0, 1):
            dtable = before.clone()
            ws = torch.full((b.tf_embedding_backward_workspace_size(rows, vocab, 8),), 0xff, dtype=torch.uint8, device="cuda")
            b.tf_embedding_backward(dy, 8, tokens if wide else tokens.int(), wide, dtable, rows, vocab, 8, 1.5, padding,
                                    accumulate, b.TF_FP16, ws, ws.numel())
            assert b.tf_read_device_error() == ((b.TF_ERR_TIMEOUT, b.TF_DEVERR_INDEX) if outside else (0, 0))
            _check_grad(dtable, before, dy, keep, 1.5, accumulate)


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
@pytest.mark.parametrize("shape", [(4097, 1500, 328), (9001, 9001, 72), (100, 140001, 200), (140, 70001, 1002), (9000, 300, 65)],
                         ids=str)
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


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", [(3, 500, 64), (33, 700, 200), (600, 1111, 77)], ids=str)
def test_dlse_without_dloss(b, shape, dtype):
    x, w, targets = _inputs(*shape, dtype, "some", seed=19)
    loss, lse = _forward(b, x, w, targets, dtype)
    dlse = 0.5 * torch.randn(shape[0], device="cuda")
    dlse[targets == IGNORE] = float("nan")
    dx, dw = _grads(b, x, w, targets, lse, None, dlse, dtype, dw_dtype="fp32")
    _check_grads(x, w, targets, lse, None, dlse, dtype, 1.0, dx, dw, "fp32")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(4000, 40001, 40), (4200, 40001, 72), (5, 140001, 1003)], ids=str)
def test_accumulates_over_pieces(b, shape):
    """Each piece of the vocabulary (of gradients of logits, or of copied weights) adds to its own rows of dw, once."""
    x, w, targets = _inputs(*shape, "bf16", "some", seed=20)
    loss, lse = _forward(b, x, w, targets, "bf16")
    dloss, dlse = _weights(targets)
    before = torch.randn(shape[1], shape[2], device="cuda")
    dw = before.clone()
    dx, _ = _grads(b, x, w, targets, lse, dloss, dlse, "bf16", dw=dw, dw_dtype="fp32", accumulate=1)
    _check_grads(x, w, targets, lse, dloss, dlse, "bf16", 1.0, dx, dw, "fp32", before)


@pytest.mark.gpu
@pytest.mark.parametrize("offset", [1, 2, 3])
@pytest.mark.parametrize("shape", [(40, 333, 64), (300, 500, 264), (5000, 300, 72), (40, 333, 65)], ids=str)
def test_accumulates_at_odd_addresses(b, shape, offset):
    """A dw inside a 16-byte word, whose values are added one by one; nothing beside it is touched."""
    rows, vocab, hidden = shape
    x, w, targets = _inputs(*shape, "bf16", "some", seed=21)
    loss, lse = _forward(b, x, w, targets, "bf16")
    before = torch.randn(vocab, hidden, device="cuda")
    flat = torch.full((vocab * hidden + offset + 8,), 7.0, device="cuda")
    dw = flat[offset:offset + vocab * hidden].view(vocab, hidden)
    dw.copy_(before)
    _grads(b, x, w, targets, lse, None, None, "bf16", dw=dw, dw_dtype="fp32", accumulate=1)
    _check_grads(x, w, targets, lse, None, None, "bf16", 1.0, None, dw, "fp32", before)
    assert (flat[:offset] == 7.0).all() and (flat[offset + vocab * hidden:] == 7.0).all()


@pytest.mark.gpu
def test_input_gradient_of_weights_past_2_31(b):
    """Only the last two words, past 2^31 elements, have weights: dx is their two gradients of logits times those."""
    vocab, hidden, rows = 2_100_000, 1040, 3
    w = torch.zeros(vocab, hidden, dtype=torch.bfloat16, device="cuda")
    w[-1, :4], w[-2, :4] = 1.0, -0.5
    x = torch.zeros(rows, hidden, dtype=torch.bfloat16, device="cuda")
    x[:, :4] = torch.tensor([[2.0], [4.0], [0.0]], device="cuda")
    targets = torch.tensor([vocab - 1, 7, vocab - 2], device="cuda")
    loss, lse = _forward(b, x, w, targets, "bf16")
    dx, _ = _grads(b, x, w, targets, lse, None, None, "bf16", want=("dx",))
    l = torch.stack([4 * x[:, 0].double(), -2 * x[:, 0].double()], 1)
    d = torch.exp(l - torch.log(vocab - 2 + l.exp().sum(1, keepdim=True)))
    d -= torch.tensor([[1.0, 0], [0, 0], [0, 1.0]], device="cuda")
    ref = (d * torch.tensor([1.0, -0.5], device="cuda")).sum(1)
    # one rounding of each gradient of a logit and of the result; the exponentials' own 2^-17 of their value
    off = 2.0 ** -8 * ((d.abs() * torch.tensor([1.0, 0.5], device="cuda")).sum(1) * (1 + 2.0 ** -8) + ref.abs()) + 2.0 ** -17
    assert ((dx[:, :4].double() - ref[:, None]).abs() <= off[:, None]).all() and (dx[:, 4:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("mask", ["all", "most", "last"])
def test_masks_of_many_rows(b, mask, dtype):
    """More rows than one part of dw's sums, of which none count, or fewer than a part."""
    rows, vocab, hidden = 5000, 700, 136
    x, w, targets = _inputs(rows, vocab, hidden, dtype, mask, seed=22)
    if mask == "all":
        targets[:] = IGNORE
        x[:] = float("nan")
    loss, lse = _forward(b, x, w, targets, dtype)
    dloss, dlse = _weights(targets)
    dx, dw = _grads(b, x, w, targets, lse, dloss, dlse, dtype)
    _check_grads(x, w, targets, lse, dloss, dlse, dtype, 1.0, dx, dw)
    before = torch.randn(vocab, hidden, device="cuda")
    dw = before.clone()
    _grads(b, x, w, targets, lse, dloss, dlse, dtype, dw=dw, dw_dtype="fp32", accumulate=1, want=("dw",))
    _check_grads(x, w, targets, lse, dloss, dlse, dtype, 1.0, None, dw, "fp32", before)
    if mask == "all":
        assert torch.equal(dw, before)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(5000, 3000, 200), (64, 140001, 136), (300, 140001, 72), (4200, 40001, 72)], ids=str)
def test_equal_bits_of_parts(b, shape):
    """Sums whose parts are added in registers or in memory, over splits and pieces: the same bits again, also from a
    graph, over a workspace that holds other numbers."""
    x, w, targets = _inputs(*shape, "bf16", "some", seed=23)
    loss, lse = _forward(b, x, w, targets, "bf16")
    dloss, dlse = _weights(targets)
    ws = torch.full((b.tf_linear_cross_entropy_backward_workspace_size(*shape, 1),), 0xff, dtype=torch.uint8, device="cuda")
    first = _grads(b, x, w, targets, lse, dloss, dlse, "bf16", ws=ws)
    for fill in (0x3f, 0xc1):
        ws.fill_(fill)
        again = _grads(b, x, w, targets, lse, dloss, dlse, "bf16", ws=ws)
        assert all(torch.equal(p, q) for p, q in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _grads(b, x, w, targets, lse, dloss, dlse, "bf16", ws=ws)
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(first, outs))
