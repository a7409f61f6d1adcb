"""Softmax cross entropy over a vocabulary without kept logits, and its gradients:
refusals on the host, and the kernels against 64-bit forms with derived bounds.

Bounds.  u = 2^-24, ut half a step of the operands' type.  A product's accumulator is
truncated once per 16 terms: 2*(n/16 + 32)*u*sum|terms| (the 32 for the additions outside).
A logit is off by e_l, so lse by the largest e_l, 2^-20 for the exponentials (2^-22 each) and
their sum's additions, and its own rounding; the loss by lse's and the target's.  A gradient
of a logit p*ca - cb is off by p*ca times (e_l + the rounding of its exponent + 2^-20), and is rounded to the
type; fp16 holds it in units in which its smallest step is 2^-39 of the largest |dloss| + |dlse|."""
import math

import pytest
import torch

from train_reference import CODES, TINY, TYPES, U, half_step

HALF = ("bf16", "fp16")
IGNORE = -100


# ---------------------------------------------------------------- refusals (no GPU)

def test_forward_refusals(native_lib):
    from gemm_conv_epilogues_gb300 import binding as b
    S, W, p = b.TF_ERR_INVALID_ARG, b.TF_ERR_UNSUPPORTED, 1 << 20
    size = b.tf_linear_cross_entropy_forward_workspace_size
    need = size(4, 100, 64, 1)
    assert need > 0 and size(4, 100, 64, b.TF_FP32) == 0 and size(-1, 100, 64, 1) == 0 and size(4, 0, 64, 1) == 0

    def call(x=p, stride=64, w=p, targets=p, index=1, loss=p, lse=p, rows=4, vocab=100, hidden=64, scale=1.0, dtype=1, ws=p,
             wsb=need):
        return b.tf_linear_cross_entropy_forward(x, stride, w, targets, index, loss, lse, rows, vocab, hidden, scale, IGNORE,
                                                 dtype, ws, wsb, 0, check=False)

    n0 = b.tf_launch_count()
    for name in ("x", "w", "targets", "loss", "lse", "ws"):
        assert call(**{name: None}) == S, name
    assert call(rows=-1) == S and call(vocab=0) == S and call(hidden=0) == S and call(stride=63) == S
    assert call(index=2) == S and call(dtype=3) == S and call(wsb=need - 1) == S
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert call(scale=scale) == S, scale
    assert call(dtype=b.TF_FP32) == W and call(rows=(1 << 22) + 1) == W and call(vocab=(1 << 22) + 1) == W
    assert call(hidden=65537, stride=1 << 20) == W and call(stride=(1 << 31) + 1) == W
    assert call(x=p + 1) == W and call(w=p + 8) == W and call(w=p + 1, hidden=63) == W and call(targets=p + 4) == W
    assert call(loss=p + 2) == W and call(lse=p + 2) == W and call(ws=p + 8) == W
    assert call(rows=0, x=None, targets=None, loss=None, lse=None, ws=None, wsb=0) == b.TF_OK
    assert b.tf_launch_count() == n0


def test_backward_refusals(native_lib):
    from gemm_conv_epilogues_gb300 import binding as b
    S, W, p = b.TF_ERR_INVALID_ARG, b.TF_ERR_UNSUPPORTED, 1 << 20
    size = b.tf_linear_cross_entropy_backward_workspace_size
    need = size(4, 100, 64, 1)
    assert need > 0 and size(4, 100, 64, b.TF_FP32) == 0

    def call(x=p, stride=64, w=p, targets=p, index=1, lse=p, dloss=p, dlse=p, dx=p, dx_stride=64, dw=p, rows=4, vocab=100,
             hidden=64, scale=1.0, acc=0, dw_dtype=1, dtype=1, ws=p, wsb=need):
        return b.tf_linear_cross_entropy_backward(x, stride, w, targets, index, lse, dloss, dlse, dx, dx_stride, dw, rows,
                                                  vocab, hidden, scale, IGNORE, acc, dw_dtype, dtype, ws, wsb, 0, check=False)

    n0 = b.tf_launch_count()
    for name in ("x", "w", "targets", "lse", "ws"):
        assert call(**{name: None}) == S, name
    assert call(dx=None, dw=None) == S and call(dx_stride=63) == S and call(stride=63) == S and call(scale=0.0) == S
    assert call(rows=-1) == S and call(vocab=0) == S and call(hidden=0) == S and call(dw_dtype=3) == S and call(wsb=need - 1) == S
    assert call(dtype=b.TF_FP32, dw_dtype=b.TF_FP32) == W and call(dw_dtype=b.TF_FP16) == W and call(acc=1) == W
    assert call(dx_stride=(1 << 31) + 1) == W and call(rows=(1 << 22) + 1) == W and call(vocab=(1 << 22) + 1) == W
    assert call(x=p + 1) == W and call(dx=p + 1) == W and call(dw=p + 1) == W and call(dw=p + 2, dw_dtype=b.TF_FP32) == W
    assert call(lse=p + 2) == W and call(dloss=p + 2) == W and call(dlse=p + 2) == W and call(ws=p + 8) == W
    assert call(rows=0, x=None, targets=None, lse=None, dw=None, ws=None, wsb=0) == b.TF_OK
    assert call(rows=0, x=None, targets=None, lse=None, acc=1, dw_dtype=b.TF_FP32, ws=None, wsb=0) == b.TF_OK
    assert b.tf_launch_count() == n0


@pytest.mark.parametrize("vocab,hidden", [(1, 1), (100, 64), (10007, 1002), (32000, 2048), (128000, 4096), (262144, 65536),
                                          (1 << 22, 128)])
def test_workspaces_do_not_fall(native_lib, vocab, hidden):
    from gemm_conv_epilogues_gb300 import binding as b
    rows = sorted({r + d for k in range(0, 23) for r in (1 << k, 3 << max(k - 2, 0), 5 << max(k - 3, 0)) for d in (-1, 0, 1)
                   if 0 <= r + d <= 1 << 22})
    for size in (b.tf_linear_cross_entropy_forward_workspace_size, b.tf_linear_cross_entropy_backward_workspace_size):
        sizes = [size(r, vocab, hidden, 1) for r in rows]
        assert sizes == sorted(sizes) and sizes[0] > 0


# ---------------------------------------------------------------- numerics

@pytest.fixture(scope="module")
def b(cuda_ready):
    from gemm_conv_epilogues_gb300 import binding
    yield binding
    assert binding.tf_read_device_error() == (0, 0)


def _inputs(rows, vocab, hidden, dtype, mask="none", pad=0, offset=0, seed=0, spread=1.5):
    """x (in a wider buffer), w, targets: words outside `mask`, IGNORE in it."""
    g = torch.Generator("cuda").manual_seed(seed)
    t = TYPES[dtype]
    flat = torch.full((rows * (hidden + pad) + offset + 8,), float("nan"), device="cuda", dtype=t)
    x = flat[offset:offset + rows * (hidden + pad)].view(rows, hidden + pad)[:, :hidden]
    x.copy_(torch.randn(rows, hidden, generator=g, device="cuda"))
    w = (spread * hidden ** -0.5 * torch.randn(vocab, hidden, generator=g, device="cuda")).to(t)
    targets = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    targets[0], targets[-1] = 0, vocab - 1
    share = {"none": 0.0, "some": 0.4, "most": 0.9, "all": 2.0, "last": 0.0}[mask]
    targets[torch.rand(rows, generator=g, device="cuda") < share] = IGNORE
    if mask == "last":
        targets[rows // 2:] = IGNORE
    x[targets == IGNORE] = float("nan")   # what is masked reaches nothing
    return x, w, targets


def _space(size):
    return torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")   # NaN, whatever the type


def _forward(b, x, w, targets, dtype, scale=1.0, wide=1, ws=None, stream=None):
    rows, hidden, vocab = x.shape[0], x.shape[1], w.shape[0]
    loss, lse = (torch.full((rows,), float("nan"), device="cuda") for _ in range(2))
    if ws is None:
        ws = _space(b.tf_linear_cross_entropy_forward_workspace_size(rows, vocab, hidden, CODES[dtype]))
    b.tf_linear_cross_entropy_forward(x, x.stride(0), w, targets if wide else targets.int(), wide, loss, lse, rows, vocab,
                                      hidden, scale, IGNORE, CODES[dtype], ws, ws.numel(), stream)
    return loss, lse


def _logits(x, w, scale):
    """64-bit logits and what they are off by, of rows that count."""
    xd, wd, n = x.double(), w.double(), x.shape[1]
    return scale * xd @ wd.t(), scale * 2 * (n / 16 + 32) * U * (xd.abs() @ wd.abs().t())


def _check_forward(x, w, targets, scale, loss, lse):
    keep = targets != IGNORE
    assert (loss[~keep] == 0).all() and (lse[~keep] == 0).all()
    l, e = _logits(x[keep], w, scale)
    want = torch.logsumexp(l, 1)
    at = targets[keep, None]
    off = e.amax(1) + 2.0 ** -20 + 4 * U * want.abs()
    assert ((lse[keep].double() - want).abs() <= off).all()
    hit = l.gather(1, at)[:, 0]
    off = off + e.gather(1, at)[:, 0] + 4 * U * (want - hit).abs()
    assert ((loss[keep].double() - (want - hit)).abs() <= off).all()


# rows about the tiles' ends (128 on single CTAs up to 256 rows, 512 on pairs), odd vocabularies and widths
SHAPES = [(1, 1, 8), (1, 1000, 64), (3, 70, 1), (5, 40000, 72), (100, 3001, 100), (127, 257, 200), (128, 256, 64),
          (129, 999, 65), (255, 511, 128), (256, 2048, 640), (257, 1025, 264), (511, 300, 63), (513, 5000, 512),
          (1100, 2999, 1000), (1536, 777, 24)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("mask", ["none", "some"])
def test_forward(b, shape, dtype, mask):
    x, w, targets = _inputs(*shape, dtype, mask, pad=8)
    _check_forward(x, w, targets, 1.0, *_forward(b, x, w, targets, dtype))


def _grads(b, x, w, targets, lse, dloss, dlse, dtype, scale=1.0, want=("dx", "dw"), dw_dtype=None, dw=None, accumulate=0, pad=0,
           wide=1, ws=None, stream=None, offset=0):
    rows, hidden, vocab = x.shape[0], x.shape[1], w.shape[0]
    t = TYPES[dtype]
    dw_dtype = dw_dtype or dtype
    flat = torch.full((rows * (hidden + pad) + offset + 8,), 7.0, device="cuda", dtype=t)
    dx = flat[offset:offset + rows * (hidden + pad)].view(rows, hidden + pad)[:, :hidden]
    if dw is None:
        dw = torch.full((vocab * hidden + offset + 8,), 7.0, device="cuda", dtype=TYPES[dw_dtype])
        dw = dw[offset:offset + vocab * hidden].view(vocab, hidden)
    if ws is None:
        ws = _space(b.tf_linear_cross_entropy_backward_workspace_size(rows, vocab, hidden, CODES[dtype]))
    b.tf_linear_cross_entropy_backward(x, x.stride(0), w, targets if wide else targets.int(), wide, lse, dloss, dlse,
                                       dx if "dx" in want else None, dx.stride(0), dw if "dw" in want else None, rows, vocab,
                                       hidden, scale, IGNORE, accumulate, CODES[dw_dtype], CODES[dtype], ws, ws.numel(),
                                       stream)
    if pad or offset:
        kept = flat.clone()
        kept[offset:offset + rows * (hidden + pad)].view(rows, -1)[:, :hidden] = 7.0
        assert (kept == 7.0).all()
    return dx, dw


def _check_grads(x, w, targets, lse, dloss, dlse, dtype, scale, dx=None, dw=None, dw_dtype=None, before=None):
    keep = targets != IGNORE
    xk, wd, at = x[keep].double(), w.double(), targets[keep, None]
    l, e = _logits(x[keep], w, scale)
    ut, z = half_step(dtype), lse.double()[keep, None]
    g = dloss.double()[keep, None] if dloss is not None else torch.ones_like(z)
    ca = g + dlse.double()[keep, None] if dlse is not None else g
    p = torch.exp(l - z) * ca
    d = p.scatter_add(1, at, -g)
    off = p.abs() * (e + 4 * U * (l.abs() + z.abs()) + 2.0 ** -20) + ut * d.abs() + 4 * U * torch.zeros_like(p).scatter_add(1, at, g.abs())
    off = (1 + ut) * off
    if dtype == "fp16" and g.numel():
        off = off + 2.0 ** -39 * (g.abs() + (ca - g).abs()).max()
    else:
        off = off + 2.0 ** -126
    if dx is not None:
        assert (dx[~keep] == 0).all()
        ref = scale * d @ wd
        bound = scale * (off @ wd.abs() + 2 * (w.shape[0] / 16 + 64) * U * (d.abs() @ wd.abs()))
        assert ((dx[keep].double() - ref).abs() <= (1 + ut) * bound + (ut + 2 * U) * ref.abs() + TINY[dtype]).all()
    if dw is not None:
        uw = half_step(dw_dtype or dtype)
        ref = scale * d.t() @ xk
        bound = scale * (off.t() @ xk.abs() + 2 * (keep.sum() / 16 + 64) * U * (d.abs().t() @ xk.abs()))
        if before is not None:
            ref, bound = ref + before.double(), bound + 2 * U * before.double().abs()
        assert ((dw.double() - ref).abs() <= (1 + uw) * bound + (uw + 2 * U) * ref.abs() + TINY[dw_dtype or dtype]).all()


def _weights(targets, seed=5, lse=True):
    """Gradients of the loss (a weighted mean) and of lse."""
    g = torch.Generator("cuda").manual_seed(seed)
    rows = targets.numel()
    dloss = (0.5 + torch.rand(rows, generator=g, device="cuda")) / max(1, int((targets != IGNORE).sum()))
    dlse = 0.1 * torch.randn(rows, generator=g, device="cuda") * dloss if lse else None
    bad = targets == IGNORE
    dloss[bad] = float("nan")
    if lse:
        dlse[bad] = float("inf")
    return dloss, dlse


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("mask", ["none", "some"])
def test_backward(b, shape, dtype, mask):
    x, w, targets = _inputs(*shape, dtype, mask, pad=8, seed=1)
    loss, lse = _forward(b, x, w, targets, dtype)
    dloss, dlse = _weights(targets, lse=mask == "some")
    lse = torch.where(targets == IGNORE, float("nan"), lse)
    dx, dw = _grads(b, x, w, targets, lse, dloss, dlse, dtype, pad=8)
    _check_grads(x, w, targets, lse, dloss, dlse, dtype, 1.0, dx, dw)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("rows", [200, 700])
@pytest.mark.parametrize("mask", ["most", "all", "last"])
def test_masks(b, rows, dtype, mask):
    """Few rows left, none, and a padded batch; dw joins what is there or replaces it."""
    vocab, hidden = 1500, 136
    x, w, targets = _inputs(rows, vocab, hidden, dtype, mask, seed=2)
    if mask == "all":
        targets[:] = IGNORE
        x[:] = float("nan")
    loss, lse = _forward(b, x, w, targets, dtype)
    _check_forward(x, w, targets, 1.0, loss, lse)
    dloss, dlse = _weights(targets)
    dx, dw = _grads(b, x, w, targets, lse, dloss, dlse, dtype)
    _check_grads(x, w, targets, lse, dloss, dlse, dtype, 1.0, dx, dw)
    before = torch.randn(vocab, hidden, device="cuda")
    dw = before.clone()
    _grads(b, x, w, targets, lse, dloss, dlse, dtype, dw=dw, dw_dtype="fp32", accumulate=1)
    _check_grads(x, w, targets, lse, dloss, dlse, dtype, 1.0, None, dw, "fp32", before)
    if mask == "all":
        assert torch.equal(dw, before)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(33, 700, 200), (600, 1111, 77), (300, 500, 1002)], ids=str)
@pytest.mark.parametrize("want", [("dx",), ("dw",), ("dx", "dw")], ids=str)
def test_results_wanted_and_types(b, shape, want):
    """dx alone, dw alone, fp32 dw, other alignments, 32-bit targets, a scale, and no dloss."""
    x, w, targets = _inputs(*shape, "bf16", "some", pad=3, offset=1, seed=3)
    scale = 0.375
    loss, lse = _forward(b, x, w, targets, "bf16", scale, wide=0)
    _check_forward(x, w, targets, scale, loss, lse)
    for dw_dtype, offset in (("bf16", 0), ("fp32", 0), ("bf16", 1), ("fp32", 1)):
        dx, dw = _grads(b, x, w, targets, lse, None, None, "bf16", scale, want, dw_dtype, wide=0, pad=offset, offset=offset)
        _check_grads(x, w, targets, lse, None, None, "bf16", scale, dx if "dx" in want else None, dw if "dw" in want else None,
                     dw_dtype)
        assert "dx" in want or (dx == 7.0).all()
        assert "dw" in want or (dw == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALF)
def test_pieces_of_the_vocabulary(b, dtype):
    """More gradients of logits than one piece holds: several pieces, the last one odd, over whole and split sums of dx."""
    for rows, vocab, hidden in ((4200, 40001, 72), (4608, 33000, 16)):
        x, w, targets = _inputs(rows, vocab, hidden, dtype, "some", seed=4)
        loss, lse = _forward(b, x, w, targets, dtype)
        _check_forward(x, w, targets, 1.0, loss, lse)
        dloss, dlse = _weights(targets)
        dx, dw = _grads(b, x, w, targets, lse, dloss, dlse, dtype, dw_dtype="fp32")
        _check_grads(x, w, targets, lse, dloss, dlse, dtype, 1.0, dx, dw, "fp32")


@pytest.mark.gpu
def test_pieces_of_odd_weights(b):
    """Weights of an odd width that are copied in more than one piece."""
    x, w, targets = _inputs(5, 140001, 1003, "bf16", seed=6)
    loss, lse = _forward(b, x, w, targets, "bf16")
    _check_forward(x, w, targets, 1.0, loss, lse)
    dloss, dlse = _weights(targets)
    dx, dw = _grads(b, x, w, targets, lse, dloss, dlse, "bf16")
    _check_grads(x, w, targets, lse, dloss, dlse, "bf16", 1.0, dx, dw)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [64, 600])
def test_far_logits(b, rows):
    """Logits of some hundred: sure targets' losses keep their digits, hopeless ones' are their logits' distance."""
    x, w, targets = _inputs(rows, 900, 128, "bf16", seed=7, spread=40.0)
    l = x.double() @ w.double().t()
    targets[: rows // 2] = l[: rows // 2].argmax(1)
    loss, lse = _forward(b, x, w, targets, "bf16")
    _check_forward(x, w, targets, 1.0, loss, lse)
    sure = (torch.topk(l, 2).values.diff(dim=1)[:, 0] < -40)[: rows // 2]
    assert sure.any() and (loss[: rows // 2][sure] == 0).all()
    dx, dw = _grads(b, x, w, targets, lse, None, None, "bf16")
    _check_grads(x, w, targets, lse, None, None, "bf16", 1.0, dx, dw)


@pytest.mark.gpu
def test_fp16_small_gradients(b):
    """A mean over many rows: shares of 1e-8 that fp16 itself could not hold; and a loss scale of 2^20."""
    for factor in (1.0, 2.0 ** 20):
        x, w, targets = _inputs(700, 9000, 64, "fp16", seed=8, spread=0.5)
        loss, lse = _forward(b, x, w, targets, "fp16")
        dloss = torch.full((700,), factor * 2.0 ** -14, device="cuda")
        dloss[3] = factor * 2.0 ** -24      # a row that weighs a thousandth
        dx, dw = _grads(b, x, w, targets, lse, dloss, None, "fp16", dw_dtype="fp32")
        _check_grads(x, w, targets, lse, dloss, None, "fp16", 1.0, dx if factor > 1 else None, dw, "fp32")


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [9, 300])
def test_targets_outside_and_nan_rows(b, rows):
    """Targets that are no words are ignored and reported; a NaN in a row that counts stays in its results."""
    vocab, hidden = 300, 64
    x, w, targets = _inputs(rows, vocab, hidden, "bf16", seed=9)
    targets[[1, 4, 5]] = torch.tensor([vocab, -1, 1 << 40], device="cuda")
    x[[1, 4, 5]] = float("nan")
    assert b.tf_read_device_error() == (0, 0)
    loss, lse = _forward(b, x, w, targets, "bf16")
    assert b.tf_read_device_error() == (b.TF_ERR_TIMEOUT, b.TF_DEVERR_INDEX)
    dx, dw = _grads(b, x, w, targets, lse, None, None, "bf16")
    assert b.tf_read_device_error() == (b.TF_ERR_TIMEOUT, b.TF_DEVERR_INDEX)
    targets[[1, 4, 5]] = IGNORE
    _check_forward(x, w, targets, 1.0, loss, lse)
    _check_grads(x, w, targets, lse, None, None, "bf16", 1.0, dx, dw)
    x[7, 3] = float("nan")
    loss, lse = _forward(b, x, w, targets, "bf16")
    assert loss[7].isnan() and lse[7].isnan()
    others = [i for i in range(rows) if i != 7]
    assert loss[others].isfinite().all() and lse[others].isfinite().all()
    dx, _ = _grads(b, x, w, targets, lse, None, None, "bf16", want=("dx",))
    assert dx[7].isnan().all() and dx[others].isfinite().all()


@pytest.mark.gpu
def test_without_rows(b):
    w = torch.randn(100, 64, device="cuda").bfloat16()
    ws = _space(b.tf_linear_cross_entropy_backward_workspace_size(0, 100, 64, 1))
    for dw in (torch.full((100, 64), 3.0, device="cuda"), torch.full((100, 64), 3.0, device="cuda").bfloat16()):
        b.tf_linear_cross_entropy_backward(None, 0, w, None, 1, None, None, None, None, 0, dw, 0, 100, 64, 1.0, IGNORE, 0,
                                           2 if dw.dtype == torch.float32 else 1, 1, ws, ws.numel())
        assert (dw == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [40, 900])
def test_equal_bits_streams_and_graphs(b, rows):
    """The same bits again, on another stream, with a workspace for more rows, and from graphs replayed side by side."""
    vocab, hidden = 3333, 192
    sets = [_inputs(rows, vocab, hidden, "bf16", "some", seed=10 + i) for i in range(2)]
    sizes = [f(2 * rows, vocab, hidden, 1) for f in (b.tf_linear_cross_entropy_forward_workspace_size,
                                                     b.tf_linear_cross_entropy_backward_workspace_size)]
    ws = [_space(max(sizes)) for _ in sets]
    weights = [_weights(t) for _, _, t in sets]

    def step(i, stream=None):
        x, w, t = sets[i]
        loss, lse = _forward(b, x, w, t, "bf16", ws=ws[i], stream=stream)
        return [loss, lse, *_grads(b, x, w, t, lse, *weights[i], "bf16", dw_dtype="fp32", ws=ws[i], stream=stream)]

    first = [step(i) for i in range(2)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = step(0)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first[0], again))
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            outs.append(step(i))
    for _ in range(2):
        for o in outs:
            for v in o:
                v.fill_(float("nan"))
        torch.cuda.synchronize()
        for i, s in enumerate((side, torch.cuda.Stream())):
            with torch.cuda.stream(s):
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(p, q) for p, q in zip(first[i], outs[i]))
    sets[0][2].copy_(torch.where(sets[0][2] == IGNORE, 3, sets[0][2]))   # other targets under the same graph
    sets[0][0].nan_to_num_()
    weights[0][0].nan_to_num_()
    weights[0][1].nan_to_num_(posinf=0.0)
    graphs[0].replay()
    x, w, t = sets[0]
    _check_forward(x, w, t, 1.0, *outs[0][:2])
    _check_grads(x, w, t, outs[0][1], *weights[0], "bf16", 1.0, *outs[0][2:], dw_dtype="fp32")


@pytest.mark.gpu
def test_gradients_against_differences(b):
    """(L(x + hd) - L(x - hd))/2h along a direction of signs.  The third derivative is a third cumulant of u = w.d
    under the softmax, at most 0.1 R^3 for u's range R; x lies on a grid that h*d does not leave."""
    rows, vocab, hidden, h = 5, 600, 64, 2.0 ** -4
    x, w, targets = _inputs(rows, vocab, hidden, "fp16", seed=11)
    x.copy_((x * 32).round() / 32)
    d = torch.where(torch.rand(rows, hidden, device="cuda") < 0.5, -1.0, 1.0).half()
    _, lse = _forward(b, x, w, targets, "fp16")
    up, down = (_forward(b, (x + s * h * d).half(), w, targets, "fp16")[0].double() for s in (1, -1))
    dx, _ = _grads(b, x, w, targets, lse, None, None, "fp16", want=("dx",))
    slope = (dx.double() * d.double()).sum(1)
    u = d.double() @ w.double().t()
    span = u.amax(1) - u.amin(1)
    _, e = _logits(x, w, 1.0)
    loss_off = 2 * e.amax() + 2.0 ** -19
    l = torch.softmax(x.double() @ w.double().t(), 1).scatter_add(1, targets[:, None], torch.full((rows, 1), -1.0, device="cuda", dtype=torch.double))
    dx_off = 4 * half_step("fp16") * (l.abs() @ w.double().abs()).sum(1)
    assert ((up - down) / (2 * h) - slope).abs().le(h * h / 60 * span ** 3 + loss_off / h + dx_off).all()


@pytest.mark.gpu
@pytest.mark.parametrize("hidden", [1, 2, 7, 9, 17, 63, 255, 1001])
@pytest.mark.parametrize("offset", [0, 1, 2, 3])
def test_weights_at_odd_addresses(b, hidden, offset):
    """Widths that are copied, from every place inside a 64-bit word; the gradient goes to such a place too."""
    rows, vocab = 40, 333
    x, w, targets = _inputs(rows, vocab, hidden, "fp16", "some", seed=12)
    flat = torch.full((vocab * hidden + offset + 8,), float("nan"), device="cuda", dtype=torch.float16)
    view = flat[offset:offset + vocab * hidden].view(vocab, hidden)
    view.copy_(w)
    loss, lse = _forward(b, x, view, targets, "fp16")
    _check_forward(x, w, targets, 1.0, loss, lse)
    for dw_dtype in ("fp16", "fp32"):
        dx, dw = _grads(b, x, view, targets, lse, None, None, "fp16", dw_dtype=dw_dtype, offset=offset)
        _check_grads(x, w, targets, lse, None, None, "fp16", 1.0, dx, dw, dw_dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("rows", [607, 609, 16385, 20011])
def test_many_rows(b, rows, dtype):
    """Rows that are brought together one per CTA, one per warp and several per warp, past the first 256 of a CTA's."""
    x, w, targets = _inputs(rows, 130, 16, dtype, "some", pad=5, seed=13)
    targets[:300] = IGNORE            # the first row that counts is not among the first
    x[:300] = float("nan")
    loss, lse = _forward(b, x, w, targets, dtype)
    _check_forward(x, w, targets, 1.0, loss, lse)
    dloss, dlse = _weights(targets)
    dx, dw = _grads(b, x, w, targets, lse, dloss, dlse, dtype, dw_dtype="fp32")
    _check_grads(x, w, targets, lse, dloss, dlse, dtype, 1.0, dx, dw, "fp32")


@pytest.mark.gpu
def test_rows_past_the_first_target_block(b):
    """More rows per CTA than threads (from 2^19 rows on)."""
    rows = (1 << 19) + 3
    x, w, targets = _inputs(rows, 3, 8, "bf16", "some", seed=14)
    loss, lse = _forward(b, x, w, targets, "bf16")
    _check_forward(x, w, targets, 1.0, loss, lse)
    dx, _ = _grads(b, x, w, targets, lse, None, None, "bf16", want=("dx",))
    _check_grads(x, w, targets, lse, None, None, "bf16", 1.0, dx)


@pytest.mark.gpu
def test_weights_of_any_size_of_dloss(b):
    """Units of the gradients: a first row's dloss of zero, tiny, huge and negative; and rows that differ by 2^20."""
    for first in (0.0, 2.0 ** -60, 2.0 ** 60, -3.0):
        for dtype in HALF:
            x, w, targets = _inputs(300, 500, 64, dtype, seed=15)
            loss, lse = _forward(b, x, w, targets, dtype)
            dloss = torch.full((300,), 0.3, device="cuda")
            dloss[0] = first
            dloss[5] = 0.3 * 2.0 ** -20
            if dtype == "fp16" and first == 2.0 ** 60:
                continue   # (dx of such a row is not an fp16 number)
            dx, dw = _grads(b, x, w, targets, lse, dloss, None, dtype, dw_dtype="fp32")
            _check_grads(x, w, targets, lse, dloss, None, dtype, 1.0, dx, dw, "fp32")


@pytest.mark.gpu
def test_large_offsets(b):
    """Weights and their gradient past 2^31 elements: zeros but for the last words."""
    vocab, hidden, rows = 2_100_000, 1040, 3
    w = torch.zeros(vocab, hidden, dtype=torch.bfloat16, device="cuda")
    w[-1, :4], w[-2, :4] = 1.0, -0.5
    x = torch.zeros(rows, hidden, dtype=torch.bfloat16, device="cuda")
    x[:, :4] = torch.tensor([[2.0], [4.0], [0.0]], device="cuda")
    targets = torch.tensor([vocab - 1, 7, vocab - 2], device="cuda")
    loss, lse = _forward(b, x, w, targets, "bf16")
    l = torch.zeros(rows, 2, dtype=torch.float64, device="cuda")
    l[:, 0], l[:, 1] = 4 * x[:, 0].double(), -2 * x[:, 0].double()   # the last word's logits, and those of the one before
    want = torch.log(vocab - 2 + l.exp().sum(1))
    assert ((lse.double() - want).abs() <= 2.0 ** -18).all()
    assert ((loss.double() - (want - torch.stack([l[0, 0], 0 * l[1, 0], l[2, 1]]))).abs() <= 2.0 ** -18).all()
    dx, dw = _grads(b, x, w, targets, lse, None, None, "bf16")
    p = torch.exp(l - want[:, None])
    d = p - torch.tensor([[1.0, 0], [0, 0], [0, 1.0]], device="cuda")
    ref = d.t() @ x[:, :4].double()
    # one rounding of each gradient of a logit, one of the result
    bound = 2.0 ** -8 * (d.abs().t() @ x[:, :4].double().abs()) + 2.0 ** -15
    assert ((dw[[-1, -2], :4].double() - ref).abs() <= bound).all()
    # the other words' shares, 1/2.1e6 or less of x
    assert (dw[:-2].abs().amax() <= 4.0 + 1e-3) and (dw[7, 0] + 4.0).abs() <= 0.02
    others = dw[8:vocab - 2]
    assert others.abs().amax() <= 6.1 / 2.0e6


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 300])
@pytest.mark.parametrize("hidden", [1024, 1032, 8200, 65536])
def test_long_sums_of_one_sign(b, rows, hidden):
    """Equal terms, whose truncation adds up: a part has 64 accumulations, each off by at most 2u of its sum, and
    the parts' sum one rounding per part."""
    vocab = 270
    x = torch.full((rows, hidden), 1.1, device="cuda").bfloat16()
    w = torch.full((vocab, hidden), 1.1, device="cuda").bfloat16()
    targets = torch.arange(rows, device="cuda") % vocab
    scale = torch.tensor(60.0 / hidden).item()
    loss, lse = _forward(b, x, w, targets, "bf16", scale)
    l = scale * hidden * float(x[0, 0]) * float(w[0, 0])
    parts = (hidden + 1023) // 1024
    assert ((lse.double() - (l + math.log(vocab))).abs() <= (2 * 64 + parts + 4) * U * l + 2.0 ** -20 + 4 * U * l).all()
    assert ((loss.double() - math.log(vocab)).abs() <= 2.0 ** -19).all()   # (every logit is off by the same)


@pytest.mark.gpu
def test_wide_rows(b):
    """The widest rows, and rows whose sums end inside a part."""
    for rows, vocab, hidden in ((3, 300, 65536), (140, 90, 9000), (5, 70, 1025)):
        x, w, targets = _inputs(rows, vocab, hidden, "bf16", "some", pad=8, seed=16)
        loss, lse = _forward(b, x, w, targets, "bf16")
        _check_forward(x, w, targets, 1.0, loss, lse)
        dx, dw = _grads(b, x, w, targets, lse, None, None, "bf16")
        _check_grads(x, w, targets, lse, None, None, "bf16", 1.0, dx, dw)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES + [(301, 10007, 8), (700, 1927, 16), (3000, 1000, 16), (3000, 257, 7), (9000, 300, 8),
                                            (4200, 40001, 24), (5, 140001, 1003)], ids=str)
def test_workspaces_are_kept_to(b, shape):
    """Nothing is written behind the bytes that the size functions ask for."""
    rows, vocab, hidden = shape
    x, w, targets = _inputs(rows, vocab, hidden, "fp16", seed=17)
    spaces = []

    def space(size):
        spaces.append((size, torch.full((size + (1 << 20),), 0xa5, dtype=torch.uint8, device="cuda")))
        return spaces[-1][1][:size]

    ws = space(b.tf_linear_cross_entropy_forward_workspace_size(rows, vocab, hidden, 0))
    loss, lse = _forward(b, x, w, targets, "fp16", ws=ws)
    ws = space(b.tf_linear_cross_entropy_backward_workspace_size(rows, vocab, hidden, 0))
    _grads(b, x, w, targets, lse, None, None, "fp16", ws=ws)
    for size, buffer in spaces:
        assert (buffer[size:] == 0xa5).all()
