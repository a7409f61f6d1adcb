"""Layer norm with saved statistics and its backward pass: refusals on the
host, and the kernels against the 64-bit formulas with derived bounds."""
import pytest
import torch

import train_reference as ref
from train_reference import CODES, TYPES

EPS = 1e-5


# ---------------------------------------------------------------- refusals (no GPU)

def test_forward_refusals(native_lib):
    from gemm_conv_epilogues_gb300 import binding as b
    S, U = b.TF_ERR_INVALID_ARG, b.TF_ERR_UNSUPPORTED
    p = 1 << 20

    def call(x=p, xs=64, res=p, rs=64, gamma=p, beta=p, y=p, ys=64, s=p, ss=64, mean=p, rstd=p, rows=4, hidden=64,
             eps=EPS, dtype=b.TF_BF16):
        return b.tf_layernorm_forward(x, xs, res, rs, gamma, beta, y, ys, s, ss, mean, rstd, rows, hidden, eps, dtype,
                                      0, check=False)

    n0 = b.tf_launch_count()
    assert call(x=None) == S and call(y=None) == S
    assert call(rows=-1) == S and call(hidden=0) == S and call(hidden=-8) == S
    assert call(eps=-1.0) == S and call(eps=float("nan")) == S
    assert call(dtype=3) == S and call(dtype=-1) == S
    assert call(xs=63) == S and call(ys=63) == S and call(rs=63) == S and call(ss=0) == S
    assert call(hidden=131073, xs=1 << 20, ys=1 << 20, rs=1 << 20, ss=1 << 20) == U
    assert call(rows=0x7fffffff) == U and call(xs=(1 << 31) + 1) == U
    for name in ("x", "res", "y", "s"):
        assert call(**{name: p + 1}) == U
        assert call(**{name: p + 2}, dtype=b.TF_FP32) == U
    for name in ("gamma", "beta", "mean", "rstd"):
        assert call(**{name: p + 2}) == U
    assert call(rows=0, x=None, y=None) == b.TF_OK     # an empty batch touches nothing
    assert b.tf_launch_count() == n0


def test_backward_refusals(native_lib):
    from gemm_conv_epilogues_gb300 import binding as b
    S, U = b.TF_ERR_INVALID_ARG, b.TF_ERR_UNSUPPORTED
    p = 1 << 20
    need = b.tf_layernorm_backward_workspace_size(4, 64, b.TF_BF16)
    assert need > 0
    assert b.tf_layernorm_backward_workspace_size(-1, 64, 1) == 0
    assert b.tf_layernorm_backward_workspace_size(4, 0, 1) == 0
    assert b.tf_layernorm_backward_workspace_size(4, 131073, 1) == 0
    assert b.tf_layernorm_backward_workspace_size(4, 64, 5) == 0

    def call(dy=p, dys=64, x=p, xs=64, gamma=p, mean=p, rstd=p, dres=p, drs=64, dx=p, dxs=64, dgamma=p, dbeta=p,
             rows=4, hidden=64, acc=0, dtype=b.TF_BF16, ws=p, wsb=need):
        return b.tf_layernorm_backward(dy, dys, x, xs, gamma, mean, rstd, dres, drs, dx, dxs, dgamma, dbeta, rows,
                                       hidden, acc, dtype, ws, wsb, 0, check=False)

    n0 = b.tf_launch_count()
    for name in ("dy", "x", "dx", "mean", "rstd", "ws"):
        assert call(**{name: None}) == S, name
    assert call(rows=-1) == S and call(hidden=0) == S and call(dtype=9) == S
    assert call(dys=63) == S and call(xs=63) == S and call(dxs=63) == S and call(drs=63) == S
    assert call(wsb=need - 1) == S and call(wsb=-1) == S
    assert call(hidden=131073, dys=1 << 20, xs=1 << 20, dxs=1 << 20, drs=1 << 20) == U
    for name in ("dy", "x", "dx", "dres"):
        assert call(**{name: p + 1}) == U
    for name in ("gamma", "mean", "rstd", "dgamma", "dbeta"):
        assert call(**{name: p + 2}) == U
    assert call(ws=p + 8) == U
    assert call(rows=0, acc=1, dy=None, x=None, dx=None, mean=None, rstd=None, ws=None, wsb=0) == b.TF_OK
    assert b.tf_launch_count() == n0


# ---------------------------------------------------------------- numerics

@pytest.fixture(scope="module")
def b(cuda_ready):
    from gemm_conv_epilogues_gb300 import binding
    yield binding
    assert binding.tf_read_device_error() == (0, 0)


def _matrix(values, pad, name):
    """`values` in a buffer with `pad` more elements per row, the padding NaN."""
    rows, cols = values.shape
    buf = torch.full((rows, cols + pad), float("nan"), dtype=TYPES[name], device="cuda")
    buf[:, :cols] = values.to(TYPES[name])
    return buf[:, :cols]


def _inputs(rows, hidden, name, pad, seed=0, offset=0.0):
    g = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    scale = 0.5 + rnd(hidden).abs()
    return dict(x=_matrix(rnd(rows, hidden) * scale + offset, pad, name), res=_matrix(rnd(rows, hidden), pad, name),
                dy=_matrix(rnd(rows, hidden), pad, name), dres=_matrix(rnd(rows, hidden), pad, name),
                gamma=1 + 0.2 * rnd(hidden), beta=0.3 * rnd(hidden))


def _forward(b, d, name, res=True, affine=True, save=True, pad=0, stream=None):
    rows, hidden = d["x"].shape
    y = _matrix(torch.zeros(rows, hidden, device="cuda"), pad, name)
    s = _matrix(torch.zeros(rows, hidden, device="cuda"), pad, name) if save else None
    mean, rstd = (torch.full((rows,), float("nan"), device="cuda") if save else None for _ in range(2))
    b.tf_layernorm_forward(d["x"], d["x"].stride(0), d["res"] if res else None, d["res"].stride(0),
                           d["gamma"] if affine else None, d["beta"] if affine else None, y, y.stride(0), s,
                           y.stride(0), mean, rstd, rows, hidden, EPS, CODES[name], stream)
    return y, s, mean, rstd


def _within(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}; worst {float((err / bound).nan_to_num(1e9).max()):.3g} of its bound"


def _check_forward(b, d, name, res=True, affine=True, save=True, pad=0):
    y, s, mean, rstd = _forward(b, d, name, res, affine, save, pad)
    gamma, beta = (d["gamma"], d["beta"]) if affine else (None, None)
    rs, rm, rr, ry = ref.norm_forward(d["x"], d["res"] if res else None, gamma, beta, EPS)
    bs, bm, br, by = ref.norm_forward_bounds(name, rs, rm, rr, ry, gamma, beta)
    _within(y, ry, by, "y")
    if save:
        _within(s, rs, bs, "sum")
        _within(mean, rm, bm, "mean")
        _within(rstd, rr, br, "rstd")
    if pad:   # the padding of the rows stays as it was
        assert torch.isnan(y.as_strided((y.shape[0], pad), y.stride(), y.storage_offset() + y.shape[1])).all()


SHAPES = [(1, 1), (3, 2), (5, 7), (7, 64), (33, 72), (257, 513), (64, 1000), (19, 1024), (11, 1032), (300, 2048),
          (5, 2501), (40, 4096), (9, 5003), (6, 8192), (4, 12296), (3, 16384), (3, 20480), (2, 30001), (2, 65536),
          (2, 131072)]


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_forward(b, shape, name):
    _check_forward(b, _inputs(*shape, name, 0), name)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [8, 3])
@pytest.mark.parametrize("shape", [(37, 640), (12, 4096), (5, 1001), (3, 20480)], ids=lambda s: f"{s[0]}x{s[1]}")
@pytest.mark.parametrize("name", ["fp16", "bf16", "fp32"])
def test_forward_strided_rows(b, shape, name, pad):
    _check_forward(b, _inputs(*shape, name, pad), name, pad=pad)


@pytest.mark.gpu
@pytest.mark.parametrize("res,affine,save", [(False, True, True), (True, False, False), (False, False, True),
                                             (True, True, False)])
@pytest.mark.parametrize("shape", [(70, 640), (9, 4096), (4, 777), (2, 20480)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_forward_left_out_operands(b, shape, res, affine, save):
    _check_forward(b, _inputs(*shape, "bf16", 0), "bf16", res, affine, save)


@pytest.mark.gpu
def test_forward_large_mean(b):
    """Rows far from zero: the variance is that of the deviations, not a difference of large sums."""
    _check_forward(b, _inputs(50, 4096, "fp32", 0, offset=1000.0), "fp32")


@pytest.mark.gpu
@pytest.mark.parametrize("hidden", [640, 4096, 777, 20480])
def test_forward_keeps_rows_apart(b, hidden):
    """NaN and infinity in one row leave the others as they are; a constant row gives beta."""
    d = _inputs(9, hidden, "bf16", 0)
    y0 = _forward(b, d, "bf16")[0].clone()
    d["x"][2, 5] = float("nan")
    d["x"][4, 0] = float("inf")
    d["x"][6] = 3.0
    d["res"][6] = -1.0
    y, s, mean, rstd = _forward(b, d, "bf16")
    keep = [0, 1, 3, 5, 7, 8]
    assert torch.equal(y[keep], y0[keep])
    assert torch.isnan(y[2]).all() and torch.isnan(y[4]).all()
    assert torch.equal(y[6], d["beta"].bfloat16()) and mean[6] == 2.0
    assert abs(float(rstd[6]) * EPS ** 0.5 - 1) < 1e-6


def _backward(b, d, name, mean, rstd, dres=True, affine=True, weights=True, pad=0, into=None, ws=None, stream=None):
    rows, hidden = d["x"].shape
    dx = _matrix(torch.zeros(rows, hidden, device="cuda"), pad, name)
    dgamma, dbeta = into or (torch.full((hidden,), float("nan"), device="cuda") for _ in range(2))
    size = b.tf_layernorm_backward_workspace_size(rows, hidden, CODES[name])
    if ws is None:
        ws = torch.full((size // 4 + 4,), float("nan"), device="cuda")
    b.tf_layernorm_backward(d["dy"], d["dy"].stride(0), d["x"], d["x"].stride(0), d["gamma"] if affine else None, mean,
                            rstd, d["dres"] if dres else None, d["dres"].stride(0), dx, dx.stride(0),
                            dgamma if weights else None, dbeta if weights else None, rows, hidden,
                            1 if into else 0, CODES[name], ws if weights else None, size if weights else 0, stream)
    return dx, dgamma, dbeta


def _check_backward(b, d, name, dres=True, affine=True, weights=True, pad=0):
    _, mean, rstd, _ = ref.norm_forward(d["x"], None, None, None, EPS)
    mean, rstd = mean.float(), rstd.float()
    dx, dgamma, dbeta = _backward(b, d, name, mean, rstd, dres, affine, weights, pad)
    gamma, dr = d["gamma"] if affine else None, d["dres"] if dres else None
    rx, rg, rb = ref.norm_backward(d["dy"], d["x"], gamma, mean, rstd, dr)
    bx, bg, bb = ref.norm_backward_bounds(name, d["dy"], d["x"], gamma, mean, rstd, dr, rx)
    _within(dx, rx, bx, "dx")
    if weights:
        _within(dgamma, rg, bg, "dgamma")
        _within(dbeta, rb, bb, "dbeta")
    if pad:
        assert torch.isnan(dx.as_strided((dx.shape[0], pad), dx.stride(), dx.storage_offset() + dx.shape[1])).all()


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES + [(5000, 640), (1999, 1003), (2500, 4096), (700, 20480)],
                         ids=lambda s: f"{s[0]}x{s[1]}")
def test_backward(b, shape, name):
    _check_backward(b, _inputs(*shape, name, 0), name)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [8, 3])
@pytest.mark.parametrize("shape", [(37, 640), (400, 4096), (5, 1001), (3, 20480)], ids=lambda s: f"{s[0]}x{s[1]}")
@pytest.mark.parametrize("name", ["fp16", "bf16", "fp32"])
def test_backward_strided_rows(b, shape, name, pad):
    _check_backward(b, _inputs(*shape, name, pad), name, pad=pad)


@pytest.mark.gpu
@pytest.mark.parametrize("dres,affine,weights", [(False, True, True), (True, False, True), (False, True, False)])
@pytest.mark.parametrize("shape", [(700, 640), (90, 4096), (44, 777), (20, 20480)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_backward_left_out_operands(b, shape, dres, affine, weights):
    _check_backward(b, _inputs(*shape, "bf16", 0), "bf16", dres, affine, weights)


@pytest.mark.gpu
@pytest.mark.parametrize("hidden", [640, 4096, 777, 20480])
def test_backward_accumulates_and_repeats(b, hidden):
    d = _inputs(333, hidden, "bf16", 0)
    _, _, mean, rstd = _forward(b, d, "bf16", res=False)
    dx, dg, db = _backward(b, d, "bf16", mean, rstd)
    dx2, dg2, db2 = _backward(b, d, "bf16", mean, rstd)
    assert torch.equal(dx, dx2) and torch.equal(dg, dg2) and torch.equal(db, db2)   # equal calls, equal bits
    base = torch.randn(2, hidden, device="cuda")
    got = (base[0].clone(), base[1].clone())
    _backward(b, d, "bf16", mean, rstd, into=got)
    assert torch.equal(got[0], base[0] + dg) and torch.equal(got[1], base[1] + db)


@pytest.mark.gpu
def test_backward_one_weight_gradient(b):
    d = _inputs(50, 1024, "bf16", 0)
    _, _, mean, rstd = _forward(b, d, "bf16", res=False)
    dx, dg, db = _backward(b, d, "bf16", mean, rstd)
    ws = torch.empty(b.tf_layernorm_backward_workspace_size(50, 1024, 1), dtype=torch.uint8, device="cuda")
    for which in (0, 1):
        out = [torch.zeros(1024, device="cuda") if which == i else None for i in range(2)]
        b.tf_layernorm_backward(d["dy"], 1024, d["x"], 1024, d["gamma"], mean, rstd, d["dres"], 1024, dx, 1024, *out,
                                50, 1024, 0, b.TF_BF16, ws, ws.numel())
        assert torch.equal(out[which], (dg, db)[which])


@pytest.mark.gpu
@pytest.mark.parametrize("hidden", [64, 1000, 2048, 9000])
@pytest.mark.parametrize("name", ["bf16", "fp32"])
def test_offsets_past_32_bits(b, name, hidden):
    """Rows 2^30 elements apart give the bits of the same rows side by side."""
    rows, stride = 5, (1 << 30) + 8
    d = _inputs(rows, hidden, name, 0)
    big = torch.empty((rows - 1) * stride + hidden, dtype=TYPES[name], device="cuda")
    far = big.as_strided((rows, hidden), (stride, 1))
    far.copy_(d["x"])
    y, s, mean, rstd = _forward(b, d, name)
    dx, dg, db = _backward(b, d, name, mean, rstd)
    near = dict(d)
    d["x"] = far
    y2, s2, mean2, rstd2 = _forward(b, d, name)
    dx2, dg2, db2 = _backward(b, d, name, mean, rstd)
    for a, c in ((y, y2), (s, s2), (mean, mean2), (rstd, rstd2), (dx, dx2), (dg, dg2), (db, db2)):
        assert torch.equal(a, c)
    b.tf_layernorm_forward(near["x"], hidden, near["res"], hidden, d["gamma"], d["beta"], far, stride, None, 0, None,
                           None, rows, hidden, EPS, CODES[name])
    assert torch.equal(far, y)


@pytest.mark.gpu
def test_no_rows(b):
    z = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    f = torch.empty(0, device="cuda")
    dg, db = (torch.full((256,), 7.0, device="cuda") for _ in range(2))
    b.tf_layernorm_forward(z, 256, None, 0, None, None, z, 256, None, 0, f, f, 0, 256, EPS, b.TF_BF16)
    args = (z, 256, z, 256, None, f, f, None, 0, z, 256, dg, db, 0, 256)
    b.tf_layernorm_backward(*args, 1, b.TF_BF16, None, 0)
    assert (dg == 7).all() and (db == 7).all()
    b.tf_layernorm_backward(*args, 0, b.TF_BF16, None, 0)
    assert (dg == 0).all() and (db == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(40, 768), (12, 4096), (6, 1001)], ids=lambda s: f"{s[0]}x{s[1]}")
def test_backward_against_differences(b, shape):
    """The gradients of L = sum(dy*y) along random directions against central differences of the
    64-bit forward formula; the slack is the outputs' own rounding along the direction."""
    d = _inputs(*shape, "fp32", 0)
    _, _, mean, rstd = _forward(b, d, "fp32", res=False)
    dx, dg, db = _backward(b, d, "fp32", mean, rstd, dres=False)
    g = torch.Generator("cuda").manual_seed(5)
    loss = lambda x, ga, be: float((d["dy"].double() * ref.norm_forward(x, None, ga, be, EPS)[3]).sum())
    h = 1e-4
    for value, grad in (("x", dx), ("gamma", dg), ("beta", db)):
        v = torch.randn(d[value].shape, generator=g, device="cuda", dtype=torch.float64)
        at = {k: d[k].double() for k in ("x", "gamma", "beta")}
        up, down = dict(at), dict(at)
        up[value], down[value] = at[value] + h * v, at[value] - h * v
        slope = (loss(up["x"], up["gamma"], up["beta"]) - loss(down["x"], down["gamma"], down["beta"])) / (2 * h)
        terms = grad.double() * v
        # h^2 of a third derivative of order one, and 1e-5 relative per gradient element (fp32 sums)
        assert abs(float(terms.sum()) - slope) <= 1e-5 * float(terms.abs().sum()) + 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("hidden", [640, 4096, 777, 20480])
def test_captured_and_replayed(b, hidden):
    """A captured step replays on new inputs, on a stream of its own, with the results of eager calls."""
    d = _inputs(60, hidden, "bf16", 0)
    mean, rstd = torch.empty(60, device="cuda"), torch.empty(60, device="cuda")
    y, s, dx = (torch.empty(60, hidden, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    dg, db = torch.empty(hidden, device="cuda"), torch.empty(hidden, device="cuda")
    size = b.tf_layernorm_backward_workspace_size(60, hidden, 1)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def step():
        b.tf_layernorm_forward(d["x"], hidden, d["res"], hidden, d["gamma"], d["beta"], y, hidden, s, hidden, mean,
                               rstd, 60, hidden, EPS, b.TF_BF16)
        b.tf_layernorm_backward(d["dy"], hidden, s, hidden, d["gamma"], mean, rstd, d["dres"], hidden, dx, hidden, dg,
                                db, 60, hidden, 0, b.TF_BF16, ws, size)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (3, 4):
        new = _inputs(60, hidden, "bf16", 0, seed=seed)
        for k in ("x", "res", "dy", "dres", "gamma", "beta"):
            d[k].copy_(new[k])
        graph.replay()
        got = [t.clone() for t in (y, s, mean, rstd, dx, dg, db)]
        step()
        for g, w in zip(got, (y, s, mean, rstd, dx, dg, db)):
            assert torch.equal(g, w)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,hidden,name,pad", [(700, 256, "bf16", 0), (400, 640, "fp16", 8), (333, 1001, "bf16", 0),
                                                  (200, 5003, "fp32", 3), (64, 9001, "fp16", 0), (64, 16384, "bf16", 0)])
def test_outputs_in_the_place_of_inputs(b, rows, hidden, name, pad):
    """The residual stream updated where it lies, and a gradient over either of its inputs: the same bits."""
    d = _inputs(rows, hidden, name, pad)
    st, code = d["x"].stride(0), CODES[name]
    place = lambda t: torch.empty_strided((rows, hidden), (st, 1), dtype=t.dtype, device="cuda").copy_(t)
    y, s, mean, rstd = _forward(b, d, name, pad=pad)
    x, res = place(d["x"]), place(d["res"])
    m, r = torch.empty_like(mean), torch.empty_like(rstd)
    b.tf_layernorm_forward(x, st, res, st, d["gamma"], d["beta"], x, st, res, st, m, r, rows, hidden, EPS, code)
    for got, want in ((x, y), (res, s), (m, mean), (r, rstd)):
        assert torch.equal(got, want)
    size = b.tf_layernorm_backward_workspace_size(rows, hidden, code)
    ws = torch.empty(size // 4, device="cuda")

    def backward(dy, xx, dres, dx):
        dg, db = torch.empty(hidden, device="cuda"), torch.empty(hidden, device="cuda")
        b.tf_layernorm_backward(dy, st, xx, st, d["gamma"], mean, rstd, dres, st, dx, st, dg, db, rows, hidden, 0, code,
                                ws, size)
        return dx.clone(), dg, db

    want = backward(place(d["dy"]), place(s), place(d["dres"]), place(d["dy"]))
    for i in range(3):
        t = [place(d["dy"]), place(s), place(d["dres"])]
        for got, w in zip(backward(*t, t[i]), want):
            assert torch.equal(got, w)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,hidden", [(9, 2), (300, 30), (257, 66), (70, 258), (900, 316), (65, 514), (400, 1002),
                                         (31, 2502), (60, 3498), (20, 5002), (7, 6146), (5, 8190), (3, 10002),
                                         (2, 65534)])
def test_rows_of_whole_words(b, rows, hidden, name):
    """16-bit rows on 4-byte boundaries that are no multiples of 16 bytes, packed and in wider rows, then shifted to 2 bytes."""
    for pad in (0, 6, 3):
        d = _inputs(rows, hidden, name, pad)
        _check_forward(b, d, name, pad=pad)
        _check_forward(b, d, name, res=False, pad=pad)
        _check_backward(b, d, name, pad=pad)
        _check_backward(b, d, name, dres=False, pad=pad)


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [1, 2, 6])
def test_rows_from_shifted_bases(b, shift):
    """Whole rows whose buffer starts 2, 4 or 12 bytes past a 16-byte boundary."""
    d = _inputs(90, 1002, "bf16", 0)
    for key in ("x", "res", "dy", "dres"):
        buf = torch.full((d[key].numel() + shift,), float("nan"), dtype=torch.bfloat16, device="cuda")
        e = dict(d)
        e[key] = buf[shift:].view(d[key].shape).copy_(d[key])
        _check_forward(b, e, "bf16")
        _check_backward(b, e, "bf16")
