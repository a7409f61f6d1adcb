"""Grouped products (forward, input gradient, weight gradient): refusals on the
host, and the kernels against 64-bit products with derived bounds."""
import pytest
import torch

import train_reference as ref
from train_reference import CODES, TYPES, U

ACTS = {"none": 0, "silu": 1, "gelu": 2}


# ---------------------------------------------------------------- refusals (no GPU)

def _refusals(b, call, matrices, aligned2, aligned4):
    S, W = b.TF_ERR_INVALID_ARG, b.TF_ERR_UNSUPPORTED
    p = 1 << 20
    n0 = b.tf_launch_count()
    for name in matrices + ["offsets"]:
        assert call(**{name: None}) == S, name
    assert call(rows=-1) == S and call(groups=0) == S and call(N=0) == S and call(K=0) == S and call(K=-8) == S
    assert call(dtype=3) == S and call(dtype=-1) == S
    assert call(dtype=b.TF_FP32) == W
    assert call(groups=1025) == W and call(rows=(1 << 22) + 1) == W
    assert call(N=65537, s1=1 << 20, s2=1 << 20, s3=1 << 20) == W
    assert call(K=65537, s1=1 << 20, s2=1 << 20, s3=1 << 20) == W
    assert call(s1=63) == S and call(s2=63) == S and call(s1=(1 << 31) + 1) == W
    for name in aligned2:
        assert call(**{name: p + 1}) == W, name
    for name in aligned4 + ["offsets"]:
        assert call(**{name: p + 2}) == W, name
    assert b.tf_launch_count() == n0


def test_forward_refusals(native_lib):
    from gemm_conv_epilogues_gb300 import binding as b
    p = 1 << 20

    def call(x=p, s1=64, w=p, bias=p, offsets=p, y=p, s2=64, pre=p, s3=64, rows=4, groups=2, N=64, K=64, act=1,
             dtype=b.TF_BF16):
        return b.tf_grouped_matmul(x, s1, w, bias, offsets, y, s2, pre, s3, rows, groups, N, K, act, dtype, 0,
                                   check=False)

    _refusals(b, call, ["x", "w", "y"], ["x", "w", "y", "pre"], ["bias"])
    assert call(act=3) == b.TF_ERR_INVALID_ARG and call(act=-1) == b.TF_ERR_INVALID_ARG
    assert call(s3=63) == b.TF_ERR_INVALID_ARG
    assert call(rows=0, x=None, y=None) == b.TF_OK


def test_dgrad_refusals(native_lib):
    from gemm_conv_epilogues_gb300 import binding as b
    p = 1 << 20

    def call(dy=p, s1=64, w=p, offsets=p, pre=p, s3=64, dx=p, s2=64, rows=4, groups=2, N=64, K=64, act=1,
             dtype=b.TF_BF16):
        return b.tf_grouped_matmul_dgrad(dy, s1, w, offsets, pre, s3, dx, s2, rows, groups, N, K, act, dtype, 0,
                                         check=False)

    _refusals(b, call, ["dy", "w", "dx", "pre"], ["dy", "w", "dx", "pre"], [])
    assert call(act=3) == b.TF_ERR_INVALID_ARG and call(s3=63) == b.TF_ERR_INVALID_ARG
    assert call(rows=0, dy=None, dx=None, pre=None) == b.TF_OK


def test_wgrad_refusals(native_lib):
    from gemm_conv_epilogues_gb300 import binding as b
    p = 1 << 20

    def call(dy=p, s1=64, x=p, s2=64, offsets=p, dw=p, dbias=p, s3=0, rows=4, groups=2, N=64, K=64, acc=0,
             dtype=b.TF_BF16, ws=p, wsb=1 << 20):
        return b.tf_grouped_matmul_wgrad(dy, s1, x, s2, offsets, dw, dbias, rows, groups, N, K, acc, dtype, ws, wsb, 0,
                                         check=False)

    _refusals(b, call, ["dy", "x", "dw"], ["dy", "x"], ["dw", "dbias"])
    assert call(ws=None) == b.TF_ERR_INVALID_ARG and call(wsb=-1) == b.TF_ERR_INVALID_ARG
    assert call(ws=p + 8) == b.TF_ERR_UNSUPPORTED
    assert b.tf_grouped_matmul_wgrad_workspace_size(4, 0, 64, 64, 1) == 0
    assert b.tf_grouped_matmul_wgrad_workspace_size(4, 2, 64, 64, 2) == 0
    assert b.tf_grouped_matmul_wgrad_workspace_size(100, 2, 64, 64, 1) >= 0


# ---------------------------------------------------------------- numerics

@pytest.fixture(scope="module")
def b(cuda_ready):
    from gemm_conv_epilogues_gb300 import binding
    yield binding
    assert binding.tf_read_device_error() == (0, 0)


def _rand(rows, cols, name, pad=0, scale=1.0, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    buf = torch.full((rows, cols + pad), float("nan"), dtype=TYPES[name], device="cuda")
    buf[:, :cols] = (torch.randn(rows, cols, generator=g, device="cuda") * scale).to(TYPES[name])
    return buf[:, :cols]


def _layout(counts, before=0, after=0):
    off = [before]
    for c in counts:
        off.append(off[-1] + c)
    return off, off[-1] + after, torch.tensor(off, dtype=torch.int32, device="cuda")


def _within(got, want, bound, what):
    """Inside the groups `want` is a number and `got` within the bound; outside it is NaN and `got` keeps its sentinel."""
    err = (got.double() - want).abs()
    bad = ~(err <= bound) & ~torch.isnan(want)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}; worst {float((err / bound).nan_to_num(0).max()):.3g} of its bound"
    assert (got[torch.isnan(want)] == 7).all(), f"{what}: rows outside the groups were written"


def _run_forward(b, x, w, bias, off, name, act, save, pad=0, rows=None, stream=None):
    rows, N = x.shape[0], w.shape[1]
    y = torch.full((rows, N + pad), 7.0, dtype=TYPES[name], device="cuda")
    pre = torch.full((rows, N + pad), 7.0, dtype=TYPES[name], device="cuda") if save else None
    b.tf_grouped_matmul(x, x.stride(0), w, bias, off, y, N + pad, pre, N + pad, rows, w.shape[0], N, w.shape[2],
                        ACTS[act], CODES[name], stream)
    if pad:
        assert (y[:, N:] == 7).all()
    return y[:, :N], pre[:, :N] if save else None


def _check_forward(b, counts, N, K, name, act="none", bias=False, save=False, pad=0, before=0, after=0, seed=0):
    off, rows, dev = _layout(counts, before, after)
    x = _rand(rows, K, name, pad, seed=seed)
    w = _rand(len(counts) * N, K, name, scale=K ** -0.5, seed=seed + 1).view(len(counts), N, K)
    bb = _rand(len(counts), N, "fp32", seed=seed + 2) if bias else None
    y, pre = _run_forward(b, x, w, bb, dev, name, act, save, pad)
    add = lambda e: bb[e].double() if bias else 0.0
    z = ref.grouped(off, rows, N, lambda e, r: x[r].double() @ w[e].double().t() + add(e))
    mag = ref.grouped(off, rows, N, lambda e, r: x[r].double().abs() @ w[e].double().abs().t() + abs(add(e)))
    e_z = ref.product_error(K, mag)
    ut, tiny = ref.half_step(name), ref.TINY[name]
    want = ref.act(act, z)
    # |act'| <= 1.13; the activation itself is good to 2e-5 of |z| at most
    _within(y, want, ut * want.abs() + 1.13 * (1 + ut) * e_z + (0 if act == "none" else 2e-5) * z.abs() + tiny, "y")
    if save:
        _within(pre, z, ut * z.abs() + (1 + ut) * e_z + tiny, "pre")


def _check_dgrad(b, counts, N, K, name, act="none", pad=0, before=0, after=0, seed=0):
    off, rows, dev = _layout(counts, before, after)
    dy = _rand(rows, N, name, pad, seed=seed)
    w = _rand(len(counts) * N, K, name, scale=N ** -0.5, seed=seed + 1).view(len(counts), N, K)
    pre = _rand(rows, K, name, pad, seed=seed + 2) if act != "none" else None
    dx = torch.full((rows, K + pad), 7.0, dtype=TYPES[name], device="cuda")
    b.tf_grouped_matmul_dgrad(dy, dy.stride(0), w, dev, pre, K + pad, dx, K + pad, rows, len(counts), N, K, ACTS[act],
                              CODES[name])
    if pad:
        assert (dx[:, K:] == 7).all()
    slope = torch.ones(rows, K, dtype=torch.float64, device="cuda") if pre is None else ref.act_slope(act, pre.double())
    prod = ref.grouped(off, rows, K, lambda e, r: dy[r].double() @ w[e].double())
    mag = ref.grouped(off, rows, K, lambda e, r: dy[r].double().abs() @ w[e].double().abs())
    want = prod * slope
    ut = ref.half_step(name)
    # the slope is good to 2e-5 absolutely
    bound = ut * want.abs() + (1 + ut) * (ref.product_error(N, mag) * slope.abs() +
                                          (0 if act == "none" else 2e-5) * prod.abs()) + ref.TINY[name]
    _within(dx[:, :K], want, bound, "dx")


def _check_wgrad(b, counts, N, K, name, bias=True, accumulate=False, pad=0, before=0, after=0, seed=0, workspace=True):
    off, rows, dev = _layout(counts, before, after)
    G = len(counts)
    dy, x = _rand(rows, N, name, pad, seed=seed), _rand(rows, K, name, pad, seed=seed + 1)
    base = torch.randn(G, N, K, device="cuda") if accumulate else torch.full((G, N, K), float("nan"), device="cuda")
    base_b = torch.randn(G, N, device="cuda") if accumulate else torch.full((G, N), float("nan"), device="cuda")
    dw, db = base.clone(), base_b.clone()
    size = b.tf_grouped_matmul_wgrad_workspace_size(rows, G, N, K, CODES[name]) if workspace else 0
    ws = torch.full((size // 4 + 4,), float("nan"), device="cuda")
    b.tf_grouped_matmul_wgrad(dy, dy.stride(0), x, x.stride(0), dev, dw, db if bias else None, rows, G, N, K,
                              1 if accumulate else 0, CODES[name], ws if size else None, size)
    for e in range(G):
        r = slice(off[e], off[e + 1])
        n = off[e + 1] - off[e]
        want = dy[r].double().t() @ x[r].double()
        bound = ref.product_error(n, dy[r].double().abs().t() @ x[r].double().abs())
        want_b, bound_b = dy[r].double().sum(0), 2 * n * U * dy[r].double().abs().sum(0)
        if accumulate:
            want, want_b = want + base[e].double(), want_b + base_b[e].double()
            bound, bound_b = bound + U * want.abs(), bound_b + U * want_b.abs()
        _within(dw[e], want, bound * (1 + U) + 1e-37, f"dw[{e}]")
        if bias:
            _within(db[e], want_b, bound_b * (1 + U) + 1e-37, f"dbias[{e}]")
    if not bias:
        assert torch.equal(db.nan_to_num(5), base_b.nan_to_num(5))


COUNTS = {
    "one_row": [1],
    "none_at_all": [0, 0, 0],
    "single": [200],
    "ragged": [3, 0, 130, 1, 0, 64, 129, 31],
    "tails": [127, 128, 129, 255, 256, 257],
    "small": [1, 2, 0, 5, 8, 9, 17, 33],
    "many": [(7 * i * i) % 23 for i in range(70)],
}
# widths: whole tiles, tiles with tails in either direction, below one tile, and (last) rows that are no multiple of 16 bytes
WIDTHS = [(64, 64), (128, 256), (256, 128), (264, 72), (8, 8), (136, 520), (512, 320), (100, 60), (33, 7), (1, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", WIDTHS)
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("name", ["fp16", "bf16"])
def test_forward(b, counts, N, K, name):
    _check_forward(b, COUNTS[counts], N, K, name)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("bias,save", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("counts,N,K", [("ragged", 264, 136), ("small", 136, 256), ("tails", 256, 128),
                                        ("ragged", 100, 60)])
def test_forward_epilogue(b, counts, N, K, act, bias, save):
    _check_forward(b, COUNTS[counts], N, K, "bf16", act, bias, save)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [8, 3])
@pytest.mark.parametrize("counts", ["ragged", "small"])
@pytest.mark.parametrize("name", ["fp16", "bf16"])
def test_strided_rows_and_rows_outside_the_groups(b, counts, name, pad):
    for before, after in ((0, 40), (13, 5)):
        _check_forward(b, COUNTS[counts], 264, 136, name, "gelu", True, True, pad, before, after)
        _check_dgrad(b, COUNTS[counts], 136, 264, name, "silu", pad, before, after)
        _check_wgrad(b, COUNTS[counts], 136, 264, name, pad=pad, before=before, after=after)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", WIDTHS)
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("name", ["fp16", "bf16"])
def test_dgrad(b, counts, N, K, name):
    _check_dgrad(b, COUNTS[counts], N, K, name)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("counts,N,K", [("ragged", 136, 264), ("small", 256, 136), ("tails", 128, 256),
                                        ("ragged", 60, 100)])
def test_dgrad_activation(b, counts, N, K, act):
    _check_dgrad(b, COUNTS[counts], N, K, "bf16", act)
    _check_dgrad(b, COUNTS[counts], N, K, "fp16", act)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", WIDTHS)
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("name", ["fp16", "bf16"])
def test_wgrad(b, counts, N, K, name):
    _check_wgrad(b, COUNTS[counts], N, K, name)


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K", [("ragged", 264, 136), ("single", 128, 128), ("small", 100, 60)])
def test_wgrad_accumulates(b, counts, N, K):
    _check_wgrad(b, COUNTS[counts], N, K, "bf16", accumulate=True)
    _check_wgrad(b, COUNTS[counts], N, K, "bf16", bias=False, accumulate=True)


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K", [([6000], 128, 256), ([2500, 0, 3111], 72, 136), ([4097], 64, 8)])
def test_wgrad_long_groups(b, counts, N, K):
    """Few tiles with long sums, with and without the workspace that lets them be split."""
    _check_wgrad(b, counts, N, K, "bf16")
    _check_wgrad(b, counts, N, K, "fp16", workspace=False)
    _check_wgrad(b, counts, N, K, "bf16", accumulate=True)


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K", [([1500, 0, 2607], 1288, 1032), ([2100], 4104, 776)])
def test_wgrad_long_groups_of_many_tiles(b, counts, N, K):
    _check_wgrad(b, counts, N, K, "bf16")
    _check_wgrad(b, counts, N, K, "fp16", pad=8, before=3, after=2)


@pytest.mark.gpu
def test_more_tiles_than_a_wave(b):
    counts = [300, 1, 777, 0, 513, 1200]
    _check_forward(b, counts, 1032, 200, "bf16", "silu", True, True)
    _check_dgrad(b, counts, 200, 1032, "bf16", "gelu")
    _check_wgrad(b, counts, 1032, 200, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("name", ["fp16", "bf16"])
def test_many_row_tiles(b, name, act):
    """Groups of many rows and enough tiles for the widest ones, in rows of a wider buffer."""
    counts = [300, 1, 777, 0, 513, 1200]
    _check_forward(b, counts, 1288, 136, name, act, True, True, 8, 5, 9)
    _check_dgrad(b, counts, 136, 1288, name, act, 8, 5, 9)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(130, 70), (75, 131), (1145, 76), (257, 129)])
@pytest.mark.parametrize("counts", [[2500, 0, 311], [300, 1, 77, 0, 513]], ids=str)
def test_unaligned_rows(b, counts, N, K):
    """Rows of 2- and 4-byte alignment, over several tiles and reduction steps in either direction."""
    for name, pad in (("fp16", 0), ("bf16", 1)):
        _check_forward(b, counts, N, K, name, "silu", True, True, pad, 3, 2)
        _check_dgrad(b, counts, N, K, name, "gelu", pad, 3, 2)
        _check_wgrad(b, counts, N, K, name, pad=pad, before=3, after=2)
    _check_wgrad(b, counts, N, K, "bf16", accumulate=True)


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_unaligned_bases(b, shift):
    """Whole 16-byte rows whose buffers start 2, 4 or 8 bytes past a 16-byte boundary."""
    counts, N, K = [70, 0, 200], 136, 72
    off, rows, dev = _layout(counts)
    whole = {"x": _rand(rows, K, "bf16"), "w": _rand(3 * N, K, "bf16", scale=0.1, seed=1).view(3, N, K),
             "dy": _rand(rows, N, "bf16", seed=2)}

    def run(t):
        y, _ = _run_forward(b, t["x"], t["w"], None, dev, "bf16", "none", False)
        dx = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
        b.tf_grouped_matmul_dgrad(t["dy"], N, t["w"], dev, None, 0, dx, K, rows, 3, N, K, 0, b.TF_BF16)
        dw = torch.empty(3, N, K, device="cuda")
        b.tf_grouped_matmul_wgrad(t["dy"], N, t["x"], K, dev, dw, None, rows, 3, N, K, 0, b.TF_BF16, None, 0)
        return y, dx, dw

    want = run(whole)
    for key in whole:
        t = dict(whole)
        buf = torch.full((t[key].numel() + shift,), float("nan"), dtype=torch.bfloat16, device="cuda")
        t[key] = buf[shift:].view(t[key].shape).copy_(t[key])
        for got, same, red in zip(run(t), want, (K, N, 200)):
            # the sums' order may differ: both are good to `red` steps of 2^-24 of sums of magnitudes below 9 * red
            assert (got.double() - same.double()).abs().max() <= 2 * red * U * 9 * red + 2.0 ** -7 * same.abs().max()


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K", [([2, 40, 0, 7, 90], 256, 320), ([1, 3, 0, 2, 5], 256, 320),
                                        ([2, 40, 0, 7, 90], 100, 60)])
def test_groups_do_not_reach_each_other(b, counts, N, K):
    """Infinities and NaN in one group's rows or weights leave every other group's results as they were."""
    off, rows, dev = _layout(counts, after=3)
    x, dy = _rand(rows, K, "bf16"), _rand(rows, N, "bf16", seed=1)
    w = _rand(len(counts) * N, K, "bf16", scale=0.1, seed=2).view(len(counts), N, K)

    def run():
        y, _ = _run_forward(b, x, w, None, dev, "bf16", "none", False)
        dx = torch.full((rows, K), 7.0, dtype=torch.bfloat16, device="cuda")
        b.tf_grouped_matmul_dgrad(dy, N, w, dev, None, 0, dx, K, rows, len(counts), N, K, 0, b.TF_BF16)
        dw, db = torch.empty(len(counts), N, K, device="cuda"), torch.empty(len(counts), N, device="cuda")
        b.tf_grouped_matmul_wgrad(dy, N, x, K, dev, dw, db, rows, len(counts), N, K, 0, b.TF_BF16, None, 0)
        return y, dx, dw, db

    clean = run()
    for bad in (1, 4):
        for v in (float("nan"), float("inf")):
            x2, dy2, w2 = x.clone(), dy.clone(), w.clone()
            for t in (x, dy):
                t[off[bad]:off[bad + 1]] = v
                t[off[-1]:] = v          # rows behind the last group too
            w[bad] = v
            got = run()
            x.copy_(x2), dy.copy_(dy2), w.copy_(w2)
            inside = torch.zeros(rows, dtype=torch.bool, device="cuda")
            inside[off[bad]:off[bad + 1]] = True
            others = [e for e in range(len(counts)) if e != bad]
            assert torch.equal(got[0][~inside], clean[0][~inside]) and torch.equal(got[1][~inside], clean[1][~inside])
            assert torch.equal(got[2][others], clean[2][others]) and torch.equal(got[3][others], clean[3][others])
            assert not torch.isfinite(got[0][inside].float()).any() and not torch.isfinite(got[2][bad]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_limits(b, act):
    """Sums far from zero, infinite or NaN: the activation's limits, and NaN stays NaN."""
    values = torch.tensor([1e30, -1e30, float("inf"), float("-inf"), float("nan"), 40.0, -40.0, 0.0], device="cuda")
    x = values.bfloat16()[:, None].repeat(1, 8)
    x[:, 1:] = 0
    w = torch.ones(1, 8, 8, dtype=torch.bfloat16, device="cuda")
    w[:, :, 1:] = 0
    _, _, dev = _layout([8])
    y, _ = _run_forward(b, x, w, None, dev, "bf16", act, False)
    got = y[:, 0].float().tolist()
    assert got[0] == float(values[0].bfloat16()) and got[2] == float("inf") and got[4] != got[4]
    assert got[5] == 40.0 and abs(got[1]) < 1e-30 and abs(got[3]) < 1e-30 and abs(got[6]) < 1e-15 and got[7] == 0
    dx = torch.empty(8, 8, dtype=torch.bfloat16, device="cuda")
    b.tf_grouped_matmul_dgrad(torch.ones(8, 8, dtype=torch.bfloat16, device="cuda"), 8, w, dev, x, 8, dx, 8, 8, 1, 8,
                              8, ACTS[act], b.TF_BF16)
    slope = (dx[:, 0].float() / 8).tolist()
    assert slope[0] == slope[2] == slope[5] == 1 and slope[4] != slope[4] and slope[7] == 0.5
    assert all(abs(slope[i]) < 1e-15 for i in (1, 3, 6))


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(64, 128), (60, 100)])
@pytest.mark.parametrize("offsets", [[0, 5, 4, 9], [-1, 3, 4, 9], [0, 3, 4, 11], [0, 1 << 30, 4, 9]], ids=str)
def test_bad_offsets_write_nothing(b, offsets, N, K):
    dev = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    x, dy = _rand(10, K, "bf16"), _rand(10, N, "bf16")
    w = _rand(3 * N, K, "bf16").view(3, N, K)
    y, dx = (torch.full((10, c), 7.0, dtype=torch.bfloat16, device="cuda") for c in (N, K))
    dw, db = torch.full((3, N, K), 7.0, device="cuda"), torch.full((3, N), 7.0, device="cuda")
    for call in (lambda: b.tf_grouped_matmul(x, K, w, None, dev, y, N, None, 0, 10, 3, N, K, 0, b.TF_BF16),
                 lambda: b.tf_grouped_matmul_dgrad(dy, N, w, dev, None, 0, dx, K, 10, 3, N, K, 0, b.TF_BF16),
                 lambda: b.tf_grouped_matmul_wgrad(dy, N, x, K, dev, dw, db, 10, 3, N, K, 0, b.TF_BF16, None, 0)):
        call()
        assert b.tf_read_device_error() == (b.TF_ERR_TIMEOUT, b.TF_DEVERR_OFFSETS)
    for t in (y, dx, dw, db):
        assert (t == 7).all()


@pytest.mark.gpu
def test_bad_offsets_with_split_sums(b):
    rows, N, K = 6000, 128, 256
    size = b.tf_grouped_matmul_wgrad_workspace_size(rows, 1, N, K, b.TF_BF16)
    assert size > 0
    dy, x = _rand(rows, N, "bf16"), _rand(rows, K, "bf16")
    ws = torch.full((size // 4,), 3.0, device="cuda")
    for accumulate in (0, 1):
        dw, db = torch.full((1, N, K), 7.0, device="cuda"), torch.full((1, N), 7.0, device="cuda")
        b.tf_grouped_matmul_wgrad(dy, N, x, K, torch.tensor([0, rows + 1], dtype=torch.int32, device="cuda"), dw, db,
                                  rows, 1, N, K, accumulate, b.TF_BF16, ws, size)
        assert b.tf_read_device_error() == (b.TF_ERR_TIMEOUT, b.TF_DEVERR_OFFSETS)
        assert (dw == 7).all() and (db == 7).all()


@pytest.mark.gpu
def test_no_rows(b):
    dev = torch.zeros(4, dtype=torch.int32, device="cuda")
    z = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = _rand(3 * 64, 64, "bf16").view(3, 64, 64)
    b.tf_grouped_matmul(z, 64, w, None, dev, z, 64, None, 0, 0, 3, 64, 64, 0, b.TF_BF16)
    b.tf_grouped_matmul_dgrad(z, 64, w, dev, None, 0, z, 64, 0, 3, 64, 64, 0, b.TF_BF16)
    for accumulate in (1, 0):
        dw, db = torch.full((3, 64, 64), 7.0, device="cuda"), torch.full((3, 64), 7.0, device="cuda")
        b.tf_grouped_matmul_wgrad(z, 64, z, 64, dev, dw, db, 0, 3, 64, 64, accumulate, b.TF_BF16, None, 0)
        assert (dw == 7 * accumulate).all() and (db == 7 * accumulate).all()


@pytest.mark.gpu
def test_gradients_against_differences(b):
    """L = sum(g*gelu(x W^T + b)) along random directions of x, W and b, against central differences
    of the 64-bit formula at the inputs' bits.  The gradients carry the bf16 rounding of the saved
    pre-activation (2^-9 relative, slope' <= 0.8) and of dx (2^-9)."""
    counts, N, K = [9, 0, 40, 3], 72, 48
    off, rows, dev = _layout(counts)
    x = _rand(rows, K, "bf16")
    w = _rand(4 * N, K, "bf16", scale=K ** -0.5, seed=1).view(4, N, K)
    bias, g = _rand(4, N, "fp32", scale=0.1, seed=2), _rand(rows, N, "bf16", seed=3)
    _, pre = _run_forward(b, x, w, bias, dev, "bf16", "gelu", True)
    # dz = g * act'(pre), through the input gradient of an identity product
    eye = torch.eye(N, dtype=torch.bfloat16, device="cuda").repeat(4, 1, 1)
    dz = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
    b.tf_grouped_matmul_dgrad(g, N, eye, dev, pre, N, dz, N, rows, 4, N, N, 2, b.TF_BF16)
    dx = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    b.tf_grouped_matmul_dgrad(dz, N, w, dev, None, 0, dx, K, rows, 4, N, K, 0, b.TF_BF16)
    dw, db = torch.empty(4, N, K, device="cuda"), torch.empty(4, N, device="cuda")
    b.tf_grouped_matmul_wgrad(dz, N, x, K, dev, dw, db, rows, 4, N, K, 0, b.TF_BF16, None, 0)

    def loss(v):
        z = ref.grouped(off, rows, N, lambda e, r: v["x"][r] @ v["w"][e].t() + v["bias"][e])
        return float((g.double() * ref.act("gelu", z)).sum())

    at = dict(x=x.double(), w=w.double(), bias=bias.double())
    gen = torch.Generator("cuda").manual_seed(9)
    h = 1e-4
    for key, grad in (("x", dx), ("w", dw), ("bias", db)):
        v = torch.randn(at[key].shape, generator=gen, device="cuda", dtype=torch.float64)
        up, down = dict(at), dict(at)
        up[key], down[key] = at[key] + h * v, at[key] - h * v
        slope = (loss(up) - loss(down)) / (2 * h)
        # every dz is off by at most 2^-9 |dz| + 0.8 * 2^-9 |pre| |g|; carried along v by absolute values
        e_dz = 2.0 ** -8 * (dz.double().abs() + pre.double().abs() * g.double().abs())
        if key == "x":
            slack = (ref.grouped(off, rows, K, lambda e, r: e_dz[r] @ w[e].double().abs()) * v.abs()).sum()
            slack = slack + 2.0 ** -8 * (dx.double() * v).abs().sum()
        else:
            slack = 0.0
            for e in range(4):
                r = slice(off[e], off[e + 1])
                slack += ((e_dz[r].t() @ x[r].double().abs()) * v[e].abs()).sum() if key == "w" else (
                    e_dz[r].sum(0) * v[e].abs()).sum()
        assert abs(float((grad.double() * v).sum()) - slope) <= float(slack) + 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K", [("ragged", 264, 136), ("small", 256, 512), ("ragged", 60, 100)])
def test_captured_and_replayed(b, counts, N, K):
    """A captured training step replays on new inputs and new offsets with the bits of eager calls."""
    off, rows, dev = _layout(COUNTS[counts], after=9)
    G = len(COUNTS[counts])
    x, dy = _rand(rows, K, "bf16"), _rand(rows, N, "bf16", seed=1)
    w = _rand(G * N, K, "bf16", scale=0.1, seed=2).view(G, N, K)
    pre_below = _rand(rows, K, "bf16", seed=3)
    y, pre = (torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dx = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    dw, db = torch.empty(G, N, K, device="cuda"), torch.empty(G, N, device="cuda")
    size = b.tf_grouped_matmul_wgrad_workspace_size(rows, G, N, K, 1)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")

    def step():
        b.tf_grouped_matmul(x, K, w, None, dev, y, N, pre, N, rows, G, N, K, 1, b.TF_BF16)
        b.tf_grouped_matmul_dgrad(dy, N, w, dev, pre_below, K, dx, K, rows, G, N, K, 2, b.TF_BF16)
        b.tf_grouped_matmul_wgrad(dy, N, x, K, dev, dw, db, rows, G, N, K, 0, b.TF_BF16, ws, size)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    outs = (y, pre, dx, dw, db)
    for seed in (5, 6):
        x.copy_(_rand(rows, K, "bf16", seed=seed))
        dy.copy_(_rand(rows, N, "bf16", seed=seed + 10))
        dev.copy_(torch.tensor(_layout(COUNTS[counts][::-1] if seed == 5 else COUNTS[counts])[0], device="cuda"))
        for t in outs:
            t.fill_(7)
        graph.replay()
        got = [t.clone() for t in outs]
        for t in outs:
            t.fill_(7)
        step()
        for g, t in zip(got, outs):
            assert torch.equal(g, t)


@pytest.mark.gpu
@pytest.mark.parametrize("G,N,K", [(512, 1024, 72), (900, 304, 520), (1024, 8, 264)])
def test_many_groups_and_tiles(b, G, N, K):
    """More work items per CTA than its lists hold at once, more groups than are sorted; every group checked."""
    counts = [(5 * i + 3) % 7 for i in range(G)]
    off, rows, dev = _layout(counts)
    x, dy = _rand(rows, K, "bf16"), _rand(rows, N, "bf16", seed=1)
    w = _rand(G * N, K, "bf16", scale=K ** -0.5, seed=2).view(G, N, K)
    y, _ = _run_forward(b, x, w, None, dev, "bf16", "none", False)
    dx = torch.full((rows, K), 7.0, dtype=torch.bfloat16, device="cuda")
    b.tf_grouped_matmul_dgrad(dy, N, w, dev, None, 0, dx, K, rows, G, N, K, 0, b.TF_BF16)
    dw, db = torch.empty(G, N, K, device="cuda"), torch.empty(G, N, device="cuda")
    b.tf_grouped_matmul_wgrad(dy, N, x, K, dev, dw, db, rows, G, N, K, 0, b.TF_BF16, None, 0)
    for e in range(G):
        r = slice(off[e], off[e + 1])
        xd, dyd, wd = x[r].double(), dy[r].double(), w[e].double()
        want, mag = xd @ wd.t(), xd.abs() @ wd.abs().t()
        _within(y[r], want, 2.0 ** -8 * want.abs() + 2 * ref.product_error(K, mag), f"y[{e}]")
        want, mag = dyd @ wd, dyd.abs() @ wd.abs()
        _within(dx[r], want, 2.0 ** -8 * want.abs() + 2 * ref.product_error(N, mag), f"dx[{e}]")
        _within(dw[e], dyd.t() @ xd, ref.product_error(counts[e], dyd.abs().t() @ xd.abs()) + 1e-37, f"dw[{e}]")
        _within(db[e], dyd.sum(0), 2 * counts[e] * U * dyd.abs().sum(0) + 1e-37, f"dbias[{e}]")


@pytest.mark.gpu
def test_offsets_past_32_bits(b):
    """Rows 2^30 elements apart, and weights of more than 2^31 elements."""
    N, K, stride, rows = 72, 64, (1 << 30) + 8, 6
    big = torch.empty((rows - 1) * stride + K, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((rows, K), (stride, 1))
    x.copy_(_rand(rows, K, "bf16"))
    w = _rand(2 * N, K, "bf16", seed=1).view(2, N, K)
    off, _, dev = _layout([2, 4])
    y, _ = _run_forward(b, x, w, None, dev, "bf16", "none", False)
    again, _ = _run_forward(b, x.contiguous(), w, None, dev, "bf16", "none", False)
    assert torch.equal(y, again)
    dy = _rand(rows, N, "bf16", seed=2)
    dx = big.as_strided((rows, K), (stride, 1), 0)
    near = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    b.tf_grouped_matmul_dgrad(dy, N, w, dev, None, 0, near, K, rows, 2, N, K, 0, b.TF_BF16)
    b.tf_grouped_matmul_dgrad(dy, N, w, dev, None, 0, dx, stride, rows, 2, N, K, 0, b.TF_BF16)
    assert torch.equal(dx, near)
    del big, x, dx
    torch.cuda.empty_cache()
    G, n = 5, 24576
    w = torch.empty(G, n, n, dtype=torch.bfloat16, device="cuda").normal_(std=n ** -0.5)   # 3.0e9 elements
    x = _rand(20, n, "bf16", seed=3)
    off, rows, dev = _layout([4, 0, 5, 1, 10])
    y, _ = _run_forward(b, x, w, None, dev, "bf16", "none", False)
    for e in (0, 3, 4):
        cols = torch.tensor([0, 1, 127, 128, n // 2, n - 2, n - 1], device="cuda")
        xd, wd = x[off[e]:off[e + 1]].double(), w[e, cols].double()
        want = xd @ wd.t()
        _within(y[off[e]:off[e + 1]][:, cols], want, 2.0 ** -8 * want.abs() + 2 * ref.product_error(n, xd.abs() @ wd.abs().t()), f"y[{e}]")


@pytest.mark.gpu
def test_first_call_captured(b, tmp_path):
    """A process whose first calls of the library are captured."""
    import subprocess
    import sys
    script = tmp_path / "first.py"
    script.write_text("""
import torch
from gemm_conv_epilogues_gb300 import binding as b
x = torch.randn(64, 128, device="cuda").bfloat16()
w = torch.randn(2, 256, 128, device="cuda").bfloat16()
off = torch.tensor([0, 40, 64], dtype=torch.int32, device="cuda")
y, s = (torch.zeros(64, c, dtype=torch.bfloat16, device="cuda") for c in (256, 128))
dw, m, r = torch.zeros(2, 256, 128, device="cuda"), torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
def step():
    b.tf_layernorm_forward(x, 128, None, 0, None, None, s, 128, None, 0, m, r, 64, 128, 1e-5, b.TF_BF16)
    b.tf_grouped_matmul(s, 128, w, None, off, y, 256, None, 0, 64, 2, 256, 128, b.TF_ACT_SILU, b.TF_BF16)
    b.tf_grouped_matmul_wgrad(y, 256, s, 128, off, dw, None, 64, 2, 256, 128, 0, b.TF_BF16, None, 0)
with torch.cuda.graph(g):
    step()
g.replay()
got = [t.clone() for t in (s, y, dw)]
step()
assert all(torch.equal(a, c) for a, c in zip(got, (s, y, dw))) and y.float().abs().sum() > 0
assert b.tf_read_device_error() == (0, 0)
""")
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, str(script)], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, PYTHONPATH=root), cwd=root)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.gpu
def test_two_streams_at_once(b):
    """Calls of different shapes overlapping on two streams give the bits of calls one after the other."""
    jobs = []
    for i, (counts, N, K) in enumerate([("tails", 512, 320), ("ragged", 264, 136)]):
        off, rows, dev = _layout(COUNTS[counts])
        x = _rand(rows, K, "bf16", seed=i)
        w = _rand(len(COUNTS[counts]) * N, K, "bf16", scale=0.1, seed=i + 5).view(-1, N, K)
        jobs.append((x, w, dev))
    alone = [_run_forward(b, x, w, None, dev, "bf16", "gelu", True) for x, w, dev in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        got = []
        for (x, w, dev), s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append(_run_forward(b, x, w, None, dev, "bf16", "gelu", True))
        torch.cuda.synchronize()
        for a, g in zip(alone, got):
            assert torch.equal(a[0], g[0]) and torch.equal(a[1], g[1])


# ---------------------------------------------------------------- the operators together

@pytest.mark.gpu
@pytest.mark.parametrize("hidden,inner", [(256, 512), (200, 72), (100, 36)])
def test_norm_and_experts_forward_and_backward(b, hidden, inner):
    """A block as a model has it: s = x + res, norm, two grouped products with GELU between them, and
    the gradients back to x and to every parameter, against 64-bit autograd of the same chain.  Every
    stored bf16 tensor adds half a step; errors are compared by norm."""
    counts = [40, 0, 7, 130, 3]
    off, rows, dev = _layout(counts)
    G, bf = len(counts), torch.bfloat16
    x, res = _rand(rows, hidden, "bf16"), _rand(rows, hidden, "bf16", seed=1)
    gamma, beta = 1 + 0.1 * torch.randn(hidden, device="cuda"), 0.1 * torch.randn(hidden, device="cuda")
    w1 = _rand(G * inner, hidden, "bf16", scale=hidden ** -0.5, seed=2).view(G, inner, hidden)
    w2 = _rand(G * hidden, inner, "bf16", scale=inner ** -0.5, seed=3).view(G, hidden, inner)
    b1, b2 = 0.1 * torch.randn(G, inner, device="cuda"), 0.1 * torch.randn(G, hidden, device="cuda")
    dout, ds = _rand(rows, hidden, "bf16", seed=4), _rand(rows, hidden, "bf16", seed=5)
    new = lambda *s: torch.empty(*s, dtype=bf, device="cuda")
    f32 = lambda *s: torch.empty(*s, device="cuda")
    y, s, mean, rstd = new(rows, hidden), new(rows, hidden), f32(rows), f32(rows)
    h, z, out = new(rows, inner), new(rows, inner), new(rows, hidden)
    dz, dyn, dx = new(rows, inner), new(rows, hidden), new(rows, hidden)
    dw1, dw2, db1, db2 = f32(G, inner, hidden), f32(G, hidden, inner), f32(G, inner), f32(G, hidden)
    dgamma, dbeta = f32(hidden), f32(hidden)
    ws = torch.empty(max(b.tf_layernorm_backward_workspace_size(rows, hidden, 1),
                         b.tf_grouped_matmul_wgrad_workspace_size(rows, G, inner, hidden, 1),
                         b.tf_grouped_matmul_wgrad_workspace_size(rows, G, hidden, inner, 1)), dtype=torch.uint8,
                     device="cuda")
    b.tf_layernorm_forward(x, hidden, res, hidden, gamma, beta, y, hidden, s, hidden, mean, rstd, rows, hidden, 1e-5, 1)
    b.tf_grouped_matmul(y, hidden, w1, b1, dev, h, inner, z, inner, rows, G, inner, hidden, 2, 1)
    b.tf_grouped_matmul(h, inner, w2, b2, dev, out, hidden, None, 0, rows, G, hidden, inner, 0, 1)
    b.tf_grouped_matmul_wgrad(dout, hidden, h, inner, dev, dw2, db2, rows, G, hidden, inner, 0, 1, ws, ws.numel())
    b.tf_grouped_matmul_dgrad(dout, hidden, w2, dev, z, inner, dz, inner, rows, G, hidden, inner, 2, 1)
    b.tf_grouped_matmul_wgrad(dz, inner, y, hidden, dev, dw1, db1, rows, G, inner, hidden, 0, 1, ws, ws.numel())
    b.tf_grouped_matmul_dgrad(dz, inner, w1, dev, None, 0, dyn, hidden, rows, G, inner, hidden, 0, 1)
    b.tf_layernorm_backward(dyn, hidden, s, hidden, gamma, mean, rstd, ds, hidden, dx, hidden, dgamma, dbeta, rows,
                            hidden, 0, 1, ws, ws.numel())
    p = {k: v.double().requires_grad_() for k, v in dict(x=x, gamma=gamma, beta=beta, w1=w1, w2=w2, b1=b1, b2=b2).items()}
    sd = p["x"] + res.double()
    d = sd - sd.mean(1, keepdim=True)
    yd = d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * p["gamma"] + p["beta"]
    outd = torch.cat([ref.act("gelu", yd[r] @ p["w1"][e].t() + p["b1"][e]) @ p["w2"][e].t() + p["b2"][e]
                      for e, r in enumerate(slice(off[i], off[i + 1]) for i in range(G))])
    ((outd * dout.double()).sum() + (sd * ds.double()).sum()).backward()
    # at most seven stored bf16 tensors (2^-9 each) lie on the longest path; random signs make the sum far smaller
    for got, want in ((out, outd), (dx, p["x"].grad), (dgamma, p["gamma"].grad), (dbeta, p["beta"].grad),
                      (dw1, p["w1"].grad), (dw2, p["w2"].grad), (db1, p["b1"].grad), (db2, p["b2"].grad)):
        assert float((got.double() - want.detach()).norm() / want.detach().norm()) <= 7 * 2.0 ** -8
