"""Layer norm with its gradients where rounding adds up or the launch changes
form."""
import pytest
import torch

import test_layernorm_grad as base
import train_reference as ref
from train_reference import U


@pytest.fixture(scope="module")
def b(cuda_ready):
    from gemm_conv_epilogues_gb300 import binding
    yield binding
    assert binding.tf_read_device_error() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("name,offset", [("fp32", 100.0), ("fp32", 1e4), ("bf16", 300.0), ("fp16", 2000.0)])
@pytest.mark.parametrize("rows,hidden,dres", [(50, 4096, True), (40, 640, False), (30, 1001, True), (9, 20480, False)])
def test_backward_far_from_zero(b, rows, hidden, dres, name, offset):
    """x - mean is one rounding of its own value, not of x: xh keeps its digits however far the row lies from zero."""
    d = base._inputs(rows, hidden, name, 0, offset=offset)
    _, mean, rstd, _ = ref.norm_forward(d["x"], None, None, None, base.EPS)
    mean, rstd = mean.float(), rstd.float()
    dx, dgamma, dbeta = base._backward(b, d, name, mean, rstd, dres)
    dr = d["dres"] if dres else None
    rx, rg, rb = ref.norm_backward(d["dy"], d["x"], d["gamma"], mean, rstd, dr)
    # the bounds of rows around zero, whose xh is off by 2u*rstd*|x - mean| and its own two roundings
    near = d["x"].double() - mean.double()[:, None]
    bx, bg, bb = ref.norm_backward_bounds(name, d["dy"], near, d["gamma"], torch.zeros_like(mean), rstd, dr, rx)
    for got, want, bound, what in ((dx, rx, bx, "dx"), (dgamma, rg, bg, "dgamma"), (dbeta, rb, bb, "dbeta")):
        base._within(got, want, bound, what)


@pytest.mark.gpu
@pytest.mark.parametrize("hidden,rows", [(8, 1 << 27), (1, (1 << 27) + 3)])
def test_weight_gradients_of_many_rows(b, hidden, rows):
    """Equal terms, whose roundings do not cancel.  No term passes more than about 1024 additions of a row
    group, 64 of the groups' and CTAs' sums and 256 of what further runs of rows add."""
    dy = torch.full((rows, hidden), 0.1, device="cuda")
    x, mean, rstd = torch.ones(rows, hidden, device="cuda"), torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dgamma, dbeta = torch.empty(hidden, device="cuda"), torch.full((hidden,), 3.0, device="cuda")
    size = b.tf_layernorm_backward_workspace_size(rows, hidden, b.TF_FP32)
    ws = torch.full((size // 4,), float("nan"), device="cuda")
    args = (dy, hidden, x, hidden, None, mean, rstd, None, 0, dy, hidden)
    # dbeta alone, added to what it holds, then both; dx takes dy's place
    keep = dy.clone()
    b.tf_layernorm_backward(*args, None, dbeta, rows, hidden, 1, b.TF_FP32, ws, size)
    dy.copy_(keep)
    del keep
    want = rows * float(torch.tensor(0.1))
    bound = (1024 + 64 + 256) * U * (want + 3)
    assert (dbeta.double() - want - 3).abs().max() <= bound
    b.tf_layernorm_backward(*args, dgamma, dbeta, rows, hidden, 0, b.TF_FP32, ws, size)
    assert (dbeta.double() - want).abs().max() <= bound
    assert (dgamma.double() - want).abs().max() <= bound


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("hidden", [8, 100, 640, 641, 1024, 4096, 5003, 20480])
def test_workspace_of_a_larger_batch_serves_a_smaller_one(native_lib, hidden, dtype):
    from gemm_conv_epilogues_gb300 import binding as b
    sizes = [b.tf_layernorm_backward_workspace_size(rows, hidden, dtype) for rows in range(6000)]
    assert sizes[0] == 0 and sizes[1] == 8 * hidden
    assert all(p <= q for p, q in zip(sizes, sizes[1:]))


# rows of every number of slices from 2 to 16, whole 16-byte rows and odd ones
CLUSTERS = [(2, 8192 * n - s) for n in range(2, 17) for s in (3000, 2991)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,hidden", CLUSTERS)
def test_every_cluster_size(b, rows, hidden):
    name = ("bf16", "fp16", "fp32")[hidden // 8192 % 3]
    d = base._inputs(rows, hidden, name, 0)
    base._check_forward(b, d, name, res=hidden % 2 == 0)
    base._check_backward(b, d, name, dres=hidden % 2 == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["bf16", "fp32"])
@pytest.mark.parametrize("hidden", [8 * g - s for g in (32, 64, 128, 192, 256, 320, 384, 448, 512, 640, 768, 896, 1024)
                                    for s in (1, 2)])
def test_every_row_group_of_single_columns(b, hidden, name):
    """Each number of threads that an unaligned row may take has its kernels, for single columns and for pairs."""
    d = base._inputs(5, hidden, name, 0)
    for extra in (False, True):
        base._check_forward(b, d, name, res=extra)
        base._check_backward(b, d, name, dres=extra)
