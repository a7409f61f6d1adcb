"""Grouped products where rounding adds up or a value lies at the end of its
type's range: bias gradients of very long groups, activations of sums far below
zero."""
import pytest
import torch

import test_grouped_matmul as base
from train_reference import CODES, TYPES, U


@pytest.fixture(scope="module")
def b(cuda_ready):
    from gemm_conv_epilogues_gb300 import binding
    yield binding
    assert binding.tf_read_device_error() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,groups,N,K", [(1 << 20, 1, 64, 8), (1 << 20, 1, 2504, 8), ((1 << 20) + 77, 3, 72, 16),
                                             (1 << 20, 1, 33, 7), (1 << 20, 2, 64, 9), (1 << 22, 1, 8, 8)])
@pytest.mark.parametrize("name", ["fp16", "bf16"])
def test_bias_gradient_of_long_groups(b, rows, groups, N, K, name):
    """Equal terms, whose roundings do not cancel.  A term passes at most 400 additions, however long its group:
    three levels of sums (of 64, 64 and at most 32 at 2^22 rows), the lanes' and warps', and the splits'."""
    dy, x = torch.full((rows, N), 0.1, dtype=TYPES[name], device="cuda"), torch.zeros(rows, K, dtype=TYPES[name], device="cuda")
    counts = [rows // groups] * (groups - 1) + [rows - rows // groups * (groups - 1)]
    off, _, dev = base._layout(counts)
    size = b.tf_grouped_matmul_wgrad_workspace_size(rows, groups, N, K, CODES[name])
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    for bytes_, accumulate in ((0, 0), (size, 1)):
        dw, db = torch.zeros(groups, N, K, device="cuda"), torch.ones(groups, N, device="cuda")
        b.tf_grouped_matmul_wgrad(dy, N, x, K, dev, dw, db, rows, groups, N, K, accumulate, CODES[name],
                                  ws if bytes_ else None, bytes_)
        for e, n in enumerate(counts):
            want = n * float(dy[0, 0]) + accumulate
            assert (db[e].double() - want).abs().max() <= 400 * U * want
        assert (dw == 0).all()


def _far_values():
    """Every negative bf16 from -1 to -110, and a few beyond."""
    bits = torch.arange(0x3f80, 0x42dd, dtype=torch.int32)
    z = (bits << 16).view(torch.float32)
    return -torch.cat([z, torch.tensor([200.0, 1e4, 1e30])])


@pytest.mark.gpu
@pytest.mark.parametrize("unaligned", [False, True])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_far_below_zero(b, act, unaligned):
    """z*sigmoid(z), z*Phi(z) and their slopes keep their relative accuracy down to the smallest bf16: half a step,
    2^-8, and 1e-4 for an fp32 exponent of up to 140 (140 * 2^-24 * ln 2, a few times) and the fits."""
    z = _far_values().bfloat16().cuda()
    rows, K = z.numel(), 9 if unaligned else 8
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = z
    w = torch.zeros(1, 8, K, dtype=torch.bfloat16, device="cuda")
    w[:, :, 0] = 1
    _, _, dev = base._layout([rows])
    y, _ = base._run_forward(b, x, w, None, dev, "bf16", act, False)
    zd = z.double()[:, None]
    tiny = 2.0 ** -134
    if act == "silu":
        want = zd * torch.exp(zd) / (1 + torch.exp(zd))
        slope = torch.exp(zd) / (1 + torch.exp(zd)) * (1 + zd / (1 + torch.exp(zd)))
        mag = torch.exp(zd) * (1 + zd.abs())
    else:
        tail = 0.5 * torch.special.erfc(-zd * 0.5 ** 0.5)
        phi = torch.exp(-0.5 * zd * zd) * 0.3989422804014327
        want, slope, mag = zd * tail, tail + zd * phi, tail + zd.abs() * phi
    base._within(y, want.expand(-1, 8), 2.0 ** -8 * want.abs() + 1.01e-4 * want.abs() + tiny, "y")
    # the slope: dy = 1 at weight 1
    dx = torch.empty(rows, 8, dtype=torch.bfloat16, device="cuda")
    n = 9 if unaligned else 8
    dy = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    dy[:, 0] = 1
    v = torch.zeros(1, n, 8, dtype=torch.bfloat16, device="cuda")
    v[:, 0] = 1
    pre = z[:, None].expand(-1, 8).contiguous()
    b.tf_grouped_matmul_dgrad(dy, n, v, dev, pre, 8, dx, 8, rows, 1, n, 8, base.ACTS[act], b.TF_BF16)
    base._within(dx, slope.expand(-1, 8), 2.0 ** -8 * slope.abs() + 1.01e-4 * mag + tiny, "slope")
