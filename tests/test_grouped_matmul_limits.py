"""Grouped products where rounding adds up: bias gradients of very long groups."""
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
