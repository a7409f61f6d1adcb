"""Two host threads calling one kernel at sizes that need different amounts of
shared memory: neither thread's launches depend on the other's sizes."""
import sys
import threading
import time

import pytest
import torch

SECONDS = 1.5


@pytest.fixture(scope="module")
def b(cuda_ready):
    from gemm_conv_epilogues_gb300 import binding
    yield binding
    assert binding.tf_read_device_error() == (0, 0)


def _refused(calls):
    """The status codes other than TF_OK that each call returned while all of them repeated, one thread each."""
    for call in calls:
        assert call() == 0
    torch.cuda.synchronize()
    codes = [[] for _ in calls]
    go, end = threading.Barrier(len(calls)), time.monotonic() + SECONDS

    def work(i):
        go.wait()
        while time.monotonic() < end and not any(codes):
            for _ in range(50):
                rc = calls[i]()
                if rc:
                    codes[i].append(rc)

    was = sys.getswitchinterval()
    sys.setswitchinterval(1e-5)
    try:
        threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(was)
    torch.cuda.synchronize()
    return codes


def _half(*shape):
    return torch.randn(*shape, device="cuda").half()


# widths (and rows) that one kernel serves with rings of different sizes
NORMS = {"cta": [(4, 2048), (4, 4096)], "words": [(4, 4098), (4, 5002)], "cluster": [(4, 9216), (4, 16384)],
         "rows": [(4, 4096), (400, 4096)]}


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", NORMS)
def test_norm_forward(b, sizes):
    def call(rows, hidden):
        x, res, y = _half(rows, hidden), _half(rows, hidden), _half(rows, hidden)
        return lambda: b.tf_layernorm_forward(x, hidden, res, hidden, None, None, y, hidden, None, 0, None, None, rows,
                                              hidden, 1e-5, b.TF_FP16, 0, check=False)

    assert _refused([call(*s) for s in NORMS[sizes]]) == [[], []]


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", NORMS)
def test_norm_backward(b, sizes):
    def call(rows, hidden):
        dy, x, dx = _half(rows, hidden), _half(rows, hidden), _half(rows, hidden)
        f = torch.ones(4, max(rows, hidden), device="cuda")
        size = b.tf_layernorm_backward_workspace_size(rows, hidden, b.TF_FP16)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        return lambda: b.tf_layernorm_backward(dy, hidden, x, hidden, None, f[0], f[1], None, 0, dx, hidden, f[2], f[3],
                                               rows, hidden, 0, b.TF_FP16, ws, size, 0, check=False)

    assert _refused([call(*s) for s in NORMS[sizes]]) == [[], []]
