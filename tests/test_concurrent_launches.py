"""Calls from several host threads: two threads that call one kernel at sizes
that need different amounts of shared memory, neither of whose launches depends
on the other's sizes, the first calls of a new thread, and graphs replayed over each
other."""
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


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["conv", "norm", "product", "input gradient", "weight gradient"])
def test_first_calls_of_a_thread(b, what):
    """A host thread that has called nothing of CUDA before gets what the main thread gets."""
    off = torch.tensor([0, 40, 64], dtype=torch.int32, device="cuda")
    x, dy = torch.randn(64, 128, device="cuda").bfloat16(), torch.randn(64, 256, device="cuda").bfloat16()
    w = torch.randn(2, 256, 128, device="cuda").bfloat16()
    shape = b.conv_shape(1, 8, 16, 64, 64, 1, 1)
    image, filt = x.view(torch.int16)[:, :64].repeat(2, 1), w.view(torch.int16)[0, :64, :64].contiguous()
    f = torch.ones(2, 64, device="cuda")
    out = {"conv": filt.new_zeros(128, 64), "norm": torch.zeros_like(x), "product": torch.zeros_like(dy),
           "input gradient": torch.zeros_like(x), "weight gradient": torch.zeros(2, 256, 128, device="cuda")}[what]
    call = {
        "conv": lambda: b.tf_conv2d_bn_silu_variant(image, filt, f[0], f[1], out, shape, b.TF_CONV_UMMA, 0, check=False),
        "norm": lambda: b.tf_layernorm_forward(x, 128, None, 0, None, None, out, 128, None, 0, None, None, 64, 128, 1e-5,
                                               b.TF_BF16, 0, check=False),
        "product": lambda: b.tf_grouped_matmul(x, 128, w, None, off, out, 256, None, 0, 64, 2, 256, 128, 0, b.TF_BF16, 0,
                                               check=False),
        "input gradient": lambda: b.tf_grouped_matmul_dgrad(dy, 256, w, off, None, 0, out, 128, 64, 2, 256, 128, 0,
                                                            b.TF_BF16, 0, check=False),
        "weight gradient": lambda: b.tf_grouped_matmul_wgrad(dy, 256, x, 128, off, out, None, 64, 2, 256, 128, 0,
                                                             b.TF_BF16, None, 0, 0, check=False)}[what]
    assert call() == 0
    torch.cuda.synchronize()
    want, codes = out.clone(), []
    out.zero_()
    torch.cuda.synchronize()
    thread = threading.Thread(target=lambda: codes.extend([call(), call()]))
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert codes == [0, 0] and torch.equal(out, want) and want.any()


@pytest.mark.gpu
@pytest.mark.parametrize("widths", [(2048, 8192), (24576, 65536)])
def test_residual_layernorm(b, widths):
    def call(hidden):
        act, res, y = _half(4, hidden), _half(4, hidden), _half(4, hidden)
        f = torch.ones(2, hidden, device="cuda")
        return lambda: b.tf_residual_layernorm(act, res, f[0], f[1], y, 4, hidden, 1e-5, 0, check=False)

    assert _refused([call(w) for w in widths]) == [[], []]


@pytest.mark.gpu
@pytest.mark.parametrize("variant,kernels", [("TF_CONV_UMMA", [(1, 64), (1, 256)]), ("TF_CONV_TILED", [(13, 8), (15, 8)])])
def test_conv(b, variant, kernels):
    def call(k, c_in):
        shape = b.conv_shape(1, 8, 16, c_in, 64, k, k, (1, 1), (k // 2, k // 2))
        x, w, y = (torch.zeros(n, dtype=torch.int16, device="cuda") for n in (128 * c_in, 64 * k * k * c_in, 128 * 64))
        f = torch.ones(2, 64, device="cuda")
        return lambda: b.tf_conv2d_bn_silu_variant(x, w, f[0], f[1], y, shape, getattr(b, variant), 0, check=False)

    assert _refused([call(*s) for s in kernels]) == [[], []]


@pytest.mark.gpu
def test_two_graphs_replayed_at_once(b):
    """Captured gradient steps with workspaces of their own, replayed over each other on two streams: the bits of
    eager calls."""
    rows, hidden, N, K = 6000, 1024, 128, 256
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    jobs = []
    for i in range(2):
        g = torch.Generator("cuda").manual_seed(i)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
        job = dict(x=rnd(rows, hidden), dy=rnd(rows, hidden), dx=rnd(rows, hidden), stats=torch.ones(2, rows, device="cuda"),
                   grads=torch.zeros(2, hidden, device="cuda"), a=rnd(rows, N), c=rnd(rows, K),
                   dw=torch.zeros(1, N, K, device="cuda"), db=torch.zeros(1, N, device="cuda"))
        job["sizes"] = (b.tf_layernorm_backward_workspace_size(rows, hidden, b.TF_BF16),
                        b.tf_grouped_matmul_wgrad_workspace_size(rows, 1, N, K, b.TF_BF16))
        assert all(job["sizes"])
        job["ws"] = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in job["sizes"]]
        jobs.append(job)

    def step(j):
        b.tf_layernorm_backward(j["dy"], hidden, j["x"], hidden, None, j["stats"][0], j["stats"][1], None, 0, j["dx"], hidden,
                                j["grads"][0], j["grads"][1], rows, hidden, 0, b.TF_BF16, j["ws"][0], j["sizes"][0])
        b.tf_grouped_matmul_wgrad(j["a"], N, j["c"], K, off, j["dw"], j["db"], rows, 1, N, K, 0, b.TF_BF16, j["ws"][1],
                                  j["sizes"][1])

    outs = lambda j: [j["dx"], j["grads"], j["dw"], j["db"]]
    for j in jobs:
        step(j)
        j["want"] = [t.clone() for t in outs(j)]
    torch.cuda.synchronize()
    for j in jobs:
        j["graph"], j["stream"] = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(j["graph"]):
            for _ in range(3):
                step(j)
        for t in outs(j):
            t.fill_(7)
    torch.cuda.synchronize()
    for _ in range(30):
        for j in jobs:
            with torch.cuda.stream(j["stream"]):
                j["graph"].replay()
    torch.cuda.synchronize()
    for j in jobs:
        assert all(torch.equal(t, w) for t, w in zip(outs(j), j["want"]))
