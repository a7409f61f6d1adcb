"""A training step over a small language model from its tokens to its loss and back: embedding lookup, norm,
an expert product, linear cross entropy, and every gradient, the table's shared by both ends."""
import pytest
import torch

from train_reference import act


@pytest.fixture(scope="module")
def b(cuda_ready):
    from gemm_conv_epilogues_gb300 import binding
    yield binding
    assert binding.tf_read_device_error() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,vocab,hidden", [(50, 130, 64), (300, 1000, 200), (700, 2500, 328)])
def test_tied_step(b, rows, vocab, hidden):
    """Against 64-bit autograd of the same chain.  At most seven stored bf16 tensors (2^-8 each) lie on the
    longest path (y0, y, h, z, dl, dh, dy); random signs make the sum far smaller; errors are compared by norm."""
    g = torch.Generator("cuda").manual_seed(rows)
    bf = torch.bfloat16
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    table = (randn(vocab, hidden) * hidden ** -0.5).to(bf)
    w1 = (randn(1, hidden, hidden) * hidden ** -0.5).to(bf)
    gamma, beta, b1 = 1 + 0.1 * randn(hidden), 0.1 * randn(hidden), 0.1 * randn(1, hidden)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    targets = torch.roll(tokens, -1).clone()
    tokens[-rows // 5:] = -1          # a padded batch
    targets[-rows // 5 - 1:] = -1
    offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    used = int((targets >= 0).sum())
    dloss = (targets >= 0).float() / used
    scale = torch.tensor(hidden ** 0.5).item()
    new = lambda *s: torch.empty(*s, dtype=bf, device="cuda")
    f32 = lambda *s: torch.empty(*s, device="cuda")
    x, y, h, z = (new(rows, hidden) for _ in range(4))
    mean, rstd, loss, lse = (f32(rows) for _ in range(4))
    dh, dz, dy, dx = (new(rows, hidden) for _ in range(4))
    dtable, dw1, db1, dgamma, dbeta = f32(vocab, hidden), f32(1, hidden, hidden), f32(1, hidden), f32(hidden), f32(hidden)
    ws = torch.empty(max(b.tf_linear_cross_entropy_forward_workspace_size(rows, vocab, hidden, 1),
                         b.tf_linear_cross_entropy_backward_workspace_size(rows, vocab, hidden, 1),
                         b.tf_embedding_backward_workspace_size(rows, vocab, hidden),
                         b.tf_layernorm_backward_workspace_size(rows, hidden, 1),
                         b.tf_grouped_matmul_wgrad_workspace_size(rows, 1, hidden, hidden, 1)), dtype=torch.uint8, device="cuda")
    size = ws.numel()

    def step():
        b.tf_embedding_forward(tokens, b.TF_INT32, table, x, hidden, rows, vocab, hidden, scale, -1, 1)
        b.tf_layernorm_forward(x, hidden, None, 0, gamma, beta, y, hidden, None, 0, mean, rstd, rows, hidden, 1e-5, 1)
        b.tf_grouped_matmul(y, hidden, w1, b1, offsets, h, hidden, z, hidden, rows, 1, hidden, hidden, b.TF_ACT_SILU, 1)
        b.tf_linear_cross_entropy_forward(h, hidden, table, targets, b.TF_INT32, loss, lse, rows, vocab, hidden, 1.0, -1, 1,
                                          ws, size)
        b.tf_linear_cross_entropy_backward(h, hidden, table, targets, b.TF_INT32, lse, dloss, None, dh, hidden, dtable, rows,
                                           vocab, hidden, 1.0, -1, 0, b.TF_FP32, 1, ws, size)
        sig = torch.sigmoid(z.float())
        dz.copy_(dh.float() * sig * (1 + z.float() * (1 - sig)))
        b.tf_grouped_matmul_wgrad(dz, hidden, y, hidden, offsets, dw1, db1, rows, 1, hidden, hidden, 0, 1, ws, size)
        b.tf_grouped_matmul_dgrad(dz, hidden, w1, offsets, None, 0, dy, hidden, rows, 1, hidden, hidden, b.TF_ACT_NONE, 1)
        b.tf_layernorm_backward(dy, hidden, x, hidden, gamma, mean, rstd, None, 0, dx, hidden, dgamma, dbeta, rows, hidden, 0,
                                1, ws, size)
        b.tf_embedding_backward(dx, hidden, tokens, b.TF_INT32, dtable, rows, vocab, hidden, scale, -1, 1, 1, ws, size)

    step()
    p = {k: v.double().requires_grad_() for k, v in dict(table=table, gamma=gamma, beta=beta, w1=w1, b1=b1).items()}
    live = (tokens >= 0).double()[:, None]
    xd = p["table"][tokens.long().clamp(min=0)] * scale * live
    d = xd - xd.mean(1, keepdim=True)
    yd = d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * p["gamma"] + p["beta"]
    hd = act("silu", yd @ p["w1"][0].t() + p["b1"][0])
    keep = targets >= 0
    logits = hd[keep] @ p["table"].t()
    lossd = torch.logsumexp(logits, 1) - logits.gather(1, targets[keep, None].long())[:, 0]
    lossd.mean().backward()
    pairs = [(loss[keep], lossd), (dtable, p["table"].grad), (dgamma, p["gamma"].grad), (dbeta, p["beta"].grad),
             (dw1, p["w1"].grad), (db1, p["b1"].grad)]
    for got, want in pairs:
        assert float((got.double() - want.detach()).norm() / want.detach().norm()) <= 7 * 2.0 ** -8
    assert (loss[~keep] == 0).all() and (dh[~keep] == 0).all()
    first = [v.clone() for v in (loss, dtable, dgamma, dbeta, dw1, db1)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for v in (loss, dtable, dgamma, dbeta, dw1, db1):
        v.fill_(float("nan"))
    graph.replay()
    assert all(torch.equal(u, v) for u, v in zip(first, (loss, dtable, dgamma, dbeta, dw1, db1)))


@pytest.mark.gpu
def test_calls_from_several_host_threads(b):
    """Threads that never called the library before, each with sizes, a stream and workspaces of its own."""
    import threading

    sizes = [(5, 900, 64), (200, 1500, 128), (700, 300000, 16), (40, 77, 1002)]

    def inputs(i):
        rows, vocab, hidden = sizes[i]
        g = torch.Generator("cuda").manual_seed(i)
        x = torch.randn(rows, hidden, generator=g, device="cuda").half()
        w = (torch.randn(vocab, hidden, generator=g, device="cuda") * hidden ** -0.5).half()
        t = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        return x, w, t

    def step(i, x, w, t):
        rows, vocab, hidden = sizes[i]
        loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        dx, dtable = torch.empty_like(x), torch.empty(vocab, hidden, device="cuda")
        y = torch.empty_like(x)
        ws = torch.empty(max(b.tf_linear_cross_entropy_forward_workspace_size(rows, vocab, hidden, 0),
                             b.tf_linear_cross_entropy_backward_workspace_size(rows, vocab, hidden, 0),
                             b.tf_embedding_backward_workspace_size(rows, vocab, hidden)), dtype=torch.uint8, device="cuda")
        n = ws.numel()
        for _ in range(10):
            b.tf_embedding_forward(t, 1, w, y, hidden, rows, vocab, hidden, 2.0, -1, 0)
            b.tf_linear_cross_entropy_forward(x, hidden, w, t, 1, loss, lse, rows, vocab, hidden, 1.0, -1, 0, ws, n)
            b.tf_linear_cross_entropy_backward(x, hidden, w, t, 1, lse, None, None, dx, hidden, dtable, rows, vocab, hidden, 1.0,
                                               -1, 0, 2, 0, ws, n)
            b.tf_embedding_backward(dx, hidden, t, 1, dtable, rows, vocab, hidden, 2.0, -1, 1, 0, ws, n)
        return y, loss, lse, dx, dtable

    data = [inputs(i) for i in range(len(sizes))]
    alone = [step(i, *data[i]) for i in range(len(sizes))]
    torch.cuda.synchronize()
    got, wrong = [None] * len(sizes), []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = step(i, *data[i])
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # (told by the thread that waits)
            wrong.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    for a, g in zip(alone, got):
        assert all(torch.equal(u, v) for u, v in zip(a, g))
