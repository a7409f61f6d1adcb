"""Embedding lookup with scaling and its gradient by sorted tokens: refusals on the
host, and the kernels against 64-bit forms with derived bounds.

Bounds.  u = 2^-24 and ut are half a step of fp32 and of the output's type.  The
lookup rounds scale*table to fp32 and then to the type: |y|(u + ut), plus half
of the type's smallest step.  A word's sum is added in levels (64 rows, the pieces
of up to 1024, eight stretches of pieces): with `depth` additions it is off
by depth*u*sum|terms|; the scale and the addition to what is there round once more each."""
import pytest
import torch

from train_reference import CODES, TYPES, U, half_step

SMALLEST = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -126, "fp32": 2.0 ** -126}   # (products below 2^-126 may be flushed)


# ---------------------------------------------------------------- refusals (no GPU)

def test_forward_refusals(native_lib):
    from gemm_conv_epilogues_gb300 import binding as b
    S, W, p = b.TF_ERR_INVALID_ARG, b.TF_ERR_UNSUPPORTED, 1 << 20

    def call(tokens=p, index=1, table=p, y=p, stride=64, rows=4, vocab=100, hidden=64, scale=1.0, padding=-1, dtype=1):
        return b.tf_embedding_forward(tokens, index, table, y, stride, rows, vocab, hidden, scale, padding, dtype, 0,
                                      check=False)

    n0 = b.tf_launch_count()
    assert call(tokens=None) == S and call(table=None) == S and call(y=None) == S
    assert call(rows=-1) == S and call(vocab=0) == S and call(hidden=0) == S and call(stride=63) == S
    assert call(dtype=3) == S and call(dtype=-1) == S and call(index=2) == S and call(index=-1) == S
    assert call(scale=float("inf")) == S and call(scale=float("nan")) == S
    assert call(rows=(1 << 30) + 1) == W and call(vocab=(1 << 31) - 1) == W and call(hidden=131073, stride=1 << 20) == W
    assert call(stride=(1 << 31) + 1) == W
    assert call(tokens=p + 4) == W and call(tokens=p + 2, index=0) == W and call(table=p + 1) == W and call(y=p + 1) == W
    assert call(dtype=b.TF_FP32, table=p + 2) == W
    assert call(rows=0, tokens=None, table=None, y=None) == b.TF_OK
    assert b.tf_launch_count() == n0


def test_backward_refusals(native_lib):
    from gemm_conv_epilogues_gb300 import binding as b
    S, W, p = b.TF_ERR_INVALID_ARG, b.TF_ERR_UNSUPPORTED, 1 << 20
    need = b.tf_embedding_backward_workspace_size(4, 100, 64)
    assert need > 0

    def call(dy=p, stride=64, tokens=p, index=1, dtable=p, rows=4, vocab=100, hidden=64, scale=1.0, padding=-1, acc=0,
             dtype=1, ws=p, wsb=need):
        return b.tf_embedding_backward(dy, stride, tokens, index, dtable, rows, vocab, hidden, scale, padding, acc, dtype,
                                       ws, wsb, 0, check=False)

    n0 = b.tf_launch_count()
    assert call(dy=None) == S and call(tokens=None) == S and call(dtable=None) == S
    assert call(rows=-1) == S and call(vocab=0) == S and call(hidden=0) == S and call(stride=63) == S
    assert call(dtype=3) == S and call(index=2) == S and call(scale=float("nan")) == S
    assert call(ws=None) == S and call(wsb=need - 1) == S and call(ws=p + 8) == W
    assert call(rows=(1 << 30) + 1, wsb=1 << 60) == W and call(vocab=(1 << 31) - 1) == W
    assert call(hidden=131073, stride=1 << 20) == W and call(stride=(1 << 31) + 1) == W
    assert call(tokens=p + 4) == W and call(dy=p + 1) == W and call(dtable=p + 2) == W
    assert call(rows=0, dy=None, tokens=None, acc=1, ws=None, wsb=0) == b.TF_OK
    assert b.tf_launch_count() == n0


@pytest.mark.parametrize("hidden", [1, 8, 100, 1000, 1024, 4096, 5000, 131072])
def test_workspace_does_not_fall(native_lib, hidden):
    from gemm_conv_epilogues_gb300 import binding as b
    rows = sorted({r + d for k in range(0, 31) for r in (1 << k, 3 << max(k - 2, 0), 38912 >> 2, 32 * 4864 >> (k % 8))
                   for d in (-1, 0, 1) if 0 <= r + d <= 1 << 30})
    sizes = [b.tf_embedding_backward_workspace_size(r, 1000, hidden) for r in rows]
    assert sizes == sorted(sizes) and sizes[0] == 0 and all(s > 0 for s in sizes[1:])


# ---------------------------------------------------------------- numerics

@pytest.fixture(scope="module")
def b(cuda_ready):
    from gemm_conv_epilogues_gb300 import binding
    yield binding
    assert binding.tf_read_device_error() == (0, 0)


def _tokens(kind, rows, vocab, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    if kind == "one":
        return torch.full((rows,), vocab // 2, device="cuda")
    if kind == "each":
        return torch.randperm(vocab, generator=g, device="cuda")[:rows]
    if kind == "ends":
        return torch.where(torch.rand(rows, generator=g, device="cuda") < 0.5, 0, vocab - 1)
    if kind == "zipf":
        u = torch.rand(rows, generator=g, device="cuda", dtype=torch.float64)
        return torch.exp(u * torch.log(torch.tensor(float(vocab)))).long().clamp(0, vocab - 1)
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    if kind == "padded":
        t[torch.rand(rows, generator=g, device="cuda") < 0.4] = -1
    if kind == "empty":
        t[:] = -1
    return t


def _wide(rows, cols, pad, t, offset=0):
    """An uninitialised-looking matrix in a wider buffer, `offset` elements from an aligned address."""
    flat = torch.full((rows * (cols + pad) + offset + 8,), 7.0, device="cuda", dtype=t)
    return flat, flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


# (rows, vocab, hidden, pad, offset): rows of whole 16-byte words, of pairs, of single elements, and less than a warp wide
SHAPES = [(1, 1, 1, 0, 0), (1, 50, 4096, 0, 0), (5, 50, 8, 0, 0), (33, 17, 24, 8, 0), (7, 1000, 1002, 2, 0), (100, 9, 63, 3, 1),
          (257, 300, 640, 0, 1), (64, 40, 5001, 0, 0), (2049, 100, 520, 8, 8), (3, 5, 131072, 0, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind", ["any", "padded"])
def test_forward(b, shape, dtype, kind):
    rows, vocab, hidden, pad, offset = shape
    t = TYPES[dtype]
    tokens = _tokens(kind, rows, vocab)
    _, table = _wide(vocab, hidden, 0, t, offset)
    table.copy_(torch.randn(vocab, hidden, device="cuda"))
    flat, y = _wide(rows, hidden, pad, t, offset)
    scale = 0.3 * hidden ** 0.5
    scale = torch.tensor(scale, dtype=torch.float32).item()
    for wide in (True, False):
        flat.fill_(7.0)
        b.tf_embedding_forward(tokens if wide else tokens.int(), int(wide), table, y, y.stride(0), rows, vocab, hidden, scale,
                               -1, CODES[dtype])
        ref = torch.where((tokens >= 0)[:, None], table.double()[tokens.clamp(min=0)] * scale, 0.0)
        assert ((y.double() - ref).abs() <= ref.abs() * (U + half_step(dtype)) + SMALLEST[dtype]).all()
        kept = flat.clone()
        kept[offset:offset + rows * (hidden + pad)].view(rows, -1)[:, :hidden] = 7.0
        assert (kept == 7.0).all()   # nothing beside the rows


@pytest.mark.gpu
def test_forward_masked_rows_read_nothing(b):
    """The padding may be a row's number; what lies in that row, NaN included, is not read."""
    table = torch.randn(10, 64, device="cuda")
    table[3] = float("nan")
    tokens = torch.tensor([3, 1, 3, 9], device="cuda")
    y = torch.full((4, 64), 5.0, device="cuda")
    b.tf_embedding_forward(tokens, 1, table, y, 64, 4, 10, 64, 2.0, 3, b.TF_FP32)
    assert (y[[0, 2]] == 0).all() and torch.equal(y[[1, 3]], 2 * table[[1, 9]])


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [1, 0])
def test_tokens_outside(b, wide):
    """Words outside the vocabulary, far outside too: zeros, no gradient, and the device error word says so."""
    far = 1 << 40 if wide else (1 << 31) - 1
    tokens = torch.tensor([0, 10, -1, far, -far, 9], device="cuda", dtype=torch.int64 if wide else torch.int32)
    table, y = torch.randn(10, 64, device="cuda"), torch.full((6, 64), 5.0, device="cuda")
    assert b.tf_read_device_error() == (0, 0)
    b.tf_embedding_forward(tokens, wide, table, y, 64, 6, 10, 64, 1.0, b.TF_NO_INDEX, b.TF_FP32)
    assert b.tf_read_device_error() == (b.TF_ERR_TIMEOUT, b.TF_DEVERR_INDEX)
    assert (y[1:5] == 0).all() and torch.equal(y[[0, 5]], table[[0, 9]])
    dtable = torch.full((10, 64), 3.0, device="cuda")
    ws = torch.empty(b.tf_embedding_backward_workspace_size(6, 10, 64), dtype=torch.uint8, device="cuda")
    dy = torch.randn(6, 64, device="cuda")
    dy[1:5] = float("nan")
    b.tf_embedding_backward(dy, 64, tokens, wide, dtable, 6, 10, 64, 1.0, b.TF_NO_INDEX, 0, b.TF_FP32, ws, ws.numel())
    assert b.tf_read_device_error() == (b.TF_ERR_TIMEOUT, b.TF_DEVERR_INDEX)
    assert (dtable[1:9] == 0).all() and torch.equal(dtable[[0, 9]], dy[[0, 5]])


def _grad(b, dy, tokens, dtable, scale, accumulate, dtype, wide=1, ws=None, stream=None):
    rows, hidden, vocab = dy.shape[0], dy.shape[1], dtable.shape[0]
    if ws is None:
        ws = torch.empty(max(16, b.tf_embedding_backward_workspace_size(rows, vocab, hidden)), dtype=torch.uint8, device="cuda")
        ws.fill_(0xff)   # NaN in every partial sum
    b.tf_embedding_backward(dy, dy.stride(0), tokens, wide, dtable, rows, vocab, hidden, scale, -1, accumulate, CODES[dtype],
                            ws, ws.numel(), stream)
    return ws


def _check_grad(dtable, before, dy, tokens, scale, accumulate):
    keep = tokens >= 0
    t, v = tokens[keep].long(), dy[keep].double() * scale
    ref = torch.zeros_like(dtable, dtype=torch.float64).index_put_((t,), v, accumulate=True)
    size = torch.zeros_like(ref).index_put_((t,), v.abs(), accumulate=True)
    rows = torch.bincount(t, minlength=dtable.shape[0]).double()[:, None]
    depth = torch.minimum(rows, 100.0 + rows / 256) + 2   # 64 rows, 16 of their sums, pieces of at least 32 in 8 stretches
    if accumulate:
        ref, size = ref + before.double(), size + before.double().abs()
    assert ((dtable.double() - ref).abs() <= depth * U * size + 2.0 ** -126).all()
    if accumulate:
        assert torch.equal(dtable[rows[:, 0] == 0], before[rows[:, 0] == 0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES + [(2048, 5000, 40, 0, 0), (5000, 60, 1024, 8, 0)], ids=str)
@pytest.mark.parametrize("kind", ["any", "padded", "zipf"])
@pytest.mark.parametrize("accumulate", [0, 1])
def test_backward(b, shape, dtype, kind, accumulate):
    rows, vocab, hidden, pad, offset = shape
    tokens = _tokens(kind, rows, vocab)
    _, dy = _wide(rows, hidden, pad, TYPES[dtype], offset)
    dy.copy_(torch.randn(rows, hidden, device="cuda"))
    flat, dtable = _wide(vocab, hidden, 0, torch.float32, offset)
    dtable.copy_(torch.randn(vocab, hidden, device="cuda"))
    before = dtable.clone()
    scale = torch.tensor(0.7 * hidden ** 0.5, dtype=torch.float32).item()
    _grad(b, dy, tokens, dtable, scale, accumulate, dtype)
    _check_grad(dtable, before, dy, tokens, scale, accumulate)
    assert (flat[:offset] == 7.0).all() and (flat[offset + vocab * hidden:] == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [31, 32, 33, 64, 65, 2047, 2048, 2049, 4097, 65535, 65536, 65537, 140000])
@pytest.mark.parametrize("kind", ["one", "each", "ends", "zipf", "empty", "padded"])
def test_backward_orders(b, rows, kind):
    """Runs of one word over many pieces, words that end at pieces' ends, and lists of one, two and three merges."""
    vocab = 150001
    tokens = _tokens(kind, rows, vocab, seed=rows)
    dy = torch.randn(rows, 8, device="cuda").bfloat16()
    dtable = torch.full((vocab, 8), float("nan"), device="cuda")
    _grad(b, dy, tokens, dtable, 1.5, 0, "bf16")
    _check_grad(dtable, None, dy, tokens, 1.5, 0)


@pytest.mark.gpu
def test_backward_long_runs_keep_their_digits(b):
    """2^21 equal terms: one running fp32 sum would stop growing in its last digits."""
    rows = 1 << 21
    dy = torch.full((rows, 8), 1.1, device="cuda").half()
    tokens = torch.full((rows,), 2, device="cuda")
    dtable = torch.empty(3, 8, device="cuda")
    _grad(b, dy, tokens, dtable, 1.0, 0, "fp16")
    ref = rows * dy[0, 0].double().item()
    # 64 + 16 additions in a piece of 1024 and 256 + 8 in the join: each rounds by u
    assert (dtable[2].double() - ref).abs().max().item() <= (64 + 16 + 256 + 8 + 1) * U * ref
    assert (dtable[:2] == 0).all()


@pytest.mark.gpu
def test_backward_equal_bits_and_masked_infinities(b):
    rows, vocab, hidden = 5000, 700, 264
    tokens = _tokens("padded", rows, vocab)
    dy = torch.randn(rows, hidden, device="cuda").bfloat16()
    dy[tokens < 0] = float("inf")
    out = []
    for _ in range(3):
        dtable = torch.full((vocab, hidden), float("nan"), device="cuda")
        _grad(b, dy, tokens, dtable, 1.0, 0, "bf16")
        out.append(dtable)
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2]) and out[0].isfinite().all()
    dy[17] = float("inf")   # of one word's row: that word's gradient alone is infinite
    tokens[17] = 5
    _grad(b, dy, tokens, out[1], 1.0, 0, "bf16")
    assert out[1][5].isinf().all() and out[1][[v for v in range(vocab) if v != 5]].isfinite().all()


@pytest.mark.gpu
def test_backward_without_rows(b):
    dtable = torch.full((5, 12), 3.0, device="cuda")
    none = torch.empty(0, 12, device="cuda")
    b.tf_embedding_backward(None, 0, None, 1, dtable, 0, 5, 12, 1.0, -1, 1, b.TF_FP32, None, 0)
    assert (dtable == 3).all()
    b.tf_embedding_backward(none, 12, None, 1, dtable, 0, 5, 12, 1.0, -1, 0, b.TF_FP32, None, 0)
    assert (dtable == 0).all()


@pytest.mark.gpu
def test_large_offsets(b):
    """Rows of the table, of y and of dy past 2^31 elements."""
    hidden, vocab = 65536, 33000          # 2.16e9 elements
    table = torch.zeros(vocab, hidden, dtype=torch.bfloat16, device="cuda")
    table[32999] = 3.0
    tokens = torch.tensor([32999, 1], device="cuda")
    stride = (1 << 31) - 8
    y = torch.zeros(stride + hidden, dtype=torch.bfloat16, device="cuda")
    b.tf_embedding_forward(tokens, 1, table, y, stride, 2, vocab, hidden, 2.0, -1, b.TF_BF16)
    assert (y[:hidden] == 6).all() and (y[stride:] == 0).all()
    del table
    y[stride:] = 1.0
    dtable = torch.ones(vocab, hidden, device="cuda")
    ws = torch.empty(b.tf_embedding_backward_workspace_size(2, vocab, hidden), dtype=torch.uint8, device="cuda")
    b.tf_embedding_backward(y, stride, tokens, 1, dtable, 2, vocab, hidden, 1.0, -1, 1, b.TF_BF16, ws, ws.numel())
    assert (dtable[32999] == 7).all() and (dtable[1] == 2).all() and (dtable[2] == 1).all()


@pytest.mark.gpu
def test_streams_and_graphs(b):
    """On another stream, and two captured calls with a workspace each, replayed with other tokens."""
    rows, vocab, hidden = 3000, 400, 512
    dy = [torch.randn(rows, hidden, device="cuda").half() for _ in range(2)]
    tokens = [_tokens("zipf", rows, vocab, seed=i) for i in range(2)]
    dtable = [torch.empty(vocab, hidden, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = [_grad(b, dy[i], tokens[i], dtable[i], 2.0, 0, "fp16", stream=side) for i in range(2)]
    side.synchronize()
    for i in range(2):
        _check_grad(dtable[i], None, dy[i], tokens[i], 2.0, 0)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            _grad(b, dy[i], tokens[i], dtable[i], 2.0, 0, "fp16", ws=ws[i])
    for i in range(2):
        tokens[i].copy_(_tokens("padded", rows, vocab, seed=7 + i))
        dtable[i].fill_(float("nan"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        _check_grad(dtable[i], None, dy[i], tokens[i], 2.0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("vocab,hidden", [(262144, 8), (262145, 8), (600001, 3), (70_000_000, 1)])
@pytest.mark.parametrize("rows", [3, 5000, 40000])
def test_backward_of_large_vocabularies(b, vocab, hidden, rows):
    """Above 2^18 words the order takes two passes; words differ in either half of their number, or in both."""
    g = torch.Generator("cuda").manual_seed(rows)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    tokens[::3] = tokens[0] % 262144 + 262144 * torch.randint(0, max(1, vocab // 262144), (tokens[::3].numel(),), generator=g, device="cuda")
    tokens[1::7] = vocab - 1
    tokens[2::11] = -1
    dy = torch.randn(rows, hidden, generator=g, device="cuda").half()
    before = torch.randn(vocab, hidden, generator=g, device="cuda")
    dtable = before.clone()
    _grad(b, dy, tokens, dtable, 0.5, 1, "fp16")
    used = torch.unique(tokens[tokens >= 0])
    place = torch.searchsorted(used, tokens.clamp(min=0))
    place[tokens < 0] = -1
    _check_grad(dtable[used], before[used], dy, place, 0.5, 1)
    dtable[used] = before[used]
    assert torch.equal(dtable, before)


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [1, 0])
def test_backward_padding_is_a_word(b, wide):
    """The padding may be a row's number: that row has no gradient, and its rows of dy are not read."""
    rows, vocab, hidden = 500, 7, 72
    tokens = torch.randint(0, vocab, (rows,), device="cuda")
    dy = torch.randn(rows, hidden, device="cuda")
    dy[tokens == 3] = float("nan")
    index = tokens if wide else tokens.int()
    ws = torch.empty(b.tf_embedding_backward_workspace_size(rows, vocab, hidden), dtype=torch.uint8, device="cuda")
    dtable = torch.full((vocab, hidden), float("nan"), device="cuda")
    b.tf_embedding_backward(dy, hidden, index, wide, dtable, rows, vocab, hidden, 1.0, 3, 0, b.TF_FP32, ws, ws.numel())
    assert (dtable[3] == 0).all()
    _check_grad(dtable, None, dy, torch.where(tokens == 3, -1, tokens), 1.0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,vocab,hidden", [(1, 5, 8), (9, 5, 8), (999, 50, 1000), (4097, 300000, 8), (5000, 3, 4096), (40000, 7, 100),
                                               (300000, 9, 8), (70000, 500, 2048)])
def test_workspace_is_kept_to(b, rows, vocab, hidden):
    """Nothing is written behind the bytes that the size function asks for."""
    for kind in ("one", "ends", "any"):
        tokens = _tokens(kind, rows, vocab)
        dy = torch.ones(rows, hidden, device="cuda").half()
        dtable = torch.empty(vocab, hidden, device="cuda")
        size = b.tf_embedding_backward_workspace_size(rows, vocab, hidden)
        buffer = torch.full((size + (1 << 20),), 0xa5, dtype=torch.uint8, device="cuda")
        _grad(b, dy, tokens, dtable, 1.0, 0, "fp16", ws=buffer[:size])
        assert (buffer[size:] == 0xa5).all()
        assert torch.equal(dtable[:, 0].double(), torch.bincount(tokens, minlength=vocab).double())
