"""Cases of the two ends of a language model: inputs, one pass, its work, its exact result.

Operators (include/tf_epilogue.h has the definitions):
  emb       y = scale * table[token]
  emb_grad  dtable (+)= scale * the sum of dy's rows by token
  score     loss = lse - logit of the target, lse = log(sum(exp(logits))), logits = scale * x W^T, none of them kept
  step      the same, then dx and dW for given gradients of loss (and of lse)

`own` selects between the plain form (elementary torch operations in 32 bits) and the library's entry points.
"""
import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
PADDING = -1     # a token that stands for none
IGNORE = -100    # a target that does not count


def _emb(op, rows, vocab, hidden, dtype, padded=0.0, pad=0, accumulate=False, wide=True):
    return dict(op=op, rows=rows, vocab=vocab, hidden=hidden, dtype=dtype, padded=padded, pad=pad, accumulate=accumulate,
                wide=wide)


def _lce(op, rows, vocab, hidden, dtype, ignored=0.0, pad=0, dlse=False, wide=True):
    return dict(op=op, rows=rows, vocab=vocab, hidden=hidden, dtype=dtype, ignored=ignored, pad=pad, dlse=dlse, wide=wide)


def listed():
    cases = [
        # a decoding step of sixteen sequences
        ("emb_decode", _emb("emb", 16, 32000, 4096, "bf16")),
        # one training batch, a tenth of it padding
        ("emb_train", _emb("emb", 16384, 128000, 4096, "bf16", padded=0.1)),
        # an odd width into a wider buffer, in full precision
        ("emb_odd", _emb("emb", 5003, 50021, 1001, "fp32", pad=6, wide=False)),
        # a micro-batch's gradient joins what the ones before (or a tied head) have left in the table's
        ("emb_grad_train", _emb("emb_grad", 16384, 32000, 4096, "bf16", accumulate=True)),
        # the step's only batch: every row of a large table's gradient is written
        ("emb_grad_fresh", _emb("emb_grad", 8192, 128000, 2048, "bf16", padded=0.1)),
        # a small fine-tuning batch
        ("emb_grad_small", _emb("emb_grad", 999, 50021, 1000, "fp16", pad=8, accumulate=True, wide=False)),
        # the likelihood of one candidate token for each of four sequences: the weights' way to the SMs
        ("score_decode", _lce("score", 4, 128000, 4096, "bf16")),
        # an evaluation batch whose prompts do not count
        ("score_eval", _lce("score", 2000, 32000, 2048, "fp16", ignored=0.3)),
        # a training batch with a penalty on lse
        ("step_train", _lce("step", 4096, 64000, 4096, "bf16", dlse=True)),
        # fine-tuning on answers only: most rows are prompts
        ("step_masked", _lce("step", 8192, 32000, 2048, "bf16", ignored=0.6)),
        # a large vocabulary over a short batch
        ("step_vocab", _lce("step", 1024, 128000, 2048, "fp16")),
        # a small batch of odd sizes, its rows in a wider buffer
        ("step_small", _lce("step", 301, 10007, 1000, "bf16", ignored=0.1, pad=8, wide=False)),
    ]
    return [dict(c, name=name) for name, c in cases]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["emb", "emb_grad", "score", "step", "step"])
    while True:
        rows, vocab = _log_uniform(rng, 1, 16384), _log_uniform(rng, 1000, 128000)
        hidden = _log_uniform(rng, 64, 4096)
        if rng.random() < 0.85:
            hidden = hidden // 8 * 8
        if op == "emb_grad" and vocab * hidden > 128000 * 2048:
            continue
        if rows * vocab * hidden * (0.25 if op == "score" else 1) <= 4096 * 64000 * 4096 or op.startswith("emb"):
            break
    pad, wide = rng.choice([0, 0, 8, 5]), rng.random() < 0.5
    if op.startswith("emb"):
        return _emb(op, rows, vocab, hidden, rng.choice(["bf16", "bf16", "fp16", "fp32"]), rng.choice([0.0, 0.1, 0.5]), pad,
                    op == "emb_grad" and rng.random() < 0.5, wide)
    return _lce(op, rows, vocab, hidden, rng.choice(["bf16", "bf16", "fp16"]), rng.choice([0.0, 0.2, 0.6]), pad,
                op == "step" and rng.random() < 0.3, wide)


def _strided(data, pad):
    """The same values in a buffer whose rows are `pad` elements longer."""
    if not pad:
        return data
    wide = torch.zeros(data.shape[0], data.shape[1] + pad, dtype=data.dtype, device=data.device)
    wide[:, :data.shape[1]] = data
    return wide[:, :data.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["dtype"]]
    rows, vocab, hidden, pad = case["rows"], case["vocab"], case["hidden"], case["pad"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(n):
        return torch.rand(n, generator=g, device="cuda", dtype=torch.float64)

    def words(n):
        """Words by frequency: the r-th most frequent one's share goes as log(1 + 1/r)."""
        rank = torch.exp(uniform(n) * math.log(vocab + 1)).long().clamp(1, vocab) - 1
        return torch.randperm(vocab, generator=g, device="cuda")[rank]

    st = dict(case=case)
    tokens = words(rows)
    share = case["padded"] if case["op"].startswith("emb") else case["ignored"]
    if share:
        tokens = torch.where(uniform(rows) < share, PADDING if case["op"].startswith("emb") else IGNORE, tokens)
    st["tokens"] = tokens if case["wide"] else tokens.int()
    if case["op"] == "emb":
        st["table"] = (normal(vocab, hidden) * hidden ** -0.5).to(t)
        st["y"] = _strided(torch.zeros(rows, hidden, dtype=t, device="cuda"), pad)
    elif case["op"] == "emb_grad":
        st["dy"] = _strided((0.02 * normal(rows, hidden)).to(t), pad)
        if case["accumulate"]:
            st["dtable"] = 0.1 * normal(vocab, hidden)
        else:
            st["dtable"] = torch.empty(vocab, hidden, device="cuda")
        if own:
            from gemm_conv_epilogues_gb300 import binding as tf
            st["ws"] = _space(tf.tf_embedding_backward_workspace_size(rows, vocab, hidden))
    else:
        # normalised rows, and weights under which the logits' deviation is between one and two
        w = normal(vocab, hidden) * (1.5 * hidden ** -0.5)
        x = normal(rows, hidden)
        # what a model has learned: the target's logit stands out by a few
        hit = st["tokens"].long().clamp(min=0)
        x = x + (w[hit] * (3.0 * uniform(rows).float()[:, None]))
        st["x"], st["w"] = _strided(x.to(t), pad), w.to(t)
        st["loss"], st["lse"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        if case["op"] == "step":
            # the mean over the targets that count; training in fp16 scales its loss
            active = (tokens != IGNORE).float()
            st["dloss"] = active * ((1024.0 if case["dtype"] == "fp16" else 1.0) / active.sum().clamp(min=1.0))
            if case["dlse"]:
                st["dlse"] = 1e-3 * st["dloss"] * (1.0 + uniform(rows).float())
            st["dx"] = _strided(torch.zeros(rows, hidden, dtype=t, device="cuda"), pad)
            st["dw"] = torch.empty(vocab, hidden, dtype=t, device="cuda")
        if own:
            from gemm_conv_epilogues_gb300 import binding as tf
            size = tf.tf_linear_cross_entropy_forward_workspace_size(rows, vocab, hidden, _dtype(tf, case))
            if case["op"] == "step":
                size = max(size, tf.tf_linear_cross_entropy_backward_workspace_size(rows, vocab, hidden, _dtype(tf, case)))
            st["ws"] = _space(size)
    return st


def _space(size):
    return torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")


def _dtype(tf, case):
    return {"fp16": tf.TF_FP16, "bf16": tf.TF_BF16, "fp32": tf.TF_FP32}[case["dtype"]]


def _emb_scale(case):
    return math.sqrt(case["hidden"])


def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    from gemm_conv_epilogues_gb300 import binding as tf
    c = st["case"]
    op, dt, rows, vocab, hidden = c["op"], _dtype(tf, c), c["rows"], c["vocab"], c["hidden"]
    index = tf.TF_INT64 if c["wide"] else tf.TF_INT32
    if op == "emb":
        tf.tf_embedding_forward(st["tokens"], index, st["table"], st["y"], st["y"].stride(0), rows, vocab, hidden,
                                _emb_scale(c), PADDING, dt)
        return [st["y"]]
    if op == "emb_grad":
        tf.tf_embedding_backward(st["dy"], st["dy"].stride(0), st["tokens"], index, st["dtable"], rows, vocab, hidden,
                                 _emb_scale(c), PADDING, int(c["accumulate"]), dt, st["ws"], st["ws"].numel())
        return [st["dtable"]]
    tf.tf_linear_cross_entropy_forward(st["x"], st["x"].stride(0), st["w"], st["tokens"], index, st["loss"], st["lse"], rows,
                                       vocab, hidden, 1.0, IGNORE, dt, st["ws"], st["ws"].numel())
    if op == "score":
        return [st["loss"], st["lse"]]
    tf.tf_linear_cross_entropy_backward(st["x"], st["x"].stride(0), st["w"], st["tokens"], index, st["lse"], st["dloss"],
                                        st.get("dlse"), st["dx"], st["dx"].stride(0), st["dw"], rows, vocab, hidden, 1.0,
                                        IGNORE, 0, dt, dt, st["ws"], st["ws"].numel())
    return [st["loss"], st["lse"], st["dx"], st["dw"]]


def _run_plain(st):
    c = st["case"]
    t = TYPES[c["dtype"]]
    op, rows, vocab, hidden = c["op"], c["rows"], c["vocab"], c["hidden"]
    tokens = st["tokens"].long()
    if op == "emb":
        y = st["table"][tokens.clamp(min=0)].float() * _emb_scale(c)
        return [torch.where((tokens != PADDING)[:, None], y, 0.0).to(t)]
    if op == "emb_grad":
        # the padding's rows go to a row behind the table
        total = torch.zeros(vocab + 1, hidden, device="cuda")
        total.index_add_(0, torch.where(tokens == PADDING, vocab, tokens), st["dy"].float())
        total = total[:vocab] * _emb_scale(c)
        if c["accumulate"]:
            st["dtable"] += total
            return [st["dtable"]]
        return [total]
    used = tokens != IGNORE
    x, w, hit = st["x"].float(), st["w"].float(), tokens.clamp(min=0)[:, None]
    logits = x @ w.t()
    top = logits.max(1, keepdim=True).values
    lse = top + torch.log(torch.exp(logits - top).sum(1, keepdim=True))
    loss = torch.where(used, (lse - logits.gather(1, hit))[:, 0], 0.0)
    out = [loss, torch.where(used, lse[:, 0], 0.0)]
    if op == "score":
        return out
    g = torch.where(used, st["dloss"], 0.0)[:, None]
    z = torch.where(used, st["dlse"], 0.0)[:, None] if c["dlse"] else 0.0
    d = torch.exp(logits - lse) * (g + z)
    d.scatter_add_(1, hit, -g)
    return out + [(d @ w).to(t), (d.t() @ x).to(t)]


def _touched(case):
    """Expected number of different words in the batch."""
    r = torch.arange(1, case["vocab"] + 1, dtype=torch.float64)
    share = torch.log1p(1.0 / r) / math.log(case["vocab"] + 1)
    return float((1.0 - torch.exp(case["rows"] * (1.0 - case["padded"]) * torch.log1p(-share))).sum())


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    rows, vocab, hidden, index = case["rows"], case["vocab"], case["hidden"], 8 if case["wide"] else 4
    if case["op"] == "emb":   # the table's rows once each, every row of y
        return {"bytes": (_touched(case) + rows) * hidden * size + rows * index, "flops": rows * hidden}
    if case["op"] == "emb_grad":
        read = rows * (1.0 - case["padded"]) * hidden
        table = 8 * hidden * _touched(case) if case["accumulate"] else 4 * hidden * vocab
        return {"bytes": read * size + rows * index + table, "flops": read}
    used = rows * (1.0 - case["ignored"])
    total = (used + vocab) * hidden * size + rows * (8 + index)
    if case["op"] == "score":
        return {"bytes": total, "flops": 2 * used * vocab * hidden}
    # three products: the logits, which the gradients need a second time where they are not kept, count once
    total += (rows + vocab) * hidden * size + 4 * rows * (2 if case["dlse"] else 1)
    return {"bytes": total, "flops": 6 * used * vocab * hidden}


def exact(case, seed):
    st = prepare(case, seed)
    op, vocab = case["op"], case["vocab"]
    tokens = st["tokens"].long()
    if op == "emb":
        keep = (tokens != PADDING).nonzero()[:, 0]
        y = torch.zeros(case["rows"], case["hidden"], dtype=torch.float64, device="cuda")
        y[keep] = torch.index_select(st["table"], 0, tokens[keep]).double() * math.sqrt(case["hidden"])
        return [y]
    if op == "emb_grad":
        out = torch.zeros(vocab, case["hidden"], dtype=torch.float64, device="cuda")
        keep = (tokens != PADDING).nonzero()[:, 0]
        out.index_put_((tokens[keep],), st["dy"][keep].double(), accumulate=True)
        out *= math.sqrt(case["hidden"])
        return [out + st["dtable"].double() if case["accumulate"] else out]
    keep = (tokens != IGNORE).nonzero()[:, 0]
    x, t = st["x"][keep].double(), tokens[keep]
    step = 8192
    spans = [slice(v, min(v + step, vocab)) for v in range(0, vocab, step)]
    lse = torch.full((keep.numel(),), -math.inf, dtype=torch.float64, device="cuda")
    for s in spans:
        lse = torch.logaddexp(lse, torch.logsumexp(torch.einsum("rh,vh->rv", x, st["w"][s].double()), dim=1))
    at = torch.einsum("rh,rh->r", x, torch.index_select(st["w"], 0, t).double())
    out = [torch.zeros(case["rows"], dtype=torch.float64, device="cuda").index_copy_(0, keep, v) for v in (lse - at, lse)]
    if op == "score":
        return out
    g = st["dloss"].double()[keep]
    both = g + st["dlse"].double()[keep] if case["dlse"] else g
    # the targets' part of the gradients apart from the probabilities'
    dx = -g[:, None] * torch.index_select(st["w"], 0, t).double()
    dw = torch.zeros(vocab, case["hidden"], dtype=torch.float64, device="cuda")
    dw.index_put_((t,), -g[:, None] * x, accumulate=True)
    for s in spans:
        w = st["w"][s].double()
        share = torch.exp(torch.einsum("rh,vh->rv", x, w) - lse[:, None]) * both[:, None]
        dx += torch.einsum("rv,vh->rh", share, w)
        dw[s] += torch.einsum("rv,rh->vh", share, x)
    full = torch.zeros(case["rows"], case["hidden"], dtype=torch.float64, device="cuda").index_copy_(0, keep, dx)
    return out + [full, dw]
