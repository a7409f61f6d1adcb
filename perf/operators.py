"""Cases of the layer-norm and grouped-product operators: inputs, one pass, its work, its exact result.

Operators (include/tf_epilogue.h has the definitions):
  ln_fwd     s = x + residual; y = (s - mean)/sqrt(var + eps)*gamma + beta, with s and the row statistics saved
  ln_bwd     dx (with the residual stream's own gradient added), dgamma and dbeta from dy, s and the statistics
  gmm        y = act(x_e W_e^T + b_e) for the rows of every expert e, with the pre-activation saved when training
  gmm_dgrad  dx = (dy_e W_e) * act'(pre), the gradient that reaches the layer below
  gmm_wgrad  dW_e = dy_e^T x_e and db_e = the sum of dy_e's rows

`own` selects between the plain form (elementary torch operations in 32 bits) and the library's entry points.
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def _ln(op, rows, hidden, dtype, residual, pad=0, **kw):
    return dict(op=op, rows=rows, hidden=hidden, dtype=dtype, residual=residual, pad=pad, **kw)


def _gmm(op, rows, used, groups, n, k, dtype, act="none", bias=False, save=False, skew=0.5):
    return dict(op=op, rows=rows, used=used, groups=groups, n=n, k=k, dtype=dtype, act=act, bias=bias, save=save,
                skew=skew)


def listed():
    cases = [
        # one decoding step of four sequences: the norm before a block, the residual stream updated, nothing saved
        ("ln_fwd_decode", _ln("ln_fwd", 4, 4096, "bf16", True, stats=False)),
        # the forward pass of one training batch: residual stream and row statistics saved for the backward pass
        ("ln_fwd_train", _ln("ln_fwd", 16384, 4096, "bf16", True, stats=True)),
        # its backward pass; the residual stream's gradient joins dx
        ("ln_bwd_train", _ln("ln_bwd", 16384, 4096, "bf16", True)),
        # a narrow norm over very many rows (patches of an image batch), where the weight's gradient is a long sum
        ("ln_bwd_narrow", _ln("ln_bwd", 50001, 640, "fp16", False)),
        # an odd width whose rows lie in a wider buffer, in full precision
        ("ln_bwd_odd", _ln("ln_bwd", 1999, 5003, "fp32", False, pad=6)),
        # a decoding step: eight tokens, two experts each, most of the time is the weights' way to the SMs
        ("gmm_decode", _gmm("gmm", 16, 16, 16, 2048, 4096, "bf16", act="silu", bias=True)),
        # the experts' first product in training, the pre-activation saved
        ("gmm_train", _gmm("gmm", 16384, 16384, 16, 4096, 2048, "bf16", act="gelu", bias=True, save=True)),
        # a short prompt over many small experts of uneven widths, in a buffer with room for more rows
        ("gmm_ragged", _gmm("gmm", 1100, 999, 24, 1000, 520, "fp16", skew=1.0)),
        # the second product's gradient, which leaves as the first one's pre-activation gradient
        ("gmm_dgrad_train", _gmm("gmm_dgrad", 16384, 16384, 16, 2048, 4096, "bf16", act="gelu")),
        # a small fine-tuning batch
        ("gmm_dgrad_ragged", _gmm("gmm_dgrad", 700, 651, 24, 520, 1000, "fp16", skew=1.0)),
        # the weights' gradients of the training batch, and of the small one
        ("gmm_wgrad_train", _gmm("gmm_wgrad", 16384, 16384, 16, 4096, 2048, "bf16", bias=True)),
        ("gmm_wgrad_ragged", _gmm("gmm_wgrad", 1100, 999, 24, 1000, 520, "fp16", bias=True, skew=1.0)),
    ]
    return [dict(c, name=name) for name, c in cases]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "gmm", "gmm_dgrad", "gmm_wgrad"])
    if op.startswith("ln"):
        while True:
            hidden = _log_uniform(rng, 64, 32768)
            if rng.random() < 0.7:
                hidden = max(64, hidden // 64 * 64)
            rows = _log_uniform(rng, 1, 60000)
            dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
            if rows * hidden * (2 if dtype == "fp32" else 1) <= 16384 * 4096:
                break
        case = _ln(op, rows, hidden, dtype, rng.random() < 0.5, pad=rng.choice([0, 0, 8, 5]))
        if op == "ln_fwd":
            case["stats"] = rng.random() < 0.6
        return case
    while True:
        groups = _log_uniform(rng, 1, 64)
        n, k = _log_uniform(rng, 64, 4096), _log_uniform(rng, 64, 4096)
        if rng.random() < 0.9:   # widths are multiples of eight but for a few
            n, k = n // 8 * 8, k // 8 * 8
        used = _log_uniform(rng, 1, 16384)
        if used * n * k <= 16384 * 4096 * 2048 and groups * n * k <= 16 * 4096 * 2048:
            break
    act = rng.choice(["none", "silu", "gelu"])
    return _gmm(op, used + rng.choice([0, 0, 37]), used, groups, n, k, rng.choice(["bf16", "fp16"]),
                act="none" if op == "gmm_wgrad" else act, bias=op != "gmm_dgrad" and rng.random() < 0.6,
                save=op == "gmm" and act != "none" and rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 1.0]))


def _counts(case):
    """Rows per expert, largest first: shares fall off as a power of the rank, and sum to the rows in use."""
    share = [(i + 1.0) ** -case["skew"] for i in range(case["groups"])]
    total = sum(share)
    exact_rows = [case["used"] * s / total for s in share]
    rows = [int(r) for r in exact_rows]
    by_rest = sorted(range(len(rows)), key=lambda i: rows[i] - exact_rows[i])
    for i in by_rest[:case["used"] - sum(rows)]:
        rows[i] += 1
    return rows


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

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    st = dict(case=case)
    if case["op"].startswith("ln"):
        rows, hidden, pad = case["rows"], case["hidden"], case["pad"]
        # a residual stream: channels of their own means and scales, a few of them large
        scale = 0.5 + normal(hidden).abs()
        scale = torch.where(torch.rand(hidden, generator=g, device="cuda") < 0.004, scale * 8, scale)
        x = (normal(rows, hidden) * scale + 0.3 * normal(hidden)).to(t)
        st.update(x=_strided(x, pad), gamma=1.0 + 0.1 * normal(hidden), beta=0.1 * normal(hidden))
        if case["op"] == "ln_fwd":
            if case["residual"]:
                st["res"] = _strided(normal(rows, hidden).to(t), pad)
                st["s"] = torch.empty(rows, hidden, dtype=t, device="cuda")
            if case["stats"]:
                st["mean"], st["rstd"] = (torch.empty(rows, device="cuda") for _ in range(2))
            st["y"] = torch.empty(rows, hidden, dtype=t, device="cuda")
        else:
            xd = x.double()
            mean = xd.mean(1)
            var = (xd * xd).mean(1) - mean * mean
            st.update(mean=mean.float(), rstd=(1.0 / (var + EPS).sqrt()).float(),
                      dy=_strided((0.05 * normal(rows, hidden)).to(t), pad))
            if case["residual"]:
                st["ds"] = (0.05 * normal(rows, hidden)).to(t)
            st.update(dx=torch.empty(rows, hidden, dtype=t, device="cuda"),
                      dgamma=torch.empty(hidden, device="cuda"), dbeta=torch.empty(hidden, device="cuda"))
            if own:
                from gemm_conv_epilogues_gb300 import binding as tf
                size = tf.tf_layernorm_backward_workspace_size(rows, hidden, _dtype(tf, case))
                st["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
        return st

    rows, groups, n, k = case["rows"], case["groups"], case["n"], case["k"]
    order = torch.randperm(groups, generator=torch.Generator().manual_seed(seed)).tolist()
    counts = _counts(case)
    offsets = [0]
    for i in order:
        offsets.append(offsets[-1] + counts[i])
    st["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    if case["op"] != "gmm_wgrad":
        st["w"] = (normal(groups, n, k) * k ** -0.5).to(t)
    if case["op"] == "gmm":
        st["x"] = normal(rows, k).to(t)
        if case["bias"]:
            st["bias"] = 0.1 * normal(groups, n)
        st["y"] = torch.zeros(rows, n, dtype=t, device="cuda")
        if case["save"]:
            st["pre"] = torch.zeros(rows, n, dtype=t, device="cuda")
    elif case["op"] == "gmm_dgrad":
        st["dy"] = (0.1 * normal(rows, n)).to(t)
        if case["act"] != "none":
            st["pre"] = normal(rows, k).to(t)
        st["dx"] = torch.zeros(rows, k, dtype=t, device="cuda")
    else:
        st["dy"] = (0.1 * normal(rows, n)).to(t)
        st["x"] = normal(rows, k).to(t)
        st["dw"] = torch.empty(groups, n, k, device="cuda")
        if case["bias"]:
            st["db"] = torch.empty(groups, n, device="cuda")
        if own:
            from gemm_conv_epilogues_gb300 import binding as tf
            size = tf.tf_grouped_matmul_wgrad_workspace_size(rows, groups, n, k, _dtype(tf, case))
            st["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    return st


def _dtype(tf, case):
    return {"fp16": tf.TF_FP16, "bf16": tf.TF_BF16, "fp32": tf.TF_FP32}[case["dtype"]]


def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    from gemm_conv_epilogues_gb300 import binding as tf
    c = st["case"]
    op, dt = c["op"], _dtype(tf, c)

    def stride(name):
        return st[name].stride(0) if name in st else 0

    if op == "ln_fwd":
        tf.tf_layernorm_forward(st["x"], stride("x"), st.get("res"), stride("res"), st["gamma"], st["beta"], st["y"],
                                stride("y"), st.get("s"), stride("s"), st.get("mean"), st.get("rstd"), c["rows"],
                                c["hidden"], EPS, dt)
        return [st[v] for v in ("y", "s", "mean", "rstd") if v in st]
    if op == "ln_bwd":
        tf.tf_layernorm_backward(st["dy"], stride("dy"), st["x"], stride("x"), st["gamma"], st["mean"], st["rstd"],
                                 st.get("ds"), stride("ds"), st["dx"], stride("dx"), st["dgamma"], st["dbeta"],
                                 c["rows"], c["hidden"], 0, dt, st["ws"], st["ws"].numel())
        return [st["dx"], st["dgamma"], st["dbeta"]]
    act = {"none": tf.TF_ACT_NONE, "silu": tf.TF_ACT_SILU, "gelu": tf.TF_ACT_GELU}[c["act"]]
    rows, groups, n, k = c["rows"], c["groups"], c["n"], c["k"]
    if op == "gmm":
        tf.tf_grouped_matmul(st["x"], stride("x"), st["w"], st.get("bias"), st["offsets"], st["y"], stride("y"),
                             st.get("pre"), stride("pre"), rows, groups, n, k, act, dt)
        return [st[v] for v in ("y", "pre") if v in st]
    if op == "gmm_dgrad":
        tf.tf_grouped_matmul_dgrad(st["dy"], stride("dy"), st["w"], st["offsets"], st.get("pre"), stride("pre"),
                                   st["dx"], stride("dx"), rows, groups, n, k, act, dt)
        return [st["dx"]]
    tf.tf_grouped_matmul_wgrad(st["dy"], stride("dy"), st["x"], stride("x"), st["offsets"], st["dw"], st.get("db"),
                               rows, groups, n, k, 0, dt, st["ws"], st["ws"].numel())
    return [st[v] for v in ("dw", "db") if v in st]


def _act(name, z):
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -(0.5 ** 0.5))
    return z


def _act_grad(name, z):
    if name == "silu":
        sig = 1.0 / (1.0 + torch.exp(-z))
        return sig * (1.0 + z * (1.0 - sig))
    if name == "gelu":
        return 0.5 * torch.erfc(z * -(0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5
    return torch.ones_like(z)


def _run_plain(st):
    c = st["case"]
    t = TYPES[c["dtype"]]
    op = c["op"]
    if op == "ln_fwd":
        s = st["x"].float()
        if "res" in st:
            s = s + st["res"].float()
        mean = s.sum(1, keepdim=True) / c["hidden"]
        d = s - mean
        rstd = 1.0 / torch.sqrt((d * d).sum(1, keepdim=True) / c["hidden"] + EPS)
        y = (d * rstd * st["gamma"] + st["beta"]).to(t)
        return [y] + ([s.to(t)] if "res" in st else []) + ([mean[:, 0], rstd[:, 0]] if "mean" in st else [])
    if op == "ln_bwd":
        dy = st["dy"].float()
        xhat = (st["x"].float() - st["mean"][:, None]) * st["rstd"][:, None]
        dgamma, dbeta = (dy * xhat).sum(0), dy.sum(0)
        w = dy * st["gamma"]
        c1 = w.sum(1, keepdim=True) / c["hidden"]
        c2 = (w * xhat).sum(1, keepdim=True) / c["hidden"]
        dx = st["rstd"][:, None] * (w - c1 - xhat * c2)
        if "ds" in st:
            dx = dx + st["ds"].float()
        return [dx.to(t), dgamma, dbeta]
    off = st["offsets"].tolist()
    if op == "gmm":
        y = torch.zeros_like(st["y"])
        pre = torch.zeros_like(st["y"]) if c["save"] else None
        for e in range(c["groups"]):
            lo, hi = off[e], off[e + 1]
            if lo == hi:
                continue
            z = st["x"][lo:hi].float() @ st["w"][e].float().t()
            if "bias" in st:
                z = z + st["bias"][e]
            y[lo:hi] = _act(c["act"], z).to(t)
            if pre is not None:
                pre[lo:hi] = z.to(t)
        return [y] if pre is None else [y, pre]
    if op == "gmm_dgrad":
        dx = torch.zeros_like(st["dx"])
        for e in range(c["groups"]):
            lo, hi = off[e], off[e + 1]
            if lo == hi:
                continue
            d = st["dy"][lo:hi].float() @ st["w"][e].float()
            if "pre" in st:
                d = d * _act_grad(c["act"], st["pre"][lo:hi].float())
            dx[lo:hi] = d.to(t)
        return [dx]
    dw = torch.zeros_like(st["dw"])
    db = torch.zeros_like(st["db"]) if "db" in st else None
    for e in range(c["groups"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        dy = st["dy"][lo:hi].float()
        dw[e] = dy.t() @ st["x"][lo:hi].float()
        if db is not None:
            db[e] = dy.sum(0)
    return [dw] if db is None else [dw, db]


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"].startswith("ln"):
        elements = case["rows"] * case["hidden"]
        if case["op"] == "ln_fwd":   # x and y, and with a residual also it and the sum
            stats = 8 * case["rows"] if case["stats"] else 0
            return {"bytes": elements * size * (4 if case["residual"] else 2) + 8 * case["hidden"] + stats,
                    "flops": 9 * elements}
        return {"bytes": elements * size * (4 if case["residual"] else 3) + 12 * case["hidden"] + 8 * case["rows"],
                "flops": 16 * elements}
    used, groups, n, k = case["used"], case["groups"], case["n"], case["k"]
    active = sum(1 for r in _counts(case) if r)
    flops = 2 * used * n * k
    if case["op"] == "gmm":
        total = used * (k + n * (2 if case["save"] else 1)) * size + active * n * k * size
        total += active * n * 4 if case["bias"] else 0
    elif case["op"] == "gmm_dgrad":
        total = used * (n + k * (2 if case["act"] != "none" else 1)) * size + active * n * k * size
    else:   # the gradient of every expert is written, of those without rows too
        total = used * (n + k) * size + groups * n * k * 4
        total += groups * n * 4 if case["bias"] else 0
    return {"bytes": total + 4 * (groups + 1), "flops": flops}


def exact(case, seed):
    st = prepare(case, seed)
    v = {name: x.double() if torch.is_tensor(x) and x.is_floating_point() else x for name, x in st.items()}
    op = case["op"]
    if op == "ln_fwd":
        s = v["x"] + v["res"] if case["residual"] else v["x"]
        var, mean = torch.var_mean(s, dim=1, correction=0, keepdim=True)
        root = (var + EPS).sqrt()
        out = [torch.addcmul(v["beta"], (s - mean) / root, v["gamma"])]
        if case["residual"]:
            out.append(s)
        if case["stats"]:
            out += [mean.flatten(), root.reciprocal().flatten()]
        return out
    if op == "ln_bwd":
        # the two projections that the norm takes out of the gradient, row by row
        rstd = v["rstd"].unsqueeze(1)
        xhat = (v["x"] - v["mean"].unsqueeze(1)) * rstd
        gx = v["dy"] * v["gamma"]
        along = torch.einsum("rh,rh->r", gx, xhat).div(case["hidden"]).unsqueeze(1)
        dx = (gx - gx.mean(1, keepdim=True) - along * xhat) * rstd
        if case["residual"]:
            dx += v["ds"]
        return [dx, torch.einsum("rh,rh->h", v["dy"], xhat), v["dy"].sum(0)]
    bounds = st["offsets"].cpu().tolist()
    spans = [(e, slice(lo, hi)) for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])) if hi > lo]
    if op == "gmm":
        z = torch.zeros_like(v["y"])
        for e, rows in spans:
            z[rows] = torch.einsum("rk,nk->rn", v["x"][rows], v["w"][e])
            if case["bias"]:
                z[rows] += v["bias"][e]
        y = {"none": lambda: z, "silu": lambda: z * torch.sigmoid(z), "gelu": lambda: z * torch.special.ndtr(z)}
        out = y[case["act"]]()
        return [out, z] if case["save"] else [out]
    if op == "gmm_dgrad":
        dx = torch.zeros_like(v["dx"])
        for e, rows in spans:
            dx[rows] = torch.einsum("rn,nk->rk", v["dy"][rows], v["w"][e])
        if case["act"] != "none":
            p = v["pre"]
            if case["act"] == "silu":
                half = torch.tanh(0.5 * p)
                dx *= 0.5 * (1 + half) + 0.25 * p * (1 - half * half)
            else:
                dx *= torch.special.ndtr(p) + p * torch.exp(torch.distributions.Normal(0.0, 1.0).log_prob(p))
        return [dx]
    dw = torch.zeros_like(v["dw"])
    for e, rows in spans:
        dw[e] = torch.einsum("rn,rk->nk", v["dy"][rows], v["x"][rows])
    if not case["bias"]:
        return [dw]
    db = torch.zeros_like(v["db"])
    for e, rows in spans:
        db[e] = torch.einsum("rn->n", v["dy"][rows])
    return [dw, db]
