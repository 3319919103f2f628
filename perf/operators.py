"""The operators around the selective scan, as measured cases.

Three operators of a language model of scan layers: the short causal
convolution before the scan ("conv"), the layer norm of the residual stream
("norm") and the softmax cross entropy over the vocabulary ("loss").  Each case
is one pass of one of them: a forward, a training pass (forward and backward)
or a step of single tokens.
"""
import torch
import torch.nn.functional as F

own = False

BF16, F32 = "bf16", "f32"
TYPES = {BF16: torch.bfloat16, F32: torch.float32}
EPS = 1e-5
IGNORE = -100


def conv(kind, dtype, batch, seqlen, dim, width=4, silu=True, bias=True, masked=False, carry=False, packed=False):
    """masked: rows have valid lengths U{1..seqlen}; carry: from a given state, returning the last one;
    packed: x is the first half of the columns of a projection's output, as in a layer whose
    projection gives x and the gate together."""
    return {"op": "conv", "kind": kind, "dtype": dtype, "batch": batch, "seqlen": seqlen, "dim": dim, "width": width, "silu": silu,
            "bias": bias, "masked": masked, "carry": carry, "packed": packed}


def norm(kind, dtype, rows, dim, rms=False, bias=True, residual=""):
    """residual: the type of the residual stream that x is added to, "" for none."""
    return {"op": "norm", "kind": kind, "dtype": dtype, "rows": rows, "dim": dim, "rms": rms, "bias": bias, "residual": residual}


def loss(kind, tokens, vocab, dim, ignored=0.0):
    """ignored: the share of the tokens whose target is the ignored one (padding, prompts)."""
    return {"op": "loss", "kind": kind, "tokens": tokens, "vocab": vocab, "dim": dim, "ignored": ignored}


def listed():
    return [
        # one sequence generating, one layer's convolution: latency
        {"name": "conv-step-b1", **conv("step", BF16, 1, 1, 2048)},
        # the same for a serving batch
        {"name": "conv-step-b1024", **conv("step", BF16, 1024, 1, 2048)},
        # a batch of padded prompts read out of the input projection, keeping the state to generate from
        {"name": "conv-prompt-varlen", **conv("fwd", BF16, 32, 2048, 1536, masked=True, carry=True, packed=True)},
        # a training step's convolution at the default scan workload's size
        {"name": "conv-train-f32", **conv("train", F32, 8, 4096, 1024)},
        # one token's norm while generating: latency
        {"name": "norm-fwd-row", **norm("fwd", BF16, 1, 2048, rms=True, bias=False, residual=F32)},
        # a training step's norm, everything in 16 bits
        {"name": "norm-train-bf16", **norm("train", BF16, 32768, 1024, residual=BF16)},
        # an odd width, fp32, no residual stream
        {"name": "norm-train-f32-odd", **norm("train", F32, 5001, 1537)},
        # a large training batch whose residual stream is kept in 32 bits
        {"name": "norm-train-mixed", **norm("train", BF16, 65536, 1536, rms=True, bias=False, residual=F32)},
        # scoring one token
        {"name": "loss-score-1", **loss("fwd", 1, 32768, 1024)},
        # scoring prompts: the forward alone, an odd vocabulary
        {"name": "loss-score-4096", **loss("fwd", 4096, 50257, 1536)},
        # a small fine-tuning batch, about half of it prompt or padding
        {"name": "loss-train-ragged", **loss("train", 1000, 32001, 768, ignored=0.5)},
        # a pre-training batch
        {"name": "loss-train-large", **loss("train", 8192, 65536, 2048)},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["conv-step", "conv-fwd", "conv-train", "norm-fwd", "norm-train", "loss-fwd", "loss-train"])
    dtype = rng.choice([BF16, BF16, F32])
    if op.startswith("conv"):
        dim = rng.choice([64, 200, 513, 768, 1000, 1024, 1536, 2048, 2560, 4096])
        width = rng.choice([2, 3, 4, 4, 4])
        more = {"width": width, "silu": rng.random() < 0.8, "bias": rng.random() < 0.8}
        if op == "conv-step":
            return conv("step", dtype, _log(rng, 1, 1024), 1, dim, **more)
        batch = _log(rng, 1, 32)
        seqlen = _log(rng, 1, max(2, min(32768, 100_000_000 // (batch * dim))))
        return conv(op[5:], dtype, batch, seqlen, dim, masked=rng.random() < 0.5, carry=rng.random() < 0.5, packed=rng.random() < 0.5, **more)
    if op.startswith("norm"):
        dim = rng.choice([64, 200, 513, 768, 1000, 1024, 1537, 2048, 2560, 4096, 6000, 8192])
        rows = _log(rng, 1, 100_000_000 // dim)
        rms = rng.random() < 0.5
        residual = rng.choice(["", dtype, F32])
        return norm(op[5:], dtype, rows, dim, rms=rms, bias=not rms and rng.random() < 0.8, residual=residual)
    dim = rng.choice([64, 200, 512, 768, 1000, 1024, 1536, 2048])
    return loss(op[5:], _log(rng, 1, 8192), _log(rng, 1000, 65536), dim, ignored=rng.choice([0.0, 0.1, 0.5]))


# ---- inputs ----------------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    f32 = torch.float32

    def randn(*shape, dtype=f32, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"case": case}
    if case["op"] == "conv":
        dt, B, L, D, K = TYPES[case["dtype"]], case["batch"], case["seqlen"], case["dim"], case["width"]
        s["w"] = (torch.rand(D, K, generator=g, device="cuda") * 2 - 1) / K ** 0.5
        s["b"] = (torch.rand(D, generator=g, device="cuda") * 2 - 1) / K ** 0.5 if case["bias"] else None
        if case["kind"] == "step":
            s["x"], s["state"] = randn(B, D, dtype=dt), randn(B, K - 1, D, dtype=dt)
            return s
        x = randn(B, L, 2 * D if case["packed"] else D, dtype=dt)
        s["x"] = x[:, :, :D]
        s["valid"] = torch.randint(1, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if case["masked"] else None
        s["state0"] = randn(B, K - 1, D, dtype=dt) if case["carry"] else None
        if case["kind"] == "train":
            s["dy"] = randn(B, L, D, dtype=dt)
    elif case["op"] == "norm":
        dt, R, D = TYPES[case["dtype"]], case["rows"], case["dim"]
        rt = TYPES[case["residual"]] if case["residual"] else None
        s["x"] = randn(R, D, dtype=dt)
        s["residual"] = (randn(R, D, scale=3.0) + 0.5).to(rt) if rt else None  # a stream that earlier layers have added to
        s["w"] = 1 + randn(D, scale=0.1)
        s["b"] = randn(D, scale=0.1) if case["bias"] else None
        if case["kind"] == "train":
            s["dy"] = randn(R, D, dtype=dt)
            s["dr"] = randn(R, D, dtype=rt) if rt else None  # the gradient that comes back along the stream
    else:
        T, V, D = case["tokens"], case["vocab"], case["dim"]
        s["h"] = randn(T, D, dtype=torch.bfloat16)
        s["w"] = randn(V, D, dtype=torch.bfloat16, scale=2 / D ** 0.5)
        s["targets"] = torch.randint(0, V, (T,), generator=g, device="cuda")
        if case["ignored"]:
            out = torch.rand(T, generator=g, device="cuda") < case["ignored"]
            s["targets"] = torch.where(out, torch.full_like(s["targets"], IGNORE), s["targets"])
        if case["kind"] == "train":
            s["dloss"] = torch.full((T,), 1.0 / T, device="cuda")
    return s


# ---- one pass ----------------------------------------------------------------------------------


def run(s):
    c = s["case"]
    return (_own if own else _plain)[c["op"], c["kind"]](s, c)


def _plain_conv_pre(xp, s, L):
    w = s["w"]
    pre = sum(w[:, k] * xp[:, k:k + L] for k in range(w.shape[1]))
    return pre if s["b"] is None else pre + s["b"]


def _plain_conv_step(s, c):
    x, state = s["x"], s["state"]
    xp = torch.cat([state.float(), x.float()[:, None]], 1)
    pre = _plain_conv_pre(xp, s, 1)[:, 0]
    y = pre / (1 + torch.exp(-pre)) if c["silu"] else pre
    state.copy_(xp[:, 1:])
    return {"y": y.to(x.dtype), "state": state}


def _plain_conv_padded(s, c):
    x, K = s["x"].float(), c["width"]
    head = s["state0"].float() if s["state0"] is not None else x.new_zeros(x.shape[0], K - 1, x.shape[2])
    return torch.cat([head, x], 1)


def _plain_conv_valid(s, c):
    if s["valid"] is None:
        return None
    return (torch.arange(c["seqlen"], device="cuda") < s["valid"][:, None])[:, :, None]


def _plain_conv_y(pre, valid, s, c):
    y = pre / (1 + torch.exp(-pre)) if c["silu"] else pre
    return (y if valid is None else torch.where(valid, y, 0.0)).to(s["x"].dtype)


def _plain_conv_fwd(s, c):
    L, K = c["seqlen"], c["width"]
    xp = _plain_conv_padded(s, c)
    out = {"y": _plain_conv_y(_plain_conv_pre(xp, s, L), _plain_conv_valid(s, c), s, c)}
    if c["carry"]:
        end = s["valid"].long() if s["valid"] is not None else torch.full((c["batch"],), L, device="cuda")
        at = end[:, None] + torch.arange(K - 1, device="cuda")
        out["final"] = torch.gather(xp, 1, at[:, :, None].expand(-1, -1, c["dim"])).to(s["x"].dtype)
    return out


def _plain_conv_train(s, c):
    L, K, w, dt = c["seqlen"], c["width"], s["w"], s["x"].dtype
    xp = _plain_conv_padded(s, c)
    pre, valid = _plain_conv_pre(xp, s, L), _plain_conv_valid(s, c)
    out = {"y": _plain_conv_y(pre, valid, s, c)}
    dpre = s["dy"].float()
    if c["silu"]:
        sig = 1 / (1 + torch.exp(-pre))
        dpre = dpre * sig * (1 + pre * (1 - sig))
    if valid is not None:
        dpre = torch.where(valid, dpre, 0.0)
    side = dpre.new_zeros(dpre.shape[0], K - 1, dpre.shape[2])
    dp = torch.cat([side, dpre, side], 1)
    dxp = sum(w[:, k] * dp[:, K - 1 - k:2 * K - 2 - k + L] for k in range(K))
    out["dx"] = dxp[:, K - 1:].to(dt)
    if s["state0"] is not None:
        out["dstate0"] = dxp[:, :K - 1].to(dt)
    out["dw"] = torch.stack([(dpre * xp[:, k:k + L]).sum((0, 1)) for k in range(K)], 1)
    if s["b"] is not None:
        out["db"] = dpre.sum((0, 1))
    return out


def _own_conv_step(s, c):
    import selective_state_space_fwd_gb300 as S
    return {"y": S.conv_step(s["x"], s["w"], s["b"], state=s["state"], silu=c["silu"]), "state": s["state"]}


def _own_conv_fwd(s, c):
    import selective_state_space_fwd_gb300 as S
    if c["carry"]:
        y, final = S.conv_fwd(s["x"], s["w"], s["b"], s["valid"], state0=s["state0"], silu=c["silu"], want_final=True)
        return {"y": y, "final": final}
    return {"y": S.conv_fwd(s["x"], s["w"], s["b"], s["valid"], silu=c["silu"])}


def _own_conv_train(s, c):
    import selective_state_space_fwd_gb300 as S
    out = {"y": S.conv_fwd(s["x"], s["w"], s["b"], s["valid"], state0=s["state0"], silu=c["silu"])}
    g = S.conv_bwd(s["x"], s["w"], s["b"], s["valid"], dy=s["dy"], state0=s["state0"], silu=c["silu"], want_dstate0=s["state0"] is not None)
    out["dx"], out["dw"] = g["dx"], g["dweight"]
    if s["state0"] is not None:
        out["dstate0"] = g["dstate0"]
    if s["b"] is not None:
        out["db"] = g["dbias"]
    return out


def _plain_norm(s, c):
    x = s["x"].float()
    out = {}
    r = x
    if s["residual"] is not None:
        out["r"] = (x + s["residual"].float()).to(s["residual"].dtype)
        r = out["r"].float()  # the norm is that of the stream as it is stored
    m = r if c["rms"] else r - r.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((m * m).mean(-1, keepdim=True) + EPS)
    xhat = m * rstd
    y = xhat * s["w"]
    out["y"] = (y if s["b"] is None else y + s["b"]).to(s["x"].dtype)
    return out, xhat, rstd


def _plain_norm_fwd(s, c):
    return _plain_norm(s, c)[0]


def _plain_norm_train(s, c):
    out, xhat, rstd = _plain_norm(s, c)
    dy = s["dy"].float()
    g = dy * s["w"]
    d = g - xhat * (g * xhat).mean(-1, keepdim=True)
    if not c["rms"]:
        d = d - g.mean(-1, keepdim=True)
    d = d * rstd
    if s["residual"] is not None:
        d = d + s["dr"].float()
        out["dresidual"] = d.to(s["residual"].dtype)
    out["dx"] = d.to(s["x"].dtype)
    out["dw"] = (dy * xhat).sum(0)
    if s["b"] is not None:
        out["db"] = dy.sum(0)
    return out


def _own_norm_fwd(s, c):
    import selective_state_space_fwd_gb300 as S
    y, r, _ = S.norm_fwd(s["x"], s["w"], s["b"], residual=s["residual"], rms=c["rms"], eps=EPS)
    return {"y": y} if r is None else {"y": y, "r": r}


def _own_norm_train(s, c):
    import selective_state_space_fwd_gb300 as S
    y, r, stats = S.norm_fwd(s["x"], s["w"], s["b"], residual=s["residual"], rms=c["rms"], eps=EPS, want_stats=True)
    g = S.norm_bwd(s["x"] if r is None else r, s["w"], stats=stats, dy=s["dy"], dr=s["dr"], rms=c["rms"], want_dbias=s["b"] is not None)
    out = {"y": y, "dx": g["dx"], "dw": g["dweight"]}
    if r is not None:
        out["r"], out["dresidual"] = r, g["dresidual"]
    if s["b"] is not None:
        out["db"] = g["dbias"]
    return out


def _plain_loss(s):
    h, w, t = s["h"].float(), s["w"].float(), s["targets"]
    kept = t != IGNORE
    logits = h @ w.T
    top = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(-1, keepdim=True)
    at = torch.where(kept, t, 0)[:, None]
    lse = torch.log(total) + top
    value = torch.where(kept, (lse - logits.gather(1, at))[:, 0], 0.0)
    return h, w, kept, at, e, total, {"loss": value, "lse": torch.where(kept, lse[:, 0], 0.0)}


def _plain_loss_fwd(s, c):
    return _plain_loss(s)[-1]


def _plain_loss_train(s, c):
    h, w, kept, at, e, total, out = _plain_loss(s)
    p = e / total
    p.scatter_add_(1, at, torch.full_like(total, -1.0))
    p = p * torch.where(kept, s["dloss"], 0.0)[:, None]
    return {**out, "dh": (p @ w).to(s["h"].dtype), "dw": (p.T @ h).to(s["w"].dtype)}


def _own_loss_fwd(s, c):
    import selective_state_space_fwd_gb300 as S
    value, lse = S.xent_fwd(s["h"], s["w"], s["targets"], ignore_index=IGNORE)
    return {"loss": value, "lse": lse}


def _own_loss_train(s, c):
    import selective_state_space_fwd_gb300 as S
    value, lse = S.xent_fwd(s["h"], s["w"], s["targets"], ignore_index=IGNORE)
    g = S.xent_bwd(s["h"], s["w"], s["targets"], lse=lse, dloss=s["dloss"], ignore_index=IGNORE)
    return {"loss": value, "lse": lse, "dh": g["dh"], "dw": g["dweight"]}


_plain = {("conv", "step"): _plain_conv_step, ("conv", "fwd"): _plain_conv_fwd, ("conv", "train"): _plain_conv_train, ("norm", "fwd"): _plain_norm_fwd,
          ("norm", "train"): _plain_norm_train, ("loss", "fwd"): _plain_loss_fwd, ("loss", "train"): _plain_loss_train}
_own = {("conv", "step"): _own_conv_step, ("conv", "fwd"): _own_conv_fwd, ("conv", "train"): _own_conv_train, ("norm", "fwd"): _own_norm_fwd,
        ("norm", "train"): _own_norm_train, ("loss", "fwd"): _own_loss_fwd, ("loss", "train"): _own_loss_train}


# ---- what a pass cannot do without ---------------------------------------------------------------


def work(case):
    if case["op"] == "conv":
        e = 2 if case["dtype"] == BF16 else 4
        B, L, D, K = case["batch"], case["seqlen"], case["dim"], case["width"]
        small = 4 * D * (K + bool(case["bias"]))
        state = B * (K - 1) * D * e
        per = 2 * K + (5 if case["silu"] else 0)
        if case["kind"] == "step":
            return {"bytes": 2 * B * D * e + 2 * state + small, "flops": B * D * per}
        valid = B * L * D * (0.5 if case["masked"] else 1.0)  # what is read; outputs are written in full
        whole = B * L * D
        carry = 2 * state if case["carry"] else 0
        if case["kind"] == "fwd":
            return {"bytes": (valid + whole) * e + small + carry, "flops": valid * per}
        return {"bytes": (valid + whole) * e + (2 * valid + whole) * e + 2 * small + carry, "flops": valid * (2 * per + 4 * K + 6)}
    if case["op"] == "norm":
        n, D = case["rows"] * case["dim"], case["dim"]
        e = 2 if case["dtype"] == BF16 else 4
        r = {"": 0, BF16: 2, F32: 4}[case["residual"]]
        small = 4 * D * (1 + bool(case["bias"]))
        fwd = n * (2 * e + 2 * r) + small
        if case["kind"] == "fwd":
            return {"bytes": fwd, "flops": 8 * n}
        same = case["residual"] == case["dtype"]  # dx and dresidual are then one tensor
        bwd = n * (e + (r or e) + r + e + (r if not same else 0)) + 2 * small  # dy, r (x without a stream), dr; dx, dresidual
        return {"bytes": fwd + bwd + 8 * case["rows"], "flops": 22 * n}
    T, V, D = case["tokens"] * (1 - case["ignored"]), case["vocab"], case["dim"]
    if case["kind"] == "fwd":
        return {"bytes": 2 * (T + V) * D + 16 * case["tokens"], "flops": 2 * T * V * D + 4 * T * V}
    return {"bytes": 4 * (T + V) * D + 24 * case["tokens"], "flops": 8 * T * V * D + 10 * T * V}


# ---- the definitions in 64 bits ---------------------------------------------------------------------


def _exact_conv_pre(x, w, b, head):
    xp = torch.cat([head, x], 1).transpose(1, 2)
    return F.conv1d(xp, w[:, None], b, groups=w.shape[0]).transpose(1, 2)


def exact(case, seed):
    s = prepare(case, seed)
    f64 = {k: v.detach().double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    leaf = {k: f64[k].requires_grad_() for k in ("x", "w", "b", "state0", "residual", "h") if k in f64}
    train = case["kind"] == "train"
    if case["op"] == "conv":
        w, b, K = leaf["w"], leaf.get("b"), case["width"]
        act = F.silu if case["silu"] else (lambda v: v)
        if case["kind"] == "step":
            y = act(_exact_conv_pre(leaf["x"][:, None], w, b, f64["state"]))[:, 0]
            return {"y": y.detach(), "state": torch.cat([f64["state"][:, 1:], f64["x"].detach()[:, None]], 1)}
        L = case["seqlen"]
        head = leaf.get("state0")
        y = act(_exact_conv_pre(leaf["x"], w, b, head if head is not None else leaf["x"].new_zeros(case["batch"], K - 1, case["dim"])))
        if s["valid"] is not None:
            y = y * (torch.arange(L, device="cuda") < s["valid"][:, None])[:, :, None]
        out = {"y": y.detach()}
        if not train:
            if case["carry"]:
                xp = torch.cat([f64["state0"], f64["x"]], 1).detach()
                end = [L] * case["batch"] if s["valid"] is None else s["valid"].tolist()
                out["final"] = torch.stack([xp[i, n:n + K - 1] for i, n in enumerate(end)])
            return out
        names = {"x": "dx", "state0": "dstate0", "w": "dw", "b": "db"}
        dy = f64["dy"]
    elif case["op"] == "norm":
        r = leaf["x"]
        out = {}
        if "residual" in leaf:
            r = leaf["x"] + leaf["residual"]
            out["r"] = r.detach()
            r = r + (out["r"].to(s["residual"].dtype).double() - out["r"])  # the stream as stored
        if case["rms"]:
            y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * leaf["w"]
        else:
            y = F.layer_norm(r, (case["dim"],), leaf["w"], None, EPS)
        y = y + leaf["b"] if "b" in leaf else y
        out["y"] = y.detach()
        if not train:
            return out
        names = {"x": "dx", "residual": "dresidual", "w": "dw", "b": "db"}
        dy = f64["dy"]
        if "residual" in leaf:
            y, dy = torch.stack([y, r]), torch.stack([dy, f64["dr"]])
    else:
        logits = leaf["h"] @ leaf["w"].T
        y = F.cross_entropy(logits, s["targets"], ignore_index=IGNORE, reduction="none")
        out = {"loss": y.detach(), "lse": torch.logsumexp(logits.detach(), 1) * (s["targets"] != IGNORE)}
        if not train:
            return out
        names = {"h": "dh", "w": "dw"}
        dy = f64["dloss"]
    have = [k for k in names if k in leaf]
    grads = torch.autograd.grad(y, [leaf[k] for k in have], dy)
    out.update({names[k]: v for k, v in zip(have, grads)})
    return out
