"""The operators at a recurrent language model's ends and middle, as measured cases.

Three operators beside the selective scan and what is around it: the gated
linear recurrence ("recur"), the embedding lookup with the gradient of its
weight ("embed") and the distillation from a teacher's top logits over the
vocabulary ("distill").  Each case is one pass of one of them: a forward, a
training pass (forward and backward) or a step of single tokens.
"""
import torch

own = False

BF16, F32 = "bf16", "f32"
TYPES = {BF16: torch.bfloat16, F32: torch.float32}
IGNORE = -100


def recur(kind, dtype, batch, seqlen, dim, floor=False, masked=False, carry=False, packed=False):
    """floor: decays have a lower bound per channel; masked: rows have valid lengths U{1..seqlen};
    carry: from a given state, returning the last one (in training its gradient arrives too);
    packed: gate and value are the halves of the columns of one projection's output."""
    return {"op": "recur", "kind": kind, "dtype": dtype, "batch": batch, "seqlen": seqlen, "dim": dim, "floor": floor,
            "masked": masked, "carry": carry, "packed": packed}


def embed(kind, dtype, tokens, vocab, dim, out="", scale=1.0, ignored=0.0, add=False):
    """out: the type of the looked up rows, "" for the weight's; ignored: the share of padding
    tokens; add: the gradient is added onto one that is there (a tied output embedding's)."""
    return {"op": "embed", "kind": kind, "dtype": dtype, "tokens": tokens, "vocab": vocab, "dim": dim, "out": out or dtype,
            "scale": scale, "ignored": ignored, "add": add}


def distill(kind, tokens, vocab, dim, top, teacher=BF16, temperature=1.0, ignored=0.0, ragged=False):
    """top: the teacher's entries per token; teacher: the type of its logits; ignored: the share of
    tokens without any (padding, prompts); ragged: tokens have 1 to top entries."""
    return {"op": "distill", "kind": kind, "tokens": tokens, "vocab": vocab, "dim": dim, "top": top, "teacher": teacher,
            "temperature": temperature, "ignored": ignored, "ragged": ragged}


def listed():
    return [
        # one sequence generating, one layer's recurrence: latency
        {"name": "recur-step-b1", **recur("step", BF16, 1, 1, 2048)},
        # the same for a serving batch, gate and value read out of the projection
        {"name": "recur-step-b1024", **recur("step", BF16, 1024, 1, 2048, floor=True, packed=True)},
        # a batch of padded prompts, keeping the state to generate from
        {"name": "recur-prompt-varlen", **recur("fwd", BF16, 32, 2048, 1536, masked=True, carry=True, packed=True)},
        # one long sequence with few channels: time is all there is to split
        {"name": "recur-long-f32", **recur("fwd", F32, 1, 65536, 256)},
        # a training step at the default scan workload's size
        {"name": "recur-train-f32", **recur("train", F32, 8, 4096, 1024)},
        # a training step on long documents, with a floor per channel
        {"name": "recur-train-bf16", **recur("train", BF16, 2, 32768, 2048, floor=True, packed=True)},
        # a serving batch's next tokens: latency
        {"name": "embed-fwd-b64", **embed("fwd", BF16, 64, 32768, 2048)},
        # a fine-tuning batch with padding, an odd width and vocabulary, fp32 weights
        {"name": "embed-train-odd", **embed("train", F32, 5001, 32001, 1537, scale=39.2, ignored=0.3)},
        # a pre-training batch with a tied embedding: onto the output embedding's gradient
        {"name": "embed-train-tied", **embed("train", BF16, 65536, 65536, 2048, add=True)},
        # measuring a student against a teacher's stored logits
        {"name": "distill-score", **distill("fwd", 4096, 50257, 1536, 64)},
        # a small fine-tuning batch, half of it prompt or padding, lists of uneven length
        {"name": "distill-train-ragged", **distill("train", 1000, 32001, 768, 16, teacher=F32, temperature=2.0, ignored=0.5, ragged=True)},
        # a large distillation batch
        {"name": "distill-train-large", **distill("train", 8192, 65536, 2048, 32)},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["recur-step", "recur-fwd", "recur-train", "embed-fwd", "embed-train", "distill-fwd", "distill-train"])
    dtype = rng.choice([BF16, BF16, F32])
    if op.startswith("recur"):
        dim = rng.choice([64, 200, 256, 513, 768, 1000, 1024, 1536, 2048, 2560, 4096])
        more = {"floor": rng.random() < 0.4, "packed": rng.random() < 0.5}
        if op == "recur-step":
            return recur("step", dtype, _log(rng, 1, 1024), 1, dim, **more)
        batch = _log(rng, 1, 32)
        seqlen = _log(rng, 1, max(2, min(65536, 130_000_000 // (batch * dim))))
        return recur(op[6:], dtype, batch, seqlen, dim, masked=rng.random() < 0.5, carry=rng.random() < 0.5, **more)
    vocab = _log(rng, 1000, 65536)
    if op.startswith("embed"):
        dim = rng.choice([64, 200, 513, 768, 1000, 1024, 1537, 2048, 2560, 4096])
        tokens = _log(rng, 1, min(65536, 130_000_000 // dim))
        return embed(op[6:], dtype, tokens, vocab, dim, out=rng.choice(["", F32]), scale=rng.choice([1.0, dim ** 0.5]),
                     ignored=rng.choice([0.0, 0.3]), add=op == "embed-train" and rng.random() < 0.5)
    dim = rng.choice([64, 200, 512, 768, 1000, 1024, 1536, 2048])
    return distill(op[8:], _log(rng, 1, 8192), vocab, dim, _log(rng, 1, 256), teacher=dtype,
                   temperature=rng.choice([1.0, 1.0, 0.7, 2.0, 4.0]), ignored=rng.choice([0.0, 0.1, 0.5]), ragged=rng.random() < 0.5)


# ---- inputs ----------------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    f32 = torch.float32

    def randn(*shape, dtype=f32, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"case": case}
    if case["op"] == "recur":
        dt, B, L, D = TYPES[case["dtype"]], case["batch"], case["seqlen"], case["dim"]
        shape = (B, D) if case["kind"] == "step" else (B, L, D)
        # gates as after training: most channels remember for some tens of steps, some for thousands
        bias = torch.rand(D, generator=g, device="cuda") * 7 - 1
        if case["packed"]:
            both = torch.cat([randn(*shape) + bias, randn(*shape)], -1).to(dt)
            s["gate"], s["value"] = both[..., :D], both[..., D:]
        else:
            s["gate"], s["value"] = (randn(*shape) + bias).to(dt), randn(*shape, dtype=dt)
        s["floor"] = torch.rand(D, generator=g, device="cuda") * 0.9 if case["floor"] else None
        if case["kind"] == "step":
            s["state"] = randn(B, D)
            return s
        s["valid"] = torch.randint(1, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if case["masked"] else None
        s["state0"] = randn(B, D) if case["carry"] else None
        if case["kind"] == "train":
            s["dy"] = randn(B, L, D, dtype=dt)
            s["dfinal"] = randn(B, D) if case["carry"] else None
    elif case["op"] == "embed":
        dt, T, V, D = TYPES[case["dtype"]], case["tokens"], case["vocab"], case["dim"]
        s["w"] = randn(V, D, dtype=dt, scale=0.02)
        # a token's frequency falls with its rank: a few make up much of a text
        rank = torch.exp(torch.rand(T, generator=g, device="cuda", dtype=torch.float64) * torch.log(torch.tensor(V + 1.0, dtype=torch.float64)))
        s["ids"] = (rank.long() - 1).clamp_(0, V - 1)
        if case["ignored"]:
            out = torch.rand(T, generator=g, device="cuda") < case["ignored"]
            s["ids"] = torch.where(out, torch.full_like(s["ids"], IGNORE), s["ids"])
        if case["kind"] == "train":
            s["dy"] = randn(T, D, dtype=TYPES[case["out"]])
            s["dw"] = randn(V, D, dtype=dt) if case["add"] else None
    else:
        T, V, D, K = case["tokens"], case["vocab"], case["dim"], case["top"]
        bf16 = torch.bfloat16
        s["h"] = randn(T, D, dtype=bf16)
        s["w"] = randn(V, D, dtype=bf16, scale=2 / D ** 0.5)
        # the teacher's logits are the student's but for a third of noise in what they come from
        z = (s["h"].float() + randn(T, D, scale=0.5)).to(bf16) @ s["w"].T
        top, ids = z.topk(K, dim=-1)
        s["logits"], s["ids"] = top.to(TYPES[case["teacher"]]), ids
        if case["ragged"]:
            count = torch.randint(1, K + 1, (T, 1), generator=g, device="cuda")
            s["ids"] = torch.where(torch.arange(K, device="cuda") < count, s["ids"], IGNORE)
        if case["ignored"]:
            out = torch.rand(T, 1, generator=g, device="cuda") < case["ignored"]
            s["ids"] = torch.where(out, IGNORE, s["ids"])
        if case["kind"] == "train":
            s["dloss"] = torch.full((T,), 1.0 / T, device="cuda")
    return s


# ---- one pass ----------------------------------------------------------------------------------


def run(s):
    c = s["case"]
    return (_own if own else _plain)[c["op"], c["kind"]](s, c)


def _plain_recur_gates(s, valid=None):
    """1 - a, a's derivative in the gate and the gate's complement, 0 past the valid steps."""
    gate = s["gate"].float()
    open_ = 1 / (1 + torch.exp(gate))     # sigmoid(-gate)
    hold = 1 / (1 + torch.exp(-gate))
    b = open_ if s["floor"] is None else (1 - s["floor"]) * open_
    if valid is not None:
        b = torch.where(valid, b, 0.0)
    return b, b * hold, open_


def _plain_recur_step(s, c):
    b, _, _ = _plain_recur_gates(s)
    h = s["state"]
    h.copy_(h + b * (s["value"].float() - h))
    return {"y": h.to(s["value"].dtype), "state": h}


def _plain_scan(a, u):
    """x_t = a_t x_{t-1} + u_t along axis 1, by doubling; both arguments are overwritten."""
    step = 1
    while step < u.shape[1]:
        u[:, step:] += a[:, step:] * u[:, :-step]
        a[:, step:] = a[:, step:] * a[:, :-step]
        step *= 2
    return u


def _plain_recur(s, c):
    valid = None
    if s["valid"] is not None:
        valid = (torch.arange(c["seqlen"], device="cuda") < s["valid"][:, None])[:, :, None]
    b, slope, open_ = _plain_recur_gates(s, valid)
    v = s["value"].float()
    if valid is not None:
        v = torch.where(valid, v, 0.0)
    u = b * v
    if s["state0"] is not None:
        u[:, 0] += (1 - b[:, 0]) * s["state0"]
    h = _plain_scan(1 - b, u)
    out = {"y": (h if valid is None else torch.where(valid, h, 0.0)).to(s["value"].dtype)}
    if c["carry"]:
        out["final"] = h[:, -1].clone()
    return out, valid, b, slope, open_, v, h


def _plain_recur_fwd(s, c):
    return _plain_recur(s, c)[0]


def _plain_recur_train(s, c):
    out, valid, b, slope, open_, v, h = _plain_recur(s, c)
    dt = s["value"].dtype
    lam = s["dy"].float()
    lam = lam.clone() if valid is None else torch.where(valid, lam, 0.0)
    if s["dfinal"] is not None:
        lam[:, -1] += s["dfinal"]
    a = torch.ones_like(b)
    a[:, 1:] = 1 - b.flip(1)[:, :-1]
    lam = _plain_scan(a, lam.flip(1)).flip(1)
    head = s["state0"][:, None] if s["state0"] is not None else torch.zeros_like(h[:, :1])
    apart = torch.cat([head, h[:, :-1]], 1) - v
    out["dvalue"] = (lam * b).to(dt)
    out["dgate"] = (lam * apart * slope).to(dt)
    if s["floor"] is not None:
        d = lam * apart * open_
        out["dfloor"] = (d if valid is None else torch.where(valid, d, 0.0)).sum((0, 1), dtype=torch.float64).float()
    if s["state0"] is not None:
        out["dstate0"] = (1 - b[:, 0]) * lam[:, 0]
    return out


def _own_recur_step(s, c):
    import selective_state_space_fwd_gb300 as S
    return {"y": S.recur_step(s["gate"], s["value"], s["floor"], state=s["state"]), "state": s["state"]}


def _own_recur_fwd(s, c):
    import selective_state_space_fwd_gb300 as S
    y, final, _ = S.recur_fwd(s["gate"], s["value"], s["floor"], s["valid"], state0=s["state0"], want_final=c["carry"])
    return {"y": y, "final": final} if c["carry"] else {"y": y}


def _own_recur_train(s, c):
    import selective_state_space_fwd_gb300 as S
    y, final, states = S.recur_fwd(s["gate"], s["value"], s["floor"], s["valid"], state0=s["state0"], want_final=c["carry"],
                                   want_states=True)
    g = S.recur_bwd(s["gate"], s["value"], s["floor"], s["valid"], states=states, dy=s["dy"], dfinal=s["dfinal"],
                    want_dstate0=s["state0"] is not None)
    out = {"y": y, "dvalue": g["dvalue"], "dgate": g["dgate"]}
    if c["carry"]:
        out["final"], out["dstate0"] = final, g["dstate0"]
    if s["floor"] is not None:
        out["dfloor"] = g["dfloor"]
    return out


def _plain_embed_fwd(s, c):
    kept = s["ids"] != IGNORE
    rows = s["w"][torch.where(kept, s["ids"], 0)].float() * c["scale"]
    return {"y": torch.where(kept[:, None], rows, 0.0).to(TYPES[c["out"]])}


def _plain_embed_train(s, c):
    out = _plain_embed_fwd(s, c)
    kept = s["ids"] != IGNORE
    total = torch.zeros(s["w"].shape, device="cuda")
    total.index_add_(0, torch.where(kept, s["ids"], 0), torch.where(kept[:, None], s["dy"].float(), 0.0))
    total *= c["scale"]
    if s["dw"] is None:
        out["dw"] = total.to(s["w"].dtype)
    else:
        out["dw"] = s["dw"].copy_(total + s["dw"].float())
    return out


def _own_embed_fwd(s, c):
    import selective_state_space_fwd_gb300 as S
    return {"y": S.embed_fwd(s["ids"], s["w"], scale=c["scale"], dtype=TYPES[c["out"]], ignore_index=IGNORE)}


def _own_embed_train(s, c):
    import selective_state_space_fwd_gb300 as S
    y = S.embed_fwd(s["ids"], s["w"], scale=c["scale"], dtype=TYPES[c["out"]], ignore_index=IGNORE)
    if s["dw"] is None:
        dw = S.embed_bwd(s["ids"], s["dy"], vocab=c["vocab"], scale=c["scale"], dtype=s["w"].dtype, ignore_index=IGNORE)
    else:
        dw = S.embed_bwd(s["ids"], s["dy"], scale=c["scale"], add_to=s["dw"], ignore_index=IGNORE)
    return {"y": y, "dw": dw}


def _plain_distill(s, c):
    tau = c["temperature"]
    entry = s["ids"] != IGNORE
    kept = entry.any(-1)
    at = torch.where(entry, s["ids"], 0)
    z = torch.where(entry, s["logits"].float() / tau, -torch.inf)
    z = torch.where(kept[:, None], z, 0.0)
    q = torch.exp(z - z.amax(-1, keepdim=True))
    total = q.sum(-1, keepdim=True)
    logq = z - z.amax(-1, keepdim=True) - torch.log(total)
    q = torch.where(entry, q / total, 0.0)
    h, w = s["h"].float(), s["w"].float()
    student = h @ w.T / tau
    top = student.amax(-1, keepdim=True)
    e = torch.exp(student - top)
    total = e.sum(-1, keepdim=True)
    lse = torch.log(total) + top
    apart = torch.where(entry, logq - (student.gather(1, at) - lse), 0.0)
    out = {"loss": (q * apart).sum(-1), "lse": torch.where(kept, lse[:, 0], 0.0)}
    return out, h, w, kept, at, q, e, total


def _plain_distill_fwd(s, c):
    return _plain_distill(s, c)[0]


def _plain_distill_train(s, c):
    out, h, w, kept, at, q, e, total = _plain_distill(s, c)
    p = e / total
    p.scatter_add_(1, at, -q)
    p = p * (torch.where(kept, s["dloss"], 0.0) / c["temperature"])[:, None]
    return {**out, "dh": (p @ w).to(s["h"].dtype), "dw": (p.T @ h).to(s["w"].dtype)}


def _own_distill_fwd(s, c):
    import selective_state_space_fwd_gb300 as S
    loss, lse = S.distill_fwd(s["h"], s["w"], s["ids"], s["logits"], temperature=c["temperature"], ignore_index=IGNORE)
    return {"loss": loss, "lse": lse}


def _own_distill_train(s, c):
    import selective_state_space_fwd_gb300 as S
    loss, lse = S.distill_fwd(s["h"], s["w"], s["ids"], s["logits"], temperature=c["temperature"], ignore_index=IGNORE)
    g = S.distill_bwd(s["h"], s["w"], s["ids"], s["logits"], lse=lse, dloss=s["dloss"], temperature=c["temperature"],
                      ignore_index=IGNORE)
    return {"loss": loss, "lse": lse, "dh": g["dh"], "dw": g["dweight"]}


_plain = {("recur", "step"): _plain_recur_step, ("recur", "fwd"): _plain_recur_fwd, ("recur", "train"): _plain_recur_train,
          ("embed", "fwd"): _plain_embed_fwd, ("embed", "train"): _plain_embed_train,
          ("distill", "fwd"): _plain_distill_fwd, ("distill", "train"): _plain_distill_train}
_own = {("recur", "step"): _own_recur_step, ("recur", "fwd"): _own_recur_fwd, ("recur", "train"): _own_recur_train,
        ("embed", "fwd"): _own_embed_fwd, ("embed", "train"): _own_embed_train,
        ("distill", "fwd"): _own_distill_fwd, ("distill", "train"): _own_distill_train}


# ---- what a pass cannot do without ---------------------------------------------------------------


def work(case):
    if case["op"] == "recur":
        e = 2 if case["dtype"] == BF16 else 4
        B, L, D = case["batch"], case["seqlen"], case["dim"]
        floor = 4 * D * bool(case["floor"])
        if case["kind"] == "step":
            return {"bytes": 3 * B * D * e + 8 * B * D + floor, "flops": 8 * B * D}
        whole = B * L * D
        valid = whole * (0.5 if case["masked"] else 1.0)  # what is read; outputs are written in full
        carry = 8 * B * D if case["carry"] else 0
        fwd = (2 * valid + whole) * e + floor + carry
        if case["kind"] == "fwd":
            return {"bytes": fwd, "flops": 8 * valid}
        return {"bytes": fwd + (3 * valid + 2 * whole) * e + 2 * floor + carry, "flops": 24 * valid}
    if case["op"] == "embed":
        e, o = (2 if t == BF16 else 4 for t in (case["dtype"], case["out"]))
        T, V, D = case["tokens"], case["vocab"], case["dim"]
        kept = T * (1 - case["ignored"])
        # tokens by rank: a row of rank r is missing with (1 - 1 / (r ln V))^kept, so about this many are met
        span = 1 + torch.log(torch.tensor(float(V))).item()
        met = sum(1 - (1 - min(1.0, 1 / (r * span))) ** kept for r in range(1, V + 1))
        fwd = met * D * e + T * D * o + 8 * T
        if case["kind"] == "fwd":
            return {"bytes": fwd, "flops": T * D}
        grad = 2 * met if case["add"] else V
        return {"bytes": fwd + kept * D * o + grad * D * e + 8 * T, "flops": T * D + kept * D + met * D}
    T, V, D, K = case["tokens"] * (1 - case["ignored"]), case["vocab"], case["dim"], case["top"]
    teacher = case["tokens"] * K * (8 + (2 if case["teacher"] == BF16 else 4))
    if case["kind"] == "fwd":
        return {"bytes": 2 * (T + V) * D + teacher + 8 * case["tokens"], "flops": 2 * T * V * D + 4 * T * V}
    return {"bytes": 4 * (T + V) * D + teacher + 16 * case["tokens"], "flops": 8 * T * V * D + 10 * T * V}


# ---- the definitions in 64 bits ---------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    f64 = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    return {"recur": _exact_recur, "embed": _exact_embed, "distill": _exact_distill}[case["op"]](case, s, f64)


def _exact_recur(case, s, f64):
    keep = 1 - f64["floor"] if s["floor"] is not None else torch.ones(case["dim"], dtype=torch.float64, device="cuda")
    gate, value = f64["gate"], f64["value"]
    if case["kind"] == "step":
        a = 1 - keep * torch.sigmoid(-gate)
        h = a * f64["state"] + (1 - a) * value
        return {"y": h, "state": h}
    B, L, D = gate.shape
    lens = [L] * B if s["valid"] is None else s["valid"].tolist()
    # time first, one step after the other; a row that has ended keeps its state
    live = torch.tensor(lens, device="cuda")[None, :, None] > torch.arange(L, device="cuda")[:, None, None]
    new = torch.where(live, keep * torch.sigmoid(-gate.transpose(0, 1)), 0.0)
    old = 1 - new
    value = torch.where(live, value.transpose(0, 1), 0.0)
    states = torch.empty(L + 1, B, D, dtype=torch.float64, device="cuda")
    states[0] = f64["state0"] if "state0" in f64 else 0.0
    part = new * value
    for t in range(L):
        torch.addcmul(part[t], old[t], states[t], out=states[t + 1])
    y = torch.where(live, states[1:], 0.0).transpose(0, 1)
    out = {"y": y}
    if case["carry"]:
        out["final"] = states[L]
    if case["kind"] == "fwd":
        return out
    grads = torch.where(live, f64["dy"].transpose(0, 1), 0.0).contiguous()
    if "dfinal" in f64:
        grads[L - 1] += f64["dfinal"]
    for t in range(L - 1, 0, -1):
        grads[t - 1].addcmul_(old[t], grads[t])
    dnew = grads * (value - states[:-1])
    side = torch.sigmoid(-gate.transpose(0, 1))
    out["dvalue"] = (grads * new).transpose(0, 1)
    out["dgate"] = torch.where(live, -dnew * keep * side * (1 - side), 0.0).transpose(0, 1)
    if s["floor"] is not None:
        out["dfloor"] = -torch.where(live, dnew * side, 0.0).sum((0, 1))
    if "state0" in f64:
        out["dstate0"] = grads[0] * old[0]
    return out


def _exact_embed(case, s, f64):
    hit = torch.nonzero(s["ids"] != IGNORE)[:, 0]
    ids = s["ids"][hit]
    y = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
    y[hit] = f64["w"][ids] * case["scale"]
    if case["kind"] == "fwd":
        return {"y": y}
    dw = f64["dw"].clone() if "dw" in f64 else torch.zeros_like(f64["w"])
    dw.index_put_((ids,), f64["dy"][hit] * case["scale"], accumulate=True)
    return {"y": y, "dw": dw}


def _exact_distill(case, s, f64):
    train = case["kind"] == "train"
    entry = s["ids"] != IGNORE
    rows = torch.nonzero(entry.any(1))[:, 0]
    T, tau = case["tokens"], case["temperature"]
    h, w = (f64[k].requires_grad_(train) for k in ("h", "w"))
    logits = h[rows] @ w.T / tau
    logp = torch.log_softmax(logits, 1)
    z = (f64["logits"][rows] / tau).masked_fill(~entry[rows], -torch.inf)
    logq = torch.log_softmax(z, 1)
    terms = logq.exp() * (logq - logp.gather(1, s["ids"][rows].clamp_min(0)))
    value = torch.where(entry[rows], terms, 0.0).sum(1)
    empty = torch.zeros(T, dtype=torch.float64, device="cuda")
    out = {"loss": empty.index_copy(0, rows, value.detach()),
           "lse": empty.index_copy(0, rows, torch.logsumexp(logits.detach(), 1))}
    if train:
        dh, dw = torch.autograd.grad(value, [h, w], f64["dloss"][rows])
        out["dh"], out["dw"] = dh, dw
    return out
