"""More operators around the packed ternary layer, as they are timed: the
packed product with bias, activation and residual in its epilogue, a whole
mixture-of-experts layer of packed experts for a few tokens, and the
distillation of a student from a teacher's top logits.

``own`` picks the side: the plain form (elementary torch operations in 32
bits) or the package's calls.  Both take the same state.
"""

import math

import torch

own = False

SUPERBLOCK = 128   # weights per packed record
GRAINS = ("per_group", "per_channel", "per_tensor")
ACTIVATIONS = ("none", "relu", "relu2", "silu", "gelu", "gelu_tanh")


def listed():
    return [
        # one decoded token through the 1B output projection, bias and residual: the latency case
        _linear("linear_decode_1", tokens=1, n=2048, k=2048, activation="none", gated=False, bias="float32", residual=True),
        # a full decode batch through gate and up packed as one weight
        _linear("linear_decode_16_gate_up", tokens=16, n=16384, k=2048, activation="silu", gated=True, bias="none",
                residual=False),
        # an odd batch and width on the long K, per-channel scales
        _linear("linear_decode_5_odd", tokens=5, n=1001, k=8192, activation="gelu", gated=False, bias="bfloat16",
                residual=True, grain="per_channel"),
        # a ragged prompt batch through the output projection
        _linear("linear_prefill_517", tokens=517, n=2048, k=2048, activation="relu2", gated=False, bias="float32",
                residual=True),
        # a long prompt batch through gate and up
        _linear("linear_prefill_2048_gate_up", tokens=2048, n=16384, k=2048, activation="silu", gated=True, bias="none",
                residual=False),
        # one token, two of eight wide experts
        _moe("moe_decode_1", tokens=1, experts=8, top_k=2, shared=0, dim=2048, hidden=8192, residual=True),
        # a few tokens of small experts, sigmoid scores and a selection bias, a shared expert
        _moe("moe_decode_3_sigmoid", tokens=3, experts=30, top_k=4, shared=1, dim=512, hidden=384, scoring="sigmoid",
             bias=True, grain="per_channel", residual=False),
        # a full decode batch of many narrow experts: nearly all of them are used
        _moe("moe_decode_16_of_64", tokens=16, experts=64, top_k=8, shared=0, dim=2048, hidden=1024, residual=False),
        # one held-out row: the loss by itself
        _distill("distill_eval_1", rows=1, vocab=128000, slots=32, dtype="bfloat16", tail=True, labels=False, train=False),
        # a small training batch
        _distill("distill_train_64", rows=64, vocab=32000, slots=16, dtype="bfloat16", tail=False, labels=True),
        # odd rows of a padded vocabulary in float32, ragged teachers
        _distill("distill_train_333_odd", rows=333, vocab=50001, slots=20, dtype="float32", tail=True, labels=True,
                 ragged=True, padded=True),
        # a training batch of a large vocabulary
        _distill("distill_train_2048", rows=2048, vocab=128000, slots=64, dtype="bfloat16", tail=True, labels=False),
    ]


def _linear(name, grain="per_group", **sizes):
    return {"name": name, "op": "linear", "grain": grain, **sizes}


def _moe(name, scoring="softmax", bias=False, grain="per_group", activation="silu", **sizes):
    return {"name": name, "op": "moe", "scoring": scoring, "bias": bias, "grain": grain, "activation": activation, **sizes}


def _distill(name, train=True, ragged=False, padded=False, temperature=2.0, **sizes):
    return {"name": name, "op": "distill", "train": train, "ragged": ragged, "padded": padded,
            "temperature": temperature, **sizes}


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["linear_decode", "linear_prefill", "moe", "moe", "distill", "distill"])
    if op.startswith("linear"):
        decode = op.endswith("decode")
        gated = rng.random() < 0.5
        n = _log_int(rng, 100, 16384 if decode else 8192)
        return {"op": "linear", "tokens": rng.randint(1, 16) if decode else _log_int(rng, 17, 2048),
                "n": n + n % 2 if gated else n, "k": SUPERBLOCK * _log_int(rng, 2, 64 if decode else 32),
                "activation": rng.choice(ACTIVATIONS[1:] if gated else ACTIVATIONS), "gated": gated,
                "bias": rng.choice(["none", "float32", "bfloat16"]), "residual": rng.random() < 0.5,
                "grain": rng.choice(["per_group", "per_group", "per_channel", "per_tensor"])}
    if op == "moe":
        experts = _log_int(rng, 4, 128)
        dim = SUPERBLOCK * _log_int(rng, 2, 32)
        hidden = SUPERBLOCK * _log_int(rng, 1, max(1, min(64, (1 << 27) // (experts * dim * SUPERBLOCK))))
        return {"op": "moe", "tokens": rng.randint(1, 16), "experts": experts, "top_k": rng.randint(1, min(8, experts)),
                "shared": rng.randint(0, 1), "dim": dim, "hidden": hidden,
                "scoring": rng.choice(["softmax", "softmax", "sigmoid"]), "bias": rng.random() < 0.3,
                "grain": rng.choice(["per_group", "per_group", "per_channel", "per_tensor"]),
                "activation": rng.choice(ACTIVATIONS[1:]), "residual": rng.random() < 0.5}
    vocab = _log_int(rng, 1000, 131072)
    return {"op": "distill", "rows": _log_int(rng, 1, min(8192, (1 << 27) // vocab)), "vocab": vocab,
            "slots": _log_int(rng, 1, 128), "dtype": rng.choice(["bfloat16", "bfloat16", "float32"]),
            "tail": rng.random() < 0.5, "labels": rng.random() < 0.5, "train": rng.random() < 0.8,
            "ragged": rng.random() < 0.3, "padded": rng.random() < 0.3, "temperature": rng.choice([1.0, 2.0, 3.5])}


def _scales(n, k, grain):
    return {"per_group": n * k // SUPERBLOCK, "per_channel": n, "per_tensor": 1}[grain]


def work(case):
    if case["op"] == "linear":
        m, n, k = case["tokens"], case["n"], case["k"]
        out = n // 2 if case["gated"] else n
        bias = {"none": 0, "float32": 4, "bfloat16": 2}[case["bias"]] * n
        return {"bytes": n * k * 5 // 32 + 4 * _scales(n, k, case["grain"]) + 2 * m * k + bias
                + 2 * m * out * (2 if case["residual"] else 1), "flops": 2 * m * n * k}
    if case["op"] == "moe":
        m, e, t, d, f = (case[x] for x in ("tokens", "experts", "top_k", "dim", "hidden"))
        used = e * (1 - (1 - t / e) ** m) + case["shared"]      # experts that m tokens meet
        expert = 3 * d * f * 5 // 32 + 4 * (_scales(2 * f, d, case["grain"]) + _scales(d, f, case["grain"]))
        return {"bytes": int(used * expert) + 2 * e * d + (6 if case["residual"] else 4) * m * d,
                "flops": 2 * m * (e * d + (t + case["shared"]) * 3 * d * f)}
    item = 2 if case["dtype"] == "bfloat16" else 4
    size = case["rows"] * case["vocab"]
    passes = 2 if case["train"] else 1                          # the logits in, and their gradient out
    return {"bytes": passes * size * item + 8 * case["rows"] * case["slots"], "flops": (12 if case["train"] else 6) * size}


# --------------------------------------------------------------------- inputs

def _rand(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _table():
    """The four weights of each 5-bit code."""
    table = torch.zeros(32, 4)
    for c in range(32):
        zero, first = (c >> 2) & 3, -1.0 if c >> 4 else 1.0
        signs = iter((first, first * (1 - 2 * (c & 1)), first * (1 - 2 * ((c >> 1) & 1))))
        for p in range(4):
            if p != zero:
                table[c, p] = next(signs)
    return table.cuda()


def _ternary(gen, n, k, grain, table):
    """A packed weight and what it stands for: 5-bit codes of random blocks in
    the record layout of the library (a nibble plane and a sign plane, 128
    weights a record), float32 scales, and the dense T * alpha."""
    sbs = k // SUPERBLOCK
    code = torch.randint(0, 32, (n, sbs, 32), generator=gen, device="cuda")
    by_record = code.permute(1, 0, 2)
    nib = (by_record & 15).reshape(sbs, n, 4, 4, 2).permute(0, 1, 3, 2, 4)     # block 8b + 2d + h -> dword d, byte b
    nib = (nib[..., 0] | nib[..., 1] << 4).to(torch.uint8).reshape(-1)
    sign = (by_record >> 4).reshape(sbs, n, 4, 8) << torch.arange(8, device="cuda")
    sign = sign.sum(-1).to(torch.uint8).reshape(-1)
    shape = {"per_group": (sbs, n), "per_channel": (1, n), "per_tensor": (1, 1)}[grain]
    alpha = 0.02 * (1 + 0.1 * torch.rand(*shape, generator=gen, device="cuda"))
    dense = (table[code].reshape(n, -1, k // shape[0]) * alpha.t().reshape(-1, shape[0], 1)).reshape(n, k)
    return torch.cat([nib, sign]), alpha.reshape(-1).contiguous(), dense


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    bf = torch.bfloat16
    if case["op"] == "linear":
        m, n, k = case["tokens"], case["n"], case["k"]
        out = n // 2 if case["gated"] else n
        s["packed"], s["alpha"], s["dense"] = _ternary(gen, n, k, case["grain"], _table())
        s["x"] = _rand(gen, m, k, dtype=bf)
        s["bias"] = None if case["bias"] == "none" else _rand(gen, n, std=0.5, dtype=getattr(torch, case["bias"]))
        s["residual"] = _rand(gen, m, out, std=2.0, dtype=bf) if case["residual"] else None
        s["res_scale"] = 0.8 if case["residual"] else 1.0
    elif case["op"] == "moe":
        e, d, f, total = case["experts"], case["dim"], case["hidden"], case["experts"] + case["shared"]
        table = _table()
        for name, n, k in (("up", 2 * f, d), ("down", d, f)):
            parts = [_ternary(gen, n, k, case["grain"], table) for _ in range(total)]
            s[name] = tuple(torch.stack(p) for p in zip(*parts))      # planes, scales, dense of every expert
            del parts
        s["x"] = _rand(gen, case["tokens"], d, dtype=bf)
        s["residual"] = _rand(gen, case["tokens"], d, std=2.0, dtype=bf) if case["residual"] else None
        s["router"] = _rand(gen, e, d, std=1.5 * d ** -0.5, dtype=bf)
        s["select"] = _rand(gen, e, std=0.05) if case["bias"] else None
        s["scale"] = 1.5 if case["scoring"] == "sigmoid" else 1.0
    else:
        t, v, j, dt = case["rows"], case["vocab"], case["slots"], getattr(torch, case["dtype"])
        stride = (v + 127) // 64 * 64 if case["padded"] else v        # rows of a padded vocabulary
        store = _rand(gen, t, stride, std=2.5, dtype=dt)
        s["logits"] = store[:, :v]
        teacher = torch.randn(t, v, generator=gen, device="cuda").mul_(1.5).add_(s["logits"], alpha=0.9)
        s["teacher"], ids = teacher.topk(j, dim=1)
        tau = case["temperature"]
        s["teacher_lse"] = torch.logsumexp(teacher.div_(tau), 1) if case["tail"] else None
        del teacher
        s["teacher"] = s["teacher"].to(dt)
        if case["tail"] and dt == bf:      # the rounded logits' mass stays below one
            s["teacher_lse"] = s["teacher_lse"] + 0.02
        if case["ragged"]:                 # slots past a row's own count are empty
            count = torch.randint(1, j + 1, (t, 1), generator=gen, device="cuda")
            ids = torch.where(torch.arange(j, device="cuda") < count, ids, -1)
        s["ids"] = ids.to(torch.int32).contiguous()
        s["labels"] = None
        if case["labels"]:                 # mostly what the teacher says, some others, some rows without
            other = torch.randint(0, v, (t,), generator=gen, device="cuda")
            kind = torch.rand(t, generator=gen, device="cuda")
            label = torch.where(kind < 0.6, ids[:, 0], other)
            s["labels"] = torch.where(kind > 0.9, -100, label)
        s["kd_weight"] = 0.7 if case["labels"] else 1.0
        if case["train"]:
            s["logits"].requires_grad_(True)
            # the mean over the rows, some of them left out
            s["g"] = (torch.rand(t, generator=gen, device="cuda") < 0.95).float() / t
    return s


# ----------------------------------------------------------------- the passes

def run(state):
    if own:
        return _own(state)
    with torch.no_grad():
        return {"linear": _plain_linear, "moe": _plain_moe, "distill": _plain_distill}[state["op"]](state)


def _own(s):
    import ternary_weight_quantization_sparse_amd as S
    if s["op"] == "linear":
        pw = S.PackedWeight(s["packed"], s["alpha"], s["n"], s["k"], s["grain"], SUPERBLOCK)
        f = S.linear_gemv if s["tokens"] <= 16 else S.linear_gemm
        return f(pw, s["x"], bias=s["bias"], activation=s["activation"], gated=s["gated"], residual=s["residual"],
                 res_scale=s["res_scale"])
    if s["op"] == "moe":
        f, d, total = s["hidden"], s["dim"], s["experts"] + s["shared"]
        up = S.PackedExperts(s["up"][0], s["up"][1], total, 2 * f, d, s["grain"], SUPERBLOCK)
        down = S.PackedExperts(s["down"][0], s["down"][1], total, d, f, s["grain"], SUPERBLOCK)
        return S.moe_decode(s["x"], s["router"], up, down, s["top_k"], shared=s["shared"], scoring=s["scoring"],
                            bias=s["select"], scale=s["scale"], activation=s["activation"], residual=s["residual"])
    args = (s["logits"], s["teacher"], s["ids"])
    kw = dict(temperature=s["temperature"], teacher_lse=s["teacher_lse"], labels=s["labels"], kd_weight=s["kd_weight"])
    if not s["train"]:
        return S.distill_loss(*args, **kw)
    loss = S.distill_loss_ad(*args, **kw)
    (grad,) = torch.autograd.grad(loss, s["logits"], s["g"])
    return loss.detach(), grad


def _act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "relu2":
        return z.clamp(min=0) ** 2
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def _plain_linear(s):
    z = s["x"].float() @ s["dense"].t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    if s["gated"]:
        gate, up = z.split(z.shape[1] // 2, 1)
        z = _act(gate, s["activation"]) * up
    else:
        z = _act(z, s["activation"])
    if s["residual"] is not None:
        z = z + s["res_scale"] * s["residual"].float()
    return z.to(torch.bfloat16)


def _plain_moe(s):
    x, e, m = s["x"].float(), s["experts"], s["tokens"]
    up, down = s["up"][2], s["down"][2]
    logits = x @ s["router"].float().t()
    if s["scoring"] == "softmax":
        score = torch.exp(logits - logits.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-logits))
    key = logits if s["select"] is None else score + s["select"]
    ids = key.argsort(dim=1, descending=True, stable=True)[:, :s["top_k"]]
    w = score.gather(1, ids)
    w = w / w.sum(1, keepdim=True) * s["scale"]
    if s["shared"]:
        extra = torch.arange(e, e + s["shared"], device=x.device).expand(m, -1)
        ids, w = torch.cat([ids, extra], 1), torch.cat([w, torch.ones_like(extra, dtype=w.dtype)], 1)
    if ids.numel() <= up.shape[0]:       # each token's own experts
        z = (up[ids] @ x[:, None, :, None])[..., 0]
        gate, val = z.split(s["hidden"], -1)
        h = _act(gate, s["activation"]) * val * w[..., None]
        y = (down[ids] @ h[..., None])[..., 0].sum(1)
    else:                                # every expert, those of a token kept
        z = (x @ up.reshape(-1, s["dim"]).t()).reshape(m, up.shape[0], -1)
        gate, val = z.split(s["hidden"], -1)
        full = torch.zeros(m, up.shape[0], device=x.device).scatter_(1, ids, w)
        h = _act(gate, s["activation"]) * val * full[..., None]
        y = h.reshape(m, -1) @ down.transpose(1, 2).reshape(-1, s["dim"])
    return (y if s["residual"] is None else y + s["residual"].float()).to(torch.bfloat16)


def _plain_distill(s):
    z, tau, a = s["logits"].float(), s["temperature"], s["kd_weight"]
    t, v = z.shape
    used = s["ids"] >= 0
    at = s["ids"].clamp(min=0).long()
    u = torch.where(used, s["teacher"].double() / tau, -math.inf)     # 64 bits: the tail is what they leave of 1
    if s["tail"]:
        p = torch.exp(u - s["teacher_lse"].double()[:, None])
        rest = (1 - p.sum(1)).clamp(min=0)
    else:
        p = torch.exp(u - u.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        rest = None
    zs = z / tau
    top = zs.amax(1, keepdim=True)
    ex = torch.exp(zs - top)
    total = ex.sum(1, dtype=torch.float64)     # of a row, sums and logarithms in 64 bits: their differences are the loss
    logq = (zs.gather(1, at) - top).double() - torch.log(total)[:, None]
    kd = torch.where(p > 0, p * (torch.log(p) - logq), 0).sum(1)
    mass = p.sum(1)
    if rest is not None:
        outside = torch.ones(t, v, dtype=torch.bool, device=z.device)
        outside[used.nonzero()[:, 0], at[used]] = False
        left = torch.where(outside, ex, 0).sum(1, dtype=torch.float64)
        kd = kd + torch.where(rest > 0, rest * torch.log(rest * total / left), 0)
        mass = mass + rest
    loss = a * tau * tau * kd
    if s["labels"] is not None:
        has = s["labels"] >= 0
        lab = s["labels"].clamp(min=0)[:, None]
        top1 = z.amax(1, keepdim=True)
        ex1 = torch.exp(z - top1)
        tot1 = ex1.sum(1, dtype=torch.float64)
        ce = torch.log(tot1) - (z.gather(1, lab) - top1)[:, 0]
        loss = loss + torch.where(has, (1 - a) * ce, 0)
    loss = loss.float()
    if not s["train"]:
        return loss
    grad = ex * (mass / total).float()[:, None]
    if rest is not None:
        grad = grad - torch.where(outside, ex * (rest / left).float()[:, None], 0)
    grad = grad.scatter_add(1, at, -p.float()) * (a * tau)
    if s["labels"] is not None:
        soft = ex1 / tot1.float()[:, None]
        soft = soft.scatter_add(1, lab, -torch.ones_like(lab, dtype=soft.dtype))
        grad = grad + torch.where(has[:, None], (1 - a) * soft, 0)
    return loss, (grad * s["g"][:, None]).to(s["logits"].dtype)


# ------------------------------------------------------------ the definitions

def exact(case, seed):
    """The operators by their definitions in 64 bits, on the inputs of this seed."""
    s = prepare(case, seed)
    return {"linear": _exact_linear, "moe": _exact_moe, "distill": _exact_distill}[case["op"]](s)


def _exact_act(z, name):
    f = torch.nn.functional
    return {"none": lambda: z, "relu": lambda: f.relu(z), "relu2": lambda: f.relu(z).square(), "silu": lambda: f.silu(z),
            "gelu": lambda: f.gelu(z), "gelu_tanh": lambda: f.gelu(z, approximate="tanh")}[name]()


def _exact_linear(s):
    z = s["x"].double().matmul(s["dense"].double().t())
    z = z if s["bias"] is None else z + s["bias"].double()
    if s["gated"]:
        half = z.shape[1] // 2
        z = _exact_act(z[:, :half], s["activation"]) * z[:, half:]
    else:
        z = _exact_act(z, s["activation"])
    return z if s["residual"] is None else z + s["res_scale"] * s["residual"].double()


def _exact_moe(s):
    x, f = s["x"].double(), s["hidden"]
    y = torch.zeros_like(x) if s["residual"] is None else s["residual"].double()
    logits = x.matmul(s["router"].double().t())
    score = logits.softmax(1) if s["scoring"] == "softmax" else logits.sigmoid()
    key = score if s["select"] is None else score + s["select"].double()
    for t in range(s["tokens"]):
        best = sorted(range(s["experts"]), key=lambda i, row=key[t].tolist(): (-row[i], i))[:s["top_k"]]
        w = score[t, best]
        w = (w / w.sum() * s["scale"]).tolist()
        best, w = best + [s["experts"] + i for i in range(s["shared"])], w + [1.0] * s["shared"]
        for c, weight in zip(best, w):
            z = s["up"][2][c].double().mv(x[t])
            h = _exact_act(z[:f], s["activation"]) * z[f:]
            y[t] += weight * s["down"][2][c].double().mv(h)
    return y


def _exact_distill(s):
    tau, a = s["temperature"], s["kd_weight"]
    losses, grads = [], []
    rows = max(1, (1 << 26) // s["vocab"])       # a slab of rows at a time
    for r0 in range(0, s["rows"], rows):
        z = s["logits"].detach()[r0:r0 + rows].double().requires_grad_(s["train"])
        ids, u = s["ids"][r0:r0 + rows].long(), s["teacher"][r0:r0 + rows].double() / tau
        used = ids >= 0
        u = u.masked_fill(~used, -math.inf)
        with torch.enable_grad():
            logq = (z / tau).log_softmax(1)
            if s["tail"]:
                logp = u - s["teacher_lse"][r0:r0 + rows].double()[:, None]
            else:
                logp = u.log_softmax(1)
            p = logp.exp()
            cross = torch.nn.functional.kl_div(logq.gather(1, ids.clamp(min=0)), p, reduction="none").sum(1)
            if s["tail"]:
                rest = (1 - p.sum(1)).clamp(min=0)
                mask = torch.zeros_like(z, dtype=torch.bool)
                row = torch.arange(len(ids), device=z.device)[:, None].expand_as(ids)
                mask[row[used], ids[used]] = True
                cross = cross + torch.nn.functional.kl_div(logq.masked_fill(mask, -math.inf).logsumexp(1), rest,
                                                           reduction="none")
            loss = a * tau ** 2 * cross
            if s["labels"] is not None:
                loss = loss + (1 - a) * torch.nn.functional.cross_entropy(z, s["labels"][r0:r0 + rows], ignore_index=-100,
                                                                          reduction="none")
            losses.append(loss.detach())
            if s["train"]:
                grads.append(torch.autograd.grad(loss, z, s["g"][r0:r0 + rows].double())[0])
    return (torch.cat(losses), torch.cat(grads)) if s["train"] else torch.cat(losses)
