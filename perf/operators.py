"""The operators around the packed ternary layer, as they are timed: adapters
of many requests beside a packed projection, the norms before and after a
block, and the orthogonalised update of latent weights.

``own`` picks the side: the plain form (elementary torch operations in 32
bits) or the package's calls.  Both take the same state.
"""

import math

import torch

own = False

SUPERBLOCK = 128   # weights per packed record


def listed():
    return [
        # one decoded token through the 1B query projection, one adapter: the latency case
        _adapters("adapter_decode_1", tokens=1, n=2048, k=2048, adapters=8, rank=16, grain="per_group"),
        # a full decode batch through gate and up packed as one weight, mixed adapters and requests without one
        _adapters("adapter_decode_16_gate_up", tokens=16, n=16384, k=2048, adapters=32, rank=64, grain="per_group"),
        # an odd batch on the long-K projection, per-channel scales, ragged ranks
        _adapters("adapter_decode_7_down", tokens=7, n=2048, k=8192, adapters=5, rank=24, grain="per_channel"),
        # a ragged prompt batch through the output projection
        _adapters("adapter_prefill_517", tokens=517, n=2048, k=2048, adapters=4, rank=16, grain="per_group"),
        # a long prompt batch through gate and up, the widest adapters
        _adapters("adapter_prefill_2048_gate_up", tokens=2048, n=16384, k=2048, adapters=8, rank=64, grain="per_group"),
        # one decoded token between two blocks
        _norms("norm_decode_1", rows=1, dim=2048, dtype="bfloat16", gate="channel", seqs=1, train=False),
        # a prompt of 2048 tokens between two blocks
        _norms("norm_prefill_2048", rows=2048, dim=2048, dtype="bfloat16", gate="none", seqs=1, train=False),
        # a training batch of eight sequences, a gate for each (conditioned blocks), forward and backward
        _norms("norm_train_8192", rows=8192, dim=2048, dtype="bfloat16", gate="sequence", seqs=8, train=True),
        # odd rows and width in float32, a learned gate per channel, forward and backward
        _norms("norm_train_1531_odd", rows=1531, dim=1001, dtype="float32", gate="channel", seqs=1, train=True),
        # the small single layer's latent weight: launches and latency count
        _muon("muon_256x512", count=1, n=256, k=512, dtype="float32", step=True),
        # the momenta of a 1B layer's k and v projections orthogonalised together in bfloat16
        _muon("muon_2x512x2048", count=2, n=512, k=2048, dtype="bfloat16", step=False),
        # the gate projection of a 1B layer: the largest products
        _muon("muon_8192x2048", count=1, n=8192, k=2048, dtype="float32", step=True),
    ]


def _adapters(name, **sizes):
    return {"name": name, "op": "adapter", **sizes}


def _norms(name, **sizes):
    return {"name": name, "op": "norm", **sizes}


def _muon(name, **sizes):
    return {"name": name, "op": "muon", **sizes}


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["adapter_decode", "adapter_prefill", "norm", "norm", "muon"])
    if op.startswith("adapter"):
        decode = op.endswith("decode")
        tokens = rng.randint(1, 16) if decode else _log_int(rng, 17, 2048)
        case = {"op": "adapter", "tokens": tokens,
                "n": _log_int(rng, 100, 16384 if decode else 8192), "k": SUPERBLOCK * _log_int(rng, 2, 64 if decode else 32),
                "adapters": _log_int(rng, 1, 48), "rank": 8 * rng.randint(1, 8),
                "grain": rng.choice(["per_group", "per_group", "per_channel", "per_tensor"])}
        return case
    if op == "norm":
        seqs = rng.randint(1, 9)
        dim = _log_int(rng, 64, 8192)
        rows = seqs * _log_int(rng, 1, max(2, (8192 * 2048) // (dim * seqs * 2)))
        return {"op": "norm", "rows": rows, "dim": dim, "dtype": rng.choice(["bfloat16", "bfloat16", "float32"]),
                "gate": rng.choice(["none", "channel", "token", "sequence"]), "seqs": seqs,
                "train": rng.random() < 0.5}
    small = _log_int(rng, 64, 2048)
    n, k = rng.sample([small, _log_int(rng, small, 8192)], 2)
    return {"op": "muon", "count": rng.randint(1, 3) if n * k <= 1 << 20 else 1, "n": n, "k": k,
            "dtype": rng.choice(["float32", "bfloat16"]), "step": rng.random() < 0.5}


def work(case):
    if case["op"] == "adapter":
        m, n, k, r = case["tokens"], case["n"], case["k"], case["rank"]
        scales = {"per_group": n * k // SUPERBLOCK, "per_channel": n, "per_tensor": 1}[case["grain"]]
        used = min(case["adapters"], m)
        return {"bytes": n * k * 5 // 32 + 4 * scales + 2 * m * (n + k) + 2 * used * r * (n + k),
                "flops": 2 * m * n * k + 2 * m * r * (n + k)}
    if case["op"] == "norm":
        item = 2 if case["dtype"] == "bfloat16" else 4
        size = case["rows"] * case["dim"]
        passes = 4 + (6 if case["train"] else 0)   # y, h, h', n; and y, h, dh', dn, dy, dh
        return {"bytes": passes * size * item, "flops": (12 + (30 if case["train"] else 0)) * size}
    r, l = sorted((case["n"], case["k"]))
    item = 2 if case["dtype"] == "bfloat16" else 4
    passes = 5 if case["step"] else 2   # w, grad, buf in and w, buf out; or the matrix in and out
    return {"bytes": passes * case["count"] * r * l * item,
            "flops": case["count"] * 5 * (3 * r * r * l + r ** 3)}   # both Gram products are symmetric


# --------------------------------------------------------------------- inputs

def _rand(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _ternary(gen, n, k, grain):
    """A packed weight and what it stands for: 5-bit codes of random blocks in
    the record layout of the library (a nibble plane and a sign plane, 128
    weights a record), float32 scales, and the dense T * alpha."""
    sbs = k // SUPERBLOCK
    code = torch.randint(0, 32, (n, sbs, 32), generator=gen, device="cuda")
    table = torch.zeros(32, 4)
    for c in range(32):
        zero, first = (c >> 2) & 3, -1.0 if c >> 4 else 1.0
        kept = [p for p in range(4) if p != zero]
        signs = (first, first * (1 - 2 * (c & 1)), first * (1 - 2 * ((c >> 1) & 1)))
        for p, s in zip(kept, signs):
            table[c, p] = s
    t = table.cuda()[code].reshape(n, k)
    by_record = code.permute(1, 0, 2)
    nib = (by_record & 15).reshape(sbs, n, 4, 4, 2).permute(0, 1, 3, 2, 4)     # block 8b + 2d + h -> dword d, byte b
    nib = (nib[..., 0] | nib[..., 1] << 4).to(torch.uint8).reshape(-1)
    sign = (by_record >> 4).reshape(sbs, n, 4, 8) << torch.arange(8, device="cuda")
    sign = sign.sum(-1).to(torch.uint8).reshape(-1)
    shape = {"per_group": (sbs, n), "per_channel": (1, n), "per_tensor": (1, 1)}[grain]
    alpha = 0.02 * (1 + 0.1 * torch.rand(*shape, generator=gen, device="cuda"))
    dense = (t.reshape(n, -1, k // shape[0]) * alpha.t().reshape(-1, shape[0], 1)).reshape(n, k)
    return torch.cat([nib, sign]), alpha.reshape(-1).contiguous(), dense


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = dict(case)
    bf = torch.bfloat16
    if case["op"] == "adapter":
        m, n, k, c, r = case["tokens"], case["n"], case["k"], case["adapters"], case["rank"]
        state["packed"], state["alpha"], state["dense"] = _ternary(gen, n, k, case["grain"])
        state["x"] = _rand(gen, m, k, dtype=bf)
        state["a"] = _rand(gen, c, r, k, std=k ** -0.5, dtype=bf)
        state["b"] = _rand(gen, c, n, r, std=0.1, dtype=bf)
        state["scale"] = 0.5 + torch.rand(c, generator=gen, device="cuda")
        # ranks up to the stored one, the first adapter at all of it
        state["rank"] = torch.randint((r + 1) // 2, r + 1, (c,), generator=gen, device="cuda", dtype=torch.int32)
        state["rank"][0] = r
        if m == 1:
            ids = torch.zeros(1, dtype=torch.int32, device="cuda")
        elif m <= 16:      # decode: a token of another request in each row, some without an adapter
            ids = torch.randint(-1, c, (m,), generator=gen, device="cuda", dtype=torch.int32)
        else:              # prefill: the prompts of a few requests one after another
            cuts = torch.randint(0, m, (min(c, 12),), generator=gen, device="cuda").sort().values
            owner = torch.randint(-1, c, (len(cuts) + 1,), generator=gen, device="cuda", dtype=torch.int32)
            ids = owner[torch.bucketize(torch.arange(m, device="cuda"), cuts)].contiguous()
        state["ids"] = ids
    elif case["op"] == "norm":
        m, d, dt = case["rows"], case["dim"], getattr(torch, case["dtype"])
        state["y"], state["h"] = _rand(gen, m, d, std=0.7, dtype=dt), _rand(gen, m, d, std=2.0, dtype=dt)
        for name in ("w_post", "w_pre"):
            state[name] = 1 + _rand(gen, d, std=0.1)      # norm weights are kept in float32
        shape = {"none": None, "channel": (d,), "token": (m, 1), "sequence": (case["seqs"], d)}[case["gate"]]
        state["gate"] = None if shape is None else _rand(gen, *shape, std=0.5, dtype=dt)
        state["res_scale"], state["eps"] = 0.8, 1e-6
        if case["train"]:
            state["dh"], state["dn"] = _rand(gen, m, d, std=1e-2, dtype=dt), _rand(gen, m, d, std=1e-2, dtype=dt)
            state["ask"] = [x for x in ("h", "y", "w_post", "w_pre", "gate") if state[x] is not None]
            for x in state["ask"]:
                state[x].requires_grad_(True)
    else:
        shape, dt = (case["count"], case["n"], case["k"]), getattr(torch, case["dtype"])
        rank = max(1, min(shape[1:]) // 8)

        def gradient(std):     # gradients are low-rank with a tail
            low = _rand(gen, case["count"], case["n"], rank) @ _rand(gen, case["count"], rank, case["k"], std=rank ** -0.5)
            return (std * (low + 0.3 * _rand(gen, *shape))).to(dt)

        state["w"], state["grad"], state["buf"] = _rand(gen, *shape, std=0.02, dtype=dt), gradient(1e-3), gradient(5e-3)
        state |= {"lr": 0.02, "momentum": 0.95, "weight_decay": 0.1, "steps": 5, "eps": 1e-7}
    return state


# ----------------------------------------------------------------- the passes

def run(state):
    if own:
        return _own(state)
    return {"adapter": _plain_adapter, "norm": _plain_norm, "muon": _plain_muon}[state["op"]](state)


def _own(s):
    import ternary_weight_quantization_sparse_amd as S
    if s["op"] == "adapter":
        pw = S.PackedWeight(s["packed"], s["alpha"], s["n"], s["k"], s["grain"], SUPERBLOCK)
        ad = S.AdapterSet(s["a"], s["b"], s["scale"], s["rank"])
        if s["tokens"] <= 16:
            return S.adapter_gemv(pw, s["x"], ad, s["ids"])
        return S.adapter_gemm(pw, s["x"], ad, s["ids"])
    if s["op"] == "norm":
        args = dict(y=s["y"], w_post=s["w_post"], gate=s["gate"], res_scale=s["res_scale"], eps=s["eps"])
        if not s["train"]:
            return S.block_norm(s["h"], s["w_pre"], **args)
        h, n = S.block_norm_ad(s["h"], s["w_pre"], **args)
        grads = torch.autograd.grad((h, n), [s[x] for x in s["ask"]], (s["dh"], s["dn"]))
        return (h.detach(), n.detach(), *grads)
    if not s["step"]:
        return S.orthogonalize(s["buf"], steps=s["steps"], eps=s["eps"])
    return S.muon_step(s["w"], s["grad"], s["buf"], s["lr"], momentum=s["momentum"], nesterov=True,
                       weight_decay=s["weight_decay"], steps=s["steps"], eps=s["eps"])


def _plain_adapter(s):
    x, ids = s["x"].float(), s["ids"].long()
    here = (ids >= 0) & (ids < s["adapters"])
    at = ids.clamp(0, s["adapters"] - 1)
    slot = torch.arange(s["a"].shape[1], device=x.device)
    if s["tokens"] <= 16:       # each token's own adapter
        v = (s["a"][at].float() @ x[:, :, None])[..., 0]
        keep = here[:, None] & (slot < s["rank"][at][:, None])
        v = torch.where(keep, v * s["scale"][at][:, None], 0)
        add = (s["b"][at].float() @ v[:, :, None])[..., 0]
    else:                       # every adapter's products, those of the token's own kept
        v = x @ s["a"].float().reshape(-1, s["k"]).t()
        v = v.reshape(x.shape[0], s["adapters"], -1)
        mine = here[:, None] & (at[:, None] == torch.arange(s["adapters"], device=x.device))
        keep = mine[:, :, None] & (slot < s["rank"][:, None])
        v = torch.where(keep, v * s["scale"][:, None], 0)
        add = v.reshape(x.shape[0], -1) @ s["b"].float().transpose(1, 2).reshape(-1, s["n"])
    return (x @ s["dense"].t() + add).to(torch.bfloat16)


def _plain_norm(s):
    with torch.no_grad():
        dt, scale, eps, gate = s["h"].dtype, s["res_scale"], s["eps"], s["gate"]
        rows, dim = s["h"].shape
        per_seq = gate is not None and gate.shape == (s["seqs"], dim) and gate.dim() == 2
        shape = (s["seqs"] if per_seq else 1, -1, dim)      # sequences, rows of each, channels
        y, h = s["y"].float().reshape(shape), s["h"].float().reshape(shape)
        w_post, w_pre = s["w_post"], s["w_pre"]
        g = 1.0 if gate is None else gate.float()
        if per_seq:
            g = g[:, None, :]
        r_y = torch.rsqrt((y * y).mean(-1, keepdim=True) + eps)
        y_hat = y * r_y
        p = y_hat * w_post
        h2 = scale * h + g * p
        r_h = torch.rsqrt((h2 * h2).mean(-1, keepdim=True) + eps)
        h_hat = h2 * r_h
        out = h2.to(dt).reshape(rows, dim), (h_hat * w_pre).to(dt).reshape(rows, dim)
        if not s["train"]:
            return out
        dh, dn = s["dh"].float().reshape(shape), s["dn"].float().reshape(shape)
        u = dn * w_pre
        t = dh + r_h * (u - h_hat * (u * h_hat).mean(-1, keepdim=True))
        dp = t * g
        v = dp * w_post
        dy = r_y * (v - y_hat * (v * y_hat).mean(-1, keepdim=True))
        grads = [(scale * t).to(dt).reshape(rows, dim), dy.to(dt).reshape(rows, dim),
                 (dp * y_hat).sum((0, 1)), (dn * h_hat).sum((0, 1))]
        if gate is not None:
            tp = t * p
            if per_seq:
                d_gate = tp.sum(1)
            elif gate.dim() == 1:
                d_gate = tp.sum((0, 1))
            else:
                d_gate = tp.sum(-1).reshape(rows, 1)
            grads.append(d_gate.to(dt))
        return (*out, *grads)


def _plain_muon(s):
    w, grad, buf = s["w"].float(), s["grad"].float(), s["buf"].float()
    u = buf
    if s["step"]:
        buf = s["momentum"] * buf + grad
        u = grad + s["momentum"] * buf
    wide = u.shape[-2] <= u.shape[-1]
    x = u if wide else u.transpose(-1, -2).contiguous()
    x = x / ((x * x).sum((-1, -2), keepdim=True).sqrt() + s["eps"])
    for _ in range(s["steps"]):
        a = x @ x.transpose(-1, -2).contiguous()
        x = 3.4445 * x + (-4.7750 * a + 2.0315 * (a @ a)) @ x
    x = x if wide else x.transpose(-1, -2)
    if not s["step"]:
        return x.to(s["buf"].dtype)
    scale = math.sqrt(max(1.0, s["n"] / s["k"]))
    w = w * (1 - s["lr"] * s["weight_decay"]) - (s["lr"] * scale) * x
    return w.to(s["w"].dtype), buf.to(s["buf"].dtype)


# ------------------------------------------------------------ the definitions

def exact(case, seed):
    """The operators by their definitions in 64 bits, on the inputs of this seed."""
    s = prepare(case, seed)
    with torch.no_grad():
        return {"adapter": _exact_adapter, "norm": _exact_norm, "muon": _exact_muon}[case["op"]](s)


def _exact_adapter(s):
    x = s["x"].double()
    out = x.matmul(s["dense"].double().t())
    for c in range(s["adapters"]):
        rows = (s["ids"] == c).nonzero()[:, 0]
        if len(rows):
            r = int(s["rank"][c])
            low = x[rows].matmul(s["a"][c, :r].double().t())
            out[rows] += float(s["scale"][c]) * low.matmul(s["b"][c, :, :r].double().t())
    return out


def _exact_norm(s):
    rows, dim = s["h"].shape
    names = ("h", "y", "w_post", "w_pre", "gate")
    v = {x: None if s[x] is None else s[x].detach().double().requires_grad_(True) for x in names}
    with torch.enable_grad():
        def norm(x, w):
            return x / (x.pow(2).sum(1, keepdim=True) / dim + s["eps"]).sqrt() * w

        p = norm(v["y"], v["w_post"])
        if v["gate"] is not None:
            if tuple(v["gate"].shape) in ((rows, 1), (dim,)):
                p = v["gate"] * p
            else:
                p = (v["gate"][:, None, :] * p.reshape(v["gate"].shape[0], -1, dim)).reshape(rows, dim)
        h = s["res_scale"] * v["h"] + p
        n = norm(h, v["w_pre"])
        if not s["train"]:
            return h.detach(), n.detach()
        grads = torch.autograd.grad((h, n), [v[x] for x in s["ask"]], (s["dh"].double(), s["dn"].double()))
    return (h.detach(), n.detach(), *grads)


def _exact_muon(s):
    w, grad, buf = (s[x].double() for x in ("w", "grad", "buf"))
    u = buf
    if s["step"]:
        buf = s["momentum"] * buf + grad
        u = grad + s["momentum"] * buf
    outs = []
    for x in u:
        x = x / (torch.linalg.matrix_norm(x) + s["eps"])
        for _ in range(s["steps"]):   # from the smaller side, whichever it is
            if x.shape[0] <= x.shape[1]:
                a = x.mm(x.t())
                x = 3.4445 * x + (-4.7750 * a + 2.0315 * a.mm(a)).mm(x)
            else:
                a = x.t().mm(x)
                x = 3.4445 * x + x.mm(-4.7750 * a + 2.0315 * a.mm(a))
        outs.append(x)
    if not s["step"]:
        return torch.stack(outs)
    scale = math.sqrt(max(1.0, s["n"] / s["k"]))
    return w * (1 - s["lr"] * s["weight_decay"]) - s["lr"] * scale * torch.stack(outs), buf
