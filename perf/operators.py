"""The operators of a feed-forward language model's step, as cases to measure:
the linear layer with its epilogue, the gated feed-forward block, the softmax
cross entropy over a vocabulary, and the clipping of gradients by their global
norm.  `run` computes a case in plain torch (`own` false) or with the
package's operators (`own` true)."""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One token through a projection: decoding for one user, latency counts.
        {"name": "linear_token", "op": "linear", "M": 1, "K": 4096, "N": 4096, "dtype": "bf16",
         "act": "none", "bias": True, "residual": True, "train": False, "lead": 0},
        # A batch of decoding users, the rows cut out of a wider buffer.
        {"name": "linear_users", "op": "linear", "M": 24, "K": 2048, "N": 8192, "dtype": "f16",
         "act": "gelu", "bias": True, "residual": False, "train": False, "lead": 64},
        # A prompt through a square projection.
        {"name": "linear_prompt", "op": "linear", "M": 4096, "K": 4096, "N": 4096, "dtype": "f16",
         "act": "gelu_tanh", "bias": True, "residual": True, "train": False, "lead": 0},
        # A training step at sizes that fit neither a tile nor a 16-byte row.
        {"name": "linear_train_odd", "op": "linear", "M": 2039, "K": 1025, "N": 2047,
         "dtype": "f16", "act": "silu", "bias": True, "residual": False, "train": True, "lead": 0},
        # A training step of a large layer.
        {"name": "linear_train", "op": "linear", "M": 8192, "K": 4096, "N": 4096, "dtype": "bf16",
         "act": "gelu", "bias": True, "residual": True, "train": True, "lead": 0},
        # One token through the gated block: the weights are all there is to read.
        {"name": "ffn_token", "op": "ffn", "M": 1, "D": 4096, "F": 8192, "dtype": "bf16",
         "act": "silu", "residual": True, "train": False},
        # A prompt through the gated block.
        {"name": "ffn_prompt", "op": "ffn", "M": 4096, "D": 4096, "F": 8192, "dtype": "f16",
         "act": "silu", "residual": True, "train": False},
        # A training step of the gated block on packed sequences of any length.
        {"name": "ffn_train", "op": "ffn", "M": 4093, "D": 2048, "F": 8192, "dtype": "bf16",
         "act": "gelu_tanh", "residual": True, "train": True},
        # Scoring a short text: each token's loss, an odd vocabulary.
        {"name": "xent_score", "op": "xent", "M": 509, "D": 1024, "V": 32001, "dtype": "f16",
         "ignored": 0.3, "train": False},
        # A training step on a large vocabulary, a part of the tokens masked out.
        {"name": "xent_train", "op": "xent", "M": 8192, "D": 2048, "V": 65536, "dtype": "bf16",
         "ignored": 0.1, "train": True},
        # Gradients of a small model: many short tensors, launches count.
        {"name": "clip_small", "op": "clip", "count": 60, "total": 1 << 20, "dtype": "f32",
         "clipped": True},
        # Gradients of a large model: two passes over memory.
        {"name": "clip_large", "op": "clip", "count": 290, "total": 700000001, "dtype": "bf16",
         "clipped": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size between lo and hi: even odds of a multiple of 8 and of any."""
    n = _log_int(rng, lo, hi)
    return max(8, n // 8 * 8) if rng.random() < 0.5 else n


def draw(rng):
    most = 3 * 8192 * 4096 * 4096  # multiply-adds of the largest linear step
    op = rng.choice(["linear", "ffn", "xent", "clip"])
    kind = rng.choice(["f16", "bf16"])
    if op == "linear":
        while True:
            c = {"op": op, "M": _log_int(rng, 1, 8192), "K": _size(rng, 200, 8192),
                 "N": _size(rng, 200, 8192), "dtype": kind,
                 "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                 "bias": rng.random() < 0.7, "residual": rng.random() < 0.5,
                 "train": rng.random() < 0.5, "lead": rng.choice([0, 0, 8, 37])}
            if c["M"] * c["K"] * c["N"] * (3 if c["train"] else 1) <= most:
                return c
    if op == "ffn":
        while True:
            c = {"op": op, "M": _log_int(rng, 1, 8192), "D": _size(rng, 200, 4096),
                 "F": _size(rng, 300, 8192), "dtype": kind,
                 "act": rng.choice(["silu", "gelu_tanh", "gelu", "relu"]),
                 "residual": rng.random() < 0.7, "train": rng.random() < 0.5}
            if 3 * c["M"] * c["D"] * c["F"] * (3 if c["train"] else 1) <= most:
                return c
    if op == "xent":
        while True:
            c = {"op": op, "M": _log_int(rng, 1, 8192), "D": _size(rng, 100, 2048),
                 "V": _log_int(rng, 500, 65536), "dtype": kind,
                 "ignored": rng.choice([0.0, 0.1, 0.5]), "train": rng.random() < 0.6}
            if c["M"] * c["D"] * c["V"] * (4 if c["train"] else 1) <= most:
                return c
    return {"op": op, "count": _log_int(rng, 1, 400), "total": _log_int(rng, 100000, 500000000),
            "dtype": rng.choice(["f16", "bf16", "f32"]), "clipped": rng.random() < 0.7}


def _clip_sizes(case):
    """Lengths of the gradient tensors: most of the total in a few large
    ones, the others short, odd lengths among them."""
    rng = random.Random(case["total"] * 1009 + case["count"])
    weights = [math.exp(rng.gauss(0.0, 2.0)) for _ in range(case["count"])]
    scale = case["total"] / sum(weights)
    return [max(1, int(w * scale)) for w in weights]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = {"case": case}
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        s["x"] = normal(M, K + case["lead"])[:, :K]
        s["w"] = normal(K, N, std=K ** -0.5)
        s["b"] = normal(N, std=0.2) if case["bias"] else None
        s["r"] = normal(M, N) if case["residual"] else None
        if case["train"]:
            s["dy"] = normal(M, N, std=0.05)
    elif case["op"] == "ffn":
        M, D, F = case["M"], case["D"], case["F"]
        s["x"] = normal(M, D)
        s["w_in"] = normal(D, 2 * F, std=D ** -0.5)
        s["w_out"] = normal(F, D, std=F ** -0.5)
        if case["train"]:
            s["dy"] = normal(M, D, std=0.05)
    elif case["op"] == "xent":
        M, D, V = case["M"], case["D"], case["V"]
        s["x"] = normal(M, D)
        s["w"] = normal(V, D, std=2.0 * D ** -0.5)
        target = torch.randint(0, V, (M,), generator=g, device="cuda")
        if case["ignored"]:
            masked = torch.rand(M, generator=g, device="cuda") < case["ignored"]
            masked[0] = False
            target = torch.where(masked, torch.full_like(target, -100), target)
        s["t"] = target
    else:
        # The tensors are cut out of one buffer, each on a 16-byte boundary, and
        # go into another one, so that a second pass finds the same gradients.
        sizes = _clip_sizes(case)
        starts = [0]
        for n in sizes:
            starts.append(starts[-1] + (n + 7) // 8 * 8)
        s["bucket"] = normal(starts[-1], std=0.01)
        s["clipped"] = torch.zeros_like(s["bucket"])
        s["grads"] = [s["bucket"][a:a + n] for a, n in zip(starts, sizes)]
        s["out"] = [s["clipped"][a:a + n] for a, n in zip(starts, sizes)]
        total = sum(sizes)
        s["max_norm"] = 0.01 * math.sqrt(total) * (0.4 if case["clipped"] else 3.0)
    return s


# ---- plain forms: 32 bits throughout, one rounding at the end ----------------

def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _plain(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "linear":
        x, w = s["x"].float(), s["w"].float()
        z = x @ w
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(z, case["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        if not case["train"]:
            return y.to(dt)
        dz = s["dy"].float() * _act_grad(z, case["act"])
        out = {"y": y.to(dt), "dx": (dz @ w.t()).to(dt), "dw": (x.t() @ dz).to(dt)}
        if s["b"] is not None:
            out["db"] = dz.sum(0).to(dt)
        return out
    if case["op"] == "ffn":
        x, w_in, w_out = s["x"].float(), s["w_in"].float(), s["w_out"].float()
        gate, up = (x @ w_in).split(case["F"], dim=1)
        a = _act(gate, case["act"])
        h = a * up
        y = h @ w_out
        if case["residual"]:
            y = y + x
        if not case["train"]:
            return y.to(dt)
        dy = s["dy"].float()
        dh = dy @ w_out.t()
        d_in = torch.cat([dh * up * _act_grad(gate, case["act"]), dh * a], dim=1)
        dx = d_in @ w_in.t()
        if case["residual"]:
            dx = dx + dy
        return {"y": y.to(dt), "dx": dx.to(dt), "dw_in": (x.t() @ d_in).to(dt),
                "dw_out": (h.t() @ dy).to(dt)}
    if case["op"] == "xent":
        x, w, t = s["x"].float(), s["w"].float(), s["t"]
        logits = x @ w.t()
        top = logits.max(dim=1, keepdim=True).values
        e = torch.exp(logits - top)
        total = e.sum(dim=1, keepdim=True)
        valid = t >= 0
        at = torch.where(valid, t, torch.zeros_like(t))[:, None]
        each = top + torch.log(total) - logits.gather(1, at)
        if not case["train"]:
            lse = (top + torch.log(total))[:, 0]
            return {"loss": torch.where(valid, each[:, 0], torch.zeros_like(lse)), "lse": lse}
        n = valid.sum().clamp(min=1).float()
        weight = valid.float()[:, None] / n
        loss = (each * weight).sum()
        d = e.div_(total).mul_(weight)
        d.scatter_add_(1, at, -weight)
        return {"loss": loss, "dx": (d @ w).to(dt), "dw": (d.t() @ x).to(dt)}
    total = sum((t.float() * t.float()).sum() for t in s["grads"])
    norm = torch.sqrt(total)
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    for o, t in zip(s["out"], s["grads"]):
        o.copy_(t.float() * coef)
    return {"norm": norm, "clipped": s["clipped"]}


def _own(s):
    import software_pipelined_tiled_pgemm_amd as pg
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "linear":
        x, w, act = s["x"], s["w"], case["act"]
        if not case["train"]:
            return pg.plinear(x, w, bias=s["b"], residual=s["r"], act=act)
        z = None
        if act != "none":
            z = torch.empty(case["M"], case["N"], dtype=dt, device="cuda")
        y = pg.plinear(x, w, bias=s["b"], residual=s["r"], act=act, preact=z)
        dx, dw, db = pg.plinear_bwd(s["dy"], x, w, preact=z, act=act,
                                    needs=(True, True, s["b"] is not None))
        out = {"y": y, "dx": dx, "dw": dw}
        if db is not None:
            out["db"] = db
        return out
    if case["op"] == "ffn":
        x = s["x"]
        r = x if case["residual"] else None
        if not case["train"]:
            return pg.pffn(x, s["w_in"], s["w_out"], residual=r, act=case["act"])
        gu = torch.empty(case["M"], 2 * case["F"], dtype=dt, device="cuda")
        y = pg.pffn(x, s["w_in"], s["w_out"], residual=r, act=case["act"], gate_up=gu)
        dx, dw_in, dw_out = pg.pffn_bwd(s["dy"], x, s["w_in"], s["w_out"], gu, act=case["act"],
                                        dx_residual=s["dy"] if case["residual"] else None)
        return {"y": y, "dx": dx, "dw_in": dw_in, "dw_out": dw_out}
    if case["op"] == "xent":
        if not case["train"]:
            loss, lse = pg.pxent(s["x"], s["w"], s["t"], reduction="none")
            return {"loss": loss, "lse": lse}
        loss, lse = pg.pxent(s["x"], s["w"], s["t"])
        dx, dw = pg.pxent_bwd(s["x"], s["w"], s["t"], lse)
        return {"loss": loss, "dx": dx, "dw": dw}
    norm = pg.pclip_grad_norm(s["grads"], s["max_norm"], out=s["out"])
    return {"norm": norm, "clipped": s["clipped"]}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    b = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        values = M * K + K * N + M * N
        if case["bias"]:
            values += N
        if case["residual"]:
            values += M * N
        if case["train"]:  # dy in; dx, dw and db out
            values += M * N + M * K + K * N + (N if case["bias"] else 0)
        return {"bytes": values * b, "flops": 2 * M * K * N * (3 if case["train"] else 1)}
    if case["op"] == "ffn":
        M, D, F = case["M"], case["D"], case["F"]
        values = 2 * M * D + 3 * D * F
        if case["train"]:  # dy in; dx, dw_in and dw_out out
            values += 2 * M * D + 3 * D * F
        return {"bytes": values * b, "flops": 6 * M * D * F * (3 if case["train"] else 1)}
    if case["op"] == "xent":
        M, D, V = case["M"], case["D"], case["V"]
        values = M * D + V * D
        if case["train"]:
            values *= 2
        # The gradient needs the logits again, since they are not kept.
        return {"bytes": values * b + 8 * M + (4 if case["train"] else 8 * M),
                "flops": 2 * M * D * V * (4 if case["train"] else 1)}
    n = sum(_clip_sizes(case))
    return {"bytes": 2 * n * b + 4, "flops": 3 * n}


# ---- the definitions in 64 bits ----------------------------------------------

def _definition(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":  # z times the standard normal distribution function
        return z * torch.special.ndtr(z)
    return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))


def exact(case, seed):
    s = prepare(case, seed)
    train = case.get("train", False)

    def leaf(t):
        return None if t is None else t.double().requires_grad_(train)

    if case["op"] == "linear":
        x, w, b, r = leaf(s["x"]), leaf(s["w"]), leaf(s["b"]), leaf(s["r"])
        z = torch.matmul(x, w) if b is None else torch.addmm(b, x, w)
        y = _definition(z, case["act"])
        if r is not None:
            y = y + r
        if not train:
            return y
        y.backward(s["dy"].double())
        out = {"y": y.detach(), "dx": x.grad, "dw": w.grad}
        if b is not None:
            out["db"] = b.grad
        return out
    if case["op"] == "ffn":
        x, w_in, w_out = leaf(s["x"]), leaf(s["w_in"]), leaf(s["w_out"])
        F = case["F"]
        h = _definition(x @ w_in[:, :F], case["act"]) * (x @ w_in[:, F:])
        y = h @ w_out
        if case["residual"]:
            y = y + x
        if not train:
            return y
        y.backward(s["dy"].double())
        return {"y": y.detach(), "dx": x.grad, "dw_in": w_in.grad, "dw_out": w_out.grad}
    if case["op"] == "xent":
        x, w, t = s["x"].double(), s["w"].double(), s["t"]
        if not train:
            logits = x @ w.t()
            lse = torch.logsumexp(logits, dim=1)
            rows = torch.arange(case["M"], device="cuda")
            return {"loss": torch.where(t < 0, 0.0, lse - logits[rows, t.clamp(min=0)]), "lse": lse}
        # In groups of rows, each row's loss and gradient standing alone.
        n = max(1, int((t >= 0).sum()))
        loss = torch.zeros((), dtype=torch.float64, device="cuda")
        dx, dw = torch.zeros_like(x), torch.zeros_like(w)
        for r0 in range(0, case["M"], 1024):
            xr, tr = x[r0:r0 + 1024], t[r0:r0 + 1024]
            keep = torch.nonzero(tr >= 0)[:, 0]
            if keep.numel() == 0:
                continue
            lp = torch.log_softmax(xr[keep] @ w.t(), dim=1)
            rows = torch.arange(keep.numel(), device="cuda")
            loss = loss - lp[rows, tr[keep]].sum() / n
            p = torch.exp(lp)
            p[rows, tr[keep]] -= 1.0
            dx[r0 + keep] = p @ w / n
            dw += p.t() @ xr[keep] / n
        return {"loss": loss, "dx": dx, "dw": dw}
    norm = torch.sqrt(sum(torch.linalg.vector_norm(t.double()) ** 2 for t in s["grads"]))
    coef = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    clipped = torch.zeros(s["bucket"].numel(), dtype=torch.float64, device="cuda")
    for t in s["grads"]:
        at = t.storage_offset()
        clipped[at:at + t.numel()] = t.double() * coef
    return {"norm": norm, "clipped": clipped}
