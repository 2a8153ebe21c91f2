"""Cases of the fused norms and of the linear cross-entropy, to be timed and compared.

Operators (M rows of N elements; x, residual, h, dy, dh and w of one type, float32 or bfloat16):

  add_norm      h = x + residual, kept in the inputs' type; y = h * rstd * w with rstd = 1 / sqrt(mean(h^2) + eps)
  add_norm_bwd  dx = dh + the gradient of that norm at h for dy; dw, summed over the rows, in float32
  norm_quant    y as above (with or without a residual), held in 8 bits: one scale a row or a group of columns,
                scale = max(largest |y| of the group, 2^-100) / qmax, q = y / scale rounded to nearest even
  lx_loss       logits = h w^T (h [M, K], w [V, K]), lse and loss = lse - logit of the target + z lse^2 a row, and the
                mean of the loss over the rows that are not ignored; the logits are no output
  lx_step       the same, and then the gradients dh and dw for a given gradient of each row's loss

`own` chooses between the plain forms below and the package's calls.
"""
import math

import torch

own = False

EPS = 1e-6
IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
QTYPES = {"e4m3": (torch.float8_e4m3fn, 448.0), "int8": (torch.int8, 127.0)}
SMALLEST = 2.0 ** -100  # no group's largest value counts as less than this


def listed():
    return [
        # One step of eight sequences being decoded: a launch whose time is latency.
        {"name": "add_norm decode 8x4096 bf16", "op": "add_norm", "dtype": "bf16", "M": 8, "N": 4096},
        # The norm in front of a block, training or prefill: 16384 tokens at a width of 4096.
        {"name": "add_norm 16384x4096 bf16", "op": "add_norm", "dtype": "bf16", "M": 16384, "N": 4096},
        # The same norm's backward pass, with the gradient of the residual stream joined.
        {"name": "add_norm_bwd 16384x4096 bf16", "op": "add_norm_bwd", "dtype": "bf16", "M": 16384, "N": 4096},
        # Full precision and a ragged width: rows that start off every vector boundary.
        {"name": "add_norm_bwd 4095x1023 f32", "op": "add_norm_bwd", "dtype": "f32", "M": 4095, "N": 1023},
        # In front of a product in 8 bits, prefill: a scale for each 128 columns.
        {"name": "norm_quant 16384x4096 bf16 g128", "op": "norm_quant", "dtype": "bf16", "M": 16384, "N": 4096,
         "qtype": "e4m3", "group": 128, "residual": True},
        # The same while decoding, one scale a token.
        {"name": "norm_quant 16x8192 bf16 row", "op": "norm_quant", "dtype": "bf16", "M": 16, "N": 8192,
         "qtype": "e4m3", "group": 0, "residual": True},
        # Integers, one scale a token, a norm without a residual, a ragged number of rows.
        {"name": "norm_quant 2049x2048 f32 int8", "op": "norm_quant", "dtype": "f32", "M": 2049, "N": 2048,
         "qtype": "int8", "group": 0, "residual": False},
        # Scoring one short answer: the weights are read once for a handful of tokens.
        {"name": "lx_loss 16x32000x4096 bf16", "op": "lx_loss", "dtype": "bf16", "M": 16, "V": 32000, "K": 4096,
         "z": 0.0},
        # The loss of 8192 tokens over a large vocabulary, as evaluation reads it.
        {"name": "lx_loss 8192x131072x4096 bf16", "op": "lx_loss", "dtype": "bf16", "M": 8192, "V": 131072, "K": 4096,
         "z": 0.0},
        # A training step's loss and gradients.
        {"name": "lx_step 8192x32000x4096 bf16", "op": "lx_step", "dtype": "bf16", "M": 8192, "V": 32000, "K": 4096,
         "z": 1e-4},
        # A small model's step with odd sizes everywhere, and its padding ignored.
        {"name": "lx_step 1001x50257x768 bf16", "op": "lx_step", "dtype": "bf16", "M": 1001, "V": 50257, "K": 768,
         "z": 0.0},
        # Full precision, odd sizes, with the term on the log of the partition function.
        {"name": "lx_step 2047x8191x513 f32", "op": "lx_step", "dtype": "f32", "M": 2047, "V": 8191, "K": 513,
         "z": 1e-4},
    ]


def _spread(rng, lo, hi, even=0.5):
    """A whole number between lo and hi, uniform over its logarithm; a share `even` of them multiples of 8."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, n // 8 * 8) if rng.random() < even else n


def draw(rng):
    op = rng.choice(["add_norm", "add_norm_bwd", "norm_quant", "lx_loss", "lx_step"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op.startswith("lx"):
        f32 = case["dtype"] == "f32"
        V, K = _spread(rng, 500, 131072), _spread(rng, 64, 4096, even=0.8)  # widths are multiples of 8, mostly
        most = (2e10 if f32 else 1e12) if op == "lx_step" else (4e10 if f32 else 4e12)
        M = _spread(rng, 1, max(2, min(8192, int(most / (V * K)))))
        return {**case, "M": M, "V": V, "K": K, "z": rng.choice([0.0, 1e-4])}
    N = _spread(rng, 64, 16384)
    M = _spread(rng, 1, min(32768, 16384 * 4096 // (N * (2 if case["dtype"] == "f32" else 1))))
    if op == "norm_quant":
        case |= {"qtype": rng.choice(["e4m3", "e4m3", "int8"]), "group": rng.choice([0, 32, 64, 128]),
                 "residual": rng.random() < 0.7}
    return {**case, "M": M, "N": N}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype, M = DTYPES[case["dtype"]], case["M"]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    state = {**case}
    if case["op"].startswith("lx"):
        V, K = case["V"], case["K"]
        state["h"] = normal(M, K)                          # what a norm leaves: values around one
        state["w"] = normal(V, K, scale=2.0 / math.sqrt(K))  # logits of a spread of two
        state["targets"] = torch.randint(0, V, (M,), generator=g, device="cuda")
        padding = torch.rand(M, generator=g, device="cuda") < 0.05
        padding[0] = False
        state["targets"][padding] = IGNORE
        state["dloss"] = (1.0 / (~padding).sum()).expand(M).float().contiguous()  # of the mean
        return state
    N = case["N"]
    state["w"] = 1.0 + normal(N, scale=0.1)
    if case["op"] == "add_norm_bwd":
        state["h"] = normal(M, N, scale=3.0)
        state["rstd"] = (state["h"].double().square().mean(-1) + EPS).rsqrt().float()
        state["dy"], state["dh"] = normal(M, N), normal(M, N)
        return state
    state["x"] = normal(M, N)
    state["r"] = normal(M, N, scale=3.0) if case.get("residual", True) else None
    return state


def _norm_plain(s):
    h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["x"].dtype)
    f = h.float()  # of the h that is kept
    rstd = 1.0 / torch.sqrt((f * f).mean(-1) + EPS)
    return h, f * rstd[:, None] * s["w"].float(), rstd


def _quant_plain(y, group, qtype):
    q, qmax = QTYPES[qtype]
    M, N = y.shape
    group = group or N
    pieces = (N + group - 1) // group
    wide = torch.zeros(M, pieces * group, device=y.device)
    wide[:, :N] = y
    wide = wide.view(M, pieces, group)
    scale = torch.clamp(wide.abs().amax(-1), min=SMALLEST) / qmax
    v = (wide / scale[..., None]).view(M, -1)[:, :N]
    return (v.round() if qtype == "int8" else v).to(q), scale


def _values(q):
    """8-bit integers as the numbers that they stand for (exact in bfloat16); 8-bit floats are numbers already."""
    return q.to(torch.bfloat16) if q.dtype == torch.int8 else q


def _loss_plain(s):
    h, w, t, M = s["h"].float(), s["w"].float(), s["targets"], s["M"]
    logits = h @ w.T
    top = logits.amax(-1)
    lse = top + torch.log(torch.exp(logits - top[:, None]).sum(-1))
    kept = t != IGNORE
    at = torch.where(kept, t, 0)
    loss = torch.where(kept, lse - logits[torch.arange(M, device=t.device), at] + s["z"] * lse * lse, 0.0)
    return logits, lse, loss, loss.sum() / kept.sum()


def _grad_plain(s, logits, lse):
    h, w, t, M = s["h"].float(), s["w"].float(), s["targets"], s["M"]
    kept = t != IGNORE
    p = torch.exp(logits - lse[:, None]) * (1.0 + 2.0 * s["z"] * lse)[:, None]
    p[torch.arange(M, device=t.device), torch.where(kept, t, 0)] -= 1.0
    p *= torch.where(kept, s["dloss"], 0.0)[:, None]
    return (p @ w).to(s["h"].dtype), (p.T @ h).to(s["w"].dtype)


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "add_norm":
        h, y, rstd = _norm_plain(s)
        return {"h": h, "y": y.to(h.dtype), "rstd": rstd}
    if op == "add_norm_bwd":
        h, dy, r, w = s["h"].float(), s["dy"].float(), s["rstd"][:, None], s["w"].float()
        g = dy * w
        dx = s["dh"].float() + r * g - h * (r * r * r) * (g * h).mean(-1, keepdim=True)
        return {"dx": dx.to(s["h"].dtype), "dw": (dy * h * r).sum(0)}
    if op == "norm_quant":
        h, y, rstd = _norm_plain(s)
        q, scale = _quant_plain(y, s["group"], s["qtype"])
        return {"q": _values(q), "scale": scale, "rstd": rstd, "h": h if s["r"] is not None else None}
    logits, lse, loss, mean = _loss_plain(s)
    if op == "lx_loss":
        return {"loss": loss, "lse": lse, "mean": mean}
    dh, dw = _grad_plain(s, logits, lse)
    return {"loss": loss, "lse": lse, "mean": mean, "dh": dh, "dw": dw}


def _run_own(s):
    from memory_bound_row_rmsnorm_gb300 import binding as qb
    op = s["op"]
    if op == "add_norm":
        y, h, rstd = qb.add_rmsnorm_fwd(s["x"], s["r"], s["w"], eps=EPS)
        return {"h": h, "y": y, "rstd": rstd}
    if op == "add_norm_bwd":
        dx, dw = qb.add_rmsnorm_bwd(s["h"], s["w"], s["rstd"], s["dy"], s["dh"])
        return {"dx": dx, "dw": dw}
    if op == "norm_quant":
        q, scale, h, rstd = qb.rmsnorm_quant_fwd(s["x"], s["w"], residual=s["r"], eps=EPS, group=s["group"],
                                                 qdtype=QTYPES[s["qtype"]][0])
        return {"q": _values(q), "scale": scale, "rstd": rstd, "h": h}
    loss, lse, mean = qb.linear_xent_fwd(s["h"], s["w"], s["targets"], ignore_index=IGNORE, z_loss=s["z"],
                                         want_mean=True)
    if op == "lx_loss":
        return {"loss": loss, "lse": lse, "mean": mean}
    dh, dw = qb.linear_xent_bwd(s["h"], s["w"], s["targets"], lse, dloss=s["dloss"], ignore_index=IGNORE,
                                z_loss=s["z"])
    return {"loss": loss, "lse": lse, "mean": mean, "dh": dh, "dw": dw}


def work(case):
    e, M = (2 if case["dtype"] == "bf16" else 4), case["M"]
    if case["op"].startswith("lx"):
        V, K = case["V"], case["K"]
        read = (M + V) * K * e + 8 * M
        if case["op"] == "lx_loss":
            return {"bytes": read + 8 * M + 4, "flops": 2 * M * V * K}
        # The loss needs the logits once, the gradients two products more; without keeping the logits they are made again.
        return {"bytes": read + (M + V) * K * e + 12 * M + 4, "flops": 8 * M * V * K}
    N = case["N"]
    if case["op"] == "add_norm":
        return {"bytes": 4 * M * N * e + N * e + 4 * M, "flops": 5 * M * N}
    if case["op"] == "add_norm_bwd":
        return {"bytes": 4 * M * N * e + N * e + 4 * M + 4 * N, "flops": 10 * M * N}
    groups = -(-N // (case["group"] or N))
    rows = 3 if case["residual"] else 1
    return {"bytes": rows * M * N * e + M * N + N * e + 4 * M * groups + 4 * M, "flops": 7 * M * N}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("lx"):
        kept = s["targets"] != IGNORE
        h, w = s["h"].double(), s["w"].double()
        h.requires_grad_(op == "lx_step")
        w.requires_grad_(op == "lx_step")
        logits = torch.nn.functional.linear(h, w)
        lse = torch.logsumexp(logits, -1)
        loss = torch.nn.functional.cross_entropy(logits, s["targets"], ignore_index=IGNORE, reduction="none")
        loss = loss + case["z"] * kept * lse ** 2
        out = {"loss": loss.detach(), "lse": lse.detach(), "mean": loss.detach()[kept].mean()}
        if op == "lx_step":
            out["dh"], out["dw"] = torch.autograd.grad(loss, (h, w), s["dloss"].double())
        return out
    if op == "add_norm_bwd":
        h, dy, r = s["h"].double(), s["dy"].double(), s["rstd"].double()
        unit = torch.einsum("mn,m->mn", h, r)
        back = torch.einsum("mn,n,m->mn", dy, s["w"].double(), r)
        along = torch.einsum("mn,mn->m", back, unit) / case["N"]
        return {"dx": s["dh"].double() + back - torch.einsum("mn,m->mn", unit, along),
                "dw": torch.einsum("mn,mn->n", dy, unit)}
    h = s["x"] if s["r"] is None else torch.add(s["x"].double(), s["r"].double()).to(s["x"].dtype)
    f = h.double()
    rstd = (torch.linalg.vector_norm(f, dim=-1) ** 2 / case["N"] + EPS) ** -0.5
    y = torch.einsum("mn,m,n->mn", f, rstd, s["w"].double())
    if op == "add_norm":
        return {"h": h.double(), "y": y, "rstd": rstd}
    q, qmax = QTYPES[case["qtype"]]
    N, group = case["N"], case["group"] or case["N"]
    cuts = torch.split(y.abs(), group, dim=-1)
    scale = torch.stack([c.amax(-1) for c in cuts], -1).clamp_min(SMALLEST) / qmax
    v = y / torch.repeat_interleave(scale, group, dim=-1)[:, :N]
    held = v.round() if case["qtype"] == "int8" else v.to(q).double()
    return {"q": held, "scale": scale, "rstd": rstd, "h": h.double() if s["r"] is not None else None}
