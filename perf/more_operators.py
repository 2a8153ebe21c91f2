"""Cases of the 8-bit products and of the rows sorted by expert, to be timed and compared.

Operators (8-bit values are e4m3; G(n) = ceil(n / 128) scales along an axis of n):

  quant       8-bit values of x [M, N] with a scale for each 128 columns of a row, or for each block of 128 x 128:
              scale = max(largest |x| of the group, 2^-100) / 448, q = x / scale rounded to nearest even; straight
              (groups along the rows) and turned (of x^T, groups along the columns of x)
  mm          y = sum over blocks c of 128 k of a_scale[i, c] b_scale[j, c] (sum of a b over the block); a [M, K] with a
              scale a row and block, b [N, K] with a scale a block of 128 x 128, or a row and block
  experts_mm  the same for rows sorted by expert: rows offsets[e] to offsets[e + 1] of a times the weights b[e];
              rows behind the last expert's are left as they were
  dispatch    experts [T, k] sorted (stable; an expert outside [0, E) has no row): the experts' offsets, the sorted row
              of each (token, choice), and the tokens' rows copied to their places, 8-bit rows with their scales
  combine     y[t] = sum over choices of weight[t, j] rows[slot[t, j]], or its gradients for rows and weights

`own` chooses between the plain forms below and the package's calls.
"""
import math

import torch

own = False

BLOCK = 128
QMAX = 448.0
SMALLEST = 2.0 ** -100  # no group's largest value counts as less than this
E4M3 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": E4M3}


def listed():
    return [
        # One step of eight sequences being decoded through a square projection: a launch whose time is latency.
        {"name": "mm decode 8x4096x4096", "op": "mm", "M": 8, "N": 4096, "K": 4096, "out": "bf16", "b_rows": 128},
        # A projection over the tokens of a long prompt, or of a training step.
        {"name": "mm 16384x8192x4096", "op": "mm", "M": 16384, "N": 8192, "K": 4096, "out": "bf16", "b_rows": 128},
        # Odd sizes everywhere: rows that start off every 16 bytes, a last block of 127 k.
        {"name": "mm 1001x2047x1023", "op": "mm", "M": 1001, "N": 2047, "K": 1023, "out": "f32", "b_rows": 128},
        # The gradient of a weight: both operands quantised along the tokens, a scale a row and block.
        {"name": "mm dw 4096x4096x8192", "op": "mm", "M": 4096, "N": 4096, "K": 8192, "out": "f32", "b_rows": 1},
        # 32 sequences being decoded, four experts of 32 each: the weights of nearly all experts for a few rows.
        {"name": "experts_mm decode 32x4 of 32 to 4096x2048", "op": "experts_mm", "T": 32, "k": 4, "E": 32, "N": 4096,
         "K": 2048, "out": "bf16", "dropped": 0.0},
        # A prompt's tokens, two experts of 32 each, unevenly chosen, and a part dropped for want of room.
        {"name": "experts_mm 8192x2 of 32 to 4096x4096", "op": "experts_mm", "T": 8192, "k": 2, "E": 32, "N": 4096,
         "K": 4096, "out": "bf16", "dropped": 0.02},
        # A decoding step's 8-bit rows on their way to the experts.
        {"name": "dispatch decode 16x4 of 32 rows 4096 e4m3", "op": "dispatch", "T": 16, "k": 4, "E": 32, "N": 4096,
         "dtype": "e4m3", "dropped": 0.0},
        # A training step's rows, four experts of 64 each.
        {"name": "dispatch 16384x4 of 64 rows 4096 bf16", "op": "dispatch", "T": 16384, "k": 4, "E": 64, "N": 4096,
         "dtype": "bf16", "dropped": 0.02},
        # The experts' outputs on their way back to the tokens.
        {"name": "combine 16384x4 rows 4096 bf16", "op": "combine", "T": 16384, "k": 4, "E": 64, "N": 4096,
         "dtype": "bf16", "dropped": 0.02, "backward": False},
        # The gradients of that in a training step, two experts a token.
        {"name": "combine_bwd 16384x2 rows 4096 bf16", "op": "combine", "T": 16384, "k": 2, "E": 64, "N": 4096,
         "dtype": "bf16", "dropped": 0.02, "backward": True},
        # A gradient on its way to both backward products: quantised along its rows and along its columns.
        {"name": "quant 16384x4096 bf16 both ways", "op": "quant", "M": 16384, "N": 4096, "dtype": "bf16", "rows": 1,
         "straight": True, "turned": True},
        # Weights of a small layer with odd sizes, kept in full precision, once a step in blocks for the forward product.
        {"name": "quant 4097x1023 f32 blocks", "op": "quant", "M": 4097, "N": 1023, "dtype": "f32", "rows": 128,
         "straight": True, "turned": False},
    ]


def _spread(rng, lo, hi, even=0.5, unit=8):
    """A whole number between lo and hi, uniform over its logarithm; a share `even` of them multiples of `unit`."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, n // unit * unit) if rng.random() < even else n


def draw(rng):
    op = rng.choice(["mm", "mm", "experts_mm", "experts_mm", "dispatch", "combine", "quant"])
    if op == "quant":
        N = _spread(rng, 64, 16384)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        M = _spread(rng, 1, min(32768, 16384 * 4096 // (N * (2 if dtype == "f32" else 1))))
        straight, turned = rng.choice([(True, True), (True, False), (False, True)])
        return {"op": op, "M": M, "N": N, "dtype": dtype, "rows": rng.choice([1, 128]), "straight": straight,
                "turned": turned}
    if op == "mm":
        N, K = _spread(rng, 64, 8192), _spread(rng, 64, 8192, even=0.8, unit=16)  # widths are multiples of 16, mostly
        M = _spread(rng, 1, min(16384, int(2.5e11 / (N * K))))
        return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(["bf16", "bf16", "f32"]),
                "b_rows": rng.choice([128, 128, 1])}
    E = rng.choice([4, 8, 16, 32, 64])
    k = rng.randint(1, min(8, E))
    case = {"op": op, "k": k, "E": E, "dropped": rng.choice([0.0, 0.02])}
    if op == "experts_mm":
        N, K = _spread(rng, 64, 4096), _spread(rng, 64, 4096, even=0.8, unit=16)
        T = _spread(rng, 1, max(2, min(8192, 16384 // k)))
        return {**case, "T": T, "N": N, "K": K, "out": rng.choice(["bf16", "bf16", "f32"])}
    dtype = rng.choice(["bf16", "f32"] if op == "combine" else ["e4m3", "bf16", "f32"])
    N = _spread(rng, 64, 8192)
    T = _spread(rng, 1, min(16384, 16384 * 4096 * 4 // (N * k * (4 if dtype == "f32" else 2))))
    case |= {"T": T, "N": N, "dtype": dtype}
    return {**case, "backward": rng.random() < 0.5} if op == "combine" else case


# -- inputs ---------------------------------------------------------------------------------------------------------

def _groups(n):
    return -(-n // BLOCK)


def _widen(scale, n, dim):
    """A scale for each 128 along `dim`, as one for each of its n elements."""
    return scale.repeat_interleave(BLOCK, dim).narrow(dim, 0, n)


def _held(x, rows):
    """x [..., M, N] in 8 bits: (q, scale), with a scale for each block of rows x 128."""
    M, N = x.shape[-2:]
    high, wide = -M % rows, -N % BLOCK
    f = torch.nn.functional.pad(x.float(), (0, wide, 0, high))
    cut = f.view(*x.shape[:-2], (M + high) // rows, rows, (N + wide) // BLOCK, BLOCK)
    top = torch.clamp(cut.abs().amax((-3, -1), keepdim=True), min=SMALLEST)
    # x 448 / top: bfloat16 values on a tie stay on it
    q = ((cut.double() * QMAX / top.double()).float() if x.dtype == torch.bfloat16 else cut / (top / QMAX)).to(E4M3)
    return q.view(f.shape)[..., :M, :N].contiguous(), (top / QMAX)[..., 0, :, 0].contiguous()


def _choices(g, T, k, E, dropped):
    """k different experts a token, some experts chosen more often than others; dropped choices are -1."""
    liking = torch.randn(E, generator=g, device="cuda") + torch.randn(T, E, generator=g, device="cuda")
    experts = liking.topk(k, dim=1).indices
    experts[torch.rand(T, k, generator=g, device="cuda") < dropped] = -1
    return experts.int()


def _sorted(experts, E):
    """(offsets, slot): where each expert's rows begin, and the sorted row of each choice (-1: none)."""
    flat = experts.reshape(-1).long()
    hit = torch.arange(E, device=flat.device)[:, None] == flat
    rank = hit.int().cumsum(1)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = rank[:, -1].long().cumsum(0)
    valid = (flat >= 0) & (flat < E)
    at = flat.clamp(0, E - 1)
    slot = offsets[at] + rank.gather(0, at[None])[0] - 1
    return offsets.int(), torch.where(valid, slot, -1).int().view(experts.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    state = {**case}
    if op == "quant":
        dtype = DTYPES[case["dtype"]]
        x = normal(case["M"], case["N"], scale=0.02)
        x *= torch.exp(normal(case["M"], 1))  # rows of unlike size, as gradients have
        state["x"] = x.to(dtype)
        return state
    if op == "mm":
        M, N, K = case["M"], case["N"], case["K"]
        state["a"], state["a_scale"] = _held(normal(M, K, dtype=torch.bfloat16), 1)
        state["b"], state["b_scale"] = _held(normal(N, K, scale=K ** -0.5, dtype=torch.bfloat16), case["b_rows"])
        return state
    T, k, E, N = case["T"], case["k"], case["E"], case["N"]
    experts = _choices(g, T, k, E, case["dropped"])
    if op == "experts_mm":
        K = case["K"]
        state["offsets"], _ = _sorted(experts, E)
        state["places"] = state["offsets"].tolist()  # what the plain form cuts its products by
        state["a"], state["a_scale"] = _held(normal(T * k, K, dtype=torch.bfloat16), 1)
        held = [_held(normal(N, K, scale=K ** -0.5, dtype=torch.bfloat16), 128) for _ in range(E)]
        state["b"] = torch.stack([q for q, _ in held])
        state["b_scale"] = torch.stack([s for _, s in held])
        state["y"] = torch.zeros(T * k, N, dtype=DTYPES[case["out"]], device="cuda")
        return state
    dtype = DTYPES[case["dtype"]]
    if op == "dispatch":
        state["experts"] = experts
        x = normal(T, N, dtype=torch.bfloat16 if case["dtype"] == "e4m3" else dtype)
        state["x"], state["scale"] = _held(x, 1) if case["dtype"] == "e4m3" else (x, None)
        state["rows"] = torch.zeros(T * k, N, dtype=dtype, device="cuda")
        state["row_scale"] = None
        if state["scale"] is not None:
            state["row_scale"] = torch.zeros(T * k, _groups(N), device="cuda")
        return state
    _, state["slot"] = _sorted(experts, E)
    state["rows"] = normal(T * k, N, dtype=dtype)
    state["weights"] = normal(T, k).softmax(1)
    if case["backward"]:
        state["dy"] = normal(T, N, dtype=dtype)
        state["drows"] = torch.zeros(T * k, N, dtype=dtype, device="cuda")
    return state


# -- plain forms ----------------------------------------------------------------------------------------------------

def _plain_product(a, a_scale, b, b_scale):
    N, K = b.shape
    wide = _widen(b_scale, K, 1)
    if b_scale.shape[0] != N:
        wide = _widen(wide, N, 0)
    return (a.float() * _widen(a_scale, K, 1)) @ (b.float() * wide).T


def _plain_dispatch(s):
    offsets, slot = _sorted(s["experts"], s["E"])
    P = s["T"] * s["k"]
    source = torch.full((P + 1,), -1, dtype=torch.int64, device=slot.device)
    flat = slot.reshape(-1).long()
    source[torch.where(flat >= 0, flat, P)] = torch.arange(P, device=slot.device) // s["k"]
    source = source[:P]
    filled, at = (source >= 0)[:, None], source.clamp(min=0)

    def moved(x, into):
        same = torch.uint8 if x.dtype == E4M3 else x.dtype
        into.view(same).copy_(torch.where(filled, x.view(same)[at], into.view(same)))
        return into

    return {"offsets": offsets, "slot": slot, "rows": moved(s["x"], s["rows"]),
            "row_scale": None if s["scale"] is None else moved(s["scale"], s["row_scale"])}


def _plain_combine(s):
    slot, w, T, k = s["slot"].long(), s["weights"], s["T"], s["k"]
    filled, at = slot >= 0, slot.clamp(min=0)
    dtype = s["rows"].dtype
    if not s["backward"]:
        y = torch.zeros(T, s["N"], device=slot.device)
        for j in range(k):
            y += torch.where(filled[:, j, None], s["rows"][at[:, j]].float() * w[:, j, None], 0.0)
        return {"y": y.to(dtype)}
    dy, drows = s["dy"].float(), s["drows"]
    dweights = torch.empty(T, k, device=slot.device)
    spare = torch.cat([drows, drows[:1]])  # a last row for the choices that have none
    for j in range(k):
        dweights[:, j] = torch.where(filled[:, j], (dy * s["rows"][at[:, j]].float()).sum(1), 0.0)
        spare[torch.where(filled[:, j], at[:, j], T * k)] = (dy * w[:, j, None]).to(dtype)
    drows.copy_(spare[:-1])
    return {"drows": drows, "dweights": dweights}


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "quant":
        x, out = s["x"], {}
        if s["straight"]:
            out["q"], out["scale"] = _held(x, s["rows"])
        if s["turned"]:
            out["qt"], out["scale_t"] = _held(x.T, s["rows"])
        return out
    if op == "mm":
        return {"y": _plain_product(s["a"], s["a_scale"], s["b"], s["b_scale"]).to(DTYPES[s["out"]])}
    if op == "experts_mm":
        for e, (lo, hi) in enumerate(zip(s["places"], s["places"][1:])):
            if lo < hi:
                s["y"][lo:hi] = _plain_product(s["a"][lo:hi], s["a_scale"][lo:hi], s["b"][e], s["b_scale"][e])
        return {"y": s["y"]}
    return _plain_dispatch(s) if op == "dispatch" else _plain_combine(s)


def _run_own(s):
    from memory_bound_row_rmsnorm_gb300 import binding as qb
    op = s["op"]
    if op == "quant":
        q, scale, qt, scale_t = qb.quant_fwd(s["x"], block_rows=s["rows"], want_q=s["straight"], want_t=s["turned"])
        out = {"q": q, "scale": scale} if s["straight"] else {}
        return out | ({"qt": qt, "scale_t": scale_t} if s["turned"] else {})
    if op == "mm":
        return {"y": qb.scaled_mm_fwd(s["a"], s["a_scale"], s["b"], s["b_scale"], out_dtype=DTYPES[s["out"]])}
    if op == "experts_mm":
        return {"y": qb.scaled_mm_fwd(s["a"], s["a_scale"], s["b"], s["b_scale"], offsets=s["offsets"], out=s["y"])}
    if op == "dispatch":
        offsets, slot = qb.expert_sort(s["experts"], s["E"])
        if s["scale"] is None:
            rows, row_scale = qb.expert_gather_fwd(s["x"], slot, out=s["rows"]), None
        else:
            rows, row_scale = qb.expert_gather_fwd(s["x"], slot, scale=s["scale"], out=s["rows"],
                                                   out_scale=s["row_scale"])
        return {"offsets": offsets, "slot": slot, "rows": rows, "row_scale": row_scale}
    if not s["backward"]:
        return {"y": qb.expert_combine_fwd(s["rows"], s["slot"], s["weights"])}
    drows, dweights = qb.expert_combine_bwd(s["dy"], s["rows"], s["slot"], s["weights"], out=s["drows"])
    return {"drows": drows, "dweights": dweights}


# -- what a pass cannot do without -----------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4, "e4m3": 1}
    if op == "quant":
        M, N = case["M"], case["N"]
        ways = case["straight"] + case["turned"]
        scales = 0
        if case["straight"]:
            scales += -(-M // case["rows"]) * _groups(N)
        if case["turned"]:
            scales += -(-N // case["rows"]) * _groups(M)
        return {"bytes": M * N * (size[case["dtype"]] + ways) + 4 * scales, "flops": 3 * M * N * ways}
    if op == "mm":
        M, N, K = case["M"], case["N"], case["K"]
        G = _groups(K)
        return {"bytes": (M + N) * K + 4 * G * (M + -(-N // case["b_rows"])) + M * N * size[case["out"]],
                "flops": 2 * M * N * K}
    T, k, E, N = case["T"], case["k"], case["E"], case["N"]
    P = T * k
    if op == "experts_mm":
        K = case["K"]
        G, used = _groups(K), min(E, P)
        return {"bytes": P * K + 4 * G * P + used * (N * K + 4 * G * _groups(N)) + P * N * size[case["out"]],
                "flops": 2 * P * N * K}
    row = N * size[case["dtype"]]
    if op == "dispatch":
        row += 4 * _groups(N) if case["dtype"] == "e4m3" else 0
        return {"bytes": (T + P) * row + 8 * P + 4 * (E + 1), "flops": 0}
    if case["backward"]:
        return {"bytes": (T + 2 * P) * row + 12 * P, "flops": 3 * P * N}
    return {"bytes": (T + P) * row + 8 * P, "flops": 2 * P * N}


# -- the same from the definitions, in 64 bits ------------------------------------------------------------------------

def _exact_held(x, rows):
    M, N = x.shape
    d = x.double()
    q, scale = torch.empty_like(d), torch.empty(-(-M // rows), _groups(N), dtype=torch.float64, device=x.device)
    if rows == 1:
        for c, cols in enumerate(torch.split(d, BLOCK, dim=1)):
            scale[:, c] = cols.abs().amax(1).clamp_min(SMALLEST) / QMAX
            q[:, c * BLOCK:c * BLOCK + cols.shape[1]] = (cols / scale[:, c, None]).to(E4M3).double()
        return q, scale
    for r, band in enumerate(torch.split(d, rows, dim=0)):
        for c, tile in enumerate(torch.split(band, BLOCK, dim=1)):
            scale[r, c] = tile.abs().max().clamp_min(SMALLEST) / QMAX
            q[r * rows:r * rows + tile.shape[0], c * BLOCK:c * BLOCK + tile.shape[1]] = \
                (tile / scale[r, c]).to(E4M3).double()
    return q, scale


def _exact_product(a, a_scale, b, b_scale):
    (M, K), N = a.shape, b.shape[0]
    y = torch.zeros(M, N, dtype=torch.float64, device=a.device)
    row = torch.arange(N, device=a.device) if b_scale.shape[0] == N else torch.arange(N, device=a.device) // BLOCK
    for c in range(_groups(K)):
        part = torch.nn.functional.linear(a[:, c * BLOCK:(c + 1) * BLOCK].double(),
                                          b[:, c * BLOCK:(c + 1) * BLOCK].double())
        y.addcmul_(torch.mul(part, a_scale[:, c, None].double()), b_scale[row, c].double()[None, :])
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        if case["rows"] == 128 and _groups(case["M"]) * _groups(case["N"]) > 20000:
            return None
        out = {}
        if case["straight"]:
            out["q"], out["scale"] = _exact_held(s["x"], case["rows"])
        if case["turned"]:
            out["qt"], out["scale_t"] = _exact_held(s["x"].T.contiguous(), case["rows"])
        return out
    if op == "mm":
        return {"y": _exact_product(s["a"], s["a_scale"], s["b"], s["b_scale"])}
    if op == "experts_mm":
        pieces = [_exact_product(s["a"][lo:hi], s["a_scale"][lo:hi], s["b"][e], s["b_scale"][e])
                  for e, (lo, hi) in enumerate(zip(s["places"], s["places"][1:]))]
        rest = torch.zeros(case["T"] * case["k"] - s["places"][-1], case["N"], dtype=torch.float64, device="cuda")
        return {"y": torch.cat(pieces + [rest])}
    T, k, N = case["T"], case["k"], case["N"]
    if op == "dispatch":
        flat = s["experts"].reshape(-1).cpu()
        kept = torch.nonzero((flat >= 0) & (flat < case["E"]))[:, 0]
        order = kept[torch.argsort(flat[kept], stable=True)]  # the choices as their rows stand
        counts = torch.bincount(flat[kept].long(), minlength=case["E"])
        offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).int()
        slot = torch.full((T * k,), -1, dtype=torch.int32)
        slot[order] = torch.arange(len(order), dtype=torch.int32)
        tokens = (order // k).cuda()

        def moved(x):
            out = torch.zeros(T * k, x.shape[1], dtype=torch.float64, device="cuda")
            out[:len(order)] = x.double()[tokens]
            return out

        return {"offsets": offsets.cuda(), "slot": slot.view(T, k).cuda(), "rows": moved(s["x"]),
                "row_scale": None if s["scale"] is None else moved(s["scale"])}
    slot, w = s["slot"].long(), s["weights"].double()
    token, choice = torch.nonzero(slot >= 0, as_tuple=True)
    at = slot[token, choice]
    rows = s["rows"].double()
    if not case["backward"]:
        y = torch.zeros(T, N, dtype=torch.float64, device="cuda")
        for j in range(k):
            mine = choice == j
            y[token[mine]] += torch.einsum("p,pn->pn", w[token[mine], j], rows[at[mine]])
        return {"y": y}
    dy = s["dy"].double()
    drows, dweights = torch.zeros_like(rows), torch.zeros_like(w)
    drows[at] = torch.einsum("p,pn->pn", w[token, choice], dy[token])
    dweights[token, choice] = torch.einsum("pn,pn->p", dy[token], rows[at])
    return {"drows": drows, "dweights": dweights}
