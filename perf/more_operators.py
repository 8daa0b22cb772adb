"""Timing cases of the MXFP4 linear layer, of tokens sorted by expert and back, and of the experts' MXFP4 products.

Three operators:

  linear   y = bf16(deq(q(x)) deq(W)^T + bias): both operands E2M1 with a power-of-two scale for each 32 elements
           along K, x quantized on the fly;
  tokens   the rows of a routed batch put in the order of their experts, and the experts' rows put back, weighted and
           added up; with the gradients of both where a training step asks for them;
  experts  that linear layer on the sorted rows, each with its own expert's weight, from the sorted rows themselves
           (the second projection) or from the tokens they belong to (the first).

``run`` computes them from elementary torch operations in 32 bits where ``own`` is false, and through the package
where it is true.  ``exact`` computes them in 64 bits from their definitions.
"""

import math

import torch

own = False

BLOCK = 32


def listed():
    return [
        # one user's next token through a square projection
        {"name": "linear token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "bias": False},
        # a small decode batch through a projection that is no multiple of the weight's padding
        {"name": "linear decode ragged", "op": "linear", "M": 13, "N": 4000, "K": 2048, "bias": True},
        # one prompt of a thousand tokens
        {"name": "linear prompt", "op": "linear", "M": 1000, "N": 4096, "K": 4096, "bias": True},
        # prefill of a large batch through the widest projection the benchmark knows
        {"name": "linear prefill", "op": "linear", "M": 8192, "N": 28672, "K": 8192, "bias": False},
        # a few tokens over few experts: nothing but latency
        {"name": "tokens few", "op": "tokens", "T": 16, "E": 8, "k": 2, "H": 2048, "dtype": "bf16", "drop": 0.0,
         "train": False},
        # the routed layer's own size, in a training step
        {"name": "tokens step", "op": "tokens", "T": 4096, "E": 128, "k": 8, "H": 2048, "dtype": "bf16", "drop": 0.0,
         "train": True},
        # one rank's share of the experts, sizes that divide by nothing, fp32 rows
        {"name": "tokens shard ragged", "op": "tokens", "T": 10007, "E": 60, "k": 4, "H": 1003, "dtype": "fp32",
         "drop": 0.5, "train": False},
        # a long batch over few wide experts, in a training step
        {"name": "tokens long", "op": "tokens", "T": 32768, "E": 8, "k": 2, "H": 4096, "dtype": "bf16", "drop": 0.0,
         "train": True},
        # one token through its experts' first projection
        {"name": "experts token", "op": "experts", "T": 1, "E": 128, "k": 8, "N": 1536, "K": 2048, "drop": 0.0,
         "gather": True},
        # a decode batch through the second projection of one rank's share of the experts
        {"name": "experts decode shard", "op": "experts", "T": 48, "E": 64, "k": 8, "N": 2048, "K": 768, "drop": 0.5,
         "gather": False},
        # the routed layer's own size: first and second projection
        {"name": "experts first", "op": "experts", "T": 4096, "E": 128, "k": 8, "N": 1536, "K": 2048, "drop": 0.0,
         "gather": True},
        {"name": "experts second", "op": "experts", "T": 4096, "E": 128, "k": 8, "N": 2048, "K": 768, "drop": 0.0,
         "gather": False},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(1, round(v / step)) * step


def draw(rng):
    op = rng.choice(["linear", "tokens", "experts"])
    if op == "linear":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 16384), "K": _log(rng, 256, 8192, 256),
                "bias": rng.random() < 0.5}
    E = rng.choice([4, 8, 16, 60, 64, 128, 160, 256])
    k = rng.randint(1, min(8, E))
    drop = rng.choice([0.0, 0.0, 0.5])
    if op == "tokens":
        T = _log(rng, 1, 32768)
        H = _log(rng, 64, min(8192, 2 ** 28 // (T * k)))
        return {"op": op, "T": T, "E": E, "k": k, "H": H, "dtype": rng.choice(["bf16", "bf16", "fp32"]), "drop": drop,
                "train": rng.random() < 0.5}
    N = _log(rng, 64, 4096)
    K = _log(rng, 256, min(4096, 2 ** 29 // (E * N)), 256)
    return {"op": op, "T": _log(rng, 1, 8192), "E": E, "k": k, "N": N, "K": K, "drop": drop,
            "gather": rng.random() < 0.5}


def work(case):
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + N * K // 2 + N * K // BLOCK + 2 * M * N + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    T, k = case["T"], case["k"]
    R = T * k
    kept = R * (1.0 - case["drop"])
    if case["op"] == "tokens":
        H, w = case["H"], 4 if case["dtype"] == "fp32" else 2
        # ids, weights; x in, sorted rows out; the experts' rows in, y out
        b = 8 * R + 4 * (2 * R + case["E"] + 1) + w * H * (T + R + kept + T)
        if case["train"]:
            # gradients of the sorted rows and of y in, of x and of the experts' rows and the weights out
            b += w * H * (kept + T + T + R) + 4 * R
        return {"bytes": int(b), "flops": int(kept * H * (6 if case["train"] else 2))}
    N, K = case["N"], case["K"]
    touched = min(case["E"], max(1.0, kept))
    rows = T if case["gather"] else kept
    return {"bytes": int(2 * rows * K + touched * N * (K // 2 + K // BLOCK) + 2 * R * N),
            "flops": int(2 * kept * N * K)}


_DTYPE = {"fp32": torch.float32, "bf16": torch.bfloat16}


def _inputs(case, seed):
    """The tensors a call starts from, on the GPU, from the seed alone."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    def activations(rows, width):
        # channels of unlike size, a few outliers
        x = normal(rows, width) * torch.exp(0.5 * normal(width))
        return torch.where(uniform(rows, width) < 1e-3, x * 20, x)

    if case["op"] == "linear":
        N, K = case["N"], case["K"]
        made = {"x": activations(case["M"], K).to(torch.bfloat16)}
        made["bias"] = (0.1 * normal(N)).to(torch.bfloat16) if case["bias"] else None
        made["wq"], made["ws"] = _codes(0.02 * normal(N, K) * torch.exp(0.3 * normal(N, 1)))
        return made
    T, E, k = case["T"], case["E"], case["k"]
    # a router under training: some experts are liked better than others
    score = normal(T, E) * 1.5 + normal(E)
    top, ids = torch.sort(score, dim=1, descending=True)
    weights = torch.softmax(top[:, :k], dim=1)
    ids = ids[:, :k].to(torch.int32)
    # experts of other ranks: no place here
    ids = torch.where(uniform(T, k) < case["drop"], torch.full_like(ids, -1), ids).contiguous()
    made = {"ids": ids}
    if case["op"] == "tokens":
        H, t = case["H"], _DTYPE[case["dtype"]]
        made["weights"] = weights.contiguous()
        made["x"] = activations(T, H).to(t)
        made["ys"] = normal(T * k, H).to(t)
        if case["train"]:
            made["dxs"] = (normal(T * k, H) * 1e-3).to(t)
            made["dy"] = (normal(T, H) * 1e-3 * torch.exp(normal(T, 1))).to(t)
        return made
    N, K = case["N"], case["K"]
    made["x"] = activations(T if case["gather"] else T * k, K).to(torch.bfloat16)
    wq, ws = _codes(0.02 * normal(E * N, K) * torch.exp(0.3 * normal(E * N, 1)))
    made["wq"], made["ws"] = wq.view(E, N, K // 2), ws.view(E, N, K // BLOCK)
    return made


def prepare(case, seed):
    state = dict(case)
    state.update(_inputs(case, seed))
    if case["op"] == "linear":
        # a server lays its weight out once after loading
        state["weight"] = _api().prepare_weight_fp4(state.pop("wq"), state.pop("ws")) if own else None
    if case["op"] == "experts":
        # the layer has sorted its tokens before its first product
        if own:
            state["weight"] = _api().moe_prepare_experts_fp4(state.pop("wq"), state.pop("ws"))
            state["order"] = _api().moe_sort(state["ids"], case["E"])
        else:
            offsets, _, slots = _sort(state["ids"], case["E"])
            state["offsets"], state["slots"] = offsets.tolist(), slots
    return state


def run(state):
    return (_run_own if own else _run_plain)(state)


# ------------------------------------------------------------------------------------------------ the package's calls

def _api():
    from mxfp8_block_scaled_amd import api
    return api


def _run_own(s):
    api = _api()
    if s["op"] == "linear":
        return api.linear_w4a4(s["x"], s["weight"], s["bias"])
    if s["op"] == "experts":
        return api.moe_linear_w4a4(s["x"], s["weight"], s["order"], gather=s["gather"])
    if not s["train"]:
        order = api.moe_sort(s["ids"], s["E"])
        return (order.offsets, order.rows, api.moe_permute(s["x"], order),
                api.moe_unpermute(s["ys"], order, s["weights"]))
    x, ys, weights = (s[n].detach().requires_grad_() for n in ("x", "ys", "weights"))
    order = api.moe_sort(s["ids"], s["E"])
    xs = api.moe_permute(x, order)
    y = api.moe_unpermute(ys, order, weights)
    return (order.offsets, order.rows, xs.detach(), y.detach()) + \
        torch.autograd.grad((xs, y), (x, ys, weights), (s["dxs"], s["dy"]))


# ------------------------------------------------------------------------------------------------ the plain forms

_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _round4(t):
    """fp32 values over their scale -> E2M1 codes: the nearest magnitude, ties to the even code, 6 at most."""
    a = t.abs()
    code = (a > 0.25).to(torch.uint8)
    for i, border in enumerate((0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (a >= border) if i % 2 == 0 else (a > border)
    return code | (torch.signbit(t).to(torch.uint8) << 3)


def _scaled4(x):
    """fp32 [R, K] -> (E2M1 codes [R, K / 32, 32], the blocks' exponents [R, K / 32, 1]); a block of zeros has
    exponent -127."""
    t = x.view(x.shape[0], -1, BLOCK)
    m, e = torch.frexp(t.abs().amax(dim=2, keepdim=True))
    e = torch.where(m > 0, e - 3, torch.full_like(e, -127)).clamp(min=-127)
    return _round4(torch.ldexp(t, -e)), e


def _codes(x):
    """fp32 [R, K] -> MXFP4 as a checkpoint holds it: two codes a byte [R, K / 2], a scale byte per block."""
    parts = [_scaled4(p) for p in x.split(1 << 16)]
    q = torch.cat([p.view(p.shape[0], -1) for p, _ in parts])
    s = torch.cat([(e.view(e.shape[0], -1) + 127).to(torch.uint8) for _, e in parts])
    return (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous(), s.contiguous()


def _values(code):
    table = torch.tensor(_MAGNITUDES + tuple(-v for v in _MAGNITUDES), device=code.device)
    return table[code.int()]


def _dequantized(x):
    code, e = _scaled4(x)
    return torch.ldexp(_values(code), e).view(x.shape)


def _weight(wq, ws):
    """Codes and scale bytes [R, K / 2], [R, K / 32] -> fp32 [R, K]."""
    code = torch.stack([wq & 15, wq >> 4], dim=2).view(wq.shape[0], -1, BLOCK)
    return torch.ldexp(_values(code), (ws.int() - 127)[:, :, None]).view(wq.shape[0], -1)


def _sort(ids, E):
    """(offsets [E + 1], rows [T, k]: the sorted row of each of a token's slots, slots [T k]: the slot of each row),
    the slots of one expert in their order, those without an expert here last."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    slots = torch.sort(key, stable=True).indices
    rows = torch.empty_like(slots)
    rows[slots] = torch.arange(slots.numel(), device=slots.device)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=slots.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cumsum(counts, 0) - counts
    return offsets.to(torch.int32), rows.view(ids.shape).to(torch.int32), slots


def _run_plain(s):
    if s["op"] == "linear":
        y = _dequantized(s["x"].float()) @ _weight(s["wq"], s["ws"]).t()
        return (y if s["bias"] is None else y + s["bias"].float()).to(torch.bfloat16)
    if s["op"] == "experts":
        x = _dequantized(s["x"].float())
        if s["gather"]:
            x = x[s["slots"] // s["k"]]
        y = torch.zeros(s["T"] * s["k"], s["N"], device=x.device)
        for e in range(s["E"]):
            a, b = s["offsets"][e], s["offsets"][e + 1]
            if b > a:
                y[a:b] = x[a:b] @ _weight(s["wq"][e], s["ws"][e]).t()
        return y.to(torch.bfloat16)
    T, k, t = s["T"], s["k"], s["x"].dtype
    offsets, rows, slots = _sort(s["ids"], s["E"])
    here = rows < offsets[-1]
    kept = here.reshape(-1)[slots][:, None]
    token = slots // k
    at = rows.reshape(-1).long()
    xs = torch.where(kept, s["x"].float()[token], 0.0)
    ys = torch.where(kept, s["ys"].float(), 0.0)
    w = torch.where(here, s["weights"], 0.0)
    by_slot = ys[at].view(T, k, -1)
    y = (by_slot * w[:, :, None]).sum(1)
    out = (offsets, rows, xs.to(t), y.to(t))
    if not s["train"]:
        return out
    dy = s["dy"].float()
    dx = torch.where(kept, s["dxs"].float(), 0.0)[at].view(T, k, -1).sum(1)
    dys = w.reshape(-1)[slots][:, None] * dy[token]
    dw = (by_slot * dy[:, None, :]).sum(2)
    return out + (dx.to(t), dys.to(t), dw)


# ------------------------------------------------------------------------------------------------ in 64 bits

def _grid64(x):
    """What x is worth after 4-bit quantization, from the definition of the E2M1 grid (1 mantissa bit, least
    exponent 0, largest value 6, ties to even), in 64 bits."""
    t = x.double().unflatten(-1, (-1, BLOCK))
    top = t.abs().amax(-1, keepdim=True)
    one = torch.ones_like(top)
    scale = torch.where(top > 0, torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, one))) - 2), one)
    v = t / scale
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=1.0))) - 1)
    return ((torch.round(v / step) * step).clamp(-6, 6) * scale).flatten(-2)


def _weight64(wq, ws):
    code = torch.stack([wq.remainder(16), wq.div(16, rounding_mode="floor")], dim=-1).flatten(-2).double()
    sign = torch.where(code >= 8, -1.0, 1.0)
    code = code.remainder(8)
    exponent = (code / 2).floor().clamp(min=1) - 1
    mantissa = code.remainder(2) / 2 + (code >= 2)
    return sign * mantissa * torch.exp2(exponent) * torch.exp2(ws.double() - 127).repeat_interleave(BLOCK, -1)


def exact(case, seed):
    made = _inputs(case, seed)
    if case["op"] == "linear":
        y = _grid64(made["x"]) @ _weight64(made["wq"], made["ws"]).t()
        return y if made["bias"] is None else y + made["bias"].double()
    T, E, k = case["T"], case["E"], case["k"]
    ids = made["ids"].reshape(-1).long()
    # the slots expert by expert, then those of no expert here
    groups = [torch.nonzero(ids == e)[:, 0] for e in range(E)]
    last = torch.nonzero((ids < 0) | (ids >= E))[:, 0]
    slots = torch.cat(groups + [last])
    ends = [0]
    for group in groups:
        ends.append(ends[-1] + group.numel())
    if case["op"] == "experts":
        x = _grid64(made["x"])
        y = torch.zeros(T * k, case["N"], dtype=torch.float64, device=x.device)
        for e in range(E):
            rows = slots[ends[e]:ends[e + 1]]
            if rows.numel():
                a = x[rows // k] if case["gather"] else x[ends[e]:ends[e + 1]]
                y[ends[e]:ends[e + 1]] = a @ _weight64(made["wq"][e], made["ws"][e]).t()
        return y
    offsets = torch.tensor(ends, dtype=torch.float64)
    rows = torch.argsort(slots).view(T, k).double()
    n, H = ends[-1], case["H"]
    token, mine = slots[:n] // k, slots[:n]
    x, ys = made["x"].double(), made["ys"].double()[:n]
    w = made["weights"].double().reshape(-1)[mine]
    xs = torch.zeros(T * k, H, dtype=torch.float64, device=x.device)
    xs[:n] = x[token]
    y = torch.zeros_like(x).index_add_(0, token, w[:, None] * ys)
    if not case["train"]:
        return offsets, rows, xs, y
    dy = made["dy"].double()
    dx = torch.zeros_like(x).index_add_(0, token, made["dxs"].double()[:n])
    dys = torch.zeros_like(xs)
    dys[:n] = w[:, None] * dy[token]
    dw = torch.zeros(T * k, dtype=torch.float64, device=x.device)
    dw[mine] = (ys * dy[token]).sum(1)
    return offsets, rows, xs, y, dx, dys, dw.view(T, k)
