"""Timing cases of the FP8 linear layer with 128-blocks, its training side and the router's balance loss.

Four operators:

  linear   y = bf16(deq(q(x)) deq(W)^T + bias): E4M3 operands, W with an fp32 scale for each 128 x 128 block, x
           quantized on the fly with a power-of-two scale for each 1 x 128 block;
  wgrad    dW = dY^T deq(X), db = column sums of dY, from X kept as an 8-bit activation checkpoint;
  train    one training step of the layer (forward, dX, dW, db) from a bf16 master weight;
  balance  the router's load-balance and z loss, the tokens of each expert, and the loss's gradient.

``run`` computes them from elementary torch operations in 32 bits where ``own`` is false, and through the package
where it is true.  ``exact`` computes them in 64 bits from their definitions.
"""

import math

import torch

own = False

BLOCK = 128


def listed():
    return [
        # one user's next token through a square projection
        {"name": "linear token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "bias": False},
        # a small decode batch; neither width is a multiple of the 128-block
        {"name": "linear decode ragged", "op": "linear", "M": 13, "N": 4000, "K": 2064, "bias": True},
        # one prompt of a thousand tokens
        {"name": "linear prompt", "op": "linear", "M": 1000, "N": 4096, "K": 4096, "bias": True},
        # prefill of a large batch through the widest projection the benchmark knows
        {"name": "linear prefill", "op": "linear", "M": 8192, "N": 28672, "K": 8192, "bias": False},
        # weight gradient of a small layer, 128-block checkpoint, fp32 main gradient
        {"name": "wgrad small", "op": "wgrad", "M": 512, "N": 1024, "K": 1024, "form": "b128", "out": "fp32"},
        # weight gradient from the MXFP8 layer's own quantized activations
        {"name": "wgrad mx", "op": "wgrad", "M": 4096, "N": 4096, "K": 4096, "form": "mx", "out": "fp32"},
        # many tokens, gradient in the weight's own type
        {"name": "wgrad long", "op": "wgrad", "M": 16384, "N": 5120, "K": 2048, "form": "b128", "out": "bf16"},
        # a training step whose sizes end inside a block everywhere
        {"name": "train ragged", "op": "train", "M": 1000, "N": 2064, "K": 2032},
        # a training step of a full micro-batch
        {"name": "train", "op": "train", "M": 8192, "N": 4096, "K": 4096},
        # a few tokens over few experts: nothing but latency
        {"name": "balance few", "op": "balance", "T": 16, "E": 8, "k": 2, "dtype": "fp32", "padded": False},
        # the routed layer's own size
        {"name": "balance", "op": "balance", "T": 4096, "E": 128, "k": 8, "dtype": "fp32", "padded": False},
        # a long padded batch, logits in bf16
        {"name": "balance padded", "op": "balance", "T": 50000, "E": 256, "k": 8, "dtype": "bf16", "padded": True},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(1, round(v / step)) * step


def draw(rng):
    op = rng.choice(["linear", "linear", "wgrad", "train", "balance"])
    if op == "linear":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 16384), "K": _log(rng, 128, 8192, 16),
                "bias": rng.random() < 0.5}
    if op == "wgrad":
        form = rng.choice(["b128", "mx"])
        return {"op": op, "M": _log(rng, 32, 16384), "N": _log(rng, 64, 8192, 8),
                "K": _log(rng, 256, 8192, 256 if form == "mx" else 16), "form": form,
                "out": rng.choice(["fp32", "bf16"])}
    if op == "train":
        return {"op": op, "M": _log(rng, 32, 8192), "N": _log(rng, 64, 8192, 16), "K": _log(rng, 128, 8192, 16)}
    E = rng.choice([4, 8, 16, 60, 64, 128, 160, 256])
    return {"op": op, "T": _log(rng, 1, 60000), "E": E, "k": rng.randint(1, min(8, E)),
            "dtype": rng.choice(["fp32", "bf16"]), "padded": rng.random() < 0.5}


def work(case):
    if case["op"] == "balance":
        T, E, w = case["T"], case["E"], 4 if case["dtype"] == "fp32" else 2
        return {"bytes": 2 * T * E * w + 4 * E + (T if case["padded"] else 0), "flops": 12 * T * E}
    M, N, K = case["M"], case["N"], case["K"]
    blocks = -(-N // BLOCK) * -(-K // BLOCK)
    if case["op"] == "linear":
        return {"bytes": 2 * M * K + N * K + 4 * blocks + 2 * M * N + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    if case["op"] == "wgrad":
        scales = -(-K // BLOCK) if case["form"] == "b128" else K // 32
        return {"bytes": 2 * M * N + M * K + M * scales + N * K * (4 if case["out"] == "fp32" else 2) + 4 * N,
                "flops": 2 * M * N * K}
    # x, w, bias, dy read; y, dx, dw, db written
    return {"bytes": 2 * (2 * M * K + 2 * N * K + 2 * M * N + 2 * N), "flops": 6 * M * N * K}


def _inputs(case, seed):
    """The tensors a call starts from, on the GPU, from the seed alone."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if case["op"] == "balance":
        T, E = case["T"], case["E"]
        # a router under training: some experts are liked better than others
        logits = normal(T, E) * 1.5 + normal(E)
        valid = None
        if case["padded"]:
            valid = torch.rand(T, generator=g, device=dev) < 0.8
        return {"logits": logits.to(torch.float32 if case["dtype"] == "fp32" else torch.bfloat16), "valid": valid}
    M, N, K = case["M"], case["N"], case["K"]
    # activations: channels of unlike size, a few outliers
    x = normal(M, K) * torch.exp(0.5 * normal(K))
    x = torch.where(torch.rand(M, K, generator=g, device=dev) < 1e-3, x * 20, x).to(torch.bfloat16)
    made = {"x": x}
    if case["op"] in ("wgrad", "train"):
        # gradients: small, rows (tokens) of unlike size
        made["dy"] = (normal(M, N) * 1e-3 * torch.exp(normal(M, 1))).to(torch.bfloat16)
    if case["op"] == "wgrad":
        return made
    made["bias"] = (0.1 * normal(N)).to(torch.bfloat16) if case["op"] == "train" or case["bias"] else None
    w = 0.02 * normal(N, K) * torch.exp(0.3 * normal(N, 1))
    if case["op"] == "train":
        made["w"] = w.to(torch.bfloat16)
        return made
    # a weight as a checkpoint holds it: E4M3 with an fp32 scale for each 128 x 128 block
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    tiles = torch.nn.functional.pad(w, (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(nb, BLOCK, kb, BLOCK)
    made["ws"] = tiles.abs().amax(dim=(1, 3)) / 448.0
    q = (tiles / made["ws"][:, None, :, None]).reshape(nb * BLOCK, kb * BLOCK)[:N, :K]
    made["wq"] = q.to(torch.float8_e4m3fn).view(torch.uint8).contiguous()
    return made


def prepare(case, seed):
    state = dict(case)
    state.update(_inputs(case, seed))
    if case["op"] == "linear":
        # a server lays its weight out once after loading
        state["weight"] = _api().prepare_weight_b128(state["wq"], state["ws"]) if own else None
    if case["op"] == "wgrad":
        # the forward pass left the activations as an 8-bit checkpoint
        if own:
            keep = _api().quantize_act_packed_b128 if case["form"] == "b128" else _api().quantize_act_packed
            state["kept"] = keep(state.pop("x"))
        else:
            state["kept"] = _quantize(state.pop("x").float(), BLOCK if case["form"] == "b128" else 32)
    return state


def run(state):
    return (_run_own if own else _run_plain)(state)


# ------------------------------------------------------------------------------------------------ the package's calls

def _api():
    from mxfp8_block_scaled_amd import api
    return api


_OUT = {"fp32": torch.float32, "bf16": torch.bfloat16}
COEF, Z_COEF = 1e-2, 1e-3


def _run_own(s):
    api = _api()
    if s["op"] == "linear":
        return api.linear(s["x"], s["weight"], s["bias"])
    if s["op"] == "wgrad":
        return api.linear_wgrad(s["dy"], s["kept"], dtype=_OUT[s["out"]], bias_grad=True)
    if s["op"] == "train":
        x, w, b = (s[k].detach().requires_grad_() for k in ("x", "w", "bias"))
        y = api.linear_b128(x, w, b)
        return (y.detach(),) + torch.autograd.grad(y, (x, w, b), s["dy"])
    loss, counts, used = api.moe_balance(s["logits"], s["k"], valid=s["valid"], coef=COEF, z_coef=Z_COEF)
    grad = api.moe_balance_backward(s["logits"], s["k"], counts, used, valid=s["valid"], coef=COEF, z_coef=Z_COEF)
    return loss, counts, used, grad


# ------------------------------------------------------------------------------------------------ the plain forms

def _quantize(x, block, rows=1):
    """fp32 x -> (E4M3 values, fp32 power-of-two scales spread to x's shape).  block 128: the smallest power of two
    under which nothing leaves the E4M3 range; block 32: the MX rule, whose largest elements saturate.  ``rows``:
    the rows that share a scale (128 for a weight)."""
    R, K = x.shape
    pr, pk = -(-R // rows) * rows, -(-K // block) * block
    t = torch.nn.functional.pad(x, (0, pk - K, 0, pr - R)).view(pr // rows, rows, pk // block, block)
    m, e = torch.frexp(t.abs().amax(dim=(1, 3), keepdim=True))
    j = e - 9
    if block == BLOCK:
        j = j + (m > 0.875).to(j.dtype)
    scale = torch.where(m > 0, torch.exp2(j.float()), torch.ones_like(m))
    q = (t / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    spread = scale.expand(t.shape).reshape(pr, pk)[:R, :K]
    return q.reshape(pr, pk)[:R, :K], spread


def _dequantized(x, block=BLOCK, rows=1):
    q, s = _quantize(x, block, rows)
    return q.float() * s


def _run_plain(s):
    if s["op"] == "linear":
        N, K = s["N"], s["K"]
        at_n = torch.arange(N, device=s["x"].device) // BLOCK
        at_k = torch.arange(K, device=s["x"].device) // BLOCK
        w = s["wq"].view(torch.float8_e4m3fn).float() * s["ws"][at_n][:, at_k]
        y = _dequantized(s["x"].float()) @ w.t()
        return (y if s["bias"] is None else y + s["bias"].float()).to(torch.bfloat16)
    if s["op"] == "wgrad":
        q, scale = s["kept"]
        dy = s["dy"].float()
        return (dy.t() @ (q.float() * scale)).to(_OUT[s["out"]]), dy.sum(0)
    if s["op"] == "train":
        x, w, dy = _dequantized(s["x"].float()), _dequantized(s["w"].float(), rows=BLOCK), s["dy"].float()
        y = x @ w.t() + s["bias"].float()
        dx = _dequantized(dy) @ w
        return tuple(t.to(torch.bfloat16) for t in (y, dx, dy.t() @ x, dy.sum(0)))
    logits, E, k = s["logits"].float(), s["E"], s["k"]
    top = logits.amax(1, keepdim=True)
    live = top[:, 0] > float("-inf")
    if s["valid"] is not None:
        live = live & s["valid"]
    z = torch.where(live[:, None], logits - top, torch.zeros_like(logits))
    ez = torch.exp(z)
    total = ez.sum(1, keepdim=True)
    p = ez / total * live[:, None]
    lse = torch.where(live, top[:, 0] + torch.log(total[:, 0]), torch.zeros_like(total[:, 0]))
    # equal logits: the lower expert first
    ids = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    hit = torch.zeros_like(logits).scatter_(1, ids, 1.0) * live[:, None]
    counts = hit.sum(0)
    used = live.sum()
    n = used.float().clamp(min=1)
    a, b = COEF * E / (k * n * n), Z_COEF / n
    loss = a * (counts * p.sum(0)).sum() + b * (lse * lse).sum()
    inner = (p * counts).sum(1, keepdim=True)
    grad = a * p * (counts - inner) + 2 * b * lse[:, None] * p
    return loss, counts.to(torch.int32), used.to(torch.int32).reshape(1), grad.to(s["logits"].dtype)


# ------------------------------------------------------------------------------------------------ in 64 bits

def _grid64(x, block, rows=1):
    """What x is worth after 8-bit quantization, from the definition of the E4M3 grid (3 mantissa bits, least
    exponent -6, largest value 448, ties to even), in 64 bits."""
    x = x.double()
    R, K = x.shape
    out = torch.empty_like(x)
    for k0 in range(0, K, block):
        part = x[:, k0:k0 + block]
        top = part.abs().amax(1)
        if rows > 1:
            top = torch.cat([top[r:r + rows].amax().expand(min(rows, R - r)) for r in range(0, R, rows)])
        one = torch.ones_like(top)
        floor = torch.floor(torch.log2(torch.where(top > 0, top, one)))
        e = floor - 8
        if block == BLOCK:
            e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
        scale = torch.where(top > 0, torch.exp2(e), one)[:, None]
        v = part / scale
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        out[:, k0:k0 + block] = (torch.round(v / step) * step).clamp(-448, 448) * scale
    return out


def exact(case, seed):
    made = _inputs(case, seed)
    if case["op"] == "linear":
        w = made["wq"].view(torch.float8_e4m3fn).double()
        for i in range(made["ws"].shape[0]):
            for j in range(made["ws"].shape[1]):
                w[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= made["ws"][i, j].double()
        y = _grid64(made["x"], BLOCK) @ w.t()
        return y if made["bias"] is None else y + made["bias"].double()
    if case["op"] == "wgrad":
        dy = made["dy"].double()
        return dy.t() @ _grid64(made["x"], BLOCK if case["form"] == "b128" else 32), dy.sum(0)
    if case["op"] == "train":
        x, w, dy = _grid64(made["x"], BLOCK), _grid64(made["w"], BLOCK, BLOCK), made["dy"].double()
        return x @ w.t() + made["bias"].double(), _grid64(made["dy"], BLOCK) @ w, dy.t() @ x, dy.sum(0)
    logits, k = made["logits"].double(), case["k"]
    E = logits.shape[1]
    live = torch.isfinite(logits).any(1)
    if made["valid"] is not None:
        live &= made["valid"]
    rows = logits[live]
    n = max(rows.shape[0], 1)
    prob, lse = torch.softmax(rows, 1), torch.logsumexp(rows, 1)
    left, counts = rows.clone(), torch.zeros(E, dtype=torch.float64, device=rows.device)
    index = torch.arange(E, device=rows.device).expand(rows.shape)
    for _ in range(k if rows.shape[0] else 0):
        best = left.amax(1, keepdim=True)
        first = torch.where(left == best, index, torch.full_like(index, E)).amin(1)
        counts += torch.bincount(first, minlength=E)
        left.scatter_(1, first[:, None], float("-inf"))
    a, b = COEF * E / (k * float(n) ** 2), Z_COEF / n
    loss = a * (counts * prob.sum(0)).sum() + b * (lse ** 2).sum()
    grad = torch.zeros_like(logits)
    grad[live] = prob * (a * (counts - (prob * counts).sum(1, keepdim=True)) + 2 * b * lse[:, None])
    return loss, counts, torch.tensor([rows.shape[0]], dtype=torch.float64), grad
