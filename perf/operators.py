"""Measured cases of the 8-bit operators: the coding of activations and weights (E4M3 codes, one power-of-two scale
per block of 128), the matrix product of two coded operands, and the backward pass of the weightless linear from a
coded activation checkpoint.

`own` chooses between the plain torch form and the library's kernels.  Shapes are those of the synthetic Gemma-3-1B
and Gemma-4-31B bundles, plus ragged ones.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128


def listed():
    return [
        # the checkpoint of a single decoded token: the smallest call there is
        {"name": "encode_act_token", "op": "encode_act", "T": 1, "K": 1152},
        # the MLP hidden state of a long training batch (down's input)
        {"name": "encode_act_mlp", "op": "encode_act", "T": 8192, "K": 21504},
        # coding a 31B gate block at load time
        {"name": "encode_weight_gate", "op": "encode_weight", "N": 21504, "K": 5376},
        # one token through a small projection (1B gate): launch latency
        {"name": "product_token_1b", "op": "product", "T": 1, "N": 4096, "K": 1152},
        # one token through the 31B gate: weight streaming
        {"name": "product_token_31b", "op": "product", "T": 1, "N": 21504, "K": 5376},
        # a decode batch of 16 through the 31B down: long K, few rows
        {"name": "product_batch16_down", "op": "product", "T": 16, "N": 5376, "K": 21504},
        # ragged sizes: no dimension a multiple of a tile
        {"name": "product_ragged", "op": "product", "T": 333, "N": 1001, "K": 1160},
        # a prompt of 2048 through the 31B gate: matrix-core bound
        {"name": "product_prompt_31b", "op": "product", "T": 2048, "N": 21504, "K": 5376},
        # a short ragged sequence through an odd-sized projection, every gradient
        {"name": "backward_ragged", "op": "backward", "T": 77, "rows": "1001", "K": 712, "r": 20, "dw0": True},
        # 1B training, the stacked q|k|v call
        {"name": "backward_qkv_1b", "op": "backward", "T": 2048, "rows": "1024,256,256", "K": 1152, "r": 64, "dw0": True},
        # 31B o projection at a large rank with the shared block frozen
        {"name": "backward_o_31b", "op": "backward", "T": 512, "rows": "5376", "K": 8192, "r": 1024, "dw0": False},
        # 31B gate|up with the shared block trained: the largest case
        {"name": "backward_gate_up_31b", "op": "backward", "T": 2048, "rows": "21504,21504", "K": 5376, "r": 256, "dw0": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["encode_act", "encode_weight", "product", "product", "product", "backward", "backward", "backward"])
    k = 8 * _log(rng, 8, 2688)                      # 64 .. 21504, the library's multiple of 8
    if rng.random() < 0.5:
        k = max(64, k // 128 * 128)                 # half of them whole blocks
    if op == "encode_act":
        return {"op": op, "T": _log(rng, 1, 8192), "K": k}
    if op == "encode_weight":
        return {"op": op, "N": _log(rng, 1, 21504), "K": min(k, 8192)}
    if op == "product":
        n = _log(rng, 32, 21504)
        t = rng.choice([1, rng.randint(2, 16), _log(rng, 17, 4096)])
        while t * n * k > 2048 * 21504 * 5376:
            t = max(1, t // 2)
        return {"op": op, "T": t, "N": n, "K": k}
    k = min(k, 8192)
    kids = rng.choice([1, 1, 2, 3])
    rows = [_log(rng, 40, 8192) for _ in range(kids)]
    if kids == 2:
        rows[1] = rows[0]
    t = _log(rng, 1, 4096)
    while t * sum(rows) * k > 2048 * 43008 * 2688:
        t = max(1, t // 2)
    r = min([_log(rng, 4, 512), k] + rows)
    return {"op": op, "T": t, "rows": ",".join(map(str, rows)), "K": k, "r": r, "dw0": rng.random() < 0.5}


def _gen(seed):
    return torch.Generator(DEV).manual_seed(int(seed) * 7919 + 13)


def _normal(g, *shape, std=1.0):
    return torch.empty(shape, dtype=torch.float32, device=DEV).normal_(0.0, std, generator=g)


def _activations(g, t, k):
    """Hidden states: unit normals with a few channels that run far hotter than the rest."""
    x = _normal(g, t, k)
    hot = torch.randint(0, k, (max(1, k // 256),), generator=g, device=DEV)
    x[:, hot] *= 24.0
    return x.to(torch.bfloat16)


def _rows(case):
    return [int(n) for n in case["rows"].split(",")]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "encode_act":
        return {"op": op, "x": _activations(g, case["T"], case["K"])}
    if op == "encode_weight":
        return {"op": op, "w": _normal(g, case["N"], case["K"], std=case["K"] ** -0.5).to(torch.bfloat16)}
    if op == "product":
        w = _normal(g, case["N"], case["K"], std=case["K"] ** -0.5).to(torch.bfloat16)
        x = _activations(g, case["T"], case["K"])
        if own:
            from weight_shared_rank_amd import binding
            return {"op": op, "x": x, "w": binding.encode_weight(w)}
        return {"op": op, "x": x, "w": _encode(w, BLOCK)}
    rows, k, r, t = _rows(case), case["K"], case["r"], case["T"]
    n = sum(rows)
    st = {"op": op, "rows": rows, "dw0": case["dw0"],
          "dy": _normal(g, t, n, std=t ** -0.5).to(torch.bfloat16),
          "w0": [_normal(g, m, k, std=k ** -0.5).to(torch.bfloat16) for m in rows],
          "s": [1.0 + 0.05 * _normal(g, m) for m in rows],
          "u": [_normal(g, m, r, std=0.02).to(torch.bfloat16) for m in rows],
          "v": [_normal(g, k, r, std=0.02).to(torch.bfloat16) for m in rows]}
    x = _activations(g, t, k)
    if own:
        from weight_shared_rank_amd import binding
        fams = {1: ("o",), 2: ("gate", "up"), 3: ("q", "k", "v")}[len(rows)]
        spec = binding.make_spec(1, 1, {(0, f): (m, k) for f, m in zip(fams, rows)}, {(0, f): r for f in fams})
        src = [(kind, 0, 0, f, st[kind][i]) for i, f in enumerate(fams) for kind in ("w0", "s", "u", "v")]
        st["bundle"] = binding.ThetaBundle(spec, src, device=DEV)
        st["x"] = binding.encode_act(x)
        st["w0"] = st["u"] = st["v"] = None
    else:
        st["x"] = _encode(x, 1)
    return st


# ---- plain form -------------------------------------------------------------------------------------------------

def _encode(x, tall):
    """E4M3 codes and E8M0 scale bytes of `tall` x 128 blocks: e is the smallest exponent with max|x| <= 448 * 2^e
    (at least -118; 0 for a block of zeros), a code is E4M3(x * 2^-e)."""
    m, k = x.shape
    mb, kb = -(-m // tall), -(-k // BLOCK)
    f = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - k, 0, mb * tall - m))
    f = f.view(mb, tall, kb, BLOCK)
    amax = f.abs().amax(dim=(1, 3))
    frac, ex = torch.frexp(amax)
    e = torch.where(frac <= 0.875, ex - 9, ex - 8).clamp_min(-118)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    code = torch.ldexp(f, -e[:, None, :, None]).to(torch.float8_e4m3fn)
    return code.view(mb * tall, kb * BLOCK)[:m, :k], (e + 127).to(torch.uint8)


def _values(coded, tall, dtype=torch.float32):
    """The numbers that coded blocks stand for."""
    code, scale = coded
    m, k = code.shape
    factor = torch.exp2(scale.to(dtype) - 127.0).repeat_interleave(tall, 0)[:m].repeat_interleave(BLOCK, 1)[:, :k]
    return code.to(dtype) * factor


def _plain(state):
    op = state["op"]
    if op == "encode_act":
        return _encode(state["x"], 1)
    if op == "encode_weight":
        return _encode(state["w"], BLOCK)
    if op == "product":
        x = _values(_encode(state["x"], 1), 1)
        return torch.matmul(x, _values(state["w"], BLOCK).t()).to(torch.bfloat16)
    x, dy = _values(state["x"], 1), state["dy"].float()
    out = {"ds": [], "du": [], "dv": []}
    dx, dw0, at = 0.0, [], 0
    for m, w0, s, u, v in zip(state["rows"], state["w0"], state["s"], state["u"], state["v"]):
        d, w0, u, v = dy[:, at:at + m], w0.float(), u.float(), v.float()
        at += m
        low = torch.matmul(d, u)
        dx = dx + torch.matmul(d * s, w0) + torch.matmul(low, v.t())
        full = torch.matmul(d.t(), x)
        out["ds"].append((full * w0).sum(1))
        if state["dw0"]:
            dw0.append(full * s[:, None])
        out["du"].append(torch.matmul(d.t(), torch.matmul(x, v)).to(torch.bfloat16))
        out["dv"].append(torch.matmul(x.t(), low).to(torch.bfloat16))
    out["ds"] = torch.cat(out["ds"])
    out["dx"] = dx.to(torch.bfloat16)
    if state["dw0"]:
        out["dw0"] = torch.cat(dw0)
    return out


# ---- the library's kernels --------------------------------------------------------------------------------------

def _own(state):
    from weight_shared_rank_amd import binding
    op = state["op"]
    if op == "encode_act":
        c = binding.encode_act(state["x"])
        return c.codes, c.scales
    if op == "encode_weight":
        c = binding.encode_weight(state["w"])
        return c.codes, c.scales
    if op == "product":
        return binding.coded_linear(state["w"], state["x"])
    b, rows = state["bundle"], state["rows"]
    want = ("dx", "ds", "du", "dv") + (("dw0",) if state["dw0"] else ())
    if len(rows) == 1:
        g = b.linear_backward(0, "o", state["x"], state["dy"], want=want)
        du, dv = [g.du], [g.dv]
    else:
        g = b.stacked_backward(0, "gate_up" if len(rows) == 2 else "qkv", state["x"], state["dy"], want=want)
        du, dv = list(g.du), list(g.dv)
    out = {"ds": g.ds, "du": du, "dv": dv, "dx": g.dx}
    if state["dw0"]:
        out["dw0"] = g.dw0
    return out


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, k = case["op"], case["K"]
    kb = -(-k // BLOCK)
    if op == "encode_act":
        return {"bytes": 3 * case["T"] * k + case["T"] * kb, "flops": 0}
    if op == "encode_weight":
        return {"bytes": 3 * case["N"] * k + -(-case["N"] // BLOCK) * kb, "flops": 0}
    if op == "product":
        t, n = case["T"], case["N"]
        return {"bytes": n * k + -(-n // BLOCK) * kb + 2 * t * (k + n), "flops": 2 * t * n * k}
    t, n, r, kids = case["T"], sum(_rows(case)), case["r"], len(_rows(case))
    read = t * k + t * kb + 2 * t * n + 2 * n * k + 4 * n + 2 * r * (n + kids * k)
    write = 2 * t * k + 4 * n + 2 * r * (n + kids * k) + (4 * n * k if case["dw0"] else 0)
    return {"bytes": read + write, "flops": 4 * t * n * k + 2 * t * r * (2 * n + 3 * kids * k)}


# ---- the definition in 64 bits, written apart from the plain form ------------------------------------------------

def _exact_code(x, tall):
    """Values and scale bytes by the definition: exponents by search from log2, codes by rounding to E4M3's grid."""
    x = x.double()
    m, k = x.shape
    mb, kb = -(-m // tall), -(-k // BLOCK)
    full = torch.zeros(mb * tall, kb * BLOCK, dtype=torch.float64, device=x.device)
    full[:m, :k] = x
    blocks = full.reshape(mb, tall, kb, BLOCK).permute(0, 2, 1, 3)
    top = blocks.abs().flatten(2).max(dim=2).values
    e = torch.ceil(torch.log2(top.clamp_min(1e-300) / 448.0))
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)          # log2's own rounding, either way
    e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(top == 0, torch.zeros_like(e), e.clamp_min(-118))
    v = blocks * torch.exp2(-e)[:, :, None, None]
    mag = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -40)))
    mag = torch.where(torch.exp2(mag) > v.abs(), mag - 1, mag)
    mag = torch.where(torch.exp2(mag + 1) <= v.abs(), mag + 1, mag).clamp_min(-6)
    step = torch.exp2(mag - 3)
    code = (torch.round(v / step) * step)
    lay = lambda b: b.permute(0, 2, 1, 3).reshape(mb * tall, kb * BLOCK)[:m, :k]  # noqa: E731
    return lay(code), (e + 127).to(torch.uint8), lay(code * torch.exp2(e)[:, :, None, None])


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "encode_act":
        return _exact_code(st["x"], 1)[:2]
    if op == "encode_weight":
        return _exact_code(st["w"], BLOCK)[:2]
    if op == "product":
        x = _exact_code(st["x"], 1)[2]
        return torch.matmul(x, _values(st["w"], BLOCK, torch.float64).t().contiguous())
    x, dy = _values(st["x"], 1, torch.float64), st["dy"].double()
    w0, s = torch.cat(st["w0"]).double(), torch.cat(st["s"]).double()
    edges = [0]
    for m in st["rows"]:
        edges.append(edges[-1] + m)
    grad = torch.matmul(dy.t().contiguous(), x)                      # d loss / d (W0 as it enters, unscaled)
    out = {"ds": torch.einsum("nk,nk->n", grad, w0),
           "dx": torch.matmul(dy * s[None, :], w0), "du": [], "dv": []}
    for i, (u, v) in enumerate(zip(st["u"], st["v"])):
        block = grad[edges[i]:edges[i + 1]]                          # G = dy^T x: dU = G V, dV = G^T U
        out["du"].append(torch.matmul(block, v.double()))
        out["dv"].append(torch.matmul(block.t().contiguous(), u.double()))
        delta = torch.matmul(u.double(), v.double().t().contiguous())
        out["dx"] += torch.matmul(dy[:, edges[i]:edges[i + 1]].contiguous(), delta)
    if st["dw0"]:
        out["dw0"] = grad * s[:, None]
    return out
