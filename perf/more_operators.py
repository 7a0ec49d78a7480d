"""Measured cases of what stands before and beside a projection: the root-mean-square norm with the residual's addition
and an 8-bit coded output, its backward pass, and the low-rank adapters of many requests at once beside one shared
projection, with their gradients.

`own` chooses between the plain torch form and the library's kernels.  Shapes are those of the synthetic Gemma-3-1B
and Gemma-4-31B bundles, plus ragged ones.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
EPS = 1e-6


def listed():
    return [
        # the norm before q|k|v of one decoded token: the smallest call there is
        {"name": "norm_token_1b", "op": "norm", "T": 1, "K": 1152, "res": True, "code": True},
        # q heads of 256 of a prompt of 2048 normed one by one: many short rows
        {"name": "norm_heads_1b", "op": "norm", "T": 8192, "K": 256, "res": False, "code": False},
        # the norm before a coded projection of a long training batch, its output also the checkpoint
        {"name": "norm_train_31b", "op": "norm", "T": 8192, "K": 5376, "res": True, "code": True},
        # a short ragged sequence, no residual branch behind the norm
        {"name": "norm_backward_ragged", "op": "norm_backward", "T": 333, "K": 1160, "res": False},
        # the same training batch backwards, the residual stream's gradient joining
        {"name": "norm_backward_31b", "op": "norm_backward", "T": 8192, "K": 5376, "res": True},
        # one request through the small model's q|k|v: launch latency
        {"name": "adapters_token_1b", "op": "adapters", "T": 1, "seqs": 1, "rows": "1024,256,256", "K": 1152, "r": 16, "n": 8},
        # a decode batch whose requests nearly all have an adapter of their own: reading the adapters
        {"name": "adapters_batch64_31b", "op": "adapters", "T": 64, "seqs": 64, "rows": "21504,21504", "K": 5376, "r": 16, "n": 64},
        # packed ragged sequences, no dimension a multiple of a tile
        {"name": "adapters_ragged", "op": "adapters", "T": 333, "seqs": 9, "rows": "1001", "K": 1160, "r": 32, "n": 5},
        # a dozen prompts packed into one call of the o projection
        {"name": "adapters_prompt_31b", "op": "adapters", "T": 4096, "seqs": 12, "rows": "5376", "K": 8192, "r": 64, "n": 32},
        # a short ragged training batch of three adapters
        {"name": "adapters_backward_ragged", "op": "adapters_backward", "T": 77, "seqs": 4, "rows": "1001", "K": 712, "r": 16, "n": 3},
        # eight adapters trained at once on the small model's q|k|v
        {"name": "adapters_backward_qkv_1b", "op": "adapters_backward", "T": 2048, "seqs": 16, "rows": "1024,256,256", "K": 1152, "r": 16, "n": 8},
        # sixteen adapters trained at once on the large gate|up: the largest case
        {"name": "adapters_backward_31b", "op": "adapters_backward", "T": 4096, "seqs": 18, "rows": "21504,21504", "K": 5376, "r": 32, "n": 16},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "norm_backward", "adapters", "adapters", "adapters", "adapters_backward", "adapters_backward"])
    if op in ("norm", "norm_backward"):
        k = 8 * _log(rng, 8, 2688)                  # 64 .. 21504
        t = _log(rng, 1, 8192)
        while t * k > 8192 * 5376:
            t = max(1, t // 2)
        case = {"op": op, "T": t, "K": k, "res": rng.random() < 0.6}
        return {**case, "code": rng.random() < 0.6} if op == "norm" else case
    k = 8 * _log(rng, 8, 1024)                      # 64 .. 8192
    if rng.random() < 0.5:
        k = max(64, k // 128 * 128)
    kids = rng.choice([1, 1, 2, 3])
    rows = [_log(rng, 40, 8192) for _ in range(kids)]
    if kids == 2:
        rows[1] = rows[0]
    t = rng.choice([1, rng.randint(2, 64), _log(rng, 65, 4096)])
    seqs = t if t <= 64 and rng.random() < 0.7 else _log(rng, 1, min(t, 40))
    r, n = 16 * rng.choice([1, 1, 2, 3, 4, 8]), _log(rng, 1, 64)
    while t * (sum(rows) + kids * k) * r * n > 4096 * 53760 * 512:
        n = n // 2
    return {"op": op, "T": t, "seqs": seqs, "rows": ",".join(map(str, rows)), "K": k, "r": r, "n": n}


def _gen(seed):
    return torch.Generator(DEV).manual_seed(int(seed) * 6151 + 29)


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


def _adapted(case):
    """How many of the sequences have an adapter: every eighth runs on the shared projection alone."""
    return case["seqs"] - case["seqs"] // 8


def _ranks(case):
    """Ranks of the slots in use, in the order in which the sequences take them: pools hold mixed ranks."""
    return [max(4, case["r"] // (1, 2, 1, 4)[j % 4]) for j in range(min(case["n"], _adapted(case)))]


def prepare(case, seed):
    g = _gen(seed)
    op, t, k = case["op"], case["T"], case["K"]
    if op in ("norm", "norm_backward"):
        st = {"op": op, "x": _activations(g, t, k), "w": (0.5 * _normal(g, k)).to(torch.bfloat16)}
        if op == "norm":
            st["res"] = _activations(g, t, k) if case["res"] else None
            st["code"] = case["code"]
        else:
            # what a forward pass keeps, and the gradients that reach the norm
            st["rstd"] = torch.rsqrt(st["x"].float().square().mean(1) + EPS)
            st["dy"] = _normal(g, t, k, std=t ** -0.5).to(torch.bfloat16)
            st["dh"] = _normal(g, t, k, std=t ** -0.5).to(torch.bfloat16) if case["res"] else None
        return st
    rows, r, n, seqs = _rows(case), case["r"], case["n"], case["seqs"]
    # slots: the sequences with an adapter take them in a random order, over and over where there are fewer
    order = torch.randperm(n, generator=g, device=DEV)
    turn = torch.arange(seqs, device=DEV)
    slot = torch.where(turn % 8 == 7, torch.full_like(turn, -1), order[(turn - turn // 8) % n])
    cuts = torch.randperm(t - 1, generator=g, device=DEV)[:seqs - 1].sort().values + 1   # lengths of at least one token
    index = slot[torch.bucketize(torch.arange(t, device=DEV), cuts, right=True)].to(torch.int32)
    rank = torch.full((n,), r, dtype=torch.int32, device=DEV)
    used = _ranks(case)
    rank[order[:len(used)]] = torch.tensor(used, dtype=torch.int32, device=DEV)
    live = torch.arange(r, device=DEV)[None, :] < rank[:, None]                           # [n, r]
    vt = _normal(g, n, len(rows), r, k, std=k ** -0.5) * live[:, None, :, None]
    u = _normal(g, n, sum(rows), r, std=0.05) * live[:, None, :]
    st = {"op": op, "rows": rows, "r": r, "n": n, "index": index, "rank": rank,
          "vt": vt.view(n, len(rows) * r, k).to(torch.bfloat16), "u": u.to(torch.bfloat16),
          "scale": 0.5 + torch.rand(n, generator=g, device=DEV)}
    x = _activations(g, t, k)
    if op == "adapters":
        st["x"], st["base"] = x, _normal(g, t, sum(rows)).to(torch.bfloat16)
    else:
        st["dy"] = _normal(g, t, sum(rows), std=t ** -0.5).to(torch.bfloat16)
        st["base"] = _normal(g, t, k, std=t ** -0.5).to(torch.bfloat16)
        st["x"] = _encode(x)
    if own:
        from weight_shared_rank_amd import binding
        st["pool"] = binding.AdapterPool(st["vt"], st["u"], st["scale"], rows, rank=rank)
        if op == "adapters_backward":
            st["x"] = binding.encode_act(x)
    return st


# ---- plain form -------------------------------------------------------------------------------------------------

def _encode(x):
    """E4M3 codes and E8M0 scale bytes of token rows in blocks of 128: e is the smallest exponent with
    max|x| <= 448 * 2^e (at least -118; 0 for a block of zeros), a code is E4M3(x * 2^-e)."""
    m, k = x.shape
    kb = -(-k // BLOCK)
    f = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - k)).view(m, kb, BLOCK)
    amax = f.abs().amax(dim=2)
    frac, ex = torch.frexp(amax)
    e = torch.where(frac <= 0.875, ex - 9, ex - 8).clamp_min(-118)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    code = torch.ldexp(f, -e[:, :, None]).to(torch.float8_e4m3fn)
    return code.view(m, kb * BLOCK)[:, :k], (e + 127).to(torch.uint8)


def _values(coded, dtype=torch.float32):
    """The numbers that coded rows stand for."""
    code, scale = coded
    return code.to(dtype) * torch.exp2(scale.to(dtype) - 127.0).repeat_interleave(BLOCK, 1)[:, :code.shape[1]]


def _plain_norm(state):
    h = state["x"].float()
    out = {}
    if state["res"] is not None:
        out["h"] = (h + state["res"].float()).to(torch.bfloat16)
        h = out["h"].float()
    out["rstd"] = torch.rsqrt(h.square().mean(1) + EPS)
    out["y"] = (h * out["rstd"][:, None] * (1.0 + state["w"].float())).to(torch.bfloat16)
    if state["code"]:
        code, scale = _encode(out["y"])
        out["code"], out["scale"] = code, scale.view(torch.float8_e8m0fnu)
    return out


def _plain_norm_backward(state):
    dy, rstd = state["dy"].float(), state["rstd"][:, None]
    xh = state["x"].float() * rstd
    gw = dy * (1.0 + state["w"].float())
    dx = rstd * (gw - xh * (gw * xh).mean(1, keepdim=True))
    if state["dh"] is not None:
        dx = dx + state["dh"].float()
    return {"dx": dx.to(torch.bfloat16), "dw": (dy * xh).sum(0)}


def _chosen(state):
    """[T, n]: the scale of a token's slot in that slot's column, zero elsewhere."""
    slots = torch.arange(state["n"], device=DEV)
    return (state["index"][:, None] == slots[None, :]).float() * state["scale"][None, :]


def _plain_adapters(state):
    """All slots at once: the thin products of every slot, those of the other slots masked out."""
    n, r, rows = state["n"], state["r"], state["rows"]
    z = torch.matmul(state["x"].float(), state["vt"].float().view(-1, state["vt"].shape[2]).t())
    z = z.view(-1, n, len(rows), r) * _chosen(state)[:, :, None, None]
    y = [torch.matmul(z[:, :, c].reshape(-1, n * r), u.float().transpose(1, 2).reshape(n * r, -1))
         for c, u in enumerate(state["u"].split(rows, dim=1))]
    return (state["base"].float() + torch.cat(y, 1)).to(torch.bfloat16)


def _plain_adapters_backward(state):
    n, r, rows = state["n"], state["r"], state["rows"]
    x, dy, chosen = _values(state["x"]), state["dy"].float(), _chosen(state)[:, :, None]
    k = x.shape[1]
    dx, du, dv = state["base"].float(), [], []
    for v, u, d in zip(state["vt"].float().view(n, len(rows), r, k).unbind(1), state["u"].float().split(rows, dim=1), dy.split(rows, dim=1)):
        flat = v.reshape(n * r, k)
        z = (torch.matmul(x, flat.t()).view(-1, n, r) * chosen).view(-1, n * r)
        g = (torch.matmul(d, u.transpose(0, 1).reshape(-1, n * r)).view(-1, n, r) * chosen).view(-1, n * r)
        dx = dx + torch.matmul(g, flat)
        du.append(torch.matmul(d.t(), z).view(-1, n, r).transpose(0, 1))
        dv.append(torch.matmul(g.t(), x).view(n, r, k))
    return {"dx": dx.to(torch.bfloat16), "du": torch.cat(du, 1).to(torch.bfloat16), "dv": torch.cat(dv, 1).to(torch.bfloat16)}


# ---- the library's kernels --------------------------------------------------------------------------------------

def _own(state):
    from weight_shared_rank_amd import binding
    op = state["op"]
    if op == "norm":
        want = ("y", "rstd") + (("h",) if state["res"] is not None else ()) + (("code",) if state["code"] else ())
        o = binding.norm_act(state["x"], state["w"], eps=EPS, residual=state["res"], offset=1.0, want=want)
        out = {"y": o.y, "rstd": o.rstd}
        if state["res"] is not None:
            out["h"] = o.h
        if state["code"]:
            out["code"], out["scale"] = o.code.codes, o.code.scales.view(torch.float8_e8m0fnu)
        return out
    if op == "norm_backward":
        o = binding.norm_backward(state["dy"], state["x"], state["rstd"], state["w"], offset=1.0, dh=state["dh"])
        return {"dx": o.dx, "dw": o.dw}
    if op == "adapters":
        return state["pool"].add(state["x"], state["index"], state["base"])
    o = state["pool"].backward(state["x"], state["dy"], state["index"], state["base"])
    return {"dx": o.dx, "du": o.du, "dv": o.dv}


_PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "adapters": _plain_adapters,
          "adapters_backward": _plain_adapters_backward}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


def work(case):
    op, t, k = case["op"], case["T"], case["K"]
    if op == "norm":
        each = 2 + (4 if case["res"] else 0) + 2 + (1 if case["code"] else 0)
        return {"bytes": each * t * k + 2 * k + 4 * t + (t * -(-k // BLOCK) if case["code"] else 0), "flops": 6 * t * k}
    if op == "norm_backward":
        return {"bytes": (8 if case["res"] else 6) * t * k + 6 * k + 4 * t, "flops": 10 * t * k}
    n, kids, r = sum(_rows(case)), len(_rows(case)), case["r"]
    held = sum(_ranks(case))                                   # ranks of the slots in use
    rank = held / max(1, len(_ranks(case)))
    hit = t * _adapted(case) / case["seqs"]                    # tokens with an adapter, about
    weights = 2 * held * (kids * k + n)
    if op == "adapters":
        return {"bytes": weights + 2 * hit * k + 4 * t * n + 4 * t, "flops": 2 * hit * rank * (kids * k + n)}
    grads = 2 * case["n"] * r * (kids * k + n)
    return {"bytes": weights + grads + hit * k * (1 + 1 / BLOCK) + 2 * hit * n + 4 * t * k + 4 * t,
            "flops": 6 * hit * rank * (kids * k + n) - 2 * hit * rank * n}


# ---- the definition in 64 bits, written apart from the plain form ------------------------------------------------

def _round(x, bits, least):
    """x to `bits` significant bits, nearest with ties to even; steps no finer than 2^least."""
    _, e = torch.frexp(x)
    step = torch.exp2((e.double() - bits).clamp_min(least))
    return torch.where(x == 0, x, torch.round(x / step) * step)


def _exact_code(y):
    """Codes (as E4M3's values) and scales (as powers of two) by the definition, exponents by search from log2."""
    t, k = y.shape
    kb = -(-k // BLOCK)
    full = torch.zeros(t, kb * BLOCK, dtype=torch.float64, device=y.device)
    full[:, :k] = y
    b = full.view(t, kb, BLOCK)
    top = b.abs().max(dim=2).values
    e = torch.ceil(torch.log2(top.clamp_min(1e-300) / 448.0))
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)          # log2's own rounding, either way
    e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(top == 0, torch.zeros_like(e), e.clamp_min(-118))
    return _round(b * torch.exp2(-e)[:, :, None], 4, -9).view(t, kb * BLOCK)[:, :k], torch.exp2(e)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "norm":
        h, out = st["x"].double(), {}
        if st["res"] is not None:
            h = _round(h + st["res"].double(), 8, -133)
            out["h"] = h
        out["rstd"] = (torch.einsum("tk,tk->t", h, h) / case["K"] + EPS) ** -0.5
        out["y"] = torch.einsum("tk,t,k->tk", h, out["rstd"], 1.0 + st["w"].double())
        if st["code"]:
            out["code"], out["scale"] = _exact_code(_round(out["y"], 8, -133))
        return out
    if op == "norm_backward":
        h, dy, a, w = st["x"].double(), st["dy"].double(), st["rstd"].double(), 1.0 + st["w"].double()
        dot = torch.einsum("tk,tk,k->t", dy, h, w)
        dx = dy * w * a[:, None] - h * (dot * a ** 3 / case["K"])[:, None]
        if st["dh"] is not None:
            dx = dx + st["dh"].double()
        return {"dx": dx, "dw": torch.einsum("tk,tk,t->k", dy, h, a)}
    # slot by slot, each slot's own tokens
    rows, r, index = st["rows"], st["r"], st["index"].tolist()
    of = {}
    for t, a in enumerate(index):
        of.setdefault(a, []).append(t)
    edges = [sum(rows[:c]) for c in range(len(rows) + 1)]
    if op == "adapters":
        y = st["base"].double()
        for a in sorted(of):
            if a < 0:
                continue
            at = torch.tensor(of[a], device=DEV)
            x = st["x"][at].double()
            for c in range(len(rows)):
                weight = torch.matmul(st["u"][a, edges[c]:edges[c + 1]].double(), st["vt"][a, c * r:(c + 1) * r].double())
                y[at, edges[c]:edges[c + 1]] += st["scale"][a].double() * torch.matmul(x, weight.t().contiguous())
        return y
    values, dx = _values(st["x"], torch.float64), st["base"].double()
    du, dv = torch.zeros(st["u"].shape, dtype=torch.float64, device=DEV), torch.zeros(st["vt"].shape, dtype=torch.float64, device=DEV)
    for a in sorted(of):
        if a < 0:
            continue
        at = torch.tensor(of[a], device=DEV)
        x = values[at]
        for c in range(len(rows)):
            u, v = st["u"][a, edges[c]:edges[c + 1]].double(), st["vt"][a, c * r:(c + 1) * r].double()
            d = st["dy"][at, edges[c]:edges[c + 1]].double() * st["scale"][a].double()
            grad = torch.matmul(d.t().contiguous(), x)              # d loss / d (U V^T): dU = G V, dV^T = U^T G
            du[a, edges[c]:edges[c + 1]] = torch.matmul(grad, v.t().contiguous())
            dv[a, c * r:(c + 1) * r] = torch.matmul(u.t().contiguous(), grad)
            dx[at] += torch.matmul(d, torch.matmul(u, v))
    return {"dx": dx, "du": du, "dv": dv}
