"""Cases for the norms around a block, adapters beside a projection, and tokens sorted by expert and back.

Operators, named by a case's "op":

* norm:     a block's output, normalised or not, times a gate and a scale, added to the residual; the sum
            normalised for the next block, as bf16 or quantized with a scale per token and 128 columns.
* lora:     the low-rank adapters of many requests added to the output of a projection they share.
* dispatch: tokens copied to rows sorted by expert.
* combine:  the experts' rows back to their tokens, summed with the routing weights.
* backward: the gradients of both.

`run` computes them in elementary torch operations in 32 bits, or (own) through the package.
"""

import math

import torch

own = False

FP8_MAX = 448.0
BLOCK = 128
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decoding token between two blocks: residual, norm and codes for the next projection
        {"name": "norm decode 1", "op": "norm", "M": 1, "H": 4096, "post": False, "gate": "none", "scale": 1.0,
         "quantize": True},
        # a chunk of no round size, norms on both sides, a gate per channel, bf16 for a router
        {"name": "norm ragged 777", "op": "norm", "M": 777, "H": 1001, "post": True, "gate": "channel", "scale": 1.0,
         "quantize": False},
        # a wide model's batch, norms on both sides, a gate of each token, a scaled residual branch
        {"name": "norm gated 4096", "op": "norm", "M": 4096, "H": 8192, "post": True, "gate": "token", "scale": 0.22,
         "quantize": True},
        # a full prompt batch before a block-scaled projection
        {"name": "norm prefill 16384", "op": "norm", "M": 16384, "H": 4096, "post": False, "gate": "none",
         "scale": 1.0, "quantize": True},
        # one decoding request with an adapter: latency
        {"name": "lora decode 1", "op": "lora", "M": 1, "K": 4096, "N": 6144, "r": 16, "L": 8, "runs": False,
         "bare": 0.0},
        # a decode batch, each token of a request of its own, some without an adapter
        {"name": "lora decode 64", "op": "lora", "M": 64, "K": 4096, "N": 4096, "r": 64, "L": 32, "runs": False,
         "bare": 0.2},
        # a few prompts of no round size, an odd rank
        {"name": "lora ragged 333", "op": "lora", "M": 333, "K": 1000, "N": 1027, "r": 12, "L": 5, "runs": True,
         "bare": 0.1},
        # a prompt batch of many requests
        {"name": "lora prefill 8192", "op": "lora", "M": 8192, "K": 4096, "N": 14336, "r": 64, "L": 16, "runs": True,
         "bare": 0.0},
        # one decoding token to its experts
        {"name": "dispatch decode 1", "op": "dispatch", "T": 1, "E": 256, "k": 8, "H": 4096, "drop": 0.0,
         "dtype": "bfloat16"},
        # a prompt batch to its experts
        {"name": "dispatch prefill 8192", "op": "dispatch", "T": 8192, "E": 64, "k": 8, "H": 4096, "drop": 0.0,
         "dtype": "bfloat16"},
        # odd sizes back in fp32, pairs of experts that live elsewhere left out
        {"name": "combine ragged 1001", "op": "combine", "T": 1001, "E": 12, "k": 3, "H": 1000, "drop": 0.25,
         "dtype": "float32"},
        # the gradients of a training batch's way to the experts and back
        {"name": "backward 8192", "op": "backward", "T": 8192, "E": 64, "k": 8, "H": 2048, "drop": 0.0,
         "dtype": "bfloat16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A model's width: mostly a multiple of 128, else any."""
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.4 else max(BLOCK, n // BLOCK * BLOCK)


def draw(rng):
    op = rng.choice(["norm", "norm", "lora", "lora", "dispatch", "combine", "backward"])
    if op == "norm":
        M, H = _log_int(rng, 1, 16384), _width(rng, 64, 16384)
        M = max(1, min(M, 16384 * 4096 // H))
        return {"op": op, "M": M, "H": H, "post": rng.random() < 0.5, "gate": rng.choice(["none", "channel", "token"]),
                "scale": rng.choice([1.0, 0.22]), "quantize": rng.random() < 0.6}
    if op == "lora":
        runs = rng.random() < 0.5
        M = _log_int(rng, 16, 8192) if runs else _log_int(rng, 1, 512)
        K, N = _width(rng, 64, 8192), _width(rng, 64, 14336)
        r = rng.choice([8, 16, 32, 64, 128, rng.randint(1, 128)])
        if M * r * (K + N) > 8192 * 64 * (4096 + 14336):
            M = max(1, 8192 * 64 * (4096 + 14336) // (r * (K + N)))
        return {"op": op, "M": M, "K": K, "N": N, "r": r, "L": _log_int(rng, 1, 16 if M > 1024 else 64), "runs": runs,
                "bare": rng.choice([0.0, 0.0, 0.2])}
    E = _log_int(rng, 4, 256)
    k = rng.randint(1, min(8, E))
    T, H = _log_int(rng, 1, 8192), _width(rng, 64, 7168)
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    most = 8192 * 8 * (4096 if op == "dispatch" else 2048) // (2 if dtype == "float32" else 1)
    T = max(1, min(T, most // (k * H)))
    return {"op": op, "T": T, "E": E, "k": k, "H": H, "drop": rng.choice([0.0, 0.0, 0.25]), "dtype": dtype}


def _blocks(n):
    return -(-n // BLOCK)


def _size(case):
    return 4 if case["dtype"] == "float32" else 2


def work(case):
    if case["op"] == "norm":
        M, H = case["M"], case["H"]
        read = 4 * M * H + 2 * H * (2 if case["post"] else 1)
        read += {"none": 0, "channel": 2 * H, "token": 2 * M * H}[case["gate"]]
        n = M * H + 4 * M * _blocks(H) if case["quantize"] else 2 * M * H
        return {"bytes": read + 2 * M * H + n, "flops": 12 * M * H}
    if case["op"] == "lora":
        M, K, N, r, L = case["M"], case["K"], case["N"], case["r"], case["L"]
        with_one = M * (1.0 - case["bare"])
        touched = L * (1.0 - (1.0 - 1.0 / L) ** (_requests(case) * (1.0 - case["bare"])))
        return {"bytes": 2 * with_one * K + 4 * M * N + touched * 2 * r * (K + N) + 4 * M,
                "flops": 2 * with_one * r * (K + N)}
    T, k, H, size = case["T"], case["k"], case["H"], _size(case)
    pairs = T * k * (1.0 - case["drop"])
    if case["op"] == "dispatch":
        return {"bytes": size * H * (T + pairs) + 8 * T * k + 4 * (case["E"] + 1), "flops": T * k}
    if case["op"] == "combine":
        return {"bytes": size * H * (T + pairs) + 8 * T * k, "flops": 2 * pairs * H}
    # dy, ys -> dys, dw; dxs -> dx
    return {"bytes": size * H * (T + 2 * pairs) + size * H * (T + pairs) + 16 * T * k, "flops": 4 * pairs * H}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _requests(case):
    """Requests in the batch: a prompt each of about 512 tokens (at least four of them), or one token each."""
    return min(case["M"], max(4, case["M"] // 512)) if case["runs"] else case["M"]


def _activations(rows, cols, g, device):
    """Rows as a block leaves them: unit variance, a few channels much larger."""
    x = torch.randn(rows, cols, generator=g, device=device)
    loud = torch.randint(0, cols, (max(1, cols // 100),), generator=g, device=device)
    x[:, loud] *= 20.0
    return x.to(torch.bfloat16)


def _around_one(n, g, device):
    return (1.0 + 0.2 * torch.randn(n, generator=g, device=device)).to(torch.bfloat16)


def prepare(case, seed):
    device = "cuda"
    g = torch.Generator(device=device).manual_seed(int(seed))
    if case["op"] == "norm":
        M, H = case["M"], case["H"]
        gate = None
        if case["gate"] != "none":
            shape = (H,) if case["gate"] == "channel" else (M, H)
            gate = (0.5 * torch.randn(shape, generator=g, device=device)).to(torch.bfloat16)
        return {"case": dict(case), "y": _activations(M, H, g, device), "residual": 3 * _activations(M, H, g, device),
                "weight": _around_one(H, g, device), "post": _around_one(H, g, device) if case["post"] else None,
                "gate": gate}
    if case["op"] == "lora":
        M, K, N, r, L = case["M"], case["K"], case["N"], case["r"], case["L"]
        x = _activations(M, K, g, device)
        y = torch.randn(M, N, generator=g, device=device).to(torch.bfloat16)
        a = (torch.randn(L, r, K, generator=g, device=device) * K ** -0.5).to(torch.bfloat16)
        b = (torch.randn(L, N, r, generator=g, device=device) * r ** -0.5).to(torch.bfloat16)
        scales = 0.25 + torch.rand(L, generator=g, device=device)
        n = _requests(case)
        which = torch.randint(0, L, (n,), generator=g, device=device)
        which = torch.where(torch.rand(n, generator=g, device=device) < case["bare"], -torch.ones_like(which), which)
        if case["runs"]:  # prompts of uneven lengths, one after the other
            ends = torch.rand(n, generator=g, device=device).add_(0.3).cumsum(0)
            ends = (ends / ends[-1] * M).round().long()
            which = which[torch.searchsorted(ends, torch.arange(M, device=device), right=True).clamp_(max=n - 1)]
        return {"case": dict(case), "x": x, "y": y, "a": a, "b": b, "scales": scales, "ids": which.to(torch.int32)}
    T, E, k, H = case["T"], case["E"], case["k"], case["H"]
    dtype = getattr(torch, case["dtype"])
    liking = torch.randn(T, E, generator=g, device=device) + 0.3 * torch.randn(E, generator=g, device=device)
    top, ids = liking.topk(k, dim=1)
    weights = torch.softmax(top, dim=1).contiguous()
    if case["drop"]:
        gone = torch.rand(T, k, generator=g, device=device) < case["drop"]
        gone[0, 0] = False  # some pair is left
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    ids = ids.to(torch.int32).contiguous()
    s = {"case": dict(case), "ids": ids, "weights": weights}
    if case["op"] == "dispatch":
        # a program keeps the sorted rows' buffer; rows behind the kept pairs stay as they are
        return dict(s, x=torch.randn(T, H, generator=g, device=device).to(dtype),
                    xs=torch.zeros(T * k, H, dtype=dtype, device=device))
    s["pos"] = _sorted_rows(ids, E)[0]
    s["ys"] = torch.randn(T * k, H, generator=g, device=device).to(dtype)
    if case["op"] == "backward":
        s["dy"] = torch.randn(T, H, generator=g, device=device).to(dtype)
        s["dxs"] = torch.randn(T * k, H, generator=g, device=device).to(dtype)
        s["dys"] = torch.zeros(T * k, H, dtype=dtype, device=device)
    return s


# ---------------------------------------------------------------------------
# plain forms: 32-bit torch operations
# ---------------------------------------------------------------------------

def _plain_norm(s):
    c = s["case"]
    t = s["y"].float()
    if s["post"] is not None:
        t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + EPS) * s["post"].float()
    if s["gate"] is not None:
        t = t * s["gate"].float()
    r = s["residual"].float() + c["scale"] * t
    n = r / torch.sqrt((r * r).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if not c["quantize"]:
        return {"n": n.to(torch.bfloat16), "r": r.to(torch.bfloat16)}
    H = c["H"]
    p = torch.nn.functional.pad(n, (0, _blocks(H) * BLOCK - H)).unflatten(-1, (-1, BLOCK))
    amax = p.abs().amax(-1)
    scale = amax / torch.full_like(amax, FP8_MAX)
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    q = (p / scale[..., None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    # codes end at the next multiple of 16 columns, with zeros; the scales of one block are adjacent
    return {"q": q.flatten(-2)[:, :-(-H // 16) * 16], "s": scale.T, "r": r.to(torch.bfloat16)}


def _plain_lora(s):
    c = s["case"]
    M, K, N, r, L = c["M"], c["K"], c["N"], c["r"], c["L"]
    ids = s["ids"].long()
    x, y = s["x"].float(), s["y"].float()
    with_one = (ids >= 0) & (ids < L)
    at = ids.clamp(0, L - 1)
    factor = torch.where(with_one, s["scales"][at], torch.zeros_like(s["scales"][at]))
    if M <= 64:  # each token with its own adapter
        v = torch.einsum("mk,mrk->mr", x, s["a"][at].float())
        d = torch.einsum("mr,mnr->mn", v, s["b"][at].float())
    else:  # all adapters, all but the token's own set to zero
        v = (x @ s["a"].float().flatten(0, 1).T).view(M, L, r)
        mine = torch.arange(L, device=x.device)[None, :, None] == at[:, None, None]
        v = torch.where(mine, v, torch.zeros_like(v))
        d = v.flatten(1) @ s["b"].float().transpose(1, 2).reshape(L * r, N)
    return (y + d * factor[:, None]).to(torch.bfloat16)


def _sorted_rows(ids, E):
    """(pos [T, k], offsets [E + 1]): the row of each pair, sorted by expert and then by pair, -1 for none."""
    e = ids.long().flatten()
    kept = (e >= 0) & (e < E)
    e = torch.where(kept, e, torch.full_like(e, E))
    order = e.sort(stable=True).indices
    pos = torch.empty_like(e)
    pos[order] = torch.arange(e.numel(), device=e.device)
    pos = torch.where(kept, pos, torch.full_like(pos, -1))
    count = torch.zeros(E + 1, dtype=torch.int64, device=e.device).scatter_add_(0, e, torch.ones_like(e))
    return pos.view(ids.shape).to(torch.int32), (count.cumsum(0) - count).to(torch.int32)


def _plain_dispatch(s):
    c = s["case"]
    pos, offsets = _sorted_rows(s["ids"], c["E"])
    n = c["T"] * c["k"]
    to = torch.where(pos >= 0, pos, torch.full_like(pos, n)).long().flatten()
    xs = torch.zeros(n + 1, c["H"], dtype=s["x"].dtype, device=s["x"].device)
    xs[to] = s["x"].repeat_interleave(c["k"], 0)
    return {"xs": xs[:-1], "pos": pos, "offsets": offsets}


def _rows_of(rows, pos):
    """fp32 [T, k, H]: each pair's row, zeros where it has none."""
    v = rows[pos.clamp(min=0).long()].float()
    return torch.where((pos >= 0)[..., None], v, torch.zeros_like(v))


def _plain_combine(s):
    return (_rows_of(s["ys"], s["pos"]) * s["weights"][..., None]).sum(1).to(s["ys"].dtype)


def _plain_backward(s):
    c, pos, dtype = s["case"], s["pos"], s["ys"].dtype
    n = c["T"] * c["k"]
    dy = s["dy"].float()
    dw = (_rows_of(s["ys"], pos) * dy[:, None]).sum(-1)
    dys = torch.zeros(n + 1, c["H"], dtype=dtype, device=dy.device)
    dys[torch.where(pos >= 0, pos, torch.full_like(pos, n)).long()] = (dy[:, None] * s["weights"][..., None]).to(dtype)
    return {"dys": dys[:-1], "dw": dw, "dx": _rows_of(s["dxs"], pos).sum(1).to(dtype)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if not own:
        return {"norm": _plain_norm, "lora": _plain_lora, "dispatch": _plain_dispatch, "combine": _plain_combine,
                "backward": _plain_backward}[c["op"]](state)
    import fp8_w8a8_quantized_dynamic_gb300 as F
    if c["op"] == "norm":
        if c["quantize"]:
            q, s, r = F.fp8_residual_norm_quantize(state["y"], state["weight"], residual=state["residual"],
                                                   post_weight=state["post"], gate=state["gate"], scale=c["scale"],
                                                   eps=EPS)
            return {"q": q.view(torch.float8_e4m3fn), "s": s, "r": r}
        n, r = F.fp8_residual_norm(state["y"], state["weight"], residual=state["residual"], post_weight=state["post"],
                                   gate=state["gate"], scale=c["scale"], eps=EPS)
        return {"n": n, "r": r}
    if c["op"] == "lora":
        return F.fp8_lora_add(state["y"], state["x"], state["a"], state["b"], state["ids"], state["scales"])
    if c["op"] == "dispatch":
        xs, pos, offsets = F.fp8_moe_dispatch(state["x"], state["ids"], c["E"], out=state["xs"])
        return {"xs": xs, "pos": pos, "offsets": offsets}
    if c["op"] == "combine":
        return F.fp8_moe_combine(state["ys"], state["pos"], state["weights"])
    dys, dw = F.fp8_moe_combine_grad(state["dy"], state["ys"], state["pos"], state["weights"], out=state["dys"])
    return {"dys": dys, "dw": dw, "dx": F.fp8_moe_dispatch_grad(state["dxs"], state["pos"])}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _e4m3_64(x):
    """The nearest e4m3 value (ties to even, saturating) of fp64 values that are fp32 numbers."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-FP8_MAX, FP8_MAX)


def _exact_norm(s):
    c = s["case"]
    M, H = c["M"], c["H"]

    def normed(v, weight):
        return v * weight.double() * (v.square().sum(1, keepdim=True) / H + EPS).rsqrt()

    t = s["y"].double() if s["post"] is None else normed(s["y"].double(), s["post"])
    if s["gate"] is not None:
        t = t * s["gate"].double()
    r = torch.add(s["residual"].double(), t, alpha=c["scale"])
    n = normed(r, s["weight"])
    if not c["quantize"]:
        return {"n": n, "r": r}
    v = torch.zeros(M, _blocks(H) * BLOCK, dtype=torch.float64, device=n.device)
    v[:, :H] = n
    v = v.view(M, -1, BLOCK)
    scale = (v.abs().amax(2) / FP8_MAX).float().double()
    scale[scale == 0] = 1.0
    q = _e4m3_64((v / scale[..., None]).float().double()).view(M, -1)
    return {"q": q[:, :(H + 15) // 16 * 16].contiguous(), "s": scale.t().contiguous(), "r": r}


def _exact_lora(s):
    out = s["y"].double()
    for i in range(s["case"]["L"]):
        t = (s["ids"] == i).nonzero(as_tuple=True)[0]
        if t.numel():
            v = s["x"][t].double() @ s["a"][i].double().T
            out[t] += (v @ s["b"][i].double().T) * s["scales"][i].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "lora":
        return _exact_lora(s)
    if case["op"] == "dispatch":
        flat = s["ids"].flatten()
        rows = torch.cat([(flat == e).nonzero(as_tuple=True)[0] for e in range(case["E"])])
        xs = torch.zeros(flat.numel(), case["H"], dtype=torch.float64, device=flat.device)
        xs[:rows.numel()] = s["x"].double()[rows // case["k"]]
        return {"xs": xs, "pos": None, "offsets": None}
    T, k, H = case["T"], case["k"], case["H"]
    t, j = (s["pos"] >= 0).nonzero(as_tuple=True)
    row = s["pos"][t, j].long()
    back = torch.zeros(T, H, dtype=torch.float64, device=row.device)
    if case["op"] == "combine":
        return back.index_add_(0, t, s["ys"][row].double() * s["weights"][t, j].double()[:, None])
    dys = torch.zeros(T * k, H, dtype=torch.float64, device=row.device)
    dys[row] = s["dy"].double()[t] * s["weights"][t, j].double()[:, None]
    dw = torch.zeros(T, k, dtype=torch.float64, device=row.device)
    dw[t, j] = torch.linalg.vecdot(s["dy"].double()[t], s["ys"][row].double())
    return {"dys": dys, "dw": dw, "dx": back.index_add_(0, t, s["dxs"][row].double())}
