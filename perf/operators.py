"""Cases for the block-scaled FP8 linear, the routing to experts and the experts' products.

Three operators, named by a case's "op":

* linear:  bf16 activations, quantized per token and 128 values of K, times FP8 weights with a scale
           for each 128 x 128 block.
* route:   scores of E experts to the k chosen ones and their weights (softmax, or sigmoid with a
           bias for balance and limited groups).
* experts: the gated two-layer network of each chosen expert on block-scaled FP8 weights, summed with
           the routing weights.

`run` computes them in elementary torch operations in 32 bits, or (own) through the package.
"""

import math

import torch

own = False

FP8_MAX = 448.0
BLOCK = 128


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token through an attention input projection while decoding: the weight stream alone
        {"name": "linear decode 1", "op": "linear", "M": 1, "K": 4096, "N": 6144, "bias": False},
        # a decode batch on a layer with no size a multiple of 128, with a bias
        {"name": "linear decode 13 ragged", "op": "linear", "M": 13, "K": 1000, "N": 1027, "bias": True},
        # a short chunk of a prompt through a long-K projection: too few tiles for the whole GPU
        {"name": "linear chunk 200", "op": "linear", "M": 200, "K": 5632, "N": 2048, "bias": False},
        # a full prompt batch through the widest projection: tensor cores alone
        {"name": "linear prefill 16384", "op": "linear", "M": 16384, "K": 4096, "N": 28672, "bias": False},
        # one decoding token over many experts in groups, biased sigmoid scores
        {"name": "route decode 1", "op": "route", "T": 1, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "renorm": True, "factor": 2.5, "dtype": "float32"},
        # odd counts, bf16 logits with many equal ones, weights left as they are
        {"name": "route odd 1001", "op": "route", "T": 1001, "E": 60, "k": 4, "score": "softmax", "bias": False,
         "groups": 1, "keep": 1, "renorm": False, "factor": 1.0, "dtype": "bfloat16"},
        # a prompt batch, softmax scores renormalised over the chosen ones
        {"name": "route softmax 4096", "op": "route", "T": 4096, "E": 128, "k": 8, "score": "softmax", "bias": False,
         "groups": 1, "keep": 1, "renorm": True, "factor": 1.0, "dtype": "float32"},
        # the largest prompt batch over many experts in groups
        {"name": "route prefill 16384", "op": "route", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "renorm": True, "factor": 2.5, "dtype": "float32"},
        # one decoding token: the chosen experts' weights, each read once
        {"name": "experts decode 1", "op": "experts", "T": 1, "E": 64, "k": 8, "H": 2048, "I": 1408, "drop": 0.0},
        # a decode batch: most experts are touched, each by a token or two
        {"name": "experts decode 16", "op": "experts", "T": 16, "E": 64, "k": 8, "H": 2048, "I": 1408, "drop": 0.0},
        # odd sizes, and choices that another machine's experts serve (dropped here)
        {"name": "experts ragged 333", "op": "experts", "T": 333, "E": 12, "k": 3, "H": 1000, "I": 600, "drop": 0.3},
        # a prompt batch on large experts
        {"name": "experts prefill 8192", "op": "experts", "T": 8192, "E": 64, "k": 8, "H": 4096, "I": 2048, "drop": 0.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "route", "experts"])
    if op == "linear":
        M, K, N = _log_int(rng, 1, 16384), _log_int(rng, 64, 14336), _log_int(rng, 64, 28672)
        if rng.random() < 0.5:  # model widths are mostly multiples of 128
            K, N = max(128, K // 128 * 128), max(128, N // 128 * 128)
        if M * K * N > 16384 * 4096 * 28672:
            K = max(64, 16384 * 4096 * 28672 // (M * N))
        return {"op": op, "M": M, "K": K, "N": N, "bias": rng.random() < 0.5}
    if op == "route":
        sigmoid = rng.random() < 0.5
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(2, 256 // groups)
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(16, keep * (E // groups)))
        return {"op": op, "T": _log_int(rng, 1, 16384), "E": E, "k": k, "score": "sigmoid" if sigmoid else "softmax",
                "bias": sigmoid and rng.random() < 0.7, "groups": groups, "keep": keep, "renorm": rng.random() < 0.7,
                "factor": rng.choice([1.0, 2.5]), "dtype": rng.choice(["float32", "bfloat16"])}
    E = _log_int(rng, 4, 128)
    T, H, I = _log_int(rng, 1, 8192), _log_int(rng, 128, 4096), _log_int(rng, 64, 2048)
    if rng.random() < 0.5:
        H, I = max(128, H // 128 * 128), max(128, I // 128 * 128)
    if E * H * I > 64 * 4096 * 2048:
        E = 64
    return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(8, E)), "H": H, "I": I,
            "drop": rng.choice([0.0, 0.0, 0.25])}


def _blocks(n):
    return -(-n // BLOCK)


def _pairs(case):
    """Routed pairs, and the experts they touch, of an even routing."""
    pairs = case["T"] * case["k"] * (1.0 - case["drop"])
    return pairs, case["E"] * (1.0 - (1.0 - 1.0 / case["E"]) ** pairs)


def work(case):
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 2 * M * K + N * K + 4 * _blocks(N) * _blocks(K) + 2 * M * N + (2 * N if case["bias"] else 0),
                "flops": 2 * M * K * N}
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        return {"bytes": T * E * (4 if case["dtype"] == "float32" else 2) + 8 * T * case["k"], "flops": 6 * T * E}
    T, H, I = case["T"], case["H"], case["I"]
    pairs, touched = _pairs(case)
    return {"bytes": touched * 3 * H * I + 4 * T * H + 8 * T * case["k"], "flops": 6 * pairs * H * I}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed, device):
    return torch.Generator(device=device).manual_seed(int(seed))


def _activations(rows, cols, g, device):
    """Rows as a normalisation leaves them: unit variance, a few channels much larger."""
    x = torch.randn(rows, cols, generator=g, device=device)
    loud = torch.randint(0, cols, (max(1, cols // 100),), generator=g, device=device)
    x[:, loud] *= 20.0
    return x.to(torch.bfloat16)


def _block_weight(batch, N, K, g, device):
    """FP8 weights as a block-scaled checkpoint holds them: codes [batch, N, K rounded up to 16] with zero
    tails and scales [batch, N blocks, K blocks]. Whole blocks of codes span the format's range."""
    codes = torch.zeros(batch, N, -(-K // 16) * 16, dtype=torch.uint8, device=device)
    w = torch.randn(batch, N, K, generator=g, device=device).mul_(FP8_MAX / 4.0).clamp_(-FP8_MAX, FP8_MAX)
    codes[..., :K] = w.to(torch.float8_e4m3fn).view(torch.uint8)
    spread = torch.rand(batch, _blocks(N), _blocks(K), generator=g, device=device) * 1.5 + 0.25
    return codes, spread * (0.02 * 4.0 / FP8_MAX)


def prepare(case, seed):
    device = "cuda"
    g = _generator(seed, device)
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        qw, s_w = _block_weight(1, N, K, g, device)
        bias = torch.randn(N, generator=g, device=device).to(torch.bfloat16) if case["bias"] else None
        return {"case": dict(case), "a": _activations(M, K, g, device), "qw": qw[0], "s_w": s_w[0], "bias": bias}
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        logits = torch.randn(T, E, generator=g, device=device) * 1.5
        logits += 0.5 * torch.randn(E, generator=g, device=device)  # some experts are liked more
        bias = 0.1 * torch.randn(E, generator=g, device=device) if case["bias"] else None
        return {"case": dict(case), "logits": logits.to(getattr(torch, case["dtype"])), "bias": bias}
    T, E, k, H, I = case["T"], case["E"], case["k"], case["H"], case["I"]
    x = _activations(T, H, g, device)
    liking = torch.randn(T, E, generator=g, device=device) + 0.3 * torch.randn(E, generator=g, device=device)
    top, ids = liking.topk(k, dim=1)
    weights = torch.softmax(top, dim=1)
    if case["drop"]:
        gone = torch.rand(T, k, generator=g, device=device) < case["drop"]
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    qw13, s13 = _block_weight(2 * E, I, H, g, device)
    qw2, s2 = _block_weight(E, H, I, g, device)
    kept = ids[ids >= 0]
    most = int(torch.bincount(kept, minlength=E).max()) if kept.numel() else 0
    return {"case": dict(case), "x": x, "ids": ids.to(torch.int32).contiguous(), "weights": weights.contiguous(),
            "qw13": qw13.view(E, 2, I, -1), "s13": s13.view(E, 2, _blocks(I), _blocks(H)), "qw2": qw2, "s2": s2,
            "most": most}  # the busiest expert's tokens: the plain form's padding


# ---------------------------------------------------------------------------
# plain forms: 32-bit torch operations
# ---------------------------------------------------------------------------

def _through_fp8(x):
    """x [..., K] fp32 as its block-quantized values: per row and 128 columns, scale amax / 448."""
    K = x.shape[-1]
    p = torch.nn.functional.pad(x, (0, _blocks(K) * BLOCK - K)).unflatten(-1, (-1, BLOCK))
    amax = p.abs().amax(-1, keepdim=True)
    s = amax / torch.full_like(amax, FP8_MAX)
    s = torch.where(s == 0, torch.ones_like(s), s)
    q = (p / s).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).float()
    return (q * s).flatten(-2)[..., :K]


def _weight_values(codes, scales, K):
    """[..., N, ld] codes and [..., NB, KB] scales -> fp32 [..., N, K]."""
    N = codes.shape[-2]
    w = codes[..., :K].view(torch.float8_e4m3fn).float()
    s = scales.repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)[..., :K]
    return w * s


def _plain_linear(s):
    K = s["case"]["K"]
    y = _through_fp8(s["a"].float()) @ _weight_values(s["qw"], s["s_w"], K).T
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(torch.bfloat16)


def _plain_route(s):
    c = s["case"]
    E, G, k = c["E"], c["groups"], c["k"]
    x = s["logits"].float()
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-x))
        choice = p if s["bias"] is None else p + s["bias"]
    else:
        e = torch.exp(x - x.amax(-1, keepdim=True))
        p = e / e.sum(-1, keepdim=True)
        choice = x  # the same order as p
    if G > 1:
        by_group = choice.unflatten(-1, (G, E // G))
        if c["score"] == "sigmoid" and E // G > 1:
            top = by_group.sort(dim=-1, descending=True, stable=True).values
            score = top[..., 0] + top[..., 1]
        else:
            score = by_group.amax(-1)
        kept = score.sort(dim=-1, descending=True, stable=True).indices[..., :c["keep"]]
        open_ = torch.zeros_like(score, dtype=torch.bool).scatter_(-1, kept, True)
        choice = torch.where(open_.unsqueeze(-1), by_group, torch.full_like(by_group, -math.inf)).flatten(-2)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[..., :k]
    w = p.gather(-1, ids)
    if c["renorm"]:
        w = w / (w.sum(-1, keepdim=True) + 1e-20)
    return {"ids": ids.to(torch.int32), "weights": w * c["factor"]}


def _plain_experts(s):
    c = s["case"]
    T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]
    ids = s["ids"].long().flatten()
    kept = ids >= 0
    x = _through_fp8(s["x"].float()).repeat_interleave(k, 0)
    if T * k <= E:  # few pairs: each with its own expert's weights
        e = ids.clamp(min=0)
        w13, w2 = (_weight_values(s["qw13"][e], s["s13"][e], H), _weight_values(s["qw2"][e], s["s2"][e], I))
        gu = torch.einsum("ph,pnih->pni", x, w13)
        h = _through_fp8(gu[:, 0] / (1.0 + torch.exp(-gu[:, 0])) * gu[:, 1])
        y = torch.einsum("pi,phi->ph", h, w2)
    else:  # all experts, each with its tokens padded to the busiest one's count
        e = torch.where(kept, ids, torch.full_like(ids, E))  # dropped pairs after all others
        order = e.sort(stable=True).indices
        count = torch.zeros(E + 1, dtype=ids.dtype, device=ids.device).scatter_add_(0, e, torch.ones_like(e))
        place = torch.empty_like(ids)
        place[order] = torch.arange(T * k, device=ids.device) - (count.cumsum(0) - count)[e[order]]
        slot = torch.where(kept, ids * s["most"] + place, torch.full_like(ids, E * s["most"]))
        rows = torch.zeros(E * s["most"] + 1, H, device=x.device)
        rows[slot] = x
        gu = torch.einsum("emh,enih->emni", rows[:-1].view(E, s["most"], H), _weight_values(s["qw13"], s["s13"], H))
        h = _through_fp8(gu[:, :, 0] / (1.0 + torch.exp(-gu[:, :, 0])) * gu[:, :, 1])
        y = torch.bmm(h, _weight_values(s["qw2"], s["s2"], I).transpose(1, 2)).view(-1, H)
        y = torch.cat([y, torch.zeros_like(y[:1])])[slot]
    w = torch.where(kept, s["weights"].flatten(), torch.zeros_like(s["weights"].flatten()))
    y = torch.where(kept[:, None], y, torch.zeros_like(y)) * w[:, None]
    return y.view(T, k, H).sum(1).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if not own:
        return {"linear": _plain_linear, "route": _plain_route, "experts": _plain_experts}[c["op"]](state)
    import fp8_w8a8_quantized_dynamic_gb300 as F
    if c["op"] == "linear":
        return F.fp8_block_linear(state["a"], state["qw"], state["s_w"], state["bias"])
    if c["op"] == "route":
        ids, weights = F.fp8_moe_route(state["logits"], c["k"], score=c["score"], bias=state["bias"],
                                       groups=c["groups"], keep_groups=c["keep"], renormalize=c["renorm"],
                                       factor=c["factor"])
        return {"ids": ids, "weights": weights}
    return F.fp8_moe_experts(state["x"], state["ids"], state["weights"], state["qw13"], state["s13"], state["qw2"],
                             state["s2"])


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _e4m3_64(x):
    """The nearest e4m3 value (ties to even, saturating) of fp64 values that are fp32 numbers."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-FP8_MAX, FP8_MAX)


def _quantized_64(x):
    """x [R, K] fp64 -> its block-quantized values; scale and quotient are fp32 numbers by definition."""
    rows, K = x.shape
    v = torch.zeros(rows, _blocks(K) * BLOCK, dtype=torch.float64, device=x.device)
    v[:, :K] = x
    v = v.view(rows, -1, BLOCK)
    s = (v.abs().amax(2, keepdim=True) / FP8_MAX).float().double()
    s = torch.where(s == 0, 1.0, s)
    return (_e4m3_64((v / s).float().double()) * s).view(rows, -1)[:, :K]


def _decoded_64(codes, scales, K):
    """Codes [N, ld], scales [NB, KB] -> fp64 values, from the bits: sign, 4 exponent, 3 mantissa bits."""
    c = codes[:, :K].int()
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, torch.ldexp(1.0 + m / 8.0, e - 7))
    v = torch.where(c >= 128, -mag, mag)
    rows = torch.arange(v.shape[0], device=v.device) // BLOCK
    cols = torch.arange(K, device=v.device) // BLOCK
    return v * scales.double()[rows][:, cols]


def _exact_route(s):
    c = s["case"]
    E, G, k = c["E"], c["groups"], c["k"]
    x = s["logits"].double()
    if c["score"] == "sigmoid":
        p = torch.sigmoid(x)
        choice = p if s["bias"] is None else p + s["bias"].double()
    else:
        p = torch.softmax(x, -1)
        choice = x
    if G > 1:
        v = choice.view(-1, G, E // G)
        two = 2 if c["score"] == "sigmoid" and E // G > 1 else 1
        score = v.topk(two, -1).values.sum(-1)
        rank = score.argsort(dim=-1, descending=True, stable=True).argsort(-1)
        choice = v.masked_fill((rank >= c["keep"])[..., None], -math.inf).reshape(-1, E)
    ids = choice.argsort(dim=-1, descending=True, stable=True)[:, :k]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return {"ids": None, "weights": w * c["factor"]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "linear":
        a = _quantized_64(s["a"].double())
        y = a @ _decoded_64(s["qw"], s["s_w"], case["K"]).T
        return y if s["bias"] is None else y + s["bias"].double()
    T, E, H, I = case["T"], case["E"], case["H"], case["I"]
    x = _quantized_64(s["x"].double())
    out = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    for e in range(E):
        t, j = (s["ids"] == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        g = x[t] @ _decoded_64(s["qw13"][e, 0], s["s13"][e, 0], H).T
        u = x[t] @ _decoded_64(s["qw13"][e, 1], s["s13"][e, 1], H).T
        h = _quantized_64(g * torch.sigmoid(g) * u)
        out.index_add_(0, t, (h @ _decoded_64(s["qw2"][e], s["s2"][e], I).T) * s["weights"][t, j].double()[:, None])
    return out
