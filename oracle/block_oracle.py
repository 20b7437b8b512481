"""CPU oracle of the block-scaled FP8 linear, the choice of experts and the experts' networks
(numpy, float64; shares no code with the CUDA side).

Quantization reuses the e4m3 encoder and the fp32 scale rule of fp8_oracle block by block. Products are
float64: with K <= 2**17 every product of two e4m3 codes is a multiple of 2**-18 and the sum of a block
is exact; the sum over blocks carries float64 rounding only (2**-53 relative).
"""

from typing import Optional, Tuple

import numpy as np

from . import fp8_oracle as O

BLOCK = 128
U32 = 2.0 ** -23  # a bound on the relative error of one fp32 operation (round to nearest: half of it)


def blocks_of(n: int) -> int:
    return -(-n // BLOCK)


def quantize_rows(x: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """x fp32 [M, K] -> (codes uint8 [M, K], scales fp32 [KB, M])."""
    M, K = x.shape
    q = np.zeros((M, K), np.uint8)
    s = np.ones((blocks_of(K), M), np.float32)
    for b in range(blocks_of(K)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK].astype(np.float32)
        s[b] = O.scale_from_amax(np.abs(part).max(axis=1))
        q[:, b * BLOCK:(b + 1) * BLOCK] = O.quantize_with_scale(part, s[b][:, None])
    return q, s


def quantize_matrix(w: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """w fp32 [N, K] -> (codes uint8 [N, K], scales fp32 [NB, KB])."""
    N, K = w.shape
    q = np.zeros((N, K), np.uint8)
    s = np.ones((blocks_of(N), blocks_of(K)), np.float32)
    for j in range(s.shape[0]):
        for b in range(s.shape[1]):
            at = np.s_[j * BLOCK:(j + 1) * BLOCK, b * BLOCK:(b + 1) * BLOCK]
            s[j, b] = O.scale_from_amax(O.amax(w[at]))
            q[at] = O.quantize_with_scale(w[at].astype(np.float32), s[j, b])
    return q, s


def scaled_product(qa, s_a, qw, s_w) -> Tuple[np.ndarray, np.ndarray]:
    """(Y, bound) in float64: the block-scaled product and a bound on the error of an fp32 evaluation.

    Within a block the tensor core adds at most min(K, 128) products in fp32; a block then costs the
    product of the two scales, one fma and at most one more addition (K splits). Each of those
    operations is within 2**-23 of its result, whose magnitude the sum of |terms| bounds.
    """
    a, w = O.decode(qa), O.decode(qw)
    M, K = a.shape
    y = np.zeros((M, w.shape[0]))
    mag = np.zeros_like(y)
    for b in range(blocks_of(K)):
        at = slice(b * BLOCK, (b + 1) * BLOCK)
        scale = s_a[b].astype(np.float64)[:, None] * np.repeat(s_w[:, b].astype(np.float64), BLOCK)[None, :w.shape[0]]
        y += scale * (a[:, at] @ w[:, at].T)
        mag += scale * (np.abs(a[:, at]) @ np.abs(w[:, at]).T)
    return y, (min(K, BLOCK) + 3 * blocks_of(K) + 2) * U32 * mag


def linear(a: np.ndarray, qw, s_w, bias: Optional[np.ndarray] = None) -> Tuple[np.ndarray, np.ndarray]:
    """(Y, tolerance) of the linear for fp32 activations: bf16 rounding of the result and the fp32 bound."""
    qa, s_a = quantize_rows(a)
    y, bound = scaled_product(qa, s_a, qw, s_w)
    if bias is not None:
        y = y + bias.astype(np.float64)
        bound = bound + U32 * (np.abs(y) + bound)
    return y, bound + O.ulp_bf16(np.abs(y) + bound)


def route(x: np.ndarray, k: int, sigmoid: bool, bias: Optional[np.ndarray] = None, groups: int = 1, keep: int = 1,
          renorm: bool = False, factor: float = 1.0, group_max: bool = False):
    """(ids [T, k], weights float64 [T, k], margin [T]): margin is the smallest gap between choices that
    the order of the k chosen, or the kept groups, hangs on (0: an exact tie, settled by the index)."""
    x = x.astype(np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    T, E = x.shape
    top = x.max(axis=1, keepdims=True)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if sigmoid:
            p = 1.0 / (1.0 + np.exp(-x))
        else:
            e = np.where(x == top, 1.0, np.exp(x - top))
            p = np.where(np.isneginf(top), 0.0, e / e.sum(axis=1, keepdims=True))
    choice = x.copy() if not sigmoid and bias is None else p + (0.0 if bias is None else bias.astype(np.float64))
    margin = np.full(T, np.inf)
    if groups > 1:
        per = choice.reshape(T, groups, E // groups)
        ordered = -np.sort(-per, axis=2)
        pair = not group_max and (sigmoid or bias is not None) and E // groups > 1
        score = ordered[:, :, 0] + ordered[:, :, 1] if pair else ordered[:, :, 0]
        order = np.argsort(-score, axis=1, kind="stable")
        if keep < groups:
            best = np.take_along_axis(score, order, 1)
            margin = np.minimum(margin, best[:, keep - 1] - best[:, keep])
        gone = np.ones((T, groups), bool)
        np.put_along_axis(gone, order[:, :keep], False, 1)
        choice = np.where(np.repeat(gone, E // groups, axis=1), -np.inf, choice)
    order = np.argsort(-choice, axis=1, kind="stable")
    best = np.take_along_axis(choice, order, 1)
    with np.errstate(invalid="ignore"):
        gaps = best[:, :-1] - best[:, 1:]
    if E > 1:
        margin = np.minimum(margin, np.nan_to_num(gaps[:, :min(k, E - 1)], nan=0.0, posinf=np.inf).min(axis=1))
    ids = order[:, :k]
    w = np.take_along_axis(p, ids, 1)
    if renorm:
        w = w / (w.sum(axis=1, keepdims=True) + 1e-20)
    return ids, w * factor, margin


def _requantize(h, err):
    """Codes' values of h [R, I] fp64 quantized 1 x 128, and a bound on what an evaluation whose h is off by
    at most `err` may give instead: the scale moves by the relative error of the block's maximum, and a
    code moves to its neighbour only where the error reaches a rounding boundary."""
    v, dv = np.zeros_like(h), np.zeros_like(h)
    for b in range(blocks_of(h.shape[1])):
        at = slice(b * BLOCK, (b + 1) * BLOCK)
        x, e = h[:, at], err[:, at]
        amax = np.abs(x).max(axis=1, keepdims=True)
        s = np.where(amax == 0, 1.0, amax / 448.0)
        rel = np.where(amax == 0, 0.0, e.max(axis=1, keepdims=True) / np.where(amax == 0, 1.0, amax)) + 2 * U32
        q = x / s
        dq = np.abs(q) * (rel + U32) + e / s
        lo, mid, hi = (O.decode(O.encode(np.clip(t, -448, 448).astype(np.float32))) for t in (q - dq, q, q + dq))
        v[:, at] = mid * s
        dv[:, at] = np.maximum(np.abs(hi - mid), np.abs(mid - lo)) * s * (1 + rel) + np.abs(mid) * s * rel
    return v, dv


def experts(x, ids, weights, q13, s13, q2, s2) -> Tuple[np.ndarray, np.ndarray]:
    """(Y, tolerance) float64 [T, H] of the experts' networks. q13 [E, 2, I, H], q2 [E, H, I] codes.

    silu's hardware exp and division are off by at most (4 + 2 |g|) units of 2**-23 relative; its slope
    is at most 1.1.
    """
    T, H = x.shape
    E, _, I, _ = q13.shape
    y, tol = np.zeros((T, H)), np.zeros((T, H))
    qa, s_a = quantize_rows(x)
    k = ids.shape[1]
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not t.size:
            continue
        g, dg = scaled_product(qa[t], s_a[:, t], q13[e, 0], s13[e, 0])
        u, du = scaled_product(qa[t], s_a[:, t], q13[e, 1], s13[e, 1])
        silu = g / (1.0 + np.exp(-g))
        h = silu * u
        dsilu = 1.1 * dg + np.abs(silu) * (4 + 2 * np.abs(g)) * U32 + 2.0 ** -126
        dh = dsilu * (np.abs(u) + du) + np.abs(silu) * du + np.abs(h) * U32
        v, dv = _requantize(h, dh)
        w2 = O.decode(q2[e]) * np.repeat(np.repeat(s2[e].astype(np.float64), BLOCK, 0)[:H], BLOCK, 1)[:, :I]
        wt = weights[t, j].astype(np.float64)[:, None]
        out, mag = v @ w2.T, np.abs(v) @ np.abs(w2).T
        d = dv @ np.abs(w2).T + (min(I, BLOCK) + 3 * blocks_of(I) + 2) * U32 * mag
        np.add.at(y, t, wt * out)
        np.add.at(tol, t, np.abs(wt) * (d + (k + 1) * U32 * (mag + d)))
    return y, tol + O.ulp_bf16(np.abs(y) + tol)
