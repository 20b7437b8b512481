"""CPU oracle of the norms around a block, of the adapters beside a projection and of tokens sorted by
expert and back (numpy, float64; shares no code with the CUDA side). Each returns its result and a bound
on what an fp32 evaluation with the stated roundings may be off by.
"""

from typing import Optional, Tuple

import numpy as np

U = 2.0 ** -24        # half a step of fp32, relative: one rounding to nearest
HALF_BF16 = 2.0 ** -8  # half a step of bf16, relative (eps / 2)
TINY = 2.0 ** -126    # smallest normal number: below it roundings are absolute


def rounded_bf16(y: np.ndarray, err: np.ndarray) -> np.ndarray:
    """The bound of a result with bound err after its rounding to bf16."""
    return err + (np.abs(y) + err) * HALF_BF16 + TINY


def _inverse_rms(x: np.ndarray, err: np.ndarray, eps: float):
    """(1 / sqrt(mean x^2 + eps), its relative bound) per row, for x off by at most err.

    The kernel's sum of squares: two chains of at most eight fmas of packed pairs in a thread, their sum and the pair's, five
    halvings over its warp's lanes, and at most 32 warps' by fours (two and eight): 25 roundings of positive sums; then the
    rounded 1 / count, and one fma with it and eps: 27. The root halves what came before it and is
    itself correctly rounded.
    """
    mean = np.mean(x * x, axis=1, keepdims=True) + eps
    inv = 1.0 / np.sqrt(mean)
    rel = (27 / 2 + 1) * U + np.mean(np.abs(x) * err + err * err, axis=1, keepdims=True) * inv * inv
    return inv, rel


def norms(y, weight=None, residual=None, post=None, gate=None, scale: float = 1.0, eps: float = 1e-6,
          plus_one: bool = False):
    """(n, n's bound, r, r's bound) before any rounding to bf16 or to codes; n is None without a weight."""
    offset = 1.0 if plus_one else 0.0
    scale, eps = float(np.float32(scale)), float(np.float32(eps))
    t = y.astype(np.float64)
    err = np.zeros_like(t)
    if post is not None:
        inv, rel = _inverse_rms(t, err, eps)
        t = t * inv * (post.astype(np.float64) + offset)
        err = np.abs(t) * (rel + 3 * U) + TINY  # times inv, offset + weight, times that
    if gate is not None:
        t = t * gate.astype(np.float64)
        err = err * np.abs(gate.astype(np.float64)) + (np.abs(t) + err * np.abs(gate.astype(np.float64))) * U + TINY
    r = scale * t + (0.0 if residual is None else residual.astype(np.float64))
    err = abs(scale) * err + (np.abs(r) + abs(scale) * err) * U + TINY  # one fma
    if weight is None:
        return None, None, r, err
    inv, rel = _inverse_rms(r, err, eps)
    w = weight.astype(np.float64) + offset
    n = r * inv * w
    moved = err * inv * np.abs(w)
    return n, (np.abs(n) + moved) * (rel + 3 * U) + moved + TINY, r, err


def sort_rows(ids: np.ndarray, E: int) -> Tuple[np.ndarray, np.ndarray]:
    """(pos int32 [T, k], offsets int32 [E + 1])."""
    flat = ids.reshape(-1)
    pos = np.full(flat.shape, -1, np.int32)
    offsets = np.zeros(E + 1, np.int32)
    row = 0
    for e in range(E):
        offsets[e] = row
        at = np.nonzero(flat == e)[0]
        pos[at] = row + np.arange(at.size)
        row += at.size
    offsets[E] = row
    return pos.reshape(ids.shape), offsets


def combine(ys: np.ndarray, pos: np.ndarray, weights: Optional[np.ndarray]) -> Tuple[np.ndarray, np.ndarray]:
    """(y, bound): one fma a pair, in fp32."""
    T, k = pos.shape
    y = np.zeros((T, ys.shape[1]))
    mag = np.zeros_like(y)
    for j in range(k):
        t = np.nonzero((pos[:, j] >= 0) & (pos[:, j] < ys.shape[0]))[0]
        term = ys[pos[t, j]].astype(np.float64) * (1.0 if weights is None else weights[t, j].astype(np.float64)[:, None])
        y[t] += term
        mag[t] += np.abs(term)
    return y, (k + 1) * U * mag + TINY


def combine_grad(dy: np.ndarray, ys: np.ndarray, pos: np.ndarray, weights: np.ndarray):
    """(dys float64 [R, H] with NaN in rows of no pair, dw, dw's bound). dys rounds once in fp32 and once to its type. A
    dot product: ceil(H / threads) fmas of a thread (one column at a time at most H / 32), five halvings, eight warps."""
    T, k = pos.shape
    H = dy.shape[1]
    dys = np.full(ys.shape, np.nan)
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            d = pos[t, j]
            if 0 <= d < ys.shape[0]:
                dys[d] = dy[t].astype(np.float64) * float(weights[t, j])
                terms = dy[t].astype(np.float64) * ys[d].astype(np.float64)
                dw[t, j], mag[t, j] = terms.sum(), np.abs(terms).sum()
    return dys, dw, (-(-H // 32) + 14) * U * mag + TINY


def lora(y, x, a, b, ids, scales=None) -> Tuple[np.ndarray, np.ndarray]:
    """(out, bound) before the rounding to bf16. Sums of K and of 3 r products in fp32 in any order, 2**-23 a step (a
    tensor core may cut instead of round): v passes it as the sum of three bf16 numbers of eight bits each, which are all
    24 of it (what is below 2**-133, the smallest bf16 number, is part of TINY); one fma."""
    M, K = x.shape
    L, r, _ = a.shape
    out = y.astype(np.float64)
    err = np.zeros_like(out)
    for e in range(L):
        t = np.nonzero(ids == e)[0]
        if not t.size:
            continue
        A, Bm, X = (v.astype(np.float64) for v in (a[e], b[e], x[t]))
        s = 1.0 if scales is None else float(scales[e])
        v = X @ A.T
        dv = (K + 16) * 2 * U * (np.abs(X) @ np.abs(A).T) + TINY
        d = v @ Bm.T
        dd = dv @ np.abs(Bm).T + (3 * r + 8) * 2 * U * ((np.abs(v) + dv) @ np.abs(Bm).T)
        out[t] += s * d
        err[t] = abs(s) * dd
        err[t] += (np.abs(out[t]) + err[t]) * U + TINY
    return out, err
