"""Host checks of the block-scaled linear and the mixture of experts: argument validation before any
device work, and the oracle against exact rational arithmetic."""

from fractions import Fraction

import numpy as np
import pytest

import fp8_w8a8_quantized_dynamic_gb300 as F
from fp8_w8a8_quantized_dynamic_gb300 import _build
from oracle import block_oracle as B
from oracle import fp8_oracle as O

P = 0x7F0000000000  # 256-byte aligned fake address, never read
BAD, MIS, WS = F.FP8_ERR_INVALID_ARG, F.FP8_ERR_MISALIGNED, F.FP8_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    _build.build()
    return F.lib()


def call(fn, defaults, **kw):
    assert set(kw) <= set(defaults)
    return fn(*{**defaults, **kw}.values())


def test_linear_refusals(L):
    d = dict(a=P, M=64, K=200, lda=200, qw=P, N=32, ldqw=208, s_w=P, bias=None, y=P, ldy=32, ws=P, ws_bytes=1 << 20,
             stream=None)
    for kw, want in ((dict(a=None), BAD), (dict(qw=None), BAD), (dict(y=None), BAD), (dict(s_w=None), BAD),
                     (dict(M=-1), BAD), (dict(K=-1), BAD), (dict(N=-1), BAD), (dict(lda=199), BAD),
                     (dict(ldqw=192), BAD), (dict(ldqw=216), MIS), (dict(ldy=31), BAD), (dict(a=P + 1), MIS),
                     (dict(qw=P + 8), MIS), (dict(s_w=P + 2), MIS), (dict(bias=P + 1), MIS), (dict(y=P + 1), MIS),
                     (dict(ws=None), WS), (dict(ws=P + 16), WS), (dict(ws_bytes=100), WS),
                     (dict(M=2 ** 31 - 1), BAD), (dict(M=2 ** 31), BAD)):
        assert call(L.fp8_block_linear, d, **kw) == want, kw
    assert call(L.fp8_block_linear, d, M=0, a=None, y=None, ws=None) == F.FP8_OK
    assert call(L.fp8_block_linear, d, N=0, qw=None, s_w=None, ws=None) == F.FP8_OK
    assert L.fp8_block_workspace_bytes(64, 200, 32) >= 64 * 208 + 2 * 64 * 4
    assert L.fp8_block_workspace_bytes(0, 200, 32) == L.fp8_block_workspace_bytes(64, 0, 32) == 0


def test_quantize_and_mm_refusals(L):
    w = dict(w=P, B=2, N=16, K=64, ldw=64, stride=1024, qw=P, ldq=64, s_w=P, stream=None)
    for kw, want in ((dict(w=None), BAD), (dict(B=-1), BAD), (dict(ldw=63), BAD), (dict(stride=-8), BAD),
                     (dict(ldq=48), BAD), (dict(ldq=72), MIS), (dict(qw=P + 4), MIS), (dict(s_w=None), BAD),
                     (dict(s_w=P + 1), MIS)):
        assert call(L.fp8_block_quantize_weight, w, **kw) == want, kw
    assert call(L.fp8_block_quantize_weight, w, B=0) == F.FP8_OK
    a = dict(a=P, M=4, K=64, lda=64, qa=P, ldq=64, s_a=P, lds=4, stream=None)
    for kw, want in ((dict(a=None), BAD), (dict(lds=3), BAD), (dict(s_a=None), BAD), (dict(s_a=P + 2), MIS),
                     (dict(ldq=32), BAD), (dict(qa=P + 1), MIS)):
        assert call(L.fp8_block_quantize_act, a, **kw) == want, kw
    m = dict(qa=P, M=4, K=64, ldqa=64, s_a=P, lds=4, qw=P, N=8, ldqw=64, s_w=P, bias=None, y=P, ldy=8, stream=None)
    for kw, want in ((dict(qa=None), BAD), (dict(lds=3), BAD), (dict(s_a=None), BAD), (dict(ldqa=72), MIS),
                     (dict(ldqw=48), BAD), (dict(ldy=7), BAD)):
        assert call(L.fp8_block_scaled_mm, m, **kw) == want, kw


def test_route_refusals(L):
    d = dict(x=P, bf16=0, T=4, E=64, ld=64, sigmoid=0, bias=None, groups=1, keep=1, k=8, renorm=0, factor=1.0, ids=P,
             w=P, stream=None)
    for kw, want in ((dict(x=None), BAD), (dict(bf16=2), BAD), (dict(T=-1), BAD), (dict(E=0), BAD), (dict(E=513, ld=513), BAD),
                     (dict(ld=63), BAD), (dict(sigmoid=2), BAD), (dict(groups=0), BAD), (dict(groups=3), BAD),
                     (dict(groups=64, keep=64), BAD), (dict(groups=4, keep=5), BAD), (dict(groups=8, keep=0), BAD),
                     (dict(k=0), BAD), (dict(k=33), BAD), (dict(groups=16, keep=1), BAD), (dict(renorm=-1), BAD),
                     (dict(x=P + 2), MIS), (dict(bias=P + 1), MIS), (dict(ids=None), BAD), (dict(w=P + 3), MIS)):
        assert call(L.fp8_moe_route, d, **kw) == want, kw
    assert call(L.fp8_moe_route, d, T=0, x=None) == F.FP8_OK


def test_experts_refusals(L):
    d = dict(x=P, T=4, H=64, ldx=64, ids=P, w=P, k=2, q13=P, ld13=64, s13=P, q2=P, ld2=48, s2=P, E=8, I=40, y=P, ldy=64,
             ws=P, ws_bytes=1 << 24, stream=None)
    for kw, want in ((dict(x=None), BAD), (dict(T=-1), BAD), (dict(k=0), BAD), (dict(k=33), BAD), (dict(E=0), BAD),
                     (dict(E=513), BAD), (dict(I=0), BAD), (dict(H=-1), BAD), (dict(ldx=63), BAD), (dict(ids=None), BAD),
                     (dict(ids=P + 2), MIS), (dict(w=None), BAD), (dict(q13=None), BAD), (dict(q13=P + 8), MIS),
                     (dict(ld13=48), BAD), (dict(ld2=32), BAD), (dict(ld2=56), MIS), (dict(s13=None), BAD),
                     (dict(s2=P + 1), MIS), (dict(ldy=63), BAD), (dict(y=P + 1), MIS), (dict(ws=None), WS),
                     (dict(ws_bytes=1024), WS), (dict(T=2 ** 30, k=32), BAD)):
        assert call(L.fp8_moe_experts, d, **kw) == want, kw
    assert call(L.fp8_moe_experts, d, T=0, x=None, y=None, ids=None, ws=None) == F.FP8_OK
    need = L.fp8_moe_workspace_bytes(4, 2, 8, 64, 40)
    assert 0 < need <= 1 << 20 and L.fp8_moe_workspace_bytes(0, 2, 8, 64, 40) == 0


# ---------------------------------------------------------------------------
# the oracle's own pins
# ---------------------------------------------------------------------------

def test_oracle_product_is_the_formula():
    """The block-scaled product against exact fractions, and its bound against an fp32 evaluation."""
    r = np.random.default_rng(1)
    M, K, N = 3, 300, 140
    a = r.standard_normal((M, K)).astype(np.float32)
    w = (r.standard_normal((N, K)) * 0.02).astype(np.float32)
    qa, s_a = B.quantize_rows(a)
    qw, s_w = B.quantize_matrix(w)
    y, bound = B.scaled_product(qa, s_a, qw, s_w)
    da, dw = O.decode(qa), O.decode(qw)
    for m, n in ((0, 0), (1, 127), (2, 128), (0, 139)):
        want = sum(Fraction(float(s_a[k // 128, m])) * Fraction(float(s_w[n // 128, k // 128])) *
                   Fraction(float(da[m, k])) * Fraction(float(dw[n, k])) for k in range(K))
        assert abs(Fraction(float(y[m, n])) - want) <= Fraction(1, 2 ** 48) * abs(want) + Fraction(1, 2 ** 80)
    f = np.zeros((M, N), np.float32)
    for b in range(3):
        at = slice(128 * b, 128 * b + 128)
        s = s_a[b][:, None] * np.repeat(s_w[:, b], 128)[None, :N]
        f += s * (da[:, at].astype(np.float32) @ dw[:, at].astype(np.float32).T)
    assert np.all(np.abs(f - y) <= bound)
    assert not np.all(np.abs(f * np.float32(1.001) - y) <= bound)


def test_oracle_quantization_blocks():
    """Each block maps its own maximum to 448, whatever its neighbours hold."""
    x = np.ones((2, 260), np.float32)
    x[0, :128] = 3.0
    x[1, 128:256] = 0.0
    x[1, 258] = -7.0
    q, s = B.quantize_rows(x)
    assert s.shape == (3, 2) and s[1, 1] == 1.0
    assert np.all(O.decode(q)[0] == 448) and not O.decode(q)[1, 128:256].any()
    assert O.decode(q)[1, 258] == -448 and abs(O.decode(q)[1, 256] - 64) == 0
    w = np.ones((200, 130), np.float32)
    w[199, 129] = 14.0
    q, s = B.quantize_matrix(w)
    assert s.shape == (2, 2) and s[1, 1] == np.float32(14 / 448) and s[0, 1] == np.float32(1 / 448)
    assert O.decode(q)[198, 129] == 32 and O.decode(q)[0, 129] == 448


def test_oracle_route_by_hand():
    x = np.array([[0.0, 2.0, 1.0, 2.0, -1.0, 5.0]], np.float32)
    ids, w, margin = B.route(x, 3, False)
    assert ids.tolist() == [[5, 1, 3]] and margin[0] == 0.0
    p = np.exp(x[0].astype(np.float64) - 5)
    assert np.allclose(w[0], p[[5, 1, 3]] / p.sum(), rtol=1e-14)
    # groups {0, 1}, {2, 3}, {4, 5}: the two sigmoids sum to 1.38, 1.61, 1.26, so the last group goes; 1 and 3 tie
    ids, w, _ = B.route(x, 2, True, groups=3, keep=2, renorm=True)
    assert ids.tolist() == [[1, 3]] and abs(w.sum() - 1) < 1e-12
    # the bias steers the choice and not the weight
    ids, w, _ = B.route(x, 1, True, bias=np.array([9, 0, 0, 0, 0, 0], np.float32))
    assert ids.tolist() == [[0]] and w[0, 0] == 0.5


def test_oracle_experts_identity():
    """One expert with weight 1 is the plain gated network of the quantized values."""
    r = np.random.default_rng(2)
    T, H, I = 4, 160, 96
    x = r.standard_normal((T, H)).astype(np.float32)
    q13, s13 = zip(*(B.quantize_matrix((r.standard_normal((I, H)) * 0.05).astype(np.float32)) for _ in range(2)))
    q2, s2 = B.quantize_matrix((r.standard_normal((H, I)) * 0.05).astype(np.float32))
    y, tol = B.experts(x, np.zeros((T, 1), int), np.ones((T, 1), np.float32), np.stack(q13)[None], np.stack(s13)[None],
                       q2[None], s2[None])
    qa, s_a = B.quantize_rows(x)
    g, u = (B.scaled_product(qa, s_a, q13[i], s13[i])[0] for i in range(2))
    h = (g / (1 + np.exp(-g)) * u).astype(np.float32)
    want, _ = B.scaled_product(*B.quantize_rows(h), q2, s2)
    assert np.all(np.abs(y - want) <= tol)
    assert np.linalg.norm(tol) < 0.05 * np.linalg.norm(want)
