"""Offsets past 32 bits: operands and results of more than 2**31 elements, sampled rows against the oracle. Up to
about 25 GB of device memory at a time."""

import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_dynamic_gb300 as F
from fp8_w8a8_quantized_dynamic_gb300 import _build
from oracle import block_oracle as B
from parity import f32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAST = 2 ** 31


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    F.lib()
    yield
    torch.cuda.empty_cache()


def rand(shape, seed, std=1.0):
    """Random bf16 values, made on the device in pieces."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    for part in out.view(-1, shape[-1]).split(1 << 16):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV) * std)
    return out


def sampled(n, seed=0):
    return np.unique(np.r_[0, 1, n // 2, n - 2, n - 1, np.random.default_rng(seed).integers(0, n, 20)])


@pytest.mark.parametrize("M,K,N", [(530000, 4100, 4099), (530000, 4096, 4104)])
def test_linear(M, K, N):
    assert M * K > PAST and M * N > PAST
    a = rand((M, K), 1)
    qw, s_w = F.fp8_block_quantize_weight(rand((N, K), 2, 0.02))
    y = F.fp8_block_linear(a, qw, s_w)
    torch.cuda.synchronize()
    assert F.fp8_last_device_status() == F.FP8_OK
    rows = sampled(M)
    ref, tol = B.linear(f32(a[torch.from_numpy(rows).to(DEV)]), qw.cpu().numpy()[:, :K], s_w.cpu().numpy())
    err = np.abs(f32(y[torch.from_numpy(rows).to(DEV)]).astype(np.float64) - ref)
    assert np.all(err <= tol), f"max err/tol {np.max(err / tol)}"


def test_weights():
    """A batch of matrices past 2**31 elements, the last ones through the linear."""
    B_, N, K = 130, 4096, 4112
    assert B_ * N * K > PAST
    w = rand((B_, N, K), 3, 0.02)
    q, s = F.fp8_block_quantize_weight(w)
    for i, j, b in ((0, 0, 0), (B_ // 2, 31, 31), (B_ - 1, 31, 32), (B_ - 1, 0, 3)):
        at = np.s_[j * 128:(j + 1) * 128, b * 128:min(K, (b + 1) * 128)]
        q_ref, s_ref = B.quantize_matrix(f32(w[i][at]))
        assert np.array_equal(q[i][at].cpu().numpy(), q_ref)
        assert float(s[i, j, b]) == float(s_ref[0, 0])
    x = rand((40, K), 4)
    for i in (0, B_ - 1):
        assert torch.equal(F.fp8_block_linear(x, q[i], s[i]),
                           F.fp8_block_linear(x, *F.fp8_block_quantize_weight(w[i])))


def test_quantize_rows_past_the_32_bit_index():
    """2**28 rows of one column are 2**31 units of sixteen columns: the kernel's 64-bit index."""
    M = 2 ** 28 + 5
    g = torch.Generator(device=DEV).manual_seed(5)
    a = torch.empty((M, 1), dtype=torch.bfloat16, device=DEV)
    for part in a.split(1 << 24):
        part.copy_(torch.randn(part.shape, generator=g, device=DEV))
    q, s = F.fp8_block_quantize_act(a)
    torch.cuda.synchronize()
    for at in (slice(0, 1 << 20), slice(M // 2, M // 2 + (1 << 20)), slice(M - (1 << 20), M)):
        x = a[at, 0].float()
        zero, neg = x == 0, torch.signbit(x)
        code = torch.where(zero, 0, 0x7E) + torch.where(neg, 0x80, 0)
        assert torch.equal(q[at, 0].int(), code.int()) and not q[at, 1:].any()
        assert torch.equal(s[0, at], torch.where(zero, torch.ones_like(x), x.abs() / torch.full_like(x, 448.0)))


def test_experts():
    """The pairs' fp32 rows pass 2**31 elements."""
    T, E, k, H, I = 70000, 6, 8, 4096, 128
    assert T * k * H > PAST
    x = rand((T, H), 6)
    ids = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(7), dtype=torch.int32)
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(8))
    q13, s13 = F.fp8_block_quantize_weight(rand((E, 2, I, H), 9, 0.5 / H ** 0.5))
    q2, s2 = F.fp8_block_quantize_weight(rand((E, H, I), 10, I ** -0.5))
    y = F.fp8_moe_experts(x, ids.to(DEV), w.to(DEV), q13, s13, q2, s2)
    torch.cuda.synchronize()
    assert F.fp8_last_device_status() == F.FP8_OK
    rows = sampled(T)
    at = torch.from_numpy(rows).to(DEV)
    ref, tol = B.experts(f32(x[at]), ids.numpy()[rows], w.numpy()[rows], q13.cpu().numpy(), s13.cpu().numpy(),
                         q2.cpu().numpy(), s2.cpu().numpy())
    err = np.abs(f32(y[at]).astype(np.float64) - ref)
    assert np.all(err <= tol), f"max err/tol {np.max(err / tol)}"


def test_route():
    T, E, k = 4200000, 512, 8
    assert T * E > PAST
    x = rand((T, E), 11, 1.5)
    ids, w = F.fp8_moe_route(x, k, renormalize=True)
    rows = sampled(T)
    at = torch.from_numpy(rows).to(DEV)
    ref, w_ref, _ = B.route(f32(x[at]), k, False, renorm=True)
    assert np.array_equal(ids[at].cpu().numpy(), ref)
    assert np.allclose(w[at].cpu().numpy(), w_ref, rtol=(8 + E + k) * 2.0 ** -23, atol=1e-37)
