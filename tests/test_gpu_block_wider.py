"""Wider GPU tests of the block-scaled calls: the layout of wide code buffers, products of many tiles, the
linear against its two steps."""

import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_dynamic_gb300 as F
from fp8_w8a8_quantized_dynamic_gb300 import _build
from oracle import block_oracle as B
from parity import f32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    F.lib()


def rand(shape, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(torch.bfloat16)


def stream():
    return torch.cuda.current_stream().cuda_stream


# (rows, K, ld): the smallest ld, one that ends in the last block, some past it, by a little and by several blocks
WIDE = [(5, 100, 112), (5, 100, 128), (33, 100, 144), (7, 300, 400), (130, 128, 256), (200, 257, 1040), (3, 1, 4096),
        (4, 0, 16), (4, 0, 144)]


@pytest.mark.parametrize("M,K,ld", WIDE)
def test_quantize_act_writes_zeros_to_the_end_of_each_row(M, K, ld):
    a = rand((M, K), M + K)
    q = torch.full((M + 1, ld), 0xFF, dtype=torch.uint8, device=DEV)
    kb, lds = -(-K // 128), M + 3
    s = torch.full((kb + 1, lds), 7.0, device=DEV)
    ad = a.to(DEV)
    assert F.lib().fp8_block_quantize_act(ad.data_ptr(), M, K, max(K, 1), q.data_ptr(), ld, s.data_ptr(), lds, stream()) == 0
    q_ref, s_ref = B.quantize_rows(f32(a))
    got, sc = q.cpu().numpy(), s.cpu().numpy()
    assert np.array_equal(got[:M, :K], q_ref) and not got[:M, K:].any() and (got[M] == 0xFF).all()
    assert np.array_equal(sc[:kb, :M], s_ref) and (sc[:kb, M:] == 7).all() and (sc[kb] == 7).all()


@pytest.mark.parametrize("N,K,ld", WIDE)
def test_quantize_weight_writes_zeros_to_the_end_of_each_row(N, K, ld):
    w = rand((2, N, K), N + K + 1, 0.05)
    q = torch.full((2 * N + 1, ld), 0xFF, dtype=torch.uint8, device=DEV)
    nb, kb = -(-N // 128), -(-K // 128)
    s = torch.full((2 * nb * kb + 5,), 7.0, device=DEV)
    wd = w.to(DEV)
    assert F.lib().fp8_block_quantize_weight(wd.data_ptr(), 2, N, K, max(K, 1), N * K, q.data_ptr(), ld, s.data_ptr(),
                                             stream()) == 0
    got, sc = q.cpu().numpy(), s.cpu().numpy()
    for i in range(2):
        q_ref, s_ref = B.quantize_matrix(f32(w[i]))
        assert np.array_equal(got[i * N:(i + 1) * N, :K], q_ref)
        assert np.array_equal(sc[i * nb * kb:(i + 1) * nb * kb], s_ref.ravel())
    assert not got[:2 * N, K:].any() and (got[2 * N] == 0xFF).all() and (sc[2 * nb * kb:] == 7).all()


@pytest.mark.parametrize("M,K,N", [
    (5000, 384, 2048), (2500, 640, 4104),      # 256 columns a tile, 3 and 5 K blocks
    (4000, 128, 3001), (2500, 640, 4099),      # rows of any alignment
    (25000, 384, 120), (25000, 384, 121),      # 128 columns
    (40000, 640, 40), (40000, 640, 33),        # 64 columns
    (1000, 4096, 8200), (1000, 4096, 8195)])   # weights past 28 MB: two raster groups, the last one short
def test_many_tiles(M, K, N):
    """Several tiles a CTA: barriers, scale slots and tensor-memory buffers carried over the ends of tiles.
    Sampled rows and whole blocks of columns against the oracle, into a buffer with canaries around it."""
    a, b = rand((M, K), M), rand((N,), N + 1)
    w = (torch.randn((N, K), generator=torch.Generator(device=DEV).manual_seed(N), device=DEV) * 0.02).to(torch.bfloat16)
    qw, s_w = F.fp8_block_quantize_weight(w)
    pad = 8 if N % 8 == 0 else 3
    wide = torch.full((M + 2, N + 2 * pad), 768.0, dtype=torch.bfloat16, device=DEV)
    F.fp8_block_linear(a.to(DEV), qw, s_w, b.to(DEV), out=wide[1:M + 1, pad:pad + N])
    torch.cuda.synchronize()
    assert F.fp8_last_device_status() == F.FP8_OK
    assert bool((wide[0] == 768).all()) and bool((wide[M + 1] == 768).all())
    assert bool((wide[:, :pad] == 768).all()) and bool((wide[:, pad + N:] == 768).all())
    nb = -(-N // 128)
    blocks = sorted({0, nb // 3, nb // 2, max(0, nb - 2), nb - 1})  # the last, which may be short, comes last
    cols = np.concatenate([np.arange(j * 128, min(N, j * 128 + 128)) for j in blocks])
    rows = np.unique(np.r_[0, 127, 128, M // 2, M - 1, np.random.default_rng(M).integers(0, M, 40)])
    ref, tol = B.linear(f32(a)[rows], qw.cpu().numpy()[cols, :K], s_w.cpu().numpy()[blocks], f32(b)[cols])
    got = f32(wide[1:M + 1, pad:pad + N])[np.ix_(rows, cols)].astype(np.float64)
    assert np.all(np.abs(got - ref) <= tol), f"max err/tol {np.max(np.abs(got - ref) / tol)}"


@pytest.mark.parametrize("M,K,N", [(1, 1000, 330), (3, 700, 330), (4, 4096, 512), (9, 1000, 257), (16, 700, 330),
                                   (17, 700, 330), (30, 2049, 640), (200, 5632, 520), (1300, 384, 2056)])
def test_two_steps_give_the_linears_bits(M, K, N):
    """Quantizing in a kernel of its own or in the product's: the same codes, scales and order of sums."""
    a, b = rand((M, K), M).to(DEV), rand((N,), N).to(DEV)
    qw, s_w = F.fp8_block_quantize_weight(rand((N, K), K, 0.02).to(DEV))
    qa, s_a = F.fp8_block_quantize_act(a)
    assert torch.equal(F.fp8_block_scaled_mm(qa, K, s_a, qw, s_w, b), F.fp8_block_linear(a, qw, s_w, b))


def test_rows_that_overlap_are_refused():
    row = rand((1, 256), 1).to(DEV)
    qw, s_w = F.fp8_block_quantize_weight(rand((64, 256), 2).to(DEV))
    out = torch.empty((1, 64), dtype=torch.bfloat16, device=DEV)
    for call in (lambda: F.fp8_block_linear(row.expand(40, 256), qw, s_w), lambda: F.fp8_block_quantize_act(row.expand(2, 256)),
                 lambda: F.fp8_block_linear(row.expand(40, 256).contiguous(), qw, s_w, out=out.expand(40, 64)),
                 lambda: F.fp8_block_quantize_weight(row.expand(3, 256)),
                 lambda: F.fp8_moe_route(torch.zeros((1, 16), device=DEV).expand(5, 16), 2)):
        with pytest.raises(F.FP8Error) as e:
            call()
        assert e.value.status == F.FP8_ERR_INVALID_ARG
    assert torch.equal(F.fp8_block_linear(row.expand(40, 256).contiguous(), qw, s_w)[7:8],
                       F.fp8_block_linear(row.expand(40, 256).contiguous(), qw, s_w)[:1])


@pytest.mark.parametrize("M,K,N", [(16000, 128, 4096), (16000, 256, 4096), (16000, 384, 4099), (30000, 128, 120),
                                   (40000, 200, 40)])
def test_short_k_repeats(M, K, N):
    """Tiles of one to three K blocks, bound by their stores: the same bits on every run, the oracle's values."""
    a, w = rand((M, K), 1).to(DEV), rand((N, K), 2, 0.05).to(DEV)
    qw, s_w = F.fp8_block_quantize_weight(w)
    y = F.fp8_block_linear(a, qw, s_w)
    for _ in range(10):
        assert torch.equal(F.fp8_block_linear(a, qw, s_w), y)
    rows = np.unique(np.r_[0, M - 1, np.random.default_rng(M).integers(0, M, 60)])
    at = torch.from_numpy(rows).to(DEV)
    ref, tol = B.linear(f32(a[at]), qw.cpu().numpy()[:, :K], s_w.cpu().numpy())
    assert np.all(np.abs(f32(y[at]).astype(np.float64) - ref) <= tol)
