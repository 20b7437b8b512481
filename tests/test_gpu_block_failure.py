"""Failure detection of the block-scaled product without a GPU fault: one load is withheld from the waits of
its first CTA, they run out after 20 ms, the error is reported once, nothing of the tile is stored (in a
tile whose K two CTAs share, by neither of them) and the next product is right. Nothing faults or hangs."""

import time

import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_dynamic_gb300 as F
from fp8_w8a8_quantized_dynamic_gb300 import _build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    F.lib()


def rand(shape, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(torch.bfloat16).to(DEV)


def withheld(form, qa, K, s_a, qw, s_w, y, s_y=None):
    torch.cuda.synchronize()
    assert F.fp8_last_device_status() == F.FP8_OK  # nothing pending
    t0 = time.perf_counter()
    assert F.fp8_block_selftest_timeout(form, qa, K, s_a, qw, s_w, y, s_y) == F.FP8_OK
    assert F.fp8_last_device_status() == F.FP8_ERR_TIMEOUT
    assert 0.02 <= time.perf_counter() - t0 < 5.0  # the wait ran out, it did not hang
    assert F.fp8_last_device_status() == F.FP8_OK  # reported once, then cleared


@pytest.mark.parametrize("form,M,K,N,width", [
    (1, 40, 256, 64, 64),        # one tile, two CTAs: no row of it may be stored
    (1, 300, 1152, 200, 64),     # the other tiles are whole
    (0, 40, 128, 256, 256),      # one tile of one K block: nothing is loaded
    (0, 300, 700, 520, 256),     # a tile a CTA
    (0, 2600, 384, 2056, 256)])  # the CTA had a second tile to do
def test_unfinished_tile_is_not_stored(form, M, K, N, width):
    a = rand((M, K), M)
    qw, s_w = F.fp8_block_quantize_weight(rand((N, K), N, 0.02))
    qa, s_a = F.fp8_block_quantize_act(a)
    want = F.fp8_block_scaled_mm(qa, K, s_a, qw, s_w).float().cpu().numpy()
    y = torch.full((M, N), 768.0, dtype=torch.bfloat16, device=DEV)
    withheld(form, qa, K, s_a, qw, s_w, y)
    got = y.float().cpu().numpy()
    kept = got == 768.0
    assert not (want == 768.0).any() and kept[:128, :width].all()
    tiles = [(i, j) for i in range(0, M, 128) for j in range(0, N, width)]
    lost = 0
    for i, j in tiles:
        tile = np.s_[i:i + 128, j:j + width]
        if kept[tile].all():
            lost += 1
        else:  # other splits of K round differently: an ulp of bf16
            assert np.allclose(got[tile], want[tile], rtol=2.0 ** -7, atol=1e-3)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert lost == (1 if form == 1 else len(range(0, len(tiles), sms)))
    again = F.fp8_block_scaled_mm(qa, K, s_a, qw, s_w).float().cpu().numpy()
    assert F.fp8_last_device_status() == F.FP8_OK and np.array_equal(again, want)


@pytest.mark.parametrize("M,K,N", [(90, 256, 128), (300, 640, 400), (2600, 256, 1100)])
def test_unfinished_swiglu_tile_is_not_stored(M, K, N):
    """The warps that meet for a tile's rows all come to the meetings of the tiles left undone."""
    qw, s_w = F.fp8_block_quantize_weight(rand((2, N, K), N, 0.05))
    qa, s_a = F.fp8_block_quantize_act(rand((M, K), M))
    ld, nb = F.min_ld(N), (N + 127) // 128
    y = torch.full((M, ld), 0xEE, dtype=torch.uint8, device=DEV)
    s_y = torch.full((nb, M), 768.0, device=DEV)
    withheld(2, qa, K, s_a, qw, s_w, y, s_y)
    got, s = y.cpu().numpy(), s_y.cpu().numpy()
    tiles = [(i, j) for i in range(0, M, 128) for j in range(nb)]
    kept = [(s[j, i:i + 128] == 768.0).all() for i, j in tiles]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert kept[0] and sum(kept) == len(range(0, len(tiles), sms))
    for (i, j), k in zip(tiles, kept):
        assert (got[i:i + 128, 128 * j:128 * j + 128] == 0xEE).all() == k
        assert not (s[j, i:i + 128] == 768.0).any() or k
    # the experts' networks are right afterwards
    x, w = rand((M, K), 5), torch.ones((M, 1), device=DEV)
    ids = torch.zeros((M, 1), dtype=torch.int32, device=DEV)
    q2, s2 = F.fp8_block_quantize_weight(rand((1, K, N), 6, 0.05))
    args = (x, ids, w, qw[None], s_w[None], q2, s2)
    assert torch.equal(F.fp8_moe_experts(*args), F.fp8_moe_experts(*args))
    assert F.fp8_last_device_status() == F.FP8_OK


def test_refusals():
    qw, s_w = F.fp8_block_quantize_weight(rand((64, 128), 1))
    qa, s_a = F.fp8_block_quantize_act(rand((40, 128), 2))
    y = torch.empty((40, 64), dtype=torch.bfloat16, device=DEV)

    def call(form=0, M=40, K=128, N=64, ldy=64, y=y.data_ptr()):
        return F.lib().fp8_block_selftest_timeout(form, qa.data_ptr(), M, K, 128, s_a.data_ptr(), s_a.stride(0),
                                                  qw.data_ptr(), N, 128, s_w.data_ptr(), y, ldy, None, 0, None)
    for kw in (dict(form=3), dict(form=-1), dict(M=0), dict(K=0), dict(N=0), dict(N=60), dict(ldy=68), dict(form=1),
               dict(form=2), dict(y=None), dict(ldy=56)):
        assert call(**kw) == F.FP8_ERR_INVALID_ARG, kw
    assert call(y=y.data_ptr() + 2) == F.FP8_ERR_MISALIGNED
