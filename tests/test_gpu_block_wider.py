"""Wider GPU tests of the block-scaled calls: the layout of wide code buffers."""

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
