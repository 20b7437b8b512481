"""Wider GPU tests of the choice of experts and of the experts' networks: rows with nothing to choose from."""

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


@pytest.mark.parametrize("groups,keep", [(1, 1), (4, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_softmax_row_of_only_masks_follows_the_bias(groups, keep, dtype):
    """A row of only -inf has p = 0 everywhere: the bias alone orders its experts, however small its steps are."""
    E, k = 64, 5
    x = torch.randn((3, E), generator=torch.Generator().manual_seed(1)).to(dtype)
    x[1] = -float("inf")
    bias = torch.arange(E, dtype=torch.float32) * 1e-9
    ids, w = F.fp8_moe_route(x.to(DEV), k, bias=bias.to(DEV), groups=groups, keep_groups=keep, renormalize=True)
    ref, w_ref, _ = B.route(f32(x), k, False, bias.numpy(), groups, keep, True)
    assert ref[1].tolist() == [63, 62, 61, 60, 59]
    assert ids.cpu().numpy().tolist() == ref.tolist()
    assert not w[1].any() and np.allclose(w.cpu().numpy(), w_ref, rtol=(8 + E + k) * 2.0 ** -23, atol=1e-37)
