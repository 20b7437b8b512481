"""Wider GPU tests of the choice of experts and of the experts' networks: rows with nothing to choose from,
the rules of a group's score, gates far below zero."""

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


@pytest.mark.parametrize("T,E,k,groups,keep", [(1, 256, 8, 8, 4), (200, 256, 8, 8, 4), (33, 12, 3, 3, 2),
                                               (20, 96, 3, 32, 2), (11, 8, 2, 8, 2), (300, 512, 16, 16, 4)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_groups_scored_by_their_best_choice(T, E, k, groups, keep, score, with_bias):
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn((T, E), generator=g) * 1.5
    bias = torch.randn(E, generator=g) * 0.1 if with_bias else None
    kw = dict(score=score, bias=None if bias is None else bias.to(DEV), groups=groups, keep_groups=keep,
              renormalize=True, factor=2.5)
    ids, w = F.fp8_moe_route(x.to(DEV), k, group_score="max", **kw)
    ex = F.fp8_moe_route_ex(x.to(DEV), k, "max", **kw)
    assert torch.equal(ids, ex[0]) and torch.equal(w, ex[1])
    b = None if bias is None else bias.numpy()
    ref, w_ref, margin = B.route(x.numpy(), k, score == "sigmoid", b, groups, keep, True, 2.5, group_max=True)
    rows = margin > 2.0 ** -19  # scores are a few fp32 operations from the exact ones, all below 4
    assert rows.mean() > 0.9 and np.array_equal(ids.cpu().numpy()[rows], ref[rows])
    tol = (8 + E + k) * 2.0 ** -23 * np.abs(w_ref) + 1e-37
    assert np.all(np.abs(w.cpu().numpy() - w_ref)[rows] <= tol[rows])


def test_group_score_rules_differ():
    """Group 0 holds the best expert, group 1 the best two: sigmoid without a bias, one group kept."""
    x = torch.tensor([[2.0, -4.0, 1.5, 1.5]], device=DEV)
    kw = dict(score="sigmoid", groups=2, keep_groups=1)
    assert F.fp8_moe_route(x, 2, **kw)[0].tolist() == [[2, 3]]
    assert F.fp8_moe_route(x, 2, group_score="max", **kw)[0].tolist() == [[0, 1]]
    with pytest.raises(ValueError):
        F.fp8_moe_route(x, 2, group_score="sum", **kw)


@pytest.mark.parametrize("T", [1, 5, 300])
@pytest.mark.parametrize("gate", [-80.0, -88.0, 88.0])
def test_experts_far_gates(T, gate):
    """silu(g) stays itself where exp(-g) is near the largest fp32 number: -88 e^-88 = -5.3e-37 is a normal
    one. With |g| = 88 a fp32 exp of g, itself off by 2**-23 of 88, is off by about 1e-5: far below 0.01."""
    H, I, u = 128, 128, 2.0 ** 40
    x = torch.zeros((T, H))
    x[:, 0] = 1.0
    x = x.to(torch.bfloat16)
    w13 = torch.zeros((1, 2, I, H))
    w13[0, 0, :, 0], w13[0, 1, :, 0] = gate, u
    w2 = torch.randn((1, H, I), generator=torch.Generator().manual_seed(2))
    q13, s13 = F.fp8_block_quantize_weight(w13.to(torch.bfloat16).to(DEV))
    q2, s2 = F.fp8_block_quantize_weight(w2.to(torch.bfloat16).to(DEV))
    ids, w = torch.zeros((T, 1), dtype=torch.int32), torch.ones((T, 1))
    y = f32(F.fp8_moe_experts(x.to(DEV), ids.to(DEV), w.to(DEV), q13, s13, q2, s2)).astype(np.float64)
    ref, _ = B.experts(f32(x), ids.numpy(), w.numpy(), q13.cpu().numpy(), s13.cpu().numpy(), q2.cpu().numpy(),
                       s2.cpu().numpy())
    assert np.linalg.norm(ref) > 1e-24
    assert np.linalg.norm(y - ref) <= 0.01 * np.linalg.norm(ref)
