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


# ---------------------------------------------------------------------------
# the experts' networks: sorting by several CTAs, one token, many tiles
# ---------------------------------------------------------------------------

def weights_of(E, H, I, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w13 = (torch.randn((E, 2, I, H), generator=g, device=DEV) * (0.5 / H ** 0.5)).to(torch.bfloat16)
    w2 = (torch.randn((E, H, I), generator=g, device=DEV) * (1.0 / I ** 0.5)).to(torch.bfloat16)
    return (*F.fp8_block_quantize_weight(w13), *F.fp8_block_quantize_weight(w2))


def tokens_of(T, H, seed):
    x = torch.randn((T, H), generator=torch.Generator().manual_seed(seed))
    x[:, 0] *= 20
    return x.to(torch.bfloat16)


def check_experts(x, ids, w, weights, rows=None):
    """All tokens through the library, `rows` of them (default: all) against the oracle; returns the output."""
    q13, s13, q2, s2 = weights
    y = F.fp8_moe_experts(x.to(DEV), ids.to(DEV), w.to(DEV), *weights)
    torch.cuda.synchronize()
    assert F.fp8_last_device_status() == F.FP8_OK
    rows = np.arange(x.shape[0]) if rows is None else np.asarray(rows)
    ref, tol = B.experts(f32(x)[rows], ids.numpy()[rows], w.numpy()[rows], q13.cpu().numpy()[..., :x.shape[1]],
                         s13.cpu().numpy(), q2.cpu().numpy()[..., :q13.shape[2]], s2.cpu().numpy())
    err = np.abs(f32(y).astype(np.float64)[rows] - ref)
    assert np.all(err <= tol), f"max err/tol {np.max(err / tol)}"
    assert np.linalg.norm(err) <= 0.01 * np.linalg.norm(ref) + 1e-30
    return y


def choices(T, E, k, seed, how):
    g = torch.Generator().manual_seed(seed)
    like = torch.randn((T, E), generator=g)
    if how == "skewed":
        like[:, E // 2] += 10  # every token has the same first choice
    ids = like.topk(k, dim=1).indices.to(torch.int32)
    if how == "dropped":       # whole runs of tokens, longer than one CTA's share, and scattered pairs
        ids[T // 5: T // 5 + 700] = -1
        ids[torch.rand((T, k), generator=g) < 0.1] = E
    if how == "one":
        ids[:] = 3
    return ids, torch.rand((T, k), generator=g)


@pytest.mark.parametrize("how", ["even", "skewed", "dropped", "one"])
@pytest.mark.parametrize("T,E,k", [(513, 7, 4), (1500, 24, 4), (2100, 300, 8)])
def test_pairs_sorted_by_several_ctas(T, E, k, how):
    """From 2049 pairs on several CTAs sort them: every token's result is bit for bit that of a run of at most
    2048 pairs, which one CTA sorts, and the oracle's."""
    H, I = 64, 128
    ids, w = choices(T, E, k, T, how)
    x, q = tokens_of(T, H, T + 1), weights_of(E, H, I, 5)
    y = check_experts(x, ids, w, q, rows=np.arange(0, T, max(1, T // 200)))
    step = 2048 // k
    parts = [F.fp8_moe_experts(x[t:t + step].to(DEV), ids[t:t + step].contiguous().to(DEV),
                               w[t:t + step].contiguous().to(DEV), *q) for t in range(0, T, step)]
    assert torch.equal(y, torch.cat(parts))


@pytest.mark.parametrize("k,H,I", [(1, 256, 128), (4, 256, 300), (3, 200, 72), (8, 384, 200), (32, 128, 130)])
def test_one_token(k, H, I):
    """The GEMVs of one token: the blocks of all pairs' h one after the other in K, whatever pairs drop out."""
    E = max(8, k)
    x, q = tokens_of(1, H, k), weights_of(E, H, I, k + 1)
    g = torch.Generator().manual_seed(k)
    ids, w = torch.randperm(E, generator=g)[:k].to(torch.int32)[None], torch.rand((1, k), generator=g)
    y = check_experts(x, ids, w, q)
    for gone in {0, k // 2, k - 1}:          # one pair dropped, below and past the experts; its weight is not read
        for bad in (-1, E, 2 ** 31 - 1, -2 ** 31):
            some, ws = ids.clone(), w.clone()
            some[0, gone] = bad
            z = check_experts(x, some, ws, q) if k > 1 else None
            ws[0, gone] = float("nan")
            nan = F.fp8_moe_experts(x.to(DEV), some.to(DEV), ws.to(DEV), *q)
            assert not nan.any() if k == 1 else torch.equal(nan, z)
    none = F.fp8_moe_experts(x.to(DEV), torch.full((1, k), -1, dtype=torch.int32, device=DEV),
                             torch.full((1, k), float("nan"), device=DEV), *q)
    assert not none.any()
    check_experts(x, torch.full((1, k), 5, dtype=torch.int32), w, q)  # the same expert k times
    xn = x.clone()
    xn[0, H - 1] = float("nan")
    assert torch.isnan(F.fp8_moe_experts(xn.to(DEV), ids.to(DEV), w.to(DEV), *q)).all()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    xd, idd, wd = x.to(DEV), ids.to(DEV), w.to(DEV)
    with torch.cuda.stream(st):
        st.wait_stream(torch.cuda.default_stream())
        ws = torch.full((F.fp8_moe_workspace_bytes(1, k, E, H, I),), 0xFF, dtype=torch.uint8, device=DEV)
        ys = [F.fp8_moe_experts(xd, idd, wd, *q, ws=ws) for _ in range(3)]
    st.synchronize()
    assert all(torch.equal(y, other) for other in ys)


def test_one_token_too_wide_for_the_gemvs_is_sorted():
    """32 pairs of 6000 columns do not fit one SM's shared memory: the token takes the path of several."""
    k, H, I, E = 32, 128, 6000, 3
    x, q = tokens_of(1, H, 1), weights_of(E, H, I, 2)
    # the sorted path's workspace holds fp32 rows of H for each pair, the GEMVs' only their h
    gemvs = [-(-n * F.min_ld(I) * 4 // 256) * 256 for n in (2, k)]
    assert F.fp8_moe_workspace_bytes(1, 2, E, H, I) == gemvs[0]
    assert F.fp8_moe_workspace_bytes(1, k, E, H, I) != gemvs[1]
    ids = torch.arange(k, dtype=torch.int32)[None] % E
    w = torch.rand((1, k), generator=torch.Generator().manual_seed(3))
    y = check_experts(x, ids, w, q)
    ids[0, 5] = -1
    w[0, 5] = 0.0
    check_experts(x, ids, w, q)
    assert not torch.isnan(y).any()


@pytest.mark.parametrize("T,E,k,H,I", [
    (1300, 9, 4, 384, 400),     # 3 blocks of H, 4 of I: about 45 row tiles x 4 on 152 SMs
    (2600, 5, 2, 640, 1100),    # 5 and 9 blocks
    (3000, 40, 3, 1400, 130),   # 11 and 2, odd ends of both widths
    (700, 3, 8, 128, 2050),     # one block of H a tile: a scale slot each
    (5200, 4, 4, 100, 130),     # back in tiles of 128 columns, about 165 of them
    (5200, 4, 4, 64, 300)])     # back in tiles of 64
def test_experts_of_many_tiles(T, E, k, H, I):
    """Several tiles a CTA: barriers, scale slots and tensor-memory buffers carried over the ends of tiles, for
    numbers of K blocks that are no multiple of the scale ring's four."""
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    w = torch.rand((T, k), generator=g)
    rows = np.unique(np.r_[0, 1, T - 1, torch.randint(0, T, (60,), generator=g).numpy()])
    check_experts(tokens_of(T, H, T + 1), ids, w, weights_of(E, H, I, T + 2), rows)


def test_experts_of_a_prompt_batch():
    """The path at full width: about 132 row tiles of 16 columns each, 32 K blocks, against the oracle on
    sampled tokens."""
    T, E, k, H, I = 4096, 8, 4, 4096, 2048
    g = torch.Generator().manual_seed(9)
    ids = torch.randn((T, E), generator=g).topk(k, dim=1).indices.to(torch.int32)
    w = torch.rand((T, k), generator=g)
    check_experts(tokens_of(T, H, 10), ids, w, weights_of(E, H, I, 11), rows=[0, 77, 2048, 4095])


@pytest.mark.parametrize("T,E,k,H,I", [(2000, 6, 8, 4096, 128), (2000, 6, 8, 4096, 200), (3000, 6, 8, 4096, 384),
                                       (20000, 5, 4, 2048, 128), (4000, 6, 8, 128, 2048), (4000, 6, 8, 300, 2048)])
def test_short_k_behind_many_stores(T, E, k, H, I):
    """Tiles of one to three K blocks, whose scales are read while the memory pipe is full of the stores of tiles
    before: the slots of the scale ring may go back only when every lane has its scales. Every run gives the
    same bits, and the oracle's values on sampled tokens."""
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    w, x, q = torch.rand((T, k), generator=g), tokens_of(T, H, 1), weights_of(E, H, I, 2)
    rows = np.unique(np.r_[0, 1, T - 1, torch.randint(0, T, (60,), generator=g).numpy()])
    y = check_experts(x, ids, w, q, rows)
    xd, idd, wd = x.to(DEV), ids.to(DEV), w.to(DEV)
    for _ in range(10):
        assert torch.equal(F.fp8_moe_experts(xd, idd, wd, *q), y)
