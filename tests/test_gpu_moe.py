"""GPU parity of the choice of experts and of the experts' networks against the float64 oracle."""

import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_dynamic_gb300 as F
from fp8_w8a8_quantized_dynamic_gb300 import _build
from oracle import block_oracle as B
from parity import assert_guards_intact, f32, guarded

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# Scores are one or two fp32 operations from the exact ones (all below 4, so off by less than 2**-20):
# an order that hangs on less than this is not compared.
SAME = 2.0 ** -19


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    F.lib()


def logits_of(T, E, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=g) * 1.5).to(dtype)


def check_route(x, k, **kw):
    sigmoid = kw.get("score", "softmax") == "sigmoid"
    bias = kw.get("bias")
    groups = kw.get("groups", 1)
    keep = kw.get("keep_groups") or groups
    ids, w = F.fp8_moe_route(x.to(DEV), k, **{**kw, "bias": None if bias is None else bias.to(DEV)})
    ids, w = ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    T, E = x.shape
    ref, w_ref, margin = B.route(f32(x), k, sigmoid, None if bias is None else bias.numpy(), groups, keep,
                                 kw.get("renormalize", False), kw.get("factor", 1.0))
    # a choice by the logits themselves is exact; the others where the margin says so, or at an exact tie of inputs
    exact = not sigmoid and bias is None
    rows = np.ones(T, bool) if exact else margin > SAME
    assert rows.mean() > 0.9
    assert np.array_equal(ids[rows], ref[rows])
    # exp and the division: 2 ulp each; the sum of E (or k) terms: half an ulp a term
    tol = (8 + E + k) * 2.0 ** -23 * np.abs(w_ref) + 1e-37
    assert np.all(np.abs(w - w_ref)[rows] <= tol[rows])
    for row in ids:
        assert len(set(row.tolist())) == k and row.min() >= 0 and row.max() < E
    return ids, w


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 8, 8), (5, 31, 4), (7, 33, 6), (64, 60, 4), (100, 128, 8),
                                   (17, 160, 6), (333, 256, 8), (9, 300, 32), (40, 512, 10), (5000, 64, 6)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [False, True])
def test_softmax(T, E, k, dtype, renorm):
    check_route(logits_of(T, E, T + E + k, dtype), k, renormalize=renorm, factor=1.5)


@pytest.mark.parametrize("T,E,k,groups,keep", [(1, 256, 8, 8, 4), (50, 256, 8, 8, 4), (33, 64, 6, 1, 1),
                                               (20, 160, 6, 8, 3), (20, 96, 3, 32, 2), (11, 12, 4, 3, 2),
                                               (11, 8, 2, 8, 2), (2000, 512, 16, 16, 4)])
@pytest.mark.parametrize("bias", [False, True])
def test_sigmoid(T, E, k, groups, keep, bias):
    b = torch.randn(E, generator=torch.Generator().manual_seed(7)) * 0.1 if bias else None
    check_route(logits_of(T, E, T + E), k, score="sigmoid", bias=b, groups=groups, keep_groups=keep, renormalize=True,
                factor=2.5)


@pytest.mark.parametrize("groups,keep", [(1, 1), (4, 2)])
def test_softmax_groups_and_bias(groups, keep):
    b = torch.randn(64, generator=torch.Generator().manual_seed(8)) * 0.05
    check_route(logits_of(70, 64, 1), 6, groups=groups, keep_groups=keep)
    check_route(logits_of(70, 64, 2), 6, groups=groups, keep_groups=keep, bias=b)


def test_ties_go_to_the_lowest_index():
    x = torch.zeros((3, 70))
    x[1, 40:] = 1.0
    x[2, ::2] = -0.0
    for score in ("softmax", "sigmoid"):
        ids, w = F.fp8_moe_route(x.to(DEV), 5, score=score)
        assert ids.tolist() == [[0, 1, 2, 3, 4], [40, 41, 42, 43, 44], [0, 1, 2, 3, 4]]
        assert torch.equal(w[0], w[0, :1].expand(5))
    # groups of equal score: the first ones stay
    ids, _ = F.fp8_moe_route(torch.zeros((1, 64), device=DEV), 4, score="sigmoid", groups=8, keep_groups=2)
    assert ids.tolist() == [[0, 1, 2, 3]]


def test_masked_and_nonfinite_logits():
    lowest = float(torch.finfo(torch.float32).min)
    x = logits_of(6, 40, 3)
    x[0, :37] = -float("inf")          # three left for five places
    x[1, :] = -float("inf")            # none left
    x[2, 4:] = lowest                  # masks of the type's lowest value
    x[3, 11] = float("nan")
    x[4, 7] = float("inf")
    x[5, :] = lowest
    ids, w = F.fp8_moe_route(x.to(DEV), 5, renormalize=True)
    ref, w_ref, _ = B.route(x.numpy(), 5, False, renorm=True)
    assert np.array_equal(ids.cpu().numpy(), ref)
    assert np.allclose(w.cpu().numpy(), w_ref, rtol=60 * 2.0 ** -23, atol=1e-37)
    assert not torch.isnan(w).any() and torch.equal(w[1], torch.zeros(5, device=DEV))
    ids, w = F.fp8_moe_route(x.to(DEV), 5, score="sigmoid", renormalize=True)
    assert not torch.isnan(w).any() and 11 not in ids[3].tolist() and ids[4, 0] == 7


def test_route_strided_and_empty():
    x = logits_of(9, 100, 5)
    wide = x.to(DEV)[:, 20:84]
    ids, w = F.fp8_moe_route(wide, 4)
    ids2, w2 = F.fp8_moe_route(wide.contiguous(), 4)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    ids, w = F.fp8_moe_route(torch.empty((0, 16), device=DEV), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)


def test_route_refusals():
    x = torch.zeros((2, 16), device=DEV)
    for bad in (dict(k=17), dict(k=0), dict(k=2, groups=3), dict(k=2, groups=4, keep_groups=5),
                dict(k=9, groups=4, keep_groups=2), dict(k=2, score="tanh"),
                dict(k=2, bias=torch.zeros(15, device=DEV))):
        with pytest.raises((ValueError, F.FP8Error)):
            F.fp8_moe_route(x, **bad)
    with pytest.raises(ValueError):
        F.fp8_moe_route(x.double(), 2)
    with pytest.raises(F.FP8Error):
        F.fp8_moe_route(torch.zeros((2, 513), device=DEV), 2)


# ---------------------------------------------------------------------------
# the experts' networks
# ---------------------------------------------------------------------------

def weights_of(E, H, I, seed):
    g = torch.Generator().manual_seed(seed)
    w13 = (torch.randn((E, 2, I, H), generator=g) * (0.5 / H ** 0.5)).to(torch.bfloat16)
    w2 = (torch.randn((E, H, I), generator=g) * (1.0 / I ** 0.5)).to(torch.bfloat16)
    return (*F.fp8_block_quantize_weight(w13.to(DEV)), *F.fp8_block_quantize_weight(w2.to(DEV)))


def tokens_of(T, H, seed):
    x = torch.randn((T, H), generator=torch.Generator().manual_seed(seed))
    x[:, 0] *= 20
    return x.to(torch.bfloat16)


def choices(T, E, k, seed, drop=0.0, skew=False):
    g = torch.Generator().manual_seed(seed)
    like = torch.randn((T, E), generator=g)
    if skew:
        like[:, 0] += 10  # every token picks expert 0
    ids = like.topk(k, dim=1).indices.to(torch.int32)
    w = torch.rand((T, k), generator=g)
    if drop:
        ids[torch.rand((T, k), generator=g) < drop] = -1
    return ids, w


def check_experts(T, E, k, H, I, seed=0, ids=None, w=None, x=None, **kw):
    x = tokens_of(T, H, seed) if x is None else x
    if ids is None:
        ids, w = choices(T, E, k, seed + 1, **kw)
    q13, s13, q2, s2 = weights_of(E, H, I, seed + 2)
    buf, y, base, row_bytes, used = guarded((T, H), torch.bfloat16, DEV)
    F.fp8_moe_experts(x.to(DEV), ids.to(DEV), w.to(DEV), q13, s13, q2, s2, out=y)
    torch.cuda.synchronize()
    assert F.fp8_last_device_status() == F.FP8_OK
    assert_guards_intact(buf, base, row_bytes, used, T)
    y_ref, tol = B.experts(f32(x), ids.numpy(), w.numpy(), q13.cpu().numpy()[..., :H], s13.cpu().numpy(),
                           q2.cpu().numpy()[..., :I], s2.cpu().numpy())
    err = np.abs(f32(y).astype(np.float64) - y_ref)
    assert np.all(err <= tol), f"max err/tol {np.max(err / tol)}"
    # the tolerance is not a blank cheque: on the whole the outputs are within bf16 rounding of it
    assert np.linalg.norm(err) <= 0.01 * np.linalg.norm(y_ref) + 1e-30
    return y


@pytest.mark.parametrize("T,E,k,H,I", [(1, 1, 1, 128, 128), (1, 8, 2, 256, 128), (1, 16, 8, 200, 72), (2, 4, 4, 64, 300),
                                       (7, 12, 3, 384, 256), (16, 8, 2, 512, 384), (33, 5, 3, 130, 129),
                                       (64, 64, 8, 256, 128), (300, 6, 2, 384, 200), (700, 3, 2, 256, 256)])
def test_experts(T, E, k, H, I):
    check_experts(T, E, k, H, I, seed=T + E)


def test_experts_odd_sizes_and_dropped_pairs():
    check_experts(45, 6, 3, 101, 77, seed=3, drop=0.4)


def test_experts_all_tokens_to_one():
    check_experts(260, 4, 2, 128, 128, seed=4, skew=True)


def test_token_without_experts_gives_zeros():
    ids, w = choices(9, 4, 2, 5)
    ids[3] = -1
    ids[5] = torch.tensor([4, 99], dtype=torch.int32)  # past the last expert: dropped as well
    w[3] = float("nan")                                # the weight of a dropped pair is not read
    y = check_experts(9, 4, 2, 128, 128, seed=6, ids=ids, w=torch.nan_to_num(w))
    q = weights_of(4, 128, 128, 8)
    again = F.fp8_moe_experts(tokens_of(9, 128, 6).to(DEV), ids.to(DEV), w.to(DEV), *q)
    assert torch.equal(again, y)
    assert not y[3].any() and not y[5].any()
    none = F.fp8_moe_experts(tokens_of(9, 128, 6).to(DEV), torch.full((9, 2), -1, dtype=torch.int32, device=DEV),
                             w.to(DEV), *q)
    assert not none.any()


def test_experts_repeated_in_a_row():
    ids = torch.tensor([[1, 1, 1], [0, 2, 0]], dtype=torch.int32)
    check_experts(2, 3, 3, 128, 256, seed=9, ids=ids, w=torch.rand((2, 3), generator=torch.Generator().manual_seed(1)))


@pytest.mark.parametrize("T", [3, 90])
def test_nonfinite_token_stays_apart(T):
    x = tokens_of(T, 192, 11)
    ids, w = choices(T, 4, 2, 12)
    q = weights_of(4, 192, 128, 13)
    clean = F.fp8_moe_experts(x.to(DEV), ids.to(DEV), w.to(DEV), *q)
    x[1, 100] = float("nan")
    y = F.fp8_moe_experts(x.to(DEV), ids.to(DEV), w.to(DEV), *q)
    assert torch.isnan(y[1]).all()
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("T", [2, 100])
def test_experts_repeatable_on_another_stream(T):
    x, (ids, w) = tokens_of(T, 256, 14).to(DEV), choices(T, 8, 4, 15)
    ids, w = ids.to(DEV), w.to(DEV)
    q = weights_of(8, 256, 128, 16)
    y = F.fp8_moe_experts(x, ids, w, *q)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        ws = torch.full((F.fp8_moe_workspace_bytes(T, 4, 8, 256, 128),), 0xFF, dtype=torch.uint8, device=DEV)
        ys = [F.fp8_moe_experts(x, ids, w, *q, ws=ws) for _ in range(3)]
    st.synchronize()
    for other in ys:
        assert torch.equal(y, other)


def test_experts_empty_batch_and_refusals():
    q13, s13, q2, s2 = weights_of(4, 128, 128, 17)
    x = tokens_of(5, 128, 18).to(DEV)
    ids, w = (t.to(DEV) for t in choices(5, 4, 2, 19))
    assert F.fp8_moe_experts(x[:0], ids[:0], w[:0], q13, s13, q2, s2).shape == (0, 128)
    for bad in (dict(ids=ids.long()), dict(weights=w.half()), dict(ids=ids[:4]), dict(qw2=q2[:3]), dict(s13=s13[:, :1]),
                dict(x=x.float()), dict(qw13=q13[:, :1])):
        args = {**dict(x=x, ids=ids, weights=w, qw13=q13, s13=s13, qw2=q2, s2=s2), **bad}
        with pytest.raises(ValueError):
            F.fp8_moe_experts(**args)
    with pytest.raises(F.FP8Error) as e:
        F.fp8_moe_experts(x, ids, w, q13, s13, q2, s2, ws=torch.empty(256, dtype=torch.uint8, device=DEV))
    assert e.value.status == F.FP8_ERR_WORKSPACE


def test_layer_end_to_end():
    """Logits from a block-scaled linear, routing, experts: the pieces together, against the oracle."""
    T, E, k, H, I = 37, 16, 4, 256, 128
    x = tokens_of(T, H, 20)
    gate = (torch.randn((E, H), generator=torch.Generator().manual_seed(21)) * 0.1).to(torch.bfloat16)
    logits = F.fp8_block_linear(x.to(DEV), *F.fp8_block_quantize_weight(gate.to(DEV)))
    ids, w = check_route(logits.cpu(), k, renormalize=True)
    check_experts(T, E, k, H, I, seed=20, x=x, ids=torch.from_numpy(ids), w=torch.from_numpy(w.astype(np.float32)))


def test_experts_many_pairs_sorted_by_several_ctas():
    """Enough pairs that several CTAs sort them: the same result as in two halves, which one CTA sorts each."""
    T, E, k, H, I = 1500, 24, 4, 64, 128
    x, (ids, w) = tokens_of(T, H, 30).to(DEV), choices(T, E, k, 31, drop=0.1)
    ids, w = ids.to(DEV), w.to(DEV)
    q = weights_of(E, H, I, 32)
    y = F.fp8_moe_experts(x, ids, w, *q)
    parts = [F.fp8_moe_experts(x[s], ids[s].contiguous(), w[s].contiguous(), *q)
             for s in (slice(0, 700), slice(700, 1500))]
    assert torch.equal(y, torch.cat(parts))


@pytest.mark.parametrize("tokens", [1, 12, 200])
def test_example_layer(tokens):
    """The example's layer is within FP8's rounding of the same layer in fp32: two e4m3 operands (each value off
    by at most 2**-4, on average about 2**-5.8 of it) in each of two products leave about 5 percent in the norm."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")
    spec = importlib.util.spec_from_file_location("moe_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    off = m.main(["--tokens", str(tokens), "--hidden", "256", "--width", "384", "--experts", "16", "--chosen", "4",
                  "--steps", "2"])
    assert off < 0.1
