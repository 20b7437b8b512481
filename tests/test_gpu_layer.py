"""The norms, adapters and rows to experts run together with the framework's linears and routing, as a transformer
block of a serving program runs them."""

import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_dynamic_gb300 as F
from fp8_w8a8_quantized_dynamic_gb300 import _build
from oracle import block_oracle as B
from oracle import fp8_oracle as O
from oracle import layer_oracle as L
from parity import f32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
H, E, K_CHOSEN, WIDTH, RANK, ADAPTERS, EPS = 512, 8, 2, 256, 16, 4, 1e-5


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    F.lib()


class Block:
    """A mixing projection with adapters (in place of attention), then experts that are per-tensor FP8 linears of their own:
    norms on both sides of each, a gate a channel."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)

        def draw(*shape, std):
            return (torch.randn(shape, generator=g) * std).to(BF16).to(DEV)
        self.pre1, self.post1, self.pre2, self.post2 = (draw(H, std=0.2) for _ in range(4))  # offsets from one
        self.gate = draw(H, std=0.5)
        self.mix = F.fp8_block_quantize_weight(draw(H, H, std=H ** -0.5))
        self.a, self.b = draw(ADAPTERS, RANK, H, std=H ** -0.5), draw(ADAPTERS, H, RANK, std=RANK ** -0.5)
        self.scales = torch.rand(ADAPTERS, generator=g).to(DEV)
        self.router = F.fp8_block_quantize_weight(draw(E, H, std=H ** -0.5))
        self.up = [F.fp8_quantize_weight(draw(WIDTH, H, std=H ** -0.5)) for _ in range(E)]
        self.down = [F.fp8_quantize_weight(draw(H, WIDTH, std=WIDTH ** -0.5)) for _ in range(E)]

    def first_half(self, r, adapter_ids):
        """r bf16 [T, H] -> (the projection's output with adapters, the residual, the second half's input)."""
        q, s, _ = F.fp8_residual_norm_quantize(r, self.pre1, eps=EPS, plus_one=True)
        y = F.fp8_block_scaled_mm(q, H, s, *self.mix)
        # the adapters see the projection's input as bf16
        x, _ = F.fp8_residual_norm(r, self.pre1, eps=EPS, plus_one=True)
        with_adapters = F.fp8_lora_add(y, x, self.a, self.b, adapter_ids, self.scales)
        n, r1 = F.fp8_residual_norm(with_adapters, self.pre2, residual=r, post_weight=self.post1, gate=self.gate, scale=0.5,
                                    eps=EPS, plus_one=True)
        return (q, s, y, x, with_adapters, r1, n)

    def route(self, n):
        ids, w = F.fp8_moe_route(F.fp8_block_linear(n, *self.router), K_CHOSEN, renormalize=True)
        return (ids, w, *F.fp8_moe_dispatch(n, ids, E))

    def experts(self, xs, offsets):
        ys = torch.zeros_like(xs)
        for e in range(E):
            lo, hi = offsets[e], offsets[e + 1]
            h = F.fp8_linear(xs[lo:hi], *self.up[e])
            ys[lo:hi] = F.fp8_linear(torch.nn.functional.silu(h), *self.down[e])
        return ys

    def back(self, ys, pos, w, r1):
        y = F.fp8_moe_combine(ys, pos, w)
        return (y, *F.fp8_residual_norm_quantize(y, self.pre1, residual=r1, post_weight=self.post2, gate=self.gate,
                                                 eps=EPS, plus_one=True))


def within(got, ref, err):
    assert np.all(np.abs(f32(got).astype(np.float64) - ref) <= L.rounded_bf16(ref, err))


@pytest.mark.parametrize("T", [1, 7, 300, 1000])
def test_a_block_step_by_step(T):
    """Each step against the oracle on the step's own inputs."""
    m = Block(1)
    g = torch.Generator().manual_seed(T)
    r = (torch.randn((T, H), generator=g) * 2).to(BF16).to(DEV)
    aid = torch.randint(-1, ADAPTERS, (T,), generator=g, dtype=torch.int32).to(DEV)
    q, s, y, x, ya, r1, n = m.first_half(r, aid)
    ref, err, _, _ = L.norms(f32(r), f32(m.pre1), eps=EPS, plus_one=True)
    within(x, ref, err)
    v, dv = B._requantize(ref, err)
    got = O.decode(q.cpu().numpy()) * np.repeat(s.cpu().numpy().astype(np.float64), 128, 0).T
    assert np.all(np.abs(got - v) <= dv + np.abs(v) * 4 * L.U)
    within(y, *B.scaled_product(q.cpu().numpy(), s.cpu().numpy(), *(t.cpu().numpy() for t in m.mix)))
    within(ya, *L.lora(f32(y), f32(x), f32(m.a), f32(m.b), aid.cpu().numpy(), m.scales.cpu().numpy()))
    ref_n, err_n, ref_r, err_r = L.norms(f32(ya), f32(m.pre2), f32(r), f32(m.post1), f32(m.gate), 0.5, EPS, True)
    within(n, ref_n, err_n)
    within(r1, ref_r, err_r)
    ids, w, xs, pos, offsets = m.route(n)
    ref_pos, ref_off = L.sort_rows(ids.cpu().numpy(), E)
    assert np.array_equal(pos.cpu().numpy(), ref_pos) and offsets.tolist() == ref_off.tolist()
    assert torch.equal(xs[pos.long().flatten()], n.repeat_interleave(K_CHOSEN, 0))
    ys = m.experts(xs, offsets.tolist())
    y2, q2, s2, r2 = m.back(ys, pos, w, r1)
    within(y2, *L.combine(f32(ys), ref_pos, w.cpu().numpy()))
    ref_n, err_n, ref_r, err_r = L.norms(f32(y2), f32(m.pre1), f32(r1), f32(m.post2), f32(m.gate), 1.0, EPS, True)
    within(r2, ref_r, err_r)
    v, dv = B._requantize(ref_n, err_n)
    got = O.decode(q2.cpu().numpy()) * np.repeat(s2.cpu().numpy().astype(np.float64), 128, 0).T
    assert np.all(np.abs(got - v) <= dv + np.abs(v) * 4 * L.U)
    assert F.fp8_last_device_status() == F.FP8_OK


@pytest.mark.parametrize("T", [4, 700])
def test_two_graphs_of_a_block_on_their_own_streams(T):
    """Captured twice, replayed at once on two streams and again on new values: each as the eager run has it."""
    m = Block(2)
    g = torch.Generator().manual_seed(T)

    def values():
        return ((torch.randn((T, H), generator=g) * 2).to(BF16).to(DEV),
                torch.randint(-1, ADAPTERS, (T,), generator=g, dtype=torch.int32).to(DEV))

    def step(r, aid):
        first = m.first_half(r, aid)
        return (*first, *m.route(first[-1]))
    sides = []
    for _ in range(2):
        held = values()
        step(*held)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(*held)
        sides.append((held, graph, out, torch.cuda.Stream()))
    for _ in range(2):
        want = []
        for held, _, _, _ in sides:
            for old, new in zip(held, values()):
                old.copy_(new)
            want.append(step(*held))
        torch.cuda.synchronize()
        for _, graph, _, stream in sides:
            with torch.cuda.stream(stream):
                graph.replay()
                graph.replay()
        torch.cuda.synchronize()
        for (_, _, out, _), ref in zip(sides, want):
            assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert F.fp8_last_device_status() == F.FP8_OK


def test_a_router_trained_through_the_experts():
    """The gradient of a loss through dispatch, experts (here a matrix each) and combine, against autograd in fp64 of the
    same function, all choices fixed. fp32 throughout: off by the roundings of sums of H and of the pairs."""
    T, k, width = 40, 3, 96
    g = torch.Generator().manual_seed(3)
    x, dy = torch.randn((T, width), generator=g), torch.randn((T, width), generator=g)
    mats = torch.randn((E, width, width), generator=g) * width ** -0.5
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    w = torch.rand((T, k), generator=g)
    xs, pos, offsets = F.fp8_moe_dispatch(x.to(DEV), ids.to(DEV), E)
    o = offsets.tolist()
    ys = torch.cat([xs[o[e]:o[e + 1]] @ mats[e].to(DEV) for e in range(E)])
    y = F.fp8_moe_combine(ys, pos, w.to(DEV))
    dys, dw = F.fp8_moe_combine_grad(dy.to(DEV), ys, pos, w.to(DEV))
    dxs = torch.cat([dys[o[e]:o[e + 1]] @ mats[e].to(DEV).T for e in range(E)])
    dx = F.fp8_moe_dispatch_grad(dxs, pos)
    x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()
    y64 = (torch.einsum("th,tkhi->tki", x64, mats.double()[ids.long()]) * w64[..., None]).sum(1)
    (y64 * dy.double()).sum().backward()
    # magnitudes: a sum of `width` products of about unit size, twice, over k pairs, each step 2**-23
    tol = 2.0 ** -23 * (2 * width + k + 8) * 20
    assert (y.cpu().double() - y64).abs().max() <= tol
    assert (dw.cpu().double() - w64.grad).abs().max() <= tol * width ** 0.5
    assert (dx.cpu().double() - x64.grad).abs().max() <= tol
