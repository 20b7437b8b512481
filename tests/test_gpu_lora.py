"""GPU parity of the adapters beside a projection with the float64 oracle."""

import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_dynamic_gb300 as F
from fp8_w8a8_quantized_dynamic_gb300 import _build
from oracle import layer_oracle as L
from parity import f32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    F.lib()


def operands(M, K, N, r, adapters, seed, ids=None):
    g = torch.Generator().manual_seed(seed)

    def draw(*shape, std=1.0):
        return (torch.randn(shape, generator=g) * std).to(BF16)
    d = {"y": draw(M, N), "x": draw(M, K), "a": draw(adapters, r, K, std=K ** -0.5),
         "b": draw(adapters, N, r, std=r ** -0.5)}
    d["ids"] = torch.randint(-1, adapters, (M,), generator=g, dtype=torch.int32) if ids is None else ids
    d["scales"] = torch.randn(adapters, generator=g)
    return d


def run(d, **kw):
    out = F.fp8_lora_add(*(v.to(DEV) for v in d.values()), **kw)
    assert F.fp8_last_device_status() == F.FP8_OK
    return out


def check(d):
    out = run(d)
    ref, err = L.lora(*(v.numpy() if v.dtype != BF16 else f32(v) for v in d.values()))
    off = np.abs(f32(out).astype(np.float64) - ref)
    tol = L.rounded_bf16(ref, err)
    assert np.all(off <= tol), f"{np.max(off / tol):.2f} of its tolerance"
    none = (d["ids"] < 0) | (d["ids"] >= d["a"].shape[0])
    assert torch.equal(out.cpu()[none], d["y"][none])  # bit for bit
    return out


# token counts around the change of form and around tiles of 128 rows
@pytest.mark.parametrize("M", [1, 2, 16, 17, 33, 38, 39, 64, 65, 127, 128, 129, 300, 512, 513, 700])
@pytest.mark.parametrize("K,N,r,adapters", [(256, 256, 16, 3), (520, 200, 8, 1), (4096, 2048, 64, 2)])
def test_tokens(M, K, N, r, adapters):
    check(operands(M, K, N, r, adapters, M + K))


@pytest.mark.parametrize("M", [3, 60, 530])
@pytest.mark.parametrize("r", [1, 2, 7, 8, 9, 12, 16, 24, 32, 33, 48, 64, 65, 96, 100, 128, 129, 160, 192, 200, 256])
def test_ranks(M, r):
    check(operands(M, 320, 264, r, 4, r))


@pytest.mark.parametrize("M", [2, 50, 600])
@pytest.mark.parametrize("K,N", [(1, 1), (7, 9), (8, 127), (63, 128), (64, 129), (65, 130), (1000, 1027), (1001, 1000),
                                 (4096, 96), (4104, 33), (96, 4100), (2056, 2200)])
def test_odd_sizes(M, K, N):
    check(operands(M, K, N, 16, 5, K + N))
    check(operands(M, K, N, 12, 2, K + N + 1))


@pytest.mark.parametrize("M,adapters", [(1, 511), (60, 40), (130, 64), (520, 64), (600, 511), (1500, 200)])
def test_many_adapters(M, adapters):
    check(operands(M, 128, 136, 8, adapters, M))


@pytest.mark.parametrize("K", [2, 62, 66, 1002, 5142])
@pytest.mark.parametrize("r", [7, 16, 76, 130, 256])
def test_rows_of_whole_words(K, r):
    """Rows of x and A that start on 4-byte boundaries and no wider ones; more steps of K than stages; x in wider rows."""
    d = operands(530, K, 72, r, 3, r + K)
    want = check(d)
    x = torch.full((530, K + 6), float("nan"), dtype=BF16, device=DEV)
    x[:, 2:K + 2] = d["x"].to(DEV)
    rest = {k: v.to(DEV) for k, v in d.items()}
    assert torch.equal(F.fp8_lora_add(**{**rest, "x": x[:, 2:K + 2]}), want)


@pytest.mark.parametrize("r", [8, 12, 64, 100, 129, 192, 250])
@pytest.mark.parametrize("N", [12000, 12002, 12003])
def test_many_steps_of_a_cta(r, N):
    """More column steps than a CTA has buffers, for every form of B's, y's and out's loads; tiles that end within a CTA's
    run."""
    d = operands(530, 72, N, r, 3, r)
    check(d)
    one = {k: v.to(DEV) for k, v in d.items()}
    y = one["y"].clone()  # in place: rows without an adapter take no part
    assert torch.equal(F.fp8_lora_add(y, *list(one.values())[1:], out=y), run(d))
    assert F.fp8_last_device_status() == F.FP8_OK


def test_ids_outside_and_all_bare():
    M = 603
    wild = torch.tensor([-1, 3, -2 ** 31, 2 ** 31 - 1, 2, 0, 4, 511, 512], dtype=torch.int32)
    for m in (9, M):
        check(operands(m, 64, 72, 4, 3, m, wild.repeat(M // 9 + 1)[:m]))
        check(operands(m, 64, 72, 4, 3, m, torch.full((m,), -1, dtype=torch.int32)))


@pytest.mark.parametrize("lengths", [[1, 127, 1, 129], [256, 5, 0, 300], [600], [3] * 60, [3] * 200, [129, 1, 255, 128, 2]])
def test_runs_of_requests(lengths):
    ids = torch.cat([torch.full((n,), i % 7, dtype=torch.int32) for i, n in enumerate(lengths)])
    check(operands(ids.numel(), 384, 320, 32, 7, ids.numel(), ids))


@pytest.mark.parametrize("M", [5, 60, 560])
def test_in_place_strided_and_without_scales(M):
    K, N, r = 200, 160, 16
    d = operands(M, K, N, r, 3, 1)
    want = check(d)
    for shift, pad in ((0, 8), (8, 0), (1, 2)):
        wide_x = torch.zeros((M, K + shift + pad), dtype=BF16, device=DEV)
        wide_x[:, shift:shift + K] = d["x"].to(DEV)
        wide_y = torch.full((M, N + shift + pad), 7.0, dtype=BF16, device=DEV)
        wide_y[:, shift:shift + N] = d["y"].to(DEV)
        rest = [d[k].to(DEV) for k in ("a", "b", "ids", "scales")]
        x, y = wide_x[:, shift:shift + K], wide_y[:, shift:shift + N]
        wide_o = torch.full_like(wide_y, 7.0)
        out = wide_o[:, shift:shift + N]
        assert F.fp8_lora_add(y, x, *rest, out=out) is out
        assert F.fp8_lora_add(y, x, *rest, out=y) is y
        for wide in (wide_o, wide_y):
            assert torch.equal(wide[:, shift:shift + N], want)
            assert (wide[:, :shift] == 7).all() and (wide[:, shift + N:] == 7).all()
    ones = {**d, "scales": torch.ones(3)}
    assert torch.equal(run({k: v for k, v in d.items() if k != "scales"}), run(ones))


@pytest.mark.parametrize("M", [6, 520])
def test_columns_of_a_merged_projection(M):
    """Query, key and value columns of one output, each with adapters of its own."""
    K, widths = 256, (256, 64, 64)
    d = operands(M, K, sum(widths), 8, 4, 2)
    y = d["y"].to(DEV)
    at = 0
    for i, n in enumerate(widths):
        part = operands(M, K, n, 8, 4, 10 + i, d["ids"])
        part["x"], part["y"] = d["x"], d["y"][:, at:at + n].contiguous()
        want = check(part)
        cols = y[:, at:at + n]
        F.fp8_lora_add(cols, d["x"].to(DEV), part["a"].to(DEV), part["b"].to(DEV), part["ids"].to(DEV),
                       part["scales"].to(DEV), out=cols)
        assert torch.equal(cols, want)
        at += n


@pytest.mark.parametrize("M", [8, 60, 560])
def test_non_finite_values_stay_with_their_tokens(M):
    d = operands(M, 128, 144, 16, 4, 3, torch.arange(M, dtype=torch.int32) % 5 - 1)
    clean = check(d).cpu()
    d["x"][1, 5] = float("nan")
    d["x"][2, 7] = float("inf")
    d["a"][3, 2, 2] = float("nan")   # the adapter of tokens 4, 9, ...
    d["y"][0, 3] = float("inf")
    out = run(d).cpu()
    hit = (d["ids"] == 3)
    hit[[0, 1, 2]] = True
    assert torch.equal(out[~hit], clean[~hit])
    assert out[1].isnan().all() and out[d["ids"] == 3].isnan().all()
    assert not torch.isfinite(out[2]).any()
    assert out[0, 3] == float("inf") and torch.equal(out[0, 4:], clean[0, 4:])


def test_empty():
    e = torch.empty((0, 64), dtype=BF16, device=DEV)
    a, b = torch.zeros((2, 4, 64), dtype=BF16, device=DEV), torch.zeros((2, 64, 4), dtype=BF16, device=DEV)
    ids = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert F.fp8_lora_add(e, e, a, b, ids).shape == (0, 64)
    y = torch.ones((3, 64), dtype=BF16, device=DEV)
    ids = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert torch.equal(F.fp8_lora_add(y, y[:, :0], a[:, :, :0].contiguous(), b, ids), y)  # nothing to multiply
    assert torch.equal(F.fp8_lora_add(y, y, a[:0], b[:0], ids), y)                       # no adapters
    assert F.fp8_lora_add(y[:, :0], y, a, b[:, :0].contiguous(), ids).shape == (3, 0)


def test_repeats_bit_for_bit_with_a_used_workspace():
    for M in (40, 60, 900):
        d = operands(M, 1024, 512, 32, 6, M)
        need = F.fp8_lora_workspace_bytes(M, 1024, 512, 6, 32)
        ws = torch.full((max(need, 256),), 0xFF, dtype=torch.uint8, device=DEV)
        first = run(d, ws=ws)
        for _ in range(3):
            assert torch.equal(run(d, ws=ws), first)


def test_beside_a_block_linear_in_a_graph_and_on_a_side_stream():
    """A projection and its adapters as a decode step and a prompt use them, captured and replayed."""
    K, N, r, adapters = 512, 384, 16, 4
    w = (torch.randn((N, K), generator=torch.Generator().manual_seed(5)) * K ** -0.5).to(BF16)
    qw, s_w = F.fp8_block_quantize_weight(w.to(DEV))
    for M in (3, 560):
        d = {k: v.to(DEV) for k, v in operands(M, K, N, r, adapters, M).items()}

        def step():
            y = F.fp8_block_linear(d["x"], qw, s_w)
            return F.fp8_lora_add(y, d["x"], d["a"], d["b"], d["ids"], d["scales"], out=y)
        y = F.fp8_block_linear(d["x"], qw, s_w)
        ref, err = L.lora(f32(y), f32(d["x"]), f32(d["a"]), f32(d["b"]), d["ids"].cpu().numpy(), d["scales"].cpu().numpy())
        want = step()
        assert np.all(np.abs(f32(want) - ref) <= L.rounded_bf16(ref, err))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = step()
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        graph.replay()
        assert torch.equal(got, want)
        d["ids"].copy_(d["ids"].flip(0))
        d["x"].mul_(-0.5)
        want = step()
        graph.replay()
        assert torch.equal(got, want)


def test_offsets_past_32_bits():
    """y of more than 2**31 elements, adapters past 2**31 elements; the last ones compared."""
    M, K, N, r = 2 ** 17 + 5, 64, 16400, 8
    y = torch.zeros((M, N), dtype=BF16, device=DEV)
    d = {k: v.to(DEV) for k, v in operands(5, K, N, r, 1, 6, torch.zeros(5, dtype=torch.int32)).items()}
    x = torch.zeros((M, K), dtype=BF16, device=DEV)
    x[-5:] = d["x"]
    ids = torch.zeros(M, dtype=torch.int32, device=DEV)
    out = F.fp8_lora_add(y, x, d["a"], d["b"], ids, d["scales"], out=y)
    few = F.fp8_lora_add(torch.zeros((5, N), dtype=BF16, device=DEV), *(d[k] for k in ("x", "a", "b", "ids", "scales")))
    assert torch.allclose(out[-5:].float(), few.float(), rtol=2 ** -7, atol=1e-4) and not out[:-5].any()
    del y, out
    adapters, K, N, r = 40, 8192, 2 ** 18, 256
    b = torch.zeros((adapters, N, r), dtype=BF16, device=DEV)
    a = torch.zeros((adapters, r, K), dtype=BF16, device=DEV)
    one = operands(1, K, N, r, 1, 7)
    a[-1], b[-1] = one["a"][0].to(DEV), one["b"][0].to(DEV)
    for M in (1, 530):
        x = one["x"].to(DEV).expand(M, K).contiguous()
        y = one["y"].to(DEV).expand(M, N).contiguous()
        ids = torch.full((M,), adapters - 1, dtype=torch.int32, device=DEV)
        out = F.fp8_lora_add(y, x, a, b, ids)
        ref, err = L.lora(f32(one["y"]), f32(one["x"]), f32(one["a"]), f32(one["b"]), np.zeros(1, np.int32))
        tol = L.rounded_bf16(ref, err)
        assert np.all(np.abs(f32(out[-1:]) - ref) <= tol) and np.all(np.abs(f32(out[:1]) - ref) <= tol)


def formula(d):
    """The result in float64 by elementwise products, which keep infinities and NaN where the formula has them."""
    y, x, a, b = (f32(d[k]).astype(np.float64) for k in ("y", "x", "a", "b"))
    out = y.copy()
    with np.errstate(all="ignore"):
        for m, e in enumerate(d["ids"].tolist()):
            if 0 <= e < a.shape[0]:
                v = (a[e] * x[m]).sum(1)
                out[m] += float(d["scales"][e]) * (b[e] * v).sum(1)
    return out


@pytest.mark.parametrize("M,K", [(8, 128), (560, 128), (1100, 128), (600, 2056)])
@pytest.mark.parametrize("r", [12, 16, 76, 130, 256])
def test_values_of_b_that_are_not_finite(M, K, r):
    """An infinity in B gives an infinity of its product's sign, in every form, and only in its column of its adapter."""
    inf = float("inf")
    d = operands(M, K, 144, r, 4, 5, torch.arange(M, dtype=torch.int32) % 5 - 1)
    clean = run(d).cpu()
    d["b"][2, 5, 3] = inf
    d["b"][2, 6, 1] = -inf
    d["b"][1, 7, 0] = float("nan")
    d["b"][3, 143, :2] = inf       # two that may cancel
    d["a"][0, 2, 2] = inf          # A x is infinite, and so is what it meets
    d["b"][0, 9, 2] = -inf
    out, want = run(d).cpu().double().numpy(), formula(d)
    odd = ~np.isfinite(want)
    assert odd[d["ids"].numpy() == 0].all() and odd.sum() > M // 5 * 4
    assert np.array_equal(np.isnan(out), np.isnan(want))
    assert np.array_equal(out[odd & ~np.isnan(want)], want[odd & ~np.isnan(want)])
    assert np.array_equal(out[~odd], clean.double().numpy()[~odd])


@pytest.mark.parametrize("M", [3, 600])
def test_a_x_past_the_range_of_bf16(M):
    """A x = 2**127 * (2 - 2**-8): a finite fp32 number that rounds to an infinite bf16 one."""
    d = {"y": torch.zeros((M, 8), dtype=BF16), "x": torch.tensor([[2.0 ** 127, 2.0 ** 119]], dtype=BF16).repeat(M, 1),
         "a": torch.tensor([[[2 - 2.0 ** -7, 1.0]]], dtype=BF16), "b": torch.full((1, 8, 1), 2.0 ** -100, dtype=BF16),
         "ids": torch.zeros(M, dtype=torch.int32), "scales": torch.ones(1)}
    assert (run(d) == 2.0 ** 28).all()  # 2**27 * (2 - 2**-8), a tie, to even


@pytest.mark.parametrize("M", [3, 600])
@pytest.mark.parametrize("r", [2, 12, 16, 64, 76, 192, 250, 256])
def test_all_bits_of_a_x_count(M, r):
    """Pairs of A x that differ in their last bits and cancel in B's product: 1 + 2**-9 + 2**-18 less 1 + 2**-9, and the same
    one bit further down, at both ends of the rank. All sums are exact in fp32, so the result is."""
    d = {"y": torch.zeros((M, 40), dtype=BF16), "x": torch.zeros((M, 24), dtype=BF16), "a": torch.zeros((1, r, 24), dtype=BF16),
         "b": torch.zeros((1, 40, r), dtype=BF16), "ids": torch.zeros(M, dtype=torch.int32), "scales": torch.ones(1)}
    for at, bit in ((0, 18), (r - 2, 19)):
        d["b"].zero_(), d["a"].zero_()
        d["x"][:, :3] = torch.tensor([1.0, 2.0 ** -9, 2.0 ** -bit], dtype=BF16)
        d["a"][0, at, :3], d["a"][0, at + 1, :2] = 1.0, 1.0
        d["b"][0, :, at], d["b"][0, :, at + 1] = 1.0, -1.0
        assert (run(d) == 2.0 ** -bit).all()


@pytest.mark.parametrize("M", [8, 560, 1100])
@pytest.mark.parametrize("r", [7, 12, 16, 130, 256])
def test_tokens_and_adapters_that_are_not_finite(M, r):
    """Single infinite tokens, NaN late in a row of B, rows of B and a whole B that are infinite, NaN tokens beside them."""
    inf, nan = float("inf"), float("nan")
    d = operands(M, 128, 150, r, 5, 6, torch.arange(M, dtype=torch.int32) % 6 - 1)
    clean = run(d).cpu().double().numpy()
    d["x"][1, 5], d["x"][2, 3] = inf, -inf      # adapters 0 and 1
    d["x"][M - 1, 0] = nan
    d["b"][0, 11, r - 1], d["b"][0, 149, 0] = nan, nan
    d["b"][1, 33], d["b"][1, 34, r - 1] = inf, -inf
    d["b"][2] = inf
    d["b"][3, ::2] = nan
    out, want = run(d).cpu().double().numpy(), formula(d)
    odd = ~np.isfinite(want)
    assert np.array_equal(np.isnan(out), np.isnan(want))
    assert np.array_equal(out[odd & ~np.isnan(want)], want[odd & ~np.isnan(want)])
    assert np.array_equal(out[~odd], clean[~odd])


@pytest.mark.parametrize("r", [3, 8, 16, 40, 64, 128, 200, 256])
@pytest.mark.parametrize("lengths", [[1, 2, 3, 4, 5, 7, 8, 9], [15, 16, 17, 31, 32, 33], [63, 64, 65, 97]])
@pytest.mark.parametrize("K", [72, 8192])
def test_tiles_of_few_rows(K, r, lengths):
    """Rows that several lanes share, in one and in several quarters of a tile, over one and over many splits of K."""
    runs = [n for _ in range(-(-530 // sum(lengths))) for n in lengths]
    ids = torch.cat([torch.full((n,), i % 41, dtype=torch.int32) for i, n in enumerate(runs)])
    order = torch.randperm(ids.numel(), generator=torch.Generator().manual_seed(r))
    check(operands(ids.numel(), K, 140, r, 41, r, ids[order].contiguous()))
