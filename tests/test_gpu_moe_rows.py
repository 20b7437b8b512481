"""GPU parity of tokens sorted by expert and back, and of the gradients, with the float64 oracle."""

import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_dynamic_gb300 as F
from fp8_w8a8_quantized_dynamic_gb300 import _build
from oracle import layer_oracle as L
from parity import f32

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    F.lib()


def routing(T, k, E, seed, drop=0.0):
    """ids with repeats, ids outside [0, E) of every kind, and weights of either sign."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    if drop:
        wild = torch.tensor([-1, E, -2 ** 31, 2 ** 31 - 1, E + 7], dtype=torch.int32)
        gone = torch.rand((T, k), generator=g) < drop
        ids = torch.where(gone, wild[torch.randint(0, 5, (T, k), generator=g)], ids)
    return ids, torch.randn((T, k), generator=g)


def rows(n, H, seed, dtype):
    return torch.randn((n, H), generator=torch.Generator().manual_seed(seed)).to(dtype)


def check_dispatch(T, k, E, H, dtype, drop=0.0, seed=0):
    ids, _ = routing(T, k, E, seed + T + k + E, drop)
    x = rows(T, H, seed + 1, dtype)
    out = torch.full((T * k, H), 7.0, dtype=dtype, device=DEV)
    xs, pos, offsets = F.fp8_moe_dispatch(x.to(DEV), ids.to(DEV), E, out=out)
    pos_ref, off_ref = L.sort_rows(ids.numpy(), E)
    assert np.array_equal(pos.cpu().numpy(), pos_ref) and np.array_equal(offsets.cpu().numpy(), off_ref)
    want = torch.full((T * k, H), 7.0, dtype=dtype)
    for j in range(k):
        t = torch.from_numpy(np.nonzero(pos_ref[:, j] >= 0)[0])
        want[torch.from_numpy(pos_ref[t.numpy(), j]).long()] = x[t]
    assert torch.equal(xs.cpu(), want)  # rows behind the kept pairs as they were
    return pos


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (2, 32, 3), (7, 3, 12), (64, 8, 64), (100, 6, 512),
                                   (129, 8, 60), (256, 8, 8), (257, 8, 256), (1000, 2, 16), (1000, 8, 1), (5000, 8, 100)])
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_dispatch_orders(T, k, E, drop):
    check_dispatch(T, k, E, 24, BF16, drop)


@pytest.mark.parametrize("H", [1, 2, 5, 8, 31, 64, 1000, 1001, 4096])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_dispatch_widths(H, dtype):
    check_dispatch(1, 8, 16, H, dtype)
    check_dispatch(50, 3, 9, H, dtype, 0.3)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_dispatch_of_one_very_wide_row(dtype):
    H = 65535 * 256 + 3
    x = torch.arange(H, device="cuda").remainder(251).to(dtype)[None]
    xs, pos, offsets = F.fp8_moe_dispatch(x, torch.tensor([[2]], dtype=torch.int32, device="cuda"), 3)
    assert torch.equal(xs, x) and pos.tolist() == [[0]] and offsets.tolist() == [0, 0, 0, 1]


def test_dispatch_all_dropped_and_empty():
    ids = torch.full((9, 4), -1, dtype=torch.int32, device=DEV)
    out = torch.full((36, 40), 3.0, device=DEV)
    xs, pos, offsets = F.fp8_moe_dispatch(torch.ones((9, 40), device=DEV), ids, 5, out=out)
    assert (xs == 3.0).all() and (pos == -1).all() and not offsets.any()
    assert not F.fp8_moe_combine(xs, pos, torch.ones((9, 4), device=DEV)).any()
    xs, pos, offsets = F.fp8_moe_dispatch(torch.ones((0, 40), device=DEV), ids[:0], 5)
    assert xs.shape == (0, 40) and pos.shape == (0, 4) and offsets.tolist() == [0] * 6
    _, pos, offsets = F.fp8_moe_dispatch(torch.ones((9, 0), device=DEV), ids.clamp(min=2), 5)
    assert offsets.tolist() == [0, 0, 0, 36, 36, 36] and pos.flatten().tolist() == list(range(36))
    assert F.fp8_moe_combine(torch.ones((4, 8), device=DEV), pos[:0]).shape == (0, 8)


def check_back(T, k, E, H, dtype, drop=0.0, seed=0):
    ids, weights = routing(T, k, E, seed + T + k, drop)
    pos = torch.from_numpy(L.sort_rows(ids.numpy(), E)[0])
    ys, dy = rows(T * k, H, seed + 2, dtype), rows(T, H, seed + 3, dtype)
    for w in (weights, None):
        y = F.fp8_moe_combine(ys.to(DEV), pos.to(DEV), None if w is None else w.to(DEV))
        ref, err = L.combine(f32(ys), pos.numpy(), None if w is None else w.numpy())
        assert y.dtype == dtype
        tol = L.rounded_bf16(ref, err) if dtype == BF16 else err
        assert np.all(np.abs(f32(y) - ref) <= tol)
    # without weights, that is the gradient of the dispatch
    assert torch.equal(F.fp8_moe_dispatch_grad(ys.to(DEV), pos.to(DEV)), y)
    out = torch.full((T * k, H), 7.0, dtype=dtype, device=DEV)
    dys, dw = F.fp8_moe_combine_grad(dy.to(DEV), ys.to(DEV), pos.to(DEV), weights.to(DEV), out=out)
    dys_ref, dw_ref, dw_err = L.combine_grad(f32(dy), f32(ys), pos.numpy(), weights.numpy())
    got = f32(dys).astype(np.float64)
    free = np.isnan(dys_ref[:, 0])
    assert (got[free] == 7.0).all()
    half = L.HALF_BF16 if dtype == BF16 else 0.0
    tol = np.abs(dys_ref[~free]) * (half + 2 * L.U) + L.TINY
    assert np.all(np.abs(got[~free] - dys_ref[~free]) <= tol)
    assert np.all(np.abs(dw.cpu().numpy() - dw_ref) <= dw_err)
    assert not dw.cpu()[pos < 0].any()
    # over ys
    over = ys.to(DEV)
    dys2, dw2 = F.fp8_moe_combine_grad(dy.to(DEV), over, pos.to(DEV), weights.to(DEV), out=over)
    keep = torch.from_numpy(~free)
    assert torch.equal(dys2.cpu()[keep], dys.cpu()[keep]) and torch.equal(dw2, dw)
    assert torch.equal(dys2.cpu()[~keep], ys[~keep])


@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 1), (1, 8, 64, 2048), (5, 3, 4, 7), (33, 8, 16, 64), (20, 32, 64, 120),
                                     (40, 9, 20, 1000), (30, 17, 8, 1001), (64, 4, 8, 2056), (11, 2, 3, 5000)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_back_and_gradient(T, k, E, H, dtype, drop):
    check_back(T, k, E, H, dtype, drop)


def test_gradients_against_differences():
    """Central differences of <dy, combine(ys, w)>, which is linear in ys and in w: exact up to rounding."""
    T, k, E, H = 6, 2, 4, 40
    ids, w = routing(T, k, E, 3)
    pos = torch.from_numpy(L.sort_rows(ids.numpy(), E)[0]).to(DEV)
    ys, dy, w = rows(T * k, H, 4, FP32).to(DEV), rows(T, H, 5, FP32).to(DEV), w.to(DEV)
    dys, dw = F.fp8_moe_combine_grad(dy, ys, pos, w)

    def loss(ys, w):
        return float((F.fp8_moe_combine(ys, pos, w).double() * dy.double()).sum())
    size = float((ys.abs().amax() * dy.abs().amax() * w.abs().amax()).double()) * T * H * (k + 2) * L.U
    for (t, j) in ((0, 0), (3, 1), (5, 0)):
        up, down = w.clone(), w.clone()
        up[t, j] += 1.0
        down[t, j] -= 1.0
        step = float(up[t, j].double() - down[t, j].double())
        assert abs((loss(ys, up) - loss(ys, down)) / step - float(dw[t, j])) <= 4 * size
        r = int(pos[t, j])
        up, down = ys.clone(), ys.clone()
        up[r, 7] += 1.0
        down[r, 7] -= 1.0
        step = float(up[r, 7].double() - down[r, 7].double())
        assert abs((loss(up, w) - loss(down, w)) / step - float(dys[r, 7])) <= 4 * size
    # <dxs, dispatch(x)> likewise
    x, dxs = rows(T, H, 6, FP32).to(DEV), rows(T * k, H, 7, FP32).to(DEV)
    dx = F.fp8_moe_dispatch_grad(dxs, pos)
    xs, _, _ = F.fp8_moe_dispatch(x, ids.to(DEV), E)
    assert abs(float((dx.double() * x.double()).sum() - (xs.double() * dxs.double()).sum())) <= \
        float((xs.double() * dxs.double()).abs().sum()) * (k + 1) * L.U


def test_positions_outside_the_rows_have_none():
    ys = rows(6, 16, 8, FP32).to(DEV)
    pos = torch.tensor([[0, 6], [2 ** 31 - 1, -2 ** 31], [5, 1]], dtype=torch.int32, device=DEV)
    w = torch.ones((3, 2), device=DEV)
    y = F.fp8_moe_combine(ys, pos, w)
    assert torch.equal(y[0], ys[0]) and not y[1].any() and torch.equal(y[2], ys[5] + ys[1])
    _, dw = F.fp8_moe_combine_grad(torch.ones((3, 16), device=DEV), ys, pos, w)
    assert (dw.cpu() != 0).tolist() == [[True, False], [False, False], [True, True]]


def test_non_finite_rows_stay_with_their_tokens():
    ys = rows(8, 32, 9, BF16)
    ys[3] = float("nan")
    ys[5, 2] = float("inf")
    pos = torch.arange(8, dtype=torch.int32).view(4, 2)
    pos[2, 0] = -1                  # of row 4
    y = F.fp8_moe_combine(ys.to(DEV), pos.to(DEV), torch.ones((4, 2), device=DEV)).cpu()
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all()
    assert y[1].isnan().all() and y[2, 2] == float("inf") and torch.isfinite(y[2, 3:]).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shift,pad", [(1, 0), (3, 2), (8, 8)])
def test_strides_and_untouched_gaps(dtype, shift, pad):
    T, k, E, H = 21, 3, 5, 72
    ids, w = routing(T, k, E, 10, 0.2)

    def place(t):
        wide = torch.full((t.shape[0], H + shift + pad), 7.0, dtype=dtype, device=DEV)
        wide[:, shift:shift + H] = t.to(DEV)
        return wide, wide[:, shift:shift + H]
    x, ys, dy = rows(T, H, 11, dtype), rows(T * k, H, 12, dtype), rows(T, H, 13, dtype)
    sevens = torch.full((T * k, H), 7.0, dtype=dtype)
    want, pos, _ = F.fp8_moe_dispatch(x.to(DEV), ids.to(DEV), E, out=sevens.to(DEV))
    wide, out = place(sevens)
    got, _, _ = F.fp8_moe_dispatch(place(x)[1], ids.to(DEV), E, out=out)
    assert got is out and torch.equal(got, want) and (wide[:, :shift] == 7).all() and (wide[:, shift + H:] == 7).all()
    wide, out = place(rows(T, H, 1, dtype))
    assert torch.equal(F.fp8_moe_combine(place(ys)[1], pos, w.to(DEV), out=out), F.fp8_moe_combine(ys.to(DEV), pos, w.to(DEV)))
    assert (wide[:, :shift] == 7).all() and (wide[:, shift + H:] == 7).all()
    wide, out = place(sevens)
    a = F.fp8_moe_combine_grad(place(dy)[1], place(ys)[1], pos, w.to(DEV), out=out)
    b = F.fp8_moe_combine_grad(dy.to(DEV), ys.to(DEV), pos, w.to(DEV), out=sevens.to(DEV))
    assert torch.equal(a[0], b[0]) and torch.allclose(a[1], b[1], rtol=1e-5, atol=1e-5)  # another order of the sum
    assert (wide[:, :shift] == 7).all() and (wide[:, shift + H:] == 7).all()


def test_offsets_past_32_bits():
    """2**31 elements of sorted rows and more; the last token's compared."""
    T, k, H = 2 ** 15 + 1, 8, 8200
    ids = torch.arange(k, dtype=torch.int32, device=DEV).expand(T, k).contiguous()
    x = torch.zeros((T, H), dtype=BF16, device=DEV)
    x[-1] = rows(1, H, 14, BF16)[0].to(DEV)
    xs, pos, offsets = F.fp8_moe_dispatch(x, ids, k)
    assert offsets.tolist() == [T * e for e in range(k + 1)]
    last = pos[-1].long()
    assert torch.equal(xs[last], x[-1:].expand(k, H)) and not xs[last - 1].any()
    w = torch.full((T, k), 0.25, device=DEV)
    y = F.fp8_moe_combine(xs, pos, w)
    assert torch.equal(y[-1], (2 * x[-1].float()).to(BF16)) and not y[:-1].any()
    dys, dw = F.fp8_moe_combine_grad(x, xs, pos, w, out=xs)
    assert torch.equal(dys[last], (0.25 * x[-1:].float()).to(BF16).expand(k, H))
    assert not dw[:-1].any() and dw[-1, 0] > 0 and (dw[-1] == dw[-1, 0]).all()


def test_there_and_back_in_a_graph_with_a_kept_workspace():
    T, k, E, H = 600, 4, 16, 256
    ids, w = routing(T, k, E, 15)
    x, ids, w = rows(T, H, 16, BF16).to(DEV), ids.to(DEV), w.abs().to(DEV)
    need = F.fp8_moe_dispatch_workspace_bytes(T, k, E)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device=DEV)

    def step():
        xs, pos, offsets = F.fp8_moe_dispatch(x, ids, E, ws=ws)
        y = F.fp8_moe_combine(xs, pos, w)
        dys, dw = F.fp8_moe_combine_grad(x, xs, pos, w)
        return y, dys, dw, F.fp8_moe_dispatch_grad(dys, pos), offsets
    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    ids.copy_(ids.flip(0))
    x.mul_(0.5)
    want = step()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    total = w.sum(1, keepdim=True)
    assert torch.allclose(want[0].float(), x.float() * total, rtol=2 ** -6, atol=1e-30)


@pytest.mark.parametrize("at", [0, 1])
def test_rows_of_almost_two_to_the_31_columns(at):
    """The last piece of the widest rows, from column 2**31 - 8 on: what lies behind a row counts in no sum."""
    H = 2 ** 31 - 5  # three columns of the last eight

    def row(last):
        wide = torch.full((H + at + 16,), 8.0, dtype=BF16, device=DEV)
        wide[at:at + H].zero_()
        wide[at + H - 3:at + H] = torch.tensor(last, dtype=BF16, device=DEV)
        return wide, wide[None, at:at + H]
    dy, ys, (wide, out) = row([1.0, 2.0, 3.0])[1], row([1.0, 2.0, 4.0])[1], row([5.0, 5.0, 5.0])
    pos, w = torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.full((1, 1), 0.5, device=DEV)
    F.fp8_moe_combine(ys, pos, w, out=out)
    assert out[0, -4:].tolist() == [0.0, 0.5, 1.0, 2.0] and (wide[at + H:] == 8.0).all()
    _, dw = F.fp8_moe_combine_grad(dy, ys, pos, w, out=out)
    assert dw.item() == 17.0
    assert out[0, -4:].tolist() == [0.0, 0.5, 1.0, 1.5] and (wide[at + H:] == 8.0).all()
    assert not out[0, :-3].any()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_gradient_of_rows_without_a_pair_is_zero(dtype):
    """Into a buffer of the call's own, whatever the allocator's memory held before."""
    T, k, E, H = 50, 4, 8, 333
    ids, w = routing(T, k, E, 17, 0.4)
    pos = torch.from_numpy(L.sort_rows(ids.numpy(), E)[0])
    ys, dy = rows(T * k, H, 18, dtype).to(DEV), rows(T, H, 19, dtype).to(DEV)
    want, _ = F.fp8_moe_combine_grad(dy, ys, pos.to(DEV), w.to(DEV), out=torch.zeros_like(ys))
    old = [torch.full_like(ys, float("nan")) for _ in range(4)]
    del old
    dys, _ = F.fp8_moe_combine_grad(dy, ys, pos.to(DEV), w.to(DEV))
    assert (pos < 0).any() and torch.equal(dys, want)


# pairs that a cluster sorts, and that many CTAs sort after counting; rows off 16-byte boundaries
@pytest.mark.parametrize("T,k,E", [(300, 4, 9), (1037, 2, 64), (2101, 4, 16)])
@pytest.mark.parametrize("H", [1, 2, 7, 9, 31, 1001, 2047])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_dispatch_of_many_pairs_and_odd_widths(T, k, E, H, dtype, drop):
    check_dispatch(T, k, E, H, dtype, drop)


@pytest.mark.parametrize("T,k", [(600, 3), (2101, 4)])
@pytest.mark.parametrize("H", [63, 72])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("shift,out_shift,pad", [(1, 0, 0), (0, 1, 3), (3, 6, 2), (5, 7, 1), (8, 2, 6)])
def test_dispatch_of_many_pairs_with_strides(T, k, H, dtype, shift, out_shift, pad):
    """x and out start anywhere and lie in wider rows, whose other columns stay as they were."""
    ids, _ = routing(T, k, 16, 20, 0.3)
    x = rows(T, H, 21, dtype)
    sevens = torch.full((T * k, H), 7.0, dtype=dtype, device=DEV)
    want, pos, offsets = F.fp8_moe_dispatch(x.to(DEV), ids.to(DEV), 16, out=sevens)
    pos_ref, _ = L.sort_rows(ids.numpy(), 16)
    kept = torch.from_numpy(np.argwhere(pos_ref >= 0))
    at = torch.from_numpy(pos_ref[pos_ref >= 0]).long()
    assert torch.equal(want.cpu()[at], x[kept[:, 0]]) and (want[int(offsets[-1]):] == 7.0).all()
    wide_x = torch.full((T, H + shift + pad), 5.0, dtype=dtype, device=DEV)
    wide_x[:, shift:shift + H] = x.to(DEV)
    wide = torch.full((T * k, H + out_shift + pad), 7.0, dtype=dtype, device=DEV)
    out = wide[:, out_shift:out_shift + H]
    got, pos2, offsets2 = F.fp8_moe_dispatch(wide_x[:, shift:shift + H], ids.to(DEV), 16, out=out)
    assert got is out and torch.equal(got, want) and torch.equal(pos, pos2) and torch.equal(offsets, offsets2)
    assert (wide[:, :out_shift] == 7.0).all() and (wide[:, out_shift + H:] == 7.0).all()


# one and two rows a token where there is work for every SM: a thread has several pieces under way
@pytest.mark.parametrize("k", [1, 2])
@pytest.mark.parametrize("dtype,H", [(BF16, 1000), (BF16, 250), (BF16, 1001), (FP32, 500), (FP32, 125)])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_few_rows_a_token_of_many_tokens(k, dtype, H, drop):
    """125 pieces of 16 bytes a row (16-bit rows that start anywhere), of 4 bytes (250 16-bit columns, 125 of 32 bits)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = sms * 2048 // 125 + 118
    assert T * 125 % 256 and T * 125 >= sms * 2048
    ids, w = routing(T, k, 7, H + k, drop)
    pos = torch.from_numpy(L.sort_rows(ids.numpy(), 7)[0])
    ys = rows(T * k, H, 22, dtype)
    out = torch.full((T + 1, H), 7.0, dtype=dtype, device=DEV)
    for weights in (w, None):
        F.fp8_moe_combine(ys.to(DEV), pos.to(DEV), None if weights is None else weights.to(DEV), out=out[:T])
        ref, err = L.combine(f32(ys), pos.numpy(), None if weights is None else weights.numpy())
        tol = L.rounded_bf16(ref, err) if dtype == BF16 else err
        assert np.all(np.abs(f32(out[:T]) - ref) <= tol) and (out[T] == 7.0).all()
    assert torch.equal(F.fp8_moe_dispatch_grad(ys.to(DEV), pos.to(DEV)), out[:T])


@pytest.mark.parametrize("k", [1, 2, 3])
@pytest.mark.parametrize("H", [70, 1000, 2050, 2051, 9001])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_gradient_of_few_rows_a_token(k, H, dtype):
    check_back(61, k, 5, H, dtype, 0.2, seed=23)
