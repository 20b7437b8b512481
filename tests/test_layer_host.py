"""Host checks of the norms, the adapters and the rows to experts and back, without a GPU: what the C entries refuse,
workspace sizes, and what the torch wrappers check and hand on."""

import math

import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_dynamic_gb300 as F
from fp8_w8a8_quantized_dynamic_gb300 import _build
from oracle import layer_oracle as L
from test_block_wrappers_host import BF16, Fake, overlapping, rec, real, refused, zeros  # noqa: F401 (fixtures)

P = 0x7F0000000000  # aligned fake addresses, never read
Q = 0x7F1000000000


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    F.lib()


def status(name, base, **change):
    d = {**base, **change}
    return getattr(F.lib(), name)(*d.values())


NORM = dict(y=P, M=4, H=256, ldy=256, post=P, gate=P, ldg=256, scale=1.0, residual=P, ldr=256, w=P, eps=1e-6, plus_one=0,
            r=P, ldro=256, n=P, ldn=256, stream=None)
QUANT = {**{k: v for k, v in NORM.items() if k not in ("n", "ldn", "stream")}, "q": P, "ldq": 256, "s": P, "lds": 4,
         "stream": None}


@pytest.mark.parametrize("change", [
    dict(y=None), dict(M=-1), dict(H=-1), dict(H=32769, ldy=32769), dict(ldy=255), dict(ldg=255), dict(ldr=255), dict(ldro=255),
    dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(scale=math.nan), dict(scale=math.inf),
    dict(plus_one=2), dict(plus_one=-1), dict(w=None)])
def test_norm_refusals(change):
    assert status("fp8_residual_norm", NORM, **change) == F.FP8_ERR_INVALID_ARG, change
    assert status("fp8_residual_norm_quantize", QUANT, **change) == F.FP8_ERR_INVALID_ARG, change


def test_norm_refusals_of_outputs():
    assert status("fp8_residual_norm", NORM, ldn=255) == F.FP8_ERR_INVALID_ARG
    assert status("fp8_residual_norm", NORM, n=None) == F.FP8_ERR_INVALID_ARG            # a weight for no n
    assert status("fp8_residual_norm", NORM, n=None, w=None, r=None) == F.FP8_ERR_INVALID_ARG  # nothing to write
    assert status("fp8_residual_norm_quantize", QUANT, q=None) == F.FP8_ERR_INVALID_ARG
    assert status("fp8_residual_norm_quantize", QUANT, s=None) == F.FP8_ERR_INVALID_ARG
    assert status("fp8_residual_norm_quantize", QUANT, lds=3) == F.FP8_ERR_INVALID_ARG
    assert status("fp8_residual_norm_quantize", QUANT, ldq=240) == F.FP8_ERR_INVALID_ARG
    assert status("fp8_residual_norm_quantize", QUANT, ldq=264) == F.FP8_ERR_MISALIGNED
    assert status("fp8_residual_norm_quantize", QUANT, q=P + 8) == F.FP8_ERR_MISALIGNED
    assert status("fp8_residual_norm_quantize", QUANT, s=P + 2) == F.FP8_ERR_MISALIGNED


@pytest.mark.parametrize("out,ld", [("r", "ldro"), ("n", "ldn")])
@pytest.mark.parametrize("over", ["y", "residual"])
def test_norm_over_its_input_with_another_stride(out, ld, over):
    apart = {**NORM, "y": Q, "residual": Q, "r": P + 4096, "n": P + 8192, over: P, out: P}
    assert status("fp8_residual_norm", apart, **{ld: 264}) == F.FP8_ERR_INVALID_ARG
    assert status("fp8_residual_norm", apart, **{ld: 264, "M": 0}) == F.FP8_OK
    if out == "r":
        quant = {**QUANT, "y": Q, "residual": Q, over: P}
        assert status("fp8_residual_norm_quantize", quant, ldro=264) == F.FP8_ERR_INVALID_ARG


def test_norm_with_both_outputs_in_one_place():
    apart = {**NORM, "y": Q, "residual": Q, "gate": Q, "post": Q, "w": Q}
    assert status("fp8_residual_norm", apart) == F.FP8_ERR_INVALID_ARG  # r and n are the same rows
    assert status("fp8_residual_norm", apart, M=0) == F.FP8_OK


@pytest.mark.parametrize("name", ["y", "post", "gate", "residual", "w", "r"])
def test_norm_misaligned(name):
    assert status("fp8_residual_norm", NORM, **{name: P + 1}) == F.FP8_ERR_MISALIGNED
    assert status("fp8_residual_norm_quantize", QUANT, **{name: P + 1}) == F.FP8_ERR_MISALIGNED


def test_empty_norms_enqueue_nothing():
    assert status("fp8_residual_norm", NORM, M=0) == F.FP8_OK
    assert status("fp8_residual_norm", NORM, H=0) == F.FP8_OK
    assert status("fp8_residual_norm_quantize", QUANT, M=0) == F.FP8_OK


LORA = dict(y=P, M=4, N=128, ldy=128, x=P, K=256, ldx=256, a=P, b=P, L=3, r=16, ids=P, scales=P, out=Q, ldo=128, ws=P,
            ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(L=-1), dict(L=512), dict(r=0), dict(r=257), dict(ldy=127), dict(ldx=255), dict(ldo=127),
    dict(y=None), dict(x=None), dict(a=None), dict(b=None), dict(ids=None), dict(out=None), dict(out=P, ldo=136),
    dict(K=2 ** 30 + 1, ldx=2 ** 31), dict(N=2 ** 30 + 1, ldy=2 ** 31, ldo=2 ** 31), dict(M=2 ** 31 - 100)])
def test_lora_refusals(change):
    assert status("fp8_lora_add", LORA, **change) == F.FP8_ERR_INVALID_ARG, change


@pytest.mark.parametrize("name,by", [("y", 1), ("x", 1), ("a", 1), ("b", 1), ("ids", 2), ("scales", 2), ("out", 1)])
def test_lora_misaligned(name, by):
    assert status("fp8_lora_add", LORA, **{name: LORA[name] + by}) == F.FP8_ERR_MISALIGNED


def test_lora_workspace():
    many = dict(M=4096, K=4096, N=4096, L=8, r=64)
    need = F.fp8_lora_workspace_bytes(*many.values())
    assert need % 256 == 0 and need > 4096 * (64 * 4 + 8)  # A x, positions and their order
    base = {**LORA, **many, "ldy": 4096, "ldx": 4096, "ldo": 4096}
    assert status("fp8_lora_add", base, ws=None) == F.FP8_ERR_WORKSPACE
    assert status("fp8_lora_add", base, ws_bytes=need - 1) == F.FP8_ERR_WORKSPACE
    assert status("fp8_lora_add", base, ws=P + 128) == F.FP8_ERR_WORKSPACE
    assert F.fp8_lora_workspace_bytes(1, 4096, 4096, 8, 64) == 0  # a token takes none
    for none in (dict(M=0), dict(K=0), dict(N=0), dict(L=0), dict(r=0), dict(L=512)):
        assert F.fp8_lora_workspace_bytes(*{**many, **none}.values()) == 0
    assert F.fp8_lora_workspace_bytes(2 ** 31 - 256, 2 ** 30, 2 ** 30, 511, 256) > 2 ** 40  # 64-bit sizes


def test_lora_selftest_refusals():
    many = dict(form=1, **{**LORA, "M": 4096, "N": 4096, "ldy": 4096, "K": 4096, "ldx": 4096, "L": 8, "r": 64, "ldo": 4096})
    for change in (dict(form=3), dict(form=-1), dict(M=0), dict(N=0), dict(K=0), dict(L=0), dict(M=4), dict(r=72), dict(r=60),
                   dict(N=4092), dict(ldy=4100), dict(ldo=4100), dict(y=P + 8), dict(out=Q + 8), dict(b=P + 8), dict(form=0, x=P + 8),
                   dict(form=0, a=P + 8), dict(form=0, ldx=4100), dict(form=0, K=4092), dict(form=2, r=193), dict(ids=None)):
        assert status("fp8_lora_selftest_timeout", {**many, **change}) == F.FP8_ERR_INVALID_ARG, change
    assert status("fp8_lora_selftest_timeout", {**many, "ws": None}) == F.FP8_ERR_WORKSPACE


def test_lora_nothing_to_do():
    assert status("fp8_lora_add", LORA, M=0) == F.FP8_OK
    assert status("fp8_lora_add", LORA, N=0) == F.FP8_OK


DISPATCH = dict(x=P, f32=0, T=100, H=64, ldx=64, ids=P, k=8, E=16, xs=P, ldxs=64, pos=P, offsets=P, ws=P, ws_bytes=1 << 20,
                stream=None)
COMBINE = dict(ys=P, f32=0, R=32, H=64, ldys=64, pos=P, weights=P, T=4, k=8, y=P, ldy=64, stream=None)
GRAD = dict(dy=P, f32=0, T=4, H=64, lddy=64, ys=P, R=32, ldys=64, pos=P, weights=P, k=8, dys=P, lddys=64, dw=P, stream=None)


@pytest.mark.parametrize("change", [dict(T=-1), dict(H=-1), dict(k=0), dict(k=33), dict(E=0), dict(E=513), dict(f32=2), dict(f32=-1),
                                    dict(ldx=63), dict(ldxs=63), dict(x=None), dict(xs=None), dict(ids=None), dict(pos=None),
                                    dict(offsets=None), dict(T=2 ** 31 // 8)])
def test_dispatch_refusals(change):
    assert status("fp8_moe_dispatch", DISPATCH, **change) == F.FP8_ERR_INVALID_ARG, change


def test_dispatch_workspace_and_alignment():
    need = F.fp8_moe_dispatch_workspace_bytes(4096, 8, 64)
    assert need > 0 and F.fp8_moe_dispatch_workspace_bytes(16, 8, 64) == 0
    assert F.fp8_moe_dispatch_workspace_bytes(4096, 33, 64) == 0 and F.fp8_moe_dispatch_workspace_bytes(4096, 8, 513) == 0
    base = {**DISPATCH, "T": 4096, "E": 64}
    assert status("fp8_moe_dispatch", base, ws=None) == F.FP8_ERR_WORKSPACE
    assert status("fp8_moe_dispatch", base, ws_bytes=need - 1) == F.FP8_ERR_WORKSPACE
    for name, by in (("x", 1), ("xs", 1), ("ids", 2), ("pos", 1), ("offsets", 2)):
        assert status("fp8_moe_dispatch", DISPATCH, **{name: P + by}) == F.FP8_ERR_MISALIGNED
    assert status("fp8_moe_dispatch", DISPATCH, f32=1, x=P + 2) == F.FP8_ERR_MISALIGNED


@pytest.mark.parametrize("change", [dict(R=-1), dict(T=-1), dict(H=-1), dict(k=0), dict(k=33), dict(f32=2), dict(ldys=63), dict(ys=None),
                                    dict(pos=None)])
def test_combine_and_gradient_refusals(change):
    assert status("fp8_moe_combine", COMBINE, **change) == F.FP8_ERR_INVALID_ARG, change
    assert status("fp8_moe_combine_grad", GRAD, **change) == F.FP8_ERR_INVALID_ARG, change


def test_more_refusals_on_the_way_back():
    for change in (dict(ldy=63), dict(y=None)):
        assert status("fp8_moe_combine", COMBINE, **change) == F.FP8_ERR_INVALID_ARG
    for change in (dict(lddy=63), dict(lddys=63), dict(dy=None), dict(dys=None), dict(dw=None), dict(weights=None)):
        assert status("fp8_moe_combine_grad", GRAD, **change) == F.FP8_ERR_INVALID_ARG
    assert status("fp8_moe_combine_grad", GRAD, lddys=72) == F.FP8_ERR_INVALID_ARG  # over ys with another stride
    assert status("fp8_moe_combine", COMBINE, T=0) == F.FP8_OK and status("fp8_moe_combine", COMBINE, H=0) == F.FP8_OK
    assert status("fp8_moe_combine_grad", GRAD, T=0) == F.FP8_OK
    assert status("fp8_moe_combine_grad", GRAD, dw=P + 2) == F.FP8_ERR_MISALIGNED
    d = dict(dxs=P, f32=0, R=32, H=64, lddxs=64, pos=P, T=4, k=8, dx=P, lddx=64, stream=None)
    assert status("fp8_moe_dispatch_grad", d, lddx=63) == F.FP8_ERR_INVALID_ARG
    assert status("fp8_moe_dispatch_grad", d, pos=None) == F.FP8_ERR_INVALID_ARG
    assert status("fp8_moe_dispatch_grad", d, T=0) == F.FP8_OK


def test_outputs_over_rows_that_others_still_read():
    bad = F.FP8_ERR_INVALID_ARG
    assert status("fp8_moe_dispatch", DISPATCH) == bad                               # xs over x
    assert status("fp8_moe_combine", COMBINE) == bad                                 # y over ys
    assert status("fp8_moe_combine_grad", GRAD, ys=Q) == bad                         # dys over dy
    assert status("fp8_lora_add", LORA, out=LORA["x"], y=Q) == bad                   # out over x
    grad = dict(dxs=P, f32=0, R=32, H=64, lddxs=64, pos=Q, T=4, k=8, dx=P, lddx=64, stream=None)
    assert status("fp8_moe_dispatch_grad", grad) == bad                              # dx over dxs
    for name, base in (("fp8_moe_dispatch", DISPATCH), ("fp8_moe_combine", COMBINE), ("fp8_moe_combine_grad", GRAD)):
        wide = {k: 128 if k.startswith("ld") else v for k, v in base.items()}
        assert status(name, wide) == bad


# ---------------------------------------------------------------------------
# wrappers
# ---------------------------------------------------------------------------

def vec(n, dtype=BF16):
    return Fake(torch.ones(n, dtype=dtype))


def lora_operands(M=4, K=256, N=128, r=16, adapters=3, index=0):
    return [Fake(t, index) for t in (zeros(M, N), zeros(M, K), zeros(adapters, r, K), zeros(adapters, N, r),
                                     zeros(M, dtype=torch.int32), torch.ones(adapters))]


@pytest.mark.parametrize("which", [0, 1])
def test_rows_that_overlap_are_refused_here_too(real, which):
    x = Fake(overlapping(4, 256)[which])
    refused(F.fp8_residual_norm, x, vec(256))
    refused(F.fp8_residual_norm_quantize, Fake(zeros(4, 256)), vec(256), residual=x)
    refused(F.fp8_residual_norm, Fake(zeros(4, 256)), vec(256), out=x)
    y, xl, *rest = lora_operands()
    refused(F.fp8_lora_add, y, x, *rest)
    refused(F.fp8_lora_add, y, xl, *rest, out=Fake(overlapping(4, 128)[which]))
    refused(F.fp8_moe_dispatch, x, Fake(zeros(4, 2, dtype=torch.int32)), 3)
    refused(F.fp8_moe_combine, x, Fake(zeros(2, 2, dtype=torch.int32)))
    refused(F.fp8_moe_combine_grad, x, Fake(zeros(8, 256)), Fake(zeros(4, 2, dtype=torch.int32)), Fake(torch.ones(4, 2)))
    if which == 1:  # (rows that are all one row are a gate a channel, told by its shape, not by its stride)
        refused(F.fp8_residual_norm, Fake(zeros(4, 256)), vec(256), gate=x)


def test_a_gate_a_channel_has_no_row_stride(rec):
    F.fp8_residual_norm(Fake(zeros(4, 256)), vec(256), gate=vec(256))
    assert rec.calls["fp8_residual_norm"][6] == 0
    F.fp8_residual_norm(Fake(zeros(4, 256)), vec(256), gate=Fake(zeros(4, 300)[:, :256]))
    assert rec.calls["fp8_residual_norm"][6] == 300
    # a row of its own and a gate of it: the row stride means nothing, but is not 0
    F.fp8_residual_norm(Fake(zeros(1, 256)), vec(256), gate=Fake(zeros(256).as_strided((1, 256), (0, 1))))
    assert rec.calls["fp8_residual_norm"][6] == 256


def test_no_residual_where_the_norm_took_its_place(rec):
    y, w = Fake(zeros(4, 256)), vec(256)
    other = Fake(zeros(4, 256))
    assert F.fp8_residual_norm(y, w, out=y)[1] is None
    assert F.fp8_residual_norm(y, w, out=other) == (other, y)
    assert F.fp8_residual_norm(y, w, residual=Fake(zeros(4, 256)), out=y, residual_out=other)[1] is other
    for empty in (Fake(zeros(0, 256)), Fake(zeros(4, 0))):
        assert F.fp8_residual_norm(empty, vec(empty.shape[1]))[1] is empty


def bad_calls():
    y, w = Fake(zeros(4, 256)), vec(256)
    yl, xl, a, b, ids, sc = lora_operands()
    x, pos, wt = Fake(zeros(4, 64)), Fake(zeros(4, 2, dtype=torch.int32)), Fake(torch.ones(4, 2))
    ys = Fake(zeros(8, 64))
    return [
        lambda: F.fp8_residual_norm(Fake(zeros(4, 256, dtype=torch.float32)), w),
        lambda: F.fp8_residual_norm(Fake(zeros(256, 4).t()), w),
        lambda: F.fp8_residual_norm(y, vec(255)),
        lambda: F.fp8_residual_norm(y, vec(256, torch.float32)),
        lambda: F.fp8_residual_norm(y, w, residual=Fake(zeros(3, 256))),
        lambda: F.fp8_residual_norm(y, w, gate=Fake(zeros(4, 255))),
        lambda: F.fp8_residual_norm(y, w, gate=vec(4)),
        lambda: F.fp8_residual_norm(y, w, post_weight=vec(4)),
        lambda: F.fp8_residual_norm(y, w, residual_out=Fake(zeros(4, 128))),
        lambda: F.fp8_residual_norm(y, None, out=Fake(zeros(4, 256))),
        lambda: F.fp8_residual_norm(y, w, residual=Fake(zeros(4, 256), 1)),
        lambda: F.fp8_residual_norm_quantize(y, None),
        lambda: F.fp8_lora_add(yl, Fake(zeros(5, 256)), a, b, ids, sc),
        lambda: F.fp8_lora_add(yl, xl, Fake(zeros(3, 16, 255)), b, ids, sc),
        lambda: F.fp8_lora_add(yl, xl, Fake(zeros(3, 256, 16).transpose(1, 2)), b, ids, sc),
        lambda: F.fp8_lora_add(yl, xl, a, Fake(zeros(3, 16, 128)), ids, sc),
        lambda: F.fp8_lora_add(yl, xl, a, b, Fake(zeros(4, dtype=torch.int64)), sc),
        lambda: F.fp8_lora_add(yl, xl, a, b, Fake(zeros(8, dtype=torch.int32)[::2]), sc),
        lambda: F.fp8_lora_add(yl, xl, a, b, ids, Fake(torch.ones(4))),
        lambda: F.fp8_lora_add(yl, xl, a, b, ids, sc, out=Fake(zeros(4, 120))),
        lambda: F.fp8_lora_add(yl, xl, a, b, ids, sc, ws=Fake(zeros(8, dtype=torch.float32))),
        lambda: F.fp8_moe_dispatch(Fake(zeros(4, 64, dtype=torch.float16)), pos, 3),
        lambda: F.fp8_moe_dispatch(x, Fake(zeros(5, 2, dtype=torch.int32)), 3),
        lambda: F.fp8_moe_dispatch(x, Fake(zeros(4, 2, dtype=torch.int64)), 3),
        lambda: F.fp8_moe_dispatch(x, pos, 0),
        lambda: F.fp8_moe_dispatch(x, pos, 3, out=Fake(zeros(7, 64))),
        lambda: F.fp8_moe_combine(ys, Fake(zeros(4, dtype=torch.int32)), wt),
        lambda: F.fp8_moe_combine(ys, pos, Fake(torch.ones(4, 3))),
        lambda: F.fp8_moe_combine(ys, pos, wt, out=Fake(zeros(4, 64, dtype=torch.float32))),
        lambda: F.fp8_moe_combine_grad(x, Fake(zeros(8, 63)), pos, wt),
        lambda: F.fp8_moe_combine_grad(Fake(zeros(5, 64)), ys, pos, wt),
        lambda: F.fp8_moe_combine_grad(x, ys, pos, None),
        lambda: F.fp8_moe_dispatch_grad(ys, pos, out=Fake(zeros(5, 64))),
    ]


@pytest.mark.parametrize("which", range(len(bad_calls())))
def test_wrappers_refuse(rec, which):
    with pytest.raises(ValueError):
        bad_calls()[which]()
    assert not {n for n in rec.calls if not n.endswith("_bytes")}


def test_tensors_of_another_device_are_refused(rec, monkeypatch):
    from types import SimpleNamespace as NS
    monkeypatch.setattr(F, "_raw_stream", F._stream_query(NS(_C=NS(_cuda_getCurrentRawStream=lambda i: 0,
                                                                   _cuda_getDevice=lambda: 0))))
    x, w = Fake(zeros(4, 64), 1), Fake(torch.ones(64, dtype=BF16), 1)
    pos, wt, ys = Fake(zeros(4, 2, dtype=torch.int32), 1), Fake(torch.ones(4, 2), 1), Fake(zeros(8, 64), 1)
    for call in (lambda: F.fp8_residual_norm(x, w), lambda: F.fp8_residual_norm_quantize(x, w),
                 lambda: F.fp8_lora_add(*lora_operands(index=1)), lambda: F.fp8_moe_dispatch(x, pos, 3),
                 lambda: F.fp8_moe_combine(ys, pos, wt), lambda: F.fp8_moe_combine_grad(x, ys, pos, wt),
                 lambda: F.fp8_moe_dispatch_grad(ys, pos)):
        with pytest.raises(ValueError, match="current device"):
            call()
    assert not {n for n in rec.calls if not n.endswith("_bytes")}


# ---------------------------------------------------------------------------
# the oracle against small cases by hand
# ---------------------------------------------------------------------------

def test_oracle_by_hand():
    n, _, r, _ = L.norms(np.array([[3.0, 4.0]]), weight=np.array([2.0, 1.0]), eps=1e-30)
    assert np.allclose(n, [[6 / math.sqrt(12.5), 4 / math.sqrt(12.5)]]) and np.array_equal(r, [[3.0, 4.0]])
    n, _, r, _ = L.norms(np.array([[3.0, 4.0]]), post=np.array([0.0, 1.0]), residual=np.array([[1.0, 1.0]]),
                         gate=np.array([0.5, 2.0]), scale=0.5, eps=1e-30, plus_one=True)
    assert n is None and np.allclose(r, [[1 + 0.25 * 3 / math.sqrt(12.5), 1 + 2 * 4 / math.sqrt(12.5)]])
    pos, off = L.sort_rows(np.array([[2, 0], [7, 2], [0, -1]], np.int32), 3)
    assert pos.tolist() == [[2, 0], [-1, 3], [1, -1]] and off.tolist() == [0, 2, 2, 4]
    ys = np.arange(8.0).reshape(4, 2)
    y, _ = L.combine(ys, pos, np.array([[1.0, 2.0], [5.0, 3.0], [1.0, 9.0]], np.float32))
    assert y.tolist() == [[4.0, 7.0], [18.0, 21.0], [2.0, 3.0]]
    dys, dw, _ = L.combine_grad(np.ones((3, 2)), ys, pos, np.array([[1.0, 2.0], [5.0, 3.0], [1.0, 9.0]], np.float32))
    assert dys.tolist() == [[2.0, 2.0], [1.0, 1.0], [1.0, 1.0], [3.0, 3.0]]
    assert dw.tolist() == [[9.0, 1.0], [0.0, 13.0], [5.0, 0.0]]
    out, _ = L.lora(np.ones((3, 1)), np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]]), np.ones((2, 1, 2)),
                    np.array([[[2.0]], [[-1.0]]]), np.array([1, 5, 0]), np.array([1.0, 0.5], np.float32))
    assert out.tolist() == [[-0.5], [1.0], [23.0]]
