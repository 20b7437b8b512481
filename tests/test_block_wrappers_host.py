"""Host checks of the torch wrappers of the block-scaled calls, without a GPU: CPU tensors that call
themselves CUDA ones, and a library that records its arguments. What a wrapper hands to C has to be the
tensor's own layout, so that C can refuse rows that overlap."""

import pytest
import torch

import fp8_w8a8_quantized_dynamic_gb300 as F
from fp8_w8a8_quantized_dynamic_gb300 import _build

BF16 = torch.bfloat16


class Fake:
    is_cuda = True

    def __init__(self, t, index=0):
        self._t, self._index = t, index

    def __getattr__(self, name):
        return getattr(self._t, name)

    def get_device(self):
        return self._index


class Recorder:
    """Stands for the library: every call succeeds and is kept by name."""

    def __init__(self):
        self.calls = {}

    def __getattr__(self, name):
        def fn(*args):
            self.calls[name] = args
            return 0
        return fn


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(F, "_lib", r)
    monkeypatch.setattr(F, "_raw_stream", lambda index: 0)
    return r


@pytest.fixture
def real(monkeypatch):
    _build.build()
    F.lib()
    monkeypatch.setattr(F, "_raw_stream", lambda index: 0)


def refused(fn, *args, **kw):
    """The library itself says that an argument is invalid (nothing is enqueued)."""
    with pytest.raises(F.FP8Error) as e:
        fn(*args, **kw)
    assert e.value.status == F.FP8_ERR_INVALID_ARG


def zeros(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


# rows that share memory: one row broadcast, and windows that overlap
def overlapping(rows, cols, dtype=BF16):
    return [zeros(1, cols, dtype=dtype).expand(rows, cols),
            zeros(2 * rows + cols, dtype=dtype).as_strided((rows, cols), (2, 1))]


def linear_operands(K=256, N=64):
    return Fake(zeros(N, K, dtype=torch.uint8)), Fake(torch.ones((N + 127) // 128, (K + 127) // 128))


def expert_operands(T=4, E=2, k=2, H=256, I=128):
    return (Fake(zeros(T, k, dtype=torch.int32)), Fake(torch.ones(T, k)), Fake(zeros(E, 2, I, H, dtype=torch.uint8)),
            Fake(torch.ones(E, 2, 1, 2)), Fake(zeros(E, H, I, dtype=torch.uint8)), Fake(torch.ones(E, 2, 1)))


@pytest.mark.parametrize("which", [0, 1])
def test_rows_that_overlap_reach_c_as_they_are(rec, which):
    qw, s_w = linear_operands()
    a = overlapping(4, 256)[which]
    F.fp8_block_linear(Fake(a), qw, s_w)
    assert rec.calls["fp8_block_linear"][3] == a.stride(0)
    F.fp8_block_quantize_act(Fake(a))
    assert rec.calls["fp8_block_quantize_act"][3] == a.stride(0)
    F.fp8_block_quantize_weight(Fake(a))
    assert rec.calls["fp8_block_quantize_weight"][4] == a.stride(0)
    F.fp8_moe_experts(Fake(a), *expert_operands())
    assert rec.calls["fp8_moe_experts"][3] == a.stride(0)
    y = overlapping(4, 64)[which]
    F.fp8_block_linear(Fake(zeros(4, 256)), qw, s_w, out=Fake(y))
    assert rec.calls["fp8_block_linear"][10] == y.stride(0)
    qa, s_a = Fake(zeros(4, 256, dtype=torch.uint8)), Fake(torch.ones(2, 4))
    F.fp8_block_scaled_mm(qa, 256, s_a, qw, s_w, out=Fake(y))
    assert rec.calls["fp8_block_scaled_mm"][12] == y.stride(0)
    y = overlapping(4, 256)[which]
    F.fp8_moe_experts(Fake(zeros(4, 256)), *expert_operands(), out=Fake(y))
    assert rec.calls["fp8_moe_experts"][16] == y.stride(0)
    s_a = overlapping(2, 4, torch.float32)[which]
    F.fp8_block_scaled_mm(qa, 256, Fake(s_a), qw, s_w)
    assert rec.calls["fp8_block_scaled_mm"][5] == s_a.stride(0)
    x = overlapping(4, 16, torch.float32)[which]
    F.fp8_moe_route(Fake(x), 2)
    assert rec.calls["fp8_moe_route"][4] == x.stride(0)


@pytest.mark.parametrize("which", [0, 1])
def test_rows_that_overlap_are_refused(real, which):
    qw, s_w = linear_operands()
    a = Fake(overlapping(40, 256)[which])
    refused(F.fp8_block_linear, a, qw, s_w)
    refused(F.fp8_block_quantize_act, a)
    refused(F.fp8_block_quantize_weight, a)
    refused(F.fp8_moe_experts, Fake(overlapping(4, 256)[which]), *expert_operands())
    refused(F.fp8_moe_route, Fake(overlapping(4, 16, torch.float32)[which]), 2)
    qa, s_a = Fake(zeros(4, 256, dtype=torch.uint8)), Fake(torch.ones(2, 4))
    out = Fake(overlapping(4, 64)[which])
    refused(F.fp8_block_linear, Fake(zeros(4, 256)), qw, s_w, out=out)
    refused(F.fp8_block_scaled_mm, qa, 256, s_a, qw, s_w, out=out)
    refused(F.fp8_moe_experts, Fake(zeros(4, 256)), *expert_operands(), out=Fake(overlapping(4, 256)[which]))
    refused(F.fp8_block_scaled_mm, qa, 256, Fake(overlapping(2, 4, torch.float32)[which]), qw, s_w)


def test_one_row_of_any_stride_is_a_row(rec):
    """The stride of a single row (block of scales) means nothing and is not handed on."""
    qw, s_w = linear_operands()
    a = zeros(256).as_strided((1, 256), (3, 1))
    F.fp8_block_linear(Fake(a), qw, s_w, out=Fake(zeros(64).as_strided((1, 64), (1, 1))))
    assert rec.calls["fp8_block_linear"][3] == 256 and rec.calls["fp8_block_linear"][10] == 64
    F.fp8_block_quantize_act(Fake(a))
    assert rec.calls["fp8_block_quantize_act"][3] == 256
    F.fp8_block_quantize_weight(Fake(a))
    assert rec.calls["fp8_block_quantize_weight"][4] == 256
    F.fp8_moe_route(Fake(zeros(16, dtype=torch.float32).as_strided((1, 16), (2, 1))), 2)
    assert rec.calls["fp8_moe_route"][4] == 16
    F.fp8_moe_experts(Fake(a), *expert_operands(T=1))
    assert rec.calls["fp8_moe_experts"][3] == 256
    one = Fake(zeros(4, 128, dtype=torch.uint8)), 128, Fake(torch.ones(4).as_strided((1, 4), (1, 1)))
    F.fp8_block_scaled_mm(*one, *linear_operands(K=128))
    assert rec.calls["fp8_block_scaled_mm"][5] == 4


def test_wider_rows_keep_their_stride(rec):
    qw, s_w = linear_operands()
    F.fp8_block_linear(Fake(zeros(4, 300)[:, 8:264]), qw, s_w, out=Fake(zeros(4, 100)[:, :64]))
    assert rec.calls["fp8_block_linear"][3] == 300 and rec.calls["fp8_block_linear"][10] == 100
    F.fp8_block_quantize_weight(Fake(zeros(3, 2, 20, 64)[:, 1, :, :50]))
    assert rec.calls["fp8_block_quantize_weight"][1:6] == (3, 20, 50, 64, 2 * 20 * 64)


# ---------------------------------------------------------------------------
# tensors of a device that is not the current one
# ---------------------------------------------------------------------------

def test_the_stream_is_the_current_devices():
    from types import SimpleNamespace as NS
    raw = NS(_C=NS(_cuda_getCurrentRawStream=lambda i: 100 + i, _cuda_getDevice=lambda: 1))
    older = NS(_C=NS(), cuda=NS(current_device=lambda: 1, current_stream=lambda i: NS(cuda_stream=100 + i)))
    for torch_like in (raw, older):
        stream = F._stream_query(torch_like)
        assert stream(1) == 101
        with pytest.raises(ValueError, match="cuda:0.*current device is cuda:1"):
            stream(0)


def test_tensors_of_another_device_are_refused_by_every_wrapper(rec, monkeypatch):
    from types import SimpleNamespace as NS
    monkeypatch.setattr(F, "_raw_stream", F._stream_query(NS(_C=NS(_cuda_getCurrentRawStream=lambda i: 0,
                                                                   _cuda_getDevice=lambda: 0))))

    def on1(t):
        return Fake(t, 1)
    a, x = on1(zeros(4, 256)), on1(zeros(4, 16))
    qw, s_w, one = on1(zeros(64, 256, dtype=torch.uint8)), on1(torch.ones(1, 2)), on1(torch.ones(1))
    qa, s_a = on1(zeros(4, 256, dtype=torch.uint8)), on1(torch.ones(2, 4))
    experts = [on1(t._t) for t in expert_operands()]
    for call in (lambda: F.fp8_quantize_weight(a), lambda: F.fp8_quantize_act(a),
                 lambda: F.fp8_scaled_mm(qa, 256, one, qw, one), lambda: F.fp8_linear(a, qw, one, ws=zeros(1)),
                 lambda: F.fp8_linear_static(a, one, qw, one, ws=zeros(1)),
                 lambda: F.fp8_linear_ex(a, qw, one, ws=zeros(1)),
                 lambda: F.fp8_linear_weight_only(a, qw, one, ws=zeros(1)),
                 lambda: F.fp8_linear_noalloc(a, qw, one), lambda: F.fp8_block_quantize_weight(a),
                 lambda: F.fp8_block_quantize_act(a), lambda: F.fp8_block_scaled_mm(qa, 256, s_a, qw, s_w),
                 lambda: F.fp8_block_linear(a, qw, s_w), lambda: F.fp8_moe_route(x, 2),
                 lambda: F.fp8_moe_experts(a, *experts)):
        with pytest.raises(ValueError, match="current device"):
            call()
    enqueued = {name for name in rec.calls if not name.endswith("_bytes")}
    assert not enqueued


def test_route_ex_refusals(real):
    P = 0x7F0000000000  # aligned fake address, never read
    d = dict(x=P, bf16=0, T=4, E=64, ld=64, sigmoid=1, bias=None, groups=8, keep=2, group_max=1, k=8, renorm=0,
             factor=1.0, ids=P, w=P, stream=None)
    for kw in (dict(group_max=2), dict(group_max=-1), dict(groups=3), dict(keep=9), dict(k=17), dict(ld=63),
               dict(renorm=2), dict(x=None)):
        assert F.lib().fp8_moe_route_ex(*{**d, **kw}.values()) == F.FP8_ERR_INVALID_ARG, kw
    assert F.lib().fp8_moe_route_ex(*{**d, "T": 0}.values()) == F.FP8_OK
