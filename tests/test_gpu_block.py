"""GPU parity of the block-scaled linear against the float64 oracle: codes and scales bit for bit, outputs
within the oracle's bound (one bf16 ulp plus what fp32 sums may lose)."""

import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_dynamic_gb300 as F
from fp8_w8a8_quantized_dynamic_gb300 import _build
from oracle import block_oracle as B
from parity import assert_codes_equal, assert_guards_intact, f32, guarded

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    F.lib()


def rand(shape, seed, std=1.0, loud=0):
    """Seeded bf16 values on the CPU, `loud` columns 50 times larger."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * std
    if loud:
        x[..., torch.randint(0, shape[-1], (loud,), generator=g)] *= 50.0
    return x.to(torch.bfloat16)


def bits(x):
    return np.ascontiguousarray(x, np.float32).view(np.uint32)


def check(y, y_ref, tol, what=""):
    got = f32(y).astype(np.float64)
    bad = np.argwhere(~(np.abs(got - y_ref) <= tol))
    assert bad.size == 0, (f"{what}: {len(bad)} of {got.size} outside; first {bad[:3].tolist()} got "
                           f"{got[tuple(bad[:3].T)]} want {y_ref[tuple(bad[:3].T)]} tol {tol[tuple(bad[:3].T)]}")


def run(M, K, N, seed=0, bias=False, a=None, lda_pad=0, stream=None):
    """The linear into a guarded buffer, checked against the oracle on the library's own weight codes (which
    are checked bit for bit first)."""
    a = rand((M, K), seed, loud=2) if a is None else a
    w = rand((N, K), seed + 1, std=0.02)
    b = rand((N,), seed + 2) if bias else None
    qw, s_w = F.fp8_block_quantize_weight(w.to(DEV))
    q_ref, s_ref = B.quantize_matrix(f32(w))
    assert_codes_equal(qw, q_ref, K, "qw")
    assert np.array_equal(bits(s_w.cpu().numpy()), bits(s_ref))
    ad = torch.zeros((M, K + lda_pad), dtype=torch.bfloat16, device=DEV)[:, :K]
    ad.copy_(a)
    buf, y, base, row_bytes, used = guarded((M, N), torch.bfloat16, DEV)
    F.fp8_block_linear(ad, qw, s_w, None if b is None else b.to(DEV), out=y)
    torch.cuda.synchronize()
    assert F.fp8_last_device_status() == F.FP8_OK
    assert_guards_intact(buf, base, row_bytes, used, M)
    y_ref, tol = B.linear(f32(a), q_ref, s_ref, None if b is None else f32(b))
    check(y, y_ref, tol, f"{M}x{K}x{N}")
    return y


@pytest.mark.parametrize("M,K,N", [
    (1, 1, 1), (1, 16, 8), (2, 127, 129), (3, 128, 128), (5, 129, 65), (8, 256, 64), (16, 300, 200), (17, 1000, 1027),
    (1, 4100, 513), (13, 1000, 1027), (32, 2048, 320), (33, 640, 96), (64, 512, 1000), (127, 384, 257),
    (128, 1152, 256), (129, 130, 384), (200, 5632, 256), (300, 96, 2050), (515, 1280, 640)])
@pytest.mark.parametrize("bias", [False, True])
def test_linear(M, K, N, bias):
    run(M, K, N, seed=M + K + N, bias=bias)


@pytest.mark.parametrize("M,pad", [(3, 1), (19, 7), (150, 8)])
def test_strided_activations(M, pad):
    run(M, 513, 130, seed=5, lda_pad=pad)


@pytest.mark.parametrize("M,K", [(1, 1), (3, 128), (5, 200), (33, 1000), (130, 4096)])
def test_quantize_act(M, K):
    a = rand((M, K), M + K, loud=1)
    a[0] = 0  # a zero row: scale 1, codes 0
    qa, s_a = F.fp8_block_quantize_act(a.to(DEV))
    q_ref, s_ref = B.quantize_rows(f32(a))
    assert_codes_equal(qa, q_ref, K, "qa")
    assert np.array_equal(bits(s_a.cpu().numpy()), bits(s_ref))


def test_extreme_scales():
    """Blocks at the ends of the bf16 range keep their exact scale and codes."""
    a = rand((6, 384), 3)
    a[0] *= 2.0 ** 120
    a[1] *= 2.0 ** -126
    a[2, :128] = 0
    a[3, 5] = float(torch.finfo(torch.bfloat16).max)
    a[4] = 2.0 ** -133
    q_ref, s_ref = B.quantize_rows(f32(a))
    qa, s_a = F.fp8_block_quantize_act(a.to(DEV))
    assert_codes_equal(qa, q_ref, 384, "qa")
    assert np.array_equal(bits(s_a.cpu().numpy()), bits(s_ref))


def test_weight_batch():
    """A batch of matrices is quantized matrix by matrix, also from a strided view."""
    w = rand((3, 2, 200, 264), 4, std=0.05)
    q, s = F.fp8_block_quantize_weight(w.to(DEV))
    assert q.shape == (3, 2, 200, 272) and s.shape == (3, 2, 2, 3)
    view = w.to(DEV)[:, 1, :, :250]
    qv, sv = F.fp8_block_quantize_weight(view)
    for i in range(3):
        for j in range(2):
            q_ref, s_ref = B.quantize_matrix(f32(w[i, j]))
            assert_codes_equal(q[i, j], q_ref, 264, "batch")
            assert np.array_equal(bits(s[i, j].cpu().numpy()), bits(s_ref))
        q_ref, s_ref = B.quantize_matrix(f32(w[i, 1, :, :250]))
        assert_codes_equal(qv[i], q_ref, 250, "view")
        assert np.array_equal(bits(sv[i].cpu().numpy()), bits(s_ref))


@pytest.mark.parametrize("M", [1, 7, 16, 17, 40, 140])
def test_nonfinite_rows_stay_apart(M):
    """A NaN or an infinity makes its own token NaN and leaves the others as they are."""
    K, N = 320, 200
    a = rand((M, K), 8)
    clean = run(M, K, N, seed=8, a=a)
    bad = a.clone()
    bad[0, 150] = float("nan")
    if M > 2:
        bad[2, 3] = float("inf")
    qw, s_w = F.fp8_block_quantize_weight(rand((N, K), 9, std=0.02).to(DEV))
    y = F.fp8_block_linear(bad.to(DEV), qw, s_w)
    assert torch.isnan(y[0]).all()
    if M > 2:
        assert torch.isnan(y[2]).all()
    keep = [m for m in range(M) if m not in (0, 2)]
    assert torch.equal(y[keep], clean[keep])


def test_empty_and_zero_k():
    qw, s_w = F.fp8_block_quantize_weight(rand((40, 64), 1).to(DEV))
    assert F.fp8_block_linear(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV), qw, s_w).shape == (0, 40)
    b = rand((40,), 2).to(DEV)
    qz = torch.zeros((40, 16), dtype=torch.uint8, device=DEV)
    sz = torch.empty((1, 0), dtype=torch.float32, device=DEV)
    y = F.fp8_block_linear(torch.empty((3, 0), dtype=torch.bfloat16, device=DEV), qz, sz, b)
    assert torch.equal(y, b.expand(3, 40))


@pytest.mark.parametrize("M", [3, 16, 30, 200])
def test_scaled_mm_equals_linear(M):
    """The two steps apart give the linear's bits, also with scales in a wider buffer."""
    K, N = 700, 330
    a = rand((M, K), 21).to(DEV)
    qw, s_w = F.fp8_block_quantize_weight(rand((N, K), 22, std=0.02).to(DEV))
    b = rand((N,), 23).to(DEV)
    qa, s_a = F.fp8_block_quantize_act(a)
    wide = torch.full((s_a.shape[0], M + 5), 7.0, device=DEV)
    wide[:, :M] = s_a
    y = F.fp8_block_scaled_mm(qa, K, wide[:, :M], qw, s_w, b)
    y_ref, tol = B.linear(f32(a), *B.quantize_matrix(f32(rand((N, K), 22, std=0.02))), f32(b))
    check(y, y_ref, tol)
    assert torch.equal(y, F.fp8_block_scaled_mm(qa, K, s_a, qw, s_w, b))


@pytest.mark.parametrize("M,first,after", [(30, 4, 2), (130, 8, 2), (131, 4, 5), (200, 1, 3), (260, 16, 0)])
def test_scaled_mm_scales_from_inside_a_buffer(M, first, after):
    """Scales that are columns [first, first + M) of a wider buffer, filled with NaN around them."""
    K, N = 700, 330
    a = rand((M, K), 24).to(DEV)
    qw, s_w = F.fp8_block_quantize_weight(rand((N, K), 25, std=0.02).to(DEV))
    qa, s_a = F.fp8_block_quantize_act(a)
    wide = torch.full((s_a.shape[0], first + M + after), float("nan"), device=DEV)
    wide[:, first:first + M] = s_a
    assert torch.equal(F.fp8_block_scaled_mm(qa, K, wide[:, first:first + M], qw, s_w),
                       F.fp8_block_scaled_mm(qa, K, s_a, qw, s_w))


@pytest.mark.parametrize("M", [4, 24, 160])
def test_repeatable_on_another_stream(M):
    """The same bits on every call and on a side stream, with a workspace full of garbage."""
    K, N = 1536, 520
    a = rand((M, K), 31).to(DEV)
    qw, s_w = F.fp8_block_quantize_weight(rand((N, K), 32, std=0.02).to(DEV))
    y = F.fp8_block_linear(a, qw, s_w)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        need = F.fp8_block_workspace_bytes(M, K, N)
        ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device=DEV)
        ys = [F.fp8_block_linear(a, qw, s_w, ws=ws) for _ in range(4)]
    st.synchronize()
    for other in ys:
        assert torch.equal(y, other)


def test_graph_capture():
    """The linear runs inside a CUDA graph (no allocation, no synchronization of its own)."""
    for M in (4, 40):
        a = rand((M, 512), 41).to(DEV)
        qw, s_w = F.fp8_block_quantize_weight(rand((256, 512), 42, std=0.02).to(DEV))
        want = F.fp8_block_linear(a, qw, s_w)
        y = torch.zeros_like(want)
        ws = torch.empty(max(1, F.fp8_block_workspace_bytes(M, 512, 256)), dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            F.fp8_block_linear(a, qw, s_w, out=y, ws=ws)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_wrapper_refusals():
    a = rand((4, 256), 1).to(DEV)
    qw, s_w = F.fp8_block_quantize_weight(rand((64, 256), 2).to(DEV))
    with pytest.raises(ValueError):
        F.fp8_block_linear(a.float(), qw, s_w)
    with pytest.raises(ValueError):
        F.fp8_block_linear(a.t(), qw, s_w)
    with pytest.raises(ValueError):
        F.fp8_block_linear(a, qw[:, :128], s_w)
    with pytest.raises(ValueError):
        F.fp8_block_linear(a, qw, s_w[:, :1])
    with pytest.raises(ValueError):
        F.fp8_block_linear(a, qw, s_w, bias=torch.zeros(63, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        F.fp8_block_linear(a, qw, s_w, out=torch.empty((4, 63), dtype=torch.bfloat16, device=DEV))
    big = rand((64, 256), 3).to(DEV)
    with pytest.raises(F.FP8Error) as e:
        F.fp8_block_linear(big, qw, s_w, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == F.FP8_ERR_WORKSPACE


@pytest.mark.parametrize("M,K,N", [(17, 640, 64), (40, 1152, 130), (100, 2049, 512), (129, 4096, 384), (200, 5632, 320),
                                   (64, 14336, 256), (250, 1800, 1000)])
def test_few_tiles_share_k(M, K, N):
    """Shapes with few output tiles, whose K is divided among the CTAs of a cluster."""
    run(M, K, N, seed=M, bias=True)


@pytest.mark.parametrize("M,K,N", [(5, 256, 72), (40, 1152, 136), (300, 2048, 264), (1300, 128, 704), (2000, 384, 1032),
                                   (4100, 256, 2056)])
@pytest.mark.parametrize("first,after", [(0, 3), (1, 0), (2, 2), (4, 4), (8, 8), (5, 11)])
def test_output_rows_of_any_alignment(M, K, N, first, after):
    """Columns [first, first + N) of a wider output: the same bits as a gap-free one, nothing beside them touched."""
    a = rand((M, K), 41).to(DEV)
    b = rand((N,), 42).to(DEV)
    qw, s_w = F.fp8_block_quantize_weight(rand((N, K), 43, std=0.02).to(DEV))
    y = F.fp8_block_linear(a, qw, s_w, b)
    wide = torch.full((M, first + N + after), 7.0, dtype=torch.bfloat16, device=DEV)
    F.fp8_block_linear(a, qw, s_w, b, out=wide[:, first:first + N])
    assert torch.equal(wide[:, first:first + N], y)
    assert bool((wide[:, :first] == 7).all()) and bool((wide[:, first + N:] == 7).all())


@pytest.mark.parametrize("M,K,N", [(1500, 130, 1031), (3000, 257, 1153), (700, 100, 67)])
def test_odd_outputs_of_many_tiles(M, K, N):
    run(M, K, N, seed=N, bias=True)
