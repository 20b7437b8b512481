"""GPU parity of the norms around a block with the float64 oracle."""

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


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    F.lib()


def operands(M, H, seed, post=False, gate=None, residual=True):
    g = torch.Generator().manual_seed(seed)

    def draw(*shape, std=1.0):
        return (torch.randn(shape, generator=g) * std).to(BF16)
    d = {"y": draw(M, H), "weight": draw(H, std=0.5)}
    d["y"][:, ::37] *= 16
    if residual:
        d["residual"] = draw(M, H, std=3.0)
    if post:
        d["post_weight"] = draw(H, std=0.5)
    if gate:
        d["gate"] = draw(H) if gate == "channel" else draw(M, H)
    return d


def on(dev, d):
    return {k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def reference(d):
    a = {("post" if k == "post_weight" else k): (f32(v) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    with np.errstate(all="ignore"):
        return L.norms(a.pop("y"), a.pop("weight", None), **a)


def close(got, want, err, what):
    off = np.abs(f32(got).astype(np.float64) - want)
    tol = L.rounded_bf16(want, err)
    assert np.all(off <= tol), f"{what}: {np.max(off / tol):.3f} of its tolerance"


def check(d, **kw):
    """Both calls against the oracle."""
    n_ref, n_err, r_ref, r_err = reference({**d, **kw})
    args = on(DEV, {k: v for k, v in d.items() if k not in ("y", "weight")})
    y, w = d["y"].to(DEV), d["weight"].to(DEV)
    n, r = F.fp8_residual_norm(y, w, **args, **kw)
    close(n, n_ref, n_err, "n")
    close(r, r_ref, r_err, "r")
    q, s, r2 = F.fp8_residual_norm_quantize(y, w, **args, **kw)
    assert torch.equal(r2, r)
    M, H = y.shape
    assert q.shape == (M, F.min_ld(H)) and s.shape == ((H + 127) // 128, M)
    assert not q[:, H:].any()
    v, dv = B._requantize(n_ref, n_err)
    got = O.decode(q.cpu().numpy()[:, :H]) * np.repeat(s.cpu().numpy().astype(np.float64), 128, 0)[:H].T
    # the value of a code: one more rounding where the scale was divided
    assert np.all(np.abs(got - v) <= dv + np.abs(v) * 4 * L.U)
    return n, r, q, s


@pytest.mark.parametrize("H", [1, 7, 16, 100, 128, 1001, 1024, 1025, 2048, 2056, 4096, 4104, 5000, 8192, 8200, 16384,
                               16400, 32768])
@pytest.mark.parametrize("M", [1, 3, 400])
def test_sizes(M, H):
    check(operands(M if H < 9000 or M < 9 else 20, H, M + H))


@pytest.mark.parametrize("M,H", [(1, 4096), (5, 1001), (300, 1536), (200, 5120), (9, 20000)])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
def test_post_norm_gate_and_scale(M, H, post, gate):
    check(operands(M, H, M + H, post, gate), scale=0.22, eps=1e-5)
    check(operands(M, H, M + H, post, gate, residual=False), plus_one=True)


def test_without_a_weight_or_a_change():
    d = operands(6, 200, 1, post=True)
    y = d["y"].to(DEV)
    n, r = F.fp8_residual_norm(y, None, residual=d["residual"].to(DEV), post_weight=d["post_weight"].to(DEV))
    _, _, r_ref, r_err = reference({**d, "weight": None})
    assert n is None
    close(r, r_ref, r_err, "r")
    n, r = F.fp8_residual_norm(y, d["weight"].to(DEV))
    assert r is y
    n_ref, n_err, _, _ = reference({"y": d["y"], "weight": d["weight"]})
    close(n, n_ref, n_err, "n")
    assert F.fp8_residual_norm(y) == (None, y)
    q, s, r = F.fp8_residual_norm_quantize(y, d["weight"].to(DEV))
    assert r is y


def test_zero_rows_and_tiny_values():
    d = operands(5, 300, 2)
    d["y"][1], d["residual"][1] = 0, 0
    d["y"][2], d["residual"][2] = 1e-30, -1e-38
    d["y"][3, :128], d["residual"][3, :128] = 0, 0  # a block of zeros
    n, r, q, s = check(d)
    assert not n[1].any() and not (q[1] & 0x7F).any() and (s[:, 1] == 1).all() and s[0, 3] == 1


def test_squares_past_fp32():
    big = float(torch.finfo(BF16).max)
    d = operands(4, 600, 3)
    d["y"][0] *= 2.0 ** 100
    d["residual"][0] = 0
    d["y"][1] = big
    d["residual"][1] = 0
    d["y"][2, 5] = 2.0 ** 70
    n, r, q, s = check(d)
    assert torch.isfinite(n).all()
    assert (n[1].float().abs().cpu() - d["weight"].float().abs()).abs().max() < 0.02


def test_non_finite_values_stay_in_their_row():
    d = operands(6, 400, 4, post=True, gate="token")
    clean = [t.cpu() for t in check(d)]
    for row, value in ((1, float("nan")), (3, float("inf")), (4, -float("inf"))):
        d["y"][row, 250] = value
    args = on(DEV, {k: v for k, v in d.items() if k not in ("y", "weight")})
    n, r = F.fp8_residual_norm(d["y"].to(DEV), d["weight"].to(DEV), **args)
    q, s, _ = F.fp8_residual_norm_quantize(d["y"].to(DEV), d["weight"].to(DEV), **args)
    for row in (0, 2, 5):
        assert torch.equal(n[row].cpu(), clean[0][row]) and torch.equal(q[row].cpu(), clean[2][row])
        assert torch.equal(s[:, row].cpu(), clean[3][:, row])
    assert n[1].isnan().all() and s[:, 1].isnan().all()
    assert r[3, 250].isnan() and n[3].isnan().all()  # inf times 1 / sqrt(inf)
    assert r[4, 250].isnan()


def test_negative_zero_codes_keep_their_sign():
    y = torch.full((2, 128), -0.0, dtype=BF16)
    y[1, 0] = 1.0
    w = torch.ones(128, dtype=BF16)
    q, s, _ = F.fp8_residual_norm_quantize(y.to(DEV), w.to(DEV), scale=1.0)
    # r = 0 + 1 * -0: without a residual the sum starts from +0, which takes the sign away
    assert (q[0] == 0).all()
    res = torch.full((2, 128), -0.0, dtype=BF16)
    q, s, _ = F.fp8_residual_norm_quantize(y.to(DEV), w.to(DEV), residual=res.to(DEV))
    assert (q[0] == 0x80).all() and (q[1, 1:] == 0x80).all() and q[1, 0] == 0x7E


@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 0), (3, 5), (8, 24)])
def test_strides_alignments_and_untouched_gaps(shift, pad):
    M, H = 37, 260
    d = operands(M, H, 5, post=True, gate="token")

    def place(t):
        wide = torch.full((M, H + shift + pad), 7.0, dtype=BF16, device=DEV)
        wide[:, shift:shift + H] = t.to(DEV)
        return wide, wide[:, shift:shift + H]
    vec = torch.zeros(H + shift, dtype=BF16, device=DEV)
    want = check(d)
    args = {k: place(d[k])[1] for k in ("residual", "gate")}
    vec[shift:] = d["weight"].to(DEV)
    out_w, out = place(torch.zeros(M, H))
    r_w, r = place(torch.zeros(M, H))
    n, r2 = F.fp8_residual_norm(place(d["y"])[1], vec[shift:], post_weight=d["post_weight"].to(DEV), out=out,
                                residual_out=r, **args)
    assert n is out and r2 is r
    assert torch.equal(n, want[0]) and torch.equal(r, want[1])
    for wide in (out_w, r_w):
        wide[:, shift:shift + H] = 7.0
        assert (wide == 7.0).all()


@pytest.mark.parametrize("H", [96, 1000, 4096, 8192])
def test_in_place(H):
    d = operands(50, H, 6, gate="channel")
    want_n, want_r, want_q, want_s = check(d)
    for name in ("y", "residual"):
        a = on(DEV, d)
        n, r = F.fp8_residual_norm(a["y"], a["weight"], residual=a["residual"], gate=a["gate"], residual_out=a[name])
        assert r is a[name] and torch.equal(r, want_r) and torch.equal(n, want_n)
        a = on(DEV, d)
        q, s, r = F.fp8_residual_norm_quantize(a["y"], a["weight"], residual=a["residual"], gate=a["gate"],
                                               residual_out=a[name])
        assert torch.equal(r, want_r) and torch.equal(q, want_q) and torch.equal(s, want_s)


def test_longer_code_rows_end_in_zeros():
    M, H, ldq, lds = 3, 200, 4096, 10
    d = operands(M, H, 7)
    a = on(DEV, d)
    q = torch.full((M, ldq), 9, dtype=torch.uint8, device=DEV)
    s = torch.full((2, lds), 9.0, device=DEV)
    p = lambda t: t.data_ptr()  # noqa: E731
    st = F.lib().fp8_residual_norm_quantize(p(a["y"]), M, H, H, None, None, 0, 1.0, p(a["residual"]), H, p(a["weight"]),
                                            1e-6, 0, None, 0, p(q), ldq, p(s), lds,
                                            torch.cuda.current_stream().cuda_stream)
    assert st == F.FP8_OK
    want = check(d)
    assert torch.equal(q[:, :208], want[2]) and not q[:, 208:].any()
    assert torch.equal(s[:, :M], want[3]) and (s[:, M:] == 9.0).all()


def test_empty():
    w = torch.ones(64, dtype=BF16, device=DEV)
    n, r = F.fp8_residual_norm(torch.empty((0, 64), dtype=BF16, device=DEV), w)
    assert n.shape == (0, 64)
    q, s, r = F.fp8_residual_norm_quantize(torch.empty((0, 64), dtype=BF16, device=DEV), w)
    assert q.shape == (0, 64) and s.shape == (1, 0)
    none = torch.empty((4, 0), dtype=BF16, device=DEV)
    q, s, r = F.fp8_residual_norm_quantize(none, none[0])
    assert q.shape == (4, 16) and not q.any() and s.shape == (0, 4)


def test_codes_are_operands_of_the_product():
    M, H, N = 70, 640, 256
    d = operands(M, H, 8)
    a = on(DEV, d)
    w = (torch.randn((N, H), generator=torch.Generator().manual_seed(9)) * H ** -0.5).to(BF16)
    qw, s_w = F.fp8_block_quantize_weight(w.to(DEV))
    q, s, r = F.fp8_residual_norm_quantize(a["y"], a["weight"], residual=a["residual"])
    y = F.fp8_block_scaled_mm(q, H, s, qw, s_w)
    ref, bound = B.scaled_product(q.cpu().numpy(), s.cpu().numpy(), qw.cpu().numpy(), s_w.cpu().numpy())
    assert np.all(np.abs(f32(y) - ref) <= L.rounded_bf16(ref, bound))


def test_many_rows_offsets_past_32_bits():
    """Rows whose byte and element offsets pass 2**31, the last ones compared."""
    M, H = 2 ** 16 + 3, 32768
    y = torch.zeros((M, H), dtype=BF16, device=DEV)
    d = operands(3, H, 10, residual=False)
    y[-3:] = d["y"].to(DEV)
    q, s, _ = F.fp8_residual_norm_quantize(y, d["weight"].to(DEV))
    q3, s3, _ = F.fp8_residual_norm_quantize(y[-3:].clone(), d["weight"].to(DEV))
    assert torch.equal(q[-3:], q3) and torch.equal(s[:, -3:], s3) and not (q[:-3] & 0x7F).any()
    n, _ = F.fp8_residual_norm(y, d["weight"].to(DEV), out=y)  # n over y
    n3, _ = F.fp8_residual_norm(d["y"].to(DEV), d["weight"].to(DEV))
    assert torch.equal(n[-3:], n3)


def test_graph_replay_and_side_stream():
    d = on(DEV, operands(64, 2048, 11, gate="token"))
    args = dict(residual=d["residual"], gate=d["gate"])
    want = F.fp8_residual_norm_quantize(d["y"], d["weight"], **args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = F.fp8_residual_norm_quantize(d["y"], d["weight"], **args)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = F.fp8_residual_norm_quantize(d["y"], d["weight"], **args)
    fresh = on(DEV, operands(64, 2048, 12, gate="token"))
    for k in ("y", "residual", "gate"):
        d[k].copy_(fresh[k])
    d["weight"].copy_(fresh["weight"])
    graph.replay()
    want = F.fp8_residual_norm_quantize(fresh["y"], fresh["weight"], residual=fresh["residual"], gate=fresh["gate"])
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_norm_over_its_input_has_no_residual_to_give():
    d = operands(9, 300, 13, residual=False)
    y, w = d["y"].to(DEV), d["weight"].to(DEV)
    want, same = F.fp8_residual_norm(y, w)
    assert same is y
    n, r = F.fp8_residual_norm(y, w, out=y)
    assert n is y and r is None and torch.equal(n, want)


@pytest.mark.parametrize("H", [2049, 2997, 4097, 7026, 8193, 12001, 16385, 32767])
@pytest.mark.parametrize("post,gate", [(False, None), (False, "token"), (True, None), (True, "channel"), (True, "token")])
def test_wide_rows_of_any_alignment(H, post, gate):
    check(operands(7, H, H, post, gate), scale=0.22)


# a row's threads from 32 to 1024, and two units of each; several rows of each CTA
@pytest.mark.parametrize("M,H", [(20000, 101), (6000, 1001), (2600, 2997), (1300, 7026), (700, 12001), (340, 20001)])
@pytest.mark.parametrize("post,gate", [(False, None), (True, "token")])
def test_many_rows_of_any_alignment(M, H, post, gate):
    check(operands(M, H, M, post, gate))


@pytest.mark.parametrize("M,H", [(5300, 101), (1700, 1001), (900, 2997), (400, 7026), (200, 12001), (160, 20001)])
@pytest.mark.parametrize("gate", [None, "token"])
def test_in_place_of_any_alignment(M, H, gate):
    """Rows that share 16-byte pieces with their neighbours, which other threads and CTAs write meanwhile."""
    d = operands(M, H, 14, post=gate is not None, gate=gate)
    want_n, want_r, want_q, want_s = check(d)

    def fresh():
        a = on(DEV, d)
        return a, {k: v for k, v in a.items() if k not in ("y", "weight")}
    for name in ("y", "residual"):
        a, rest = fresh()
        n, r = F.fp8_residual_norm(a["y"], a["weight"], residual_out=a[name], **rest)
        assert r is a[name] and torch.equal(r, want_r) and torch.equal(n, want_n)
        a, rest = fresh()
        q, s, r = F.fp8_residual_norm_quantize(a["y"], a["weight"], residual_out=a[name], **rest)
        assert torch.equal(r, want_r) and torch.equal(q, want_q) and torch.equal(s, want_s)
        a, rest = fresh()
        n, r = F.fp8_residual_norm(a["y"], a["weight"], out=a[name], **rest)
        assert n is a[name] and torch.equal(r, want_r) and torch.equal(n, want_n)
    a, rest = fresh()  # each over the other's input
    n, r = F.fp8_residual_norm(a["y"], a["weight"], out=a["y"], residual_out=a["residual"], **rest)
    assert torch.equal(r, want_r) and torch.equal(n, want_n)


@pytest.mark.parametrize("H", [300, 1024, 4096, 8192, 20000])
@pytest.mark.parametrize("eps", [1e-45, 1e-44, 1e-40, 1e-36, 1e-30])
@pytest.mark.parametrize("post", [False, True])
def test_squares_below_fp32(H, eps, post):
    """Rows whose squares are subnormal or vanish in fp32, beside an eps as small; zeros, and a row of ordinary values."""
    d = operands(7, H, 15, post=post)
    d["y"] *= torch.tensor([2.0 ** -60, 2.0 ** -73, 2.0 ** -76, 2.0 ** -80, 2.0 ** -100, 0.0, 1.0])[:, None]
    d["residual"].mul_(d["y"].abs().amax(1, keepdim=True) > 1e-3)
    check(d, eps=eps)
