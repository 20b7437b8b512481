"""Failure detection of the adapters of many tokens without a GPU fault: one load is withheld from the waits of the first CTA of
either product, they run out after 20 ms, the error is reported once, nothing of what is left undone passes for a result, and the
next call is right. Nothing faults or hangs."""

import time

import numpy as np
import pytest
import torch

import fp8_w8a8_quantized_dynamic_gb300 as F
from fp8_w8a8_quantized_dynamic_gb300 import _build

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
TILE = 128


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    F.lib()


def operands(M, K, N, r, adapters, seed):
    g = torch.Generator().manual_seed(seed)

    def draw(*shape, std=1.0):
        return (torch.randn(shape, generator=g) * std).to(BF16).to(DEV)
    ids = torch.randint(-1, adapters, (M,), generator=g, dtype=torch.int32)
    return (draw(M, N), draw(M, K), draw(adapters, r, K, std=K ** -0.5), draw(adapters, N, r, std=r ** -0.5), ids.to(DEV),
            torch.rand(adapters, generator=g).to(DEV))


def withheld(form, args):
    """(what the call gives, what it leaves with a load withheld, into a buffer of 768), after a call that used the workspace."""
    y, x, a, b, ids, scales = args
    need = F.fp8_lora_workspace_bytes(*x.shape, y.shape[1], *a.shape[:2])
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    want = F.fp8_lora_add(*args, ws=ws)
    out = torch.full_like(y, 768.0)
    torch.cuda.synchronize()
    assert F.fp8_last_device_status() == F.FP8_OK  # nothing pending
    t0 = time.perf_counter()
    assert F.fp8_lora_selftest_timeout(form, *args, out, ws) == F.FP8_OK
    assert F.fp8_last_device_status() == F.FP8_ERR_TIMEOUT
    assert 0.02 <= time.perf_counter() - t0 < 5.0  # the wait ran out, it did not hang
    assert F.fp8_last_device_status() == F.FP8_OK  # reported once, then cleared
    assert torch.equal(F.fp8_lora_add(*args, ws=ws), want) and F.fp8_last_device_status() == F.FP8_OK
    return want, out


def tiles_of(ids, adapters):
    """The tokens of each tile: sorted by adapter, those without one last, 128 at most."""
    ids = ids.cpu().numpy()
    found = []
    for e in [*range(adapters), -1]:
        t = np.nonzero(ids == e)[0]
        found += [t[i:i + TILE] for i in range(0, t.size, TILE)]
    return found


@pytest.mark.parametrize("M,K,N,r", [(600, 64, 256, 16), (700, 512, 200, 64), (1500, 4096, 136, 8), (900, 1000, 1027, 12),
                                     (600, 2048, 64, 256)])
def test_unfinished_first_product(M, K, N, r):
    args = operands(M, K, N, r, 3, M)
    want, out = withheld(0, args)
    lost = torch.zeros(M, dtype=torch.bool)
    lost[torch.from_numpy(tiles_of(args[4], 3)[0])] = True
    assert out.cpu()[lost].isnan().all() and torch.equal(out.cpu()[~lost], want.cpu()[~lost])


@pytest.mark.parametrize("form,r,width", [(1, 64, 128), (1, 8, 128), (2, 12, 64), (2, 16, 64), (2, 190, 64)])
@pytest.mark.parametrize("M,N", [(700, 20000), (20000, 256), (40000, 64), (530, 12808)])
def test_unfinished_second_product(form, r, width, M, N):
    """Runs within a tile, on to the next, and over many tiles of one step each."""
    adapters = 3
    args = operands(M, 72, N, r, adapters, r)
    want, out = withheld(form, args)
    tiles, steps = tiles_of(args[4], adapters), -(-N // width)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ctas = min((M // TILE + adapters + 1) * steps, sms)
    run = -(-len(tiles) * steps // ctas)
    assert run > 1
    want, out = want.cpu(), out.cpu()
    left = want.clone()
    for u in range(1, run):  # the first CTA's steps from the second on
        left[torch.from_numpy(tiles[u // steps]), u % steps * width:(u % steps + 1) * width] = 768.0
    assert torch.equal(out, left)
