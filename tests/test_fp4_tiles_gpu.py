"""GPU tests of the persistent fp4 product by its tiles: the pair of CTAs (256 channels x 192 rows) and the
single CTA's 128 rows, which the products of test_fp4_gpu hardly reach.  Every shape here says which tile it
is for, and a test that got another one fails, so that a change of the rule cannot take the tests away.
Compared as in test_fp4_gpu, with the tolerance derived there.
"""
from __future__ import annotations

import ctypes

import pytest
import torch

import fp4_ref as ref
from rotated_w4a4_quantized_group_b200 import ck
from test_fp4_gpu import BF16, MX, NV

pytestmark = pytest.mark.gpu

PAIR, ONE = (2, 192), (1, 128)


def tile(M, N, K, fmt, experts=0, ragged=False):
    """(CTAs, rows) of a tile of the product; 0 CTAs: the few-tile kernel."""
    ctas, rows = ctypes.c_int(), ctypes.c_int()
    i64 = ctypes.c_int64
    ck.lib().ck_internal_fp4_tile(i64(M), i64(N), i64(K), fmt, experts, int(ragged), ctypes.byref(ctas),
                                  ctypes.byref(rows))
    return ctas.value, rows.value


def width(K, fmt):
    """K as both formats take it."""
    return K if K % ref.BLOCK[fmt] == 0 else K + 16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ck.lib()
    yield
    torch.cuda.synchronize()


# ------------------------------------------------------------------- how calls are made

def test_pairs_beside_other_calls():
    """Pairs with one to eighteen tiles each, clusters and single CTAs on as many streams, again and again:
    what a CTA sends to its peer never reaches the shared memory of the next one on that SM."""
    shapes = [(PAIR, 1500, 2049, 4112, NV), (PAIR, 1400, 2178, 4128, MX), (PAIR, 3000, 2048, 4096, NV),
              (PAIR, 2400, 3840, 4096, MX), (PAIR, 8000, 8000, 272, NV), (ONE, 2500, 2050, 544, MX),
              ((1, 64), 40, 3840, 2048, NV), ((0, 64), 100, 907, 4096, MX)]
    cases = []
    for i, (want, M, N, K, fmt) in enumerate(shapes):
        K, g = width(K, fmt), torch.Generator(device="cuda").manual_seed(110 + i)
        assert tile(M, N, K, fmt) == want
        x = torch.randn(M, K, device="cuda", generator=g, dtype=BF16)
        w, ws = ck.ck_quant_fp4(torch.randn(N, K, device="cuda", generator=g) * 0.05, fmt)
        cases.append((x, w, ws, fmt))
    want = [ck.ck_fp4_linear(*c) for c in cases]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    same = [[] for _ in cases]
    for _ in range(20):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                same[i].append((ck.ck_fp4_linear(*c, dev_status=status) == want[i]).all())
    torch.cuda.synchronize()
    assert status.item() == 0
    for i, s in enumerate(same):
        assert torch.stack(s).all(), f"case {i}"
