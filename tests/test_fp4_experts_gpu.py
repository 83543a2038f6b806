"""GPU tests of rows sorted by expert where they are not plain: activations of other layouts, whose experts
start at any address, codes in, and weights with room between matrices and rows.  Compared with float64 as in
test_fp4_gpu.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp4_ref as ref
from rotated_w4a4_quantized_group_b200 import ck
from test_fp4_gpu import BF16, DT, EXPERTS, F16, F32, FMT, NV, OFFSETS, _close, _gen, _place, _t, _weights, _x, _xvalues

pytestmark = pytest.mark.gpu

LAYOUT = pytest.mark.parametrize("layout", ["pitch", "odd", "cols", "oddcols", "second"])
# starts of every alignment, experts of one row, of none, of whole tiles and of more than one
UNEVEN = {"odd starts": [3, 40, 41, 170, 170, 305, 306], "whole tiles": [0, 128, 256, 384], "shifted tiles": [1, 129, 257, 500],
          "even starts": [2, 130, 132, 264, 328], "long": [5, 6, 700]}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ck.lib()
    yield
    torch.cuda.synchronize()


def _offsets(off):
    return torch.tensor(off, dtype=torch.int32, device="cuda")


@FMT
@DT
@LAYOUT
@pytest.mark.parametrize("name", UNEVEN)
def test_quant_by_expert_of_any_layout(fmt, dt, layout, name):
    off = UNEVEN[name]
    M, K, E = off[-1] + 7, 352, len(off) - 1
    t = 0.37 if fmt == NV and off[0] % 2 else None
    x = _x(M, K, dt, 21)
    codes = torch.full((M, K // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((ck.fp4_scales_bytes(M, K, fmt, E),), 0xA5, dtype=torch.uint8, device="cuda")
    ck.ck_quant_fp4(_place(x, layout), fmt, tensor_scale=_t(t), offsets=_offsets(off), codes=codes, scales=scales)
    rc, rs = ref.quantize(x, fmt, t)
    rows, idx = ref.expert_scale_index(off, K // ref.BLOCK[fmt])
    want = np.full((M, K // 2), 0xA5, np.uint8)
    want[rows] = ref.pack(rc)[rows]
    np.testing.assert_array_equal(codes.cpu().numpy(), want)
    np.testing.assert_array_equal(scales.cpu().numpy()[idx], rs[rows])


@FMT
@LAYOUT
@pytest.mark.parametrize("name", ["odd starts", "shifted tiles"])
def test_expert_linear_of_any_layout(fmt, layout, name):
    off = UNEVEN[name]
    M, N, K, E = off[-1] + 7, 200, 544, len(off) - 1
    x = _x(M, K, BF16, 22, spread=False)
    w, ws, _ = _weights(E, N, K, fmt, 23)
    outs = [torch.full((M, N), -7.5, dtype=BF16, device="cuda") for _ in range(2)]
    for a, out in zip((x.cuda(), _place(x, layout)), outs):
        ck.ck_fp4_expert_linear(a, _offsets(off), w, ws, fmt, out=out)
    assert torch.equal(*outs)


@FMT
@DT
@pytest.mark.parametrize("name,N,K", EXPERTS)
def test_experts_from_codes(fmt, dt, name, N, K):
    """Codes at a pitch with room behind the rows, weights with room behind rows and matrices."""
    off = OFFSETS[name]
    M, E, b = off[-1] + 9, len(off) - 1, ref.BLOCK[fmt]
    tw = [0.001 * (1 + e % 5) for e in range(E)] if fmt == NV else None
    tx = 0.02 if fmt == NV else None
    x = _x(M, K, F32, 24, spread=False)
    w, ws, wv = _weights(E, N, K, fmt, 25, tw)
    room = torch.full((E, N + 3, -(-K // 32) * 16 + 32), 0x77, dtype=torch.uint8, device="cuda")
    room[:, :N, : K // 2] = w
    buf = torch.full((M, -(-K // 32) * 16 + 48), 0x77, dtype=torch.uint8, device="cuda")
    rc, rs = ref.quantize(x, fmt, tx)
    codes = buf[:, : K // 2]
    codes.copy_(torch.from_numpy(ref.pack(rc)))
    rows, idx = ref.expert_scale_index(off, K // b)
    sb = np.zeros(ck.fp4_scales_bytes(M, K, fmt, E), np.uint8)
    sb[idx] = rs[rows]
    bias = (torch.randn(E, N, generator=_gen(26)) * 0.3).to((F16, F32, BF16)[N % 3]).cuda() if N % 2 else None
    out = torch.full((M, N + 8), -7.5, dtype=dt, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ck.ck_fp4_expert_linear(codes, _offsets(off), room[:, :N, : K // 2], ws, fmt, bias, x_scales=torch.from_numpy(sb).cuda(),
                            x_tensor_scale=_t(tx), w_tensor_scale=None if tw is None else torch.tensor(tw, device="cuda"),
                            out=out[:, :N], dev_status=status)
    assert status.item() == 0
    xv = _xvalues(x, fmt, tx)
    rest = torch.ones(M, dtype=torch.bool)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        rest[lo:hi] = False
        exact, mag = xv[lo:hi] @ wv[e].t(), xv[lo:hi].abs() @ wv[e].abs().t()
        if bias is not None:
            exact, mag = exact + bias[e].double(), mag + bias[e].double().abs()
        _close(out[lo:hi, :N], exact, mag, K, f"expert {e}")
    assert (out[rest] == -7.5).all() and (out[:, N:] == -7.5).all()


@FMT
def test_a_padded_batch_through_two_layers(fmt):
    """Rows behind the last sequence are left as they were, quantized or not, and change nothing."""
    off, M, K, N = [0, 60, 61, 200], 333, 320, 256
    x = _x(M, K, BF16, 27, spread=False).cuda()
    w1, s1, _ = _weights(3, N, K, fmt, 28)
    w2, s2, _ = _weights(3, K, N, fmt, 29)

    def layers(x):
        h = torch.full((M, N), float("nan"), dtype=BF16, device="cuda")
        ck.ck_fp4_expert_linear(x, _offsets(off), w1, s1, fmt, out=h)
        y = torch.full((M, K), -7.5, dtype=BF16, device="cuda")
        return h, ck.ck_fp4_expert_linear(h, _offsets(off), w2, s2, fmt, out=y)

    h, y = layers(x)
    assert torch.isfinite(h[:200]).all() and torch.isnan(h[200:]).all()
    assert torch.isfinite(y[:200]).all() and (y[200:] == -7.5).all()
    z = x.clone()
    z[200:] = float("nan")
    h2, y2 = layers(z)
    assert torch.equal(h[:200], h2[:200]) and torch.equal(y, y2)
